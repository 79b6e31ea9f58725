"""Norms of more rows than the GPU holds workgroups: every workgroup takes rows in turn, the third turn on the words of
LDS of the first.  Every row is checked, under the bars of test_gpu_norm_rows.
"""
import numpy as np
import pytest
import torch

import quantized_gemm_amd as qg
from oracle import layer_ops as LO
from test_gpu_norm_rows import Case, _d

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qg.lib()
    yield


# rows of 1025 to 2048 values: 1024 workgroups, to 4096: 768, to 8192: 256
SHAPES = [(1416, 2100), (2048, 3077), (2056, 1600), (4096, 2309), (4104, 700), (8192, 1030)]


@pytest.mark.parametrize("k,rows", SHAPES)
@pytest.mark.parametrize("kw", [
    dict(code="e4m3"),
    dict(kind="layer", post="rms", gate="rows", bias=True, code="int8", res="f32", res_scale=0.5, pad=8),
    dict(kind="rms", post="layer", gate="one", offset=1.0, code="e2m1", pad=24),
    dict(kind="layer", post="layer", gate="rows", dtype="f16"),
    dict(kind="", post="rms", gate="rows", res="f32"),
    dict(residual=False, code="e4m3", out=False),
], ids=["e4m3", "layer-int8-f32", "post-layer-e2m1", "both-layer-f16", "residual-f32", "codes"])
def test_rows_in_turn(k, rows, kw):
    kw = dict(kw)
    if kw.get("code") == "e2m1":
        k = k // 32 * 32
    Case(rows, k, **kw).run().check()


@pytest.mark.parametrize("k,rows", [(1416, 2100), (4096, 2309), (8192, 1030)])
@pytest.mark.parametrize("res", ["bf16", "f32"])
def test_rows_in_turn_in_place(k, rows, res):
    Case(rows, k, inplace=True, code="e4m3", pad=8, res=res, post="rms", gate="rows").run().check()


@pytest.mark.parametrize("k", [1416, 4096, 8192])
def test_rows_that_are_not_finite_or_far_up_among_others(k):
    # rows that take the slow way and those that are NaN, between others, in every turn
    rows = 2309
    c = Case(rows, k, kind="layer", code="int8", y=False, res="f32")
    special = np.arange(5, rows, 97)
    c.wide_r[special[::3], 9] = float("nan")
    c.wide_r[special[1::3], k - 1] = float("inf")
    c.wide_r[special[2::3]] *= 1e36
    c.want = LO.norm_rows(res=np.where(np.isfinite(_d(c.r)).all(axis=1)[:, None], _d(c.r), 0.0), weight=_d(c.w), **c.args)
    c.run()
    torch.cuda.synchronize()
    bad = np.concatenate([special[::3], special[1::3]])
    out, u = _d(c.out_wide), _d(c.res_wide)
    assert np.isnan(out[bad]).all() and np.isnan(_d(c.scale)[bad]).all() and not c.codes[torch.from_numpy(bad).cuda()].any()
    ok = np.setdiff1d(np.arange(rows), bad)
    z, zmag = c.want[1][ok], c.want[3][ok]
    assert (np.abs(out[ok] - z) <= 2.0 ** -8 * np.abs(z) + 2.0 ** -17 * zmag).all()
    assert np.array_equal(u[ok], _d(c.r)[ok])


@pytest.mark.parametrize("k,rows,post", [(8, 16 * (1 << 21) + 40, ""), (136, 4 * (1 << 21) + 9, "rms"), (8200, (1 << 21) + 3, "")])
def test_more_rows_than_a_launch_has_workgroups(k, rows, post):
    # rows of a workgroup (or part of one) each: 2^21 workgroups of 16, 4 and 1 rows, and a second turn of the first ones.
    # The rows repeat, in place: every repetition has the same bits, and those of the first are checked.
    base = 1 << 10
    torch.manual_seed(k)
    first = torch.randn((base, k), device="cuda").to(torch.bfloat16)
    w = torch.randn(k, device="cuda").to(torch.bfloat16)
    x = torch.empty((rows, k), dtype=torch.bfloat16, device="cuda")
    whole = rows // base * base
    x[:whole].view(-1, base, k).copy_(first.expand(rows // base, base, k))
    x[whole:].copy_(first[:rows - whole])
    d = qg.make_norm_desc(qg.N_RMS, qg.O_BF16, k, 1e-6, post_norm=qg.N_RMS if post else 0)
    qg.norm_rows(d, rows, x if post else None, None if post else x, None, x, weight=w, post_weight=w if post else None)
    torch.cuda.synchronize()
    u, z, umag, zmag = LO.norm_rows(y=_d(first) if post else None, res=None if post else _d(first), post=post, weight=_d(w),
                                    post_weight=_d(w) if post else None)
    got = x[:base].clone()
    assert (np.abs(_d(got) - z) <= 2.0 ** -8 * np.abs(z) + 2.0 ** -17 * zmag + 2.0 ** -25).all()
    step = max(base, (1 << 26) // k // base * base)
    for i in range(0, whole, step):
        part = x[i:min(i + step, whole)].view(-1, base, k)
        assert torch.equal(part, got.expand(part.shape)), i
    assert torch.equal(x[whole:], got[:rows - whole])
