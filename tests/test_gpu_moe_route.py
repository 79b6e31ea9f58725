"""GPU parity of qg_moe_route against the float64 definition.

Chosen experts: equal, in order.  Choice values are held in 64 bits on both sides; two of them
that differ by more than 2^-48 compare alike, and random rows have none closer (equal logits give
equal values on both sides and go to the lower index).
Weights: |gpu - ref| <= 2^-24 (1 + 2^-16) |ref| + 2^-149: 64-bit arithmetic of a few hundred
operations (2^-44 relative, below 2^-16 of a float32 half step) and one rounding to float32.
"""
import numpy as np
import pytest
import torch

import quantized_gemm_amd as qg
from oracle import formats as F
from oracle import route as RT
from quantized_gemm_amd import synth

pytestmark = pytest.mark.gpu

TYPE = {"f32": qg.L_F32, "bf16": qg.L_BF16, "f16": qg.L_F16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qg.lib()
    yield


def _logits(values, dtype, pad=0):
    """float32 [T, E] -> (device rows of E + pad elements, the float64 values they hold)."""
    v = np.asarray(values, np.float32)
    if dtype == "f32":
        held, bits = v.astype(np.float64), v
    elif dtype == "bf16":
        bits = synth.f32_to_bf16_bits(v)
        held = F.decode_bf16(bits)
    else:
        with np.errstate(over="ignore"):
            bits = synth.f32_to_f16_bits(v)
        held = F.decode_f16(bits)
    wide = np.zeros((v.shape[0], v.shape[1] + pad), bits.dtype)
    if dtype != "f32":
        wide[:] = 0x7B00 if dtype == "f16" else 0x7F00          # large values between the rows: never read as logits
    else:
        wide[:] = 1e30
    wide[:, :v.shape[1]] = bits
    dev = torch.from_numpy(wide.view(np.int16) if dtype != "f32" else wide).cuda()
    return dev, held


def _check(values, dtype, scoring, topk, bias=None, groups=1, topk_groups=1, group_top=1, renorm=False, scale=1.0, pad=0,
           stream=None, total=None):
    # total: so many tokens, whose rows repeat the given ones
    n, e = np.asarray(values).shape
    t = n if total is None else total
    dev, held = _logits(np.resize(np.asarray(values, np.float32), (t, e)), dtype, pad)
    held = held[:n]
    desc = qg.make_route_desc(qg.R_SOFTMAX if scoring == "softmax" else qg.R_SIGMOID, e, topk, groups, topk_groups,
                              group_top, renorm, scale)
    ids = torch.full((t + 1, topk), 77, dtype=torch.int32, device="cuda")
    w = torch.full((t + 1, topk), 77.0, dtype=torch.float32, device="cuda")
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    torch.cuda.synchronize()
    qg.moe_route(desc, dev, TYPE[dtype], t, ids, w, b, row_stride=e + pad, stream=stream)
    torch.cuda.synchronize()
    assert (ids[t] == 77).all() and (w[t] == 77).all()           # nothing behind the last token
    rid, rw = RT.route(held, scoring, topk, bias=None if bias is None else np.asarray(bias, np.float32), groups=groups,
                       topk_groups=topk_groups, group_top=group_top, renorm=renorm, scale=scale)
    rid, rw = np.resize(rid, (t, topk)), np.resize(rw, (t, topk))
    got_id, got_w = ids[:t].cpu().numpy(), w[:t].cpu().numpy()
    assert np.array_equal(got_id, rid), f"{np.count_nonzero((got_id != rid).any(1))} tokens differ: {got_id[(got_id != rid).any(1)][:2]} {rid[(got_id != rid).any(1)][:2]}"
    assert np.all(np.abs(got_w - rw) <= 2.0 ** -24 * (1 + 2.0 ** -16) * np.abs(rw) + 2.0 ** -149)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,e,topk", [(1, 1, 1), (3, 2, 2), (5, 7, 3), (64, 8, 2), (33, 60, 4), (16, 63, 6), (16, 64, 6),
                                      (17, 65, 6), (200, 128, 8), (9, 129, 9), (50, 256, 8), (7, 257, 64), (21, 384, 10),
                                      (5, 511, 16), (4, 512, 64)])
def test_plain_topk(t, e, topk, scoring, dtype):
    v = np.random.default_rng(t + e).standard_normal((t, e)) * 1.5
    _check(v, dtype, scoring, topk)
    _check(v, dtype, scoring, topk, renorm=True, scale=2.5, pad=3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups,kept,topk", [(256, 8, 4, 8), (160, 8, 3, 6), (64, 64, 5, 5), (128, 2, 1, 16), (30, 3, 2, 7),
                                                (512, 16, 5, 12), (36, 6, 6, 4), (8, 4, 1, 2)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_and_bias(e, groups, kept, topk, group_top, scoring, dtype):
    rng = np.random.default_rng(e + groups)
    v = rng.standard_normal((41, e)) * 1.5
    kw = dict(groups=groups, topk_groups=kept, group_top=group_top)
    _check(v, dtype, scoring, topk, **kw)
    _check(v, dtype, scoring, topk, bias=rng.standard_normal(e) * 0.05, renorm=True, scale=16.0, **kw)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_equal_values_go_to_the_lowest_index(scoring, bias):
    # few distinct logits: whole rows of ties, among groups too
    rng = np.random.default_rng(1)
    v = rng.integers(0, 3, size=(60, 96)).astype(np.float32)
    b = np.zeros(96, np.float32) if bias else None
    _check(v, "f32", scoring, 10, bias=b)
    _check(v, "f32", scoring, 10, bias=b, groups=8, topk_groups=3, group_top=1)
    _check(v, "f32", scoring, 10, bias=b, groups=8, topk_groups=3, group_top=2)
    _check(np.zeros((4, 96)), "bf16", scoring, 10, bias=b, groups=8, topk_groups=3, group_top=2, renorm=True)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_masked_and_extreme_logits(scoring, dtype):
    rng = np.random.default_rng(2)
    v = (rng.standard_normal((16, 40)) * 2).astype(np.float32)
    low = float(np.finfo(np.float32).min) if dtype != "f16" else -65504.0
    v[0] = -np.inf                         # nothing left
    v[1] = np.nan
    v[2, 1:] = -np.inf                     # one expert
    v[3] = low                             # the type's lowest value is a value
    v[4, ::2] = low
    v[5, ::3] = np.nan
    v[6, 7] = np.inf
    v[7, [3, 9]] = np.inf
    v[8, :36] = -np.inf                    # four experts, of one or two groups
    v[9] = 80.0                            # sigmoids of equal large logits
    v[10] = np.linspace(20, 60, 40)        # saturated sigmoids: the logits still order them
    v[11] = np.linspace(-100, -60, 40)
    v[12, 5] = -np.inf
    v[13] = np.where(np.arange(40) % 2, np.inf, -np.inf)
    bias = (rng.standard_normal(40) * 0.1).astype(np.float32)
    for kw in (dict(), dict(renorm=True), dict(groups=5, topk_groups=2), dict(groups=10, topk_groups=3, group_top=1)):
        _check(v, dtype, scoring, 6, **kw)
    for kw in (dict(), dict(renorm=True), dict(groups=5, topk_groups=2, group_top=2)):
        _check(v[:9], dtype, scoring, 6, bias=bias, **kw)
    bias[[1, 5]] = [-np.inf, np.nan]
    bias[8] = np.inf
    _check(v[:9], dtype, scoring, 6, bias=bias, renorm=True)


def test_scores_closer_than_float32_resolves():
    # the j-th logit is 1 + j * 2^-23 (one float32 step): sigmoids and softmaxes of neighbours differ by less
    # than a float32 step of theirs, and a bias of the scores' order of magnitude is added to each
    steps = np.random.default_rng(0).permutation(128)
    v = (np.float32(1) + steps.astype(np.float32) * np.float32(2.0 ** -23))[None].repeat(3, 0)
    for scoring in ("sigmoid", "softmax"):
        _check(v, "f32", scoring, 8)
        _check(v, "f32", scoring, 8, bias=np.full(128, 0.75, np.float32))
        _check(v, "f32", scoring, 8, bias=np.full(128, 0.75, np.float32), groups=8, topk_groups=4, group_top=2)
        _check(v, "f32", scoring, 8, groups=8, topk_groups=4, group_top=2)


@pytest.mark.parametrize("t", [4096, 8192, 10007])
def test_large_batches(t):
    rng = np.random.default_rng(t)
    v = (rng.standard_normal((t, 256)) * 1.5).astype(np.float32)
    _check(v, "f32", "sigmoid", 8, bias=rng.standard_normal(256) * 0.05, groups=8, topk_groups=4, group_top=2, renorm=True,
           scale=2.5)
    _check(v[:, :128], "bf16", "softmax", 8, renorm=True)


def _odd_rows(e, dtype, seed):
    """Rows that masks, ties and extremes make awkward, among ordinary ones."""
    rng = np.random.default_rng(seed)
    v = (rng.standard_normal((550, e)) * 1.5).astype(np.float32)
    v[3::50] = rng.integers(0, 3, size=v[3::50].shape)                 # ties, among groups too
    v[4::50] = np.where(rng.random(v[4::50].shape) < 0.5, 0.0, -0.0)   # zeros of both signs are equal
    v[5::50] = -np.inf
    v[6::50] = np.nan
    v[7::50, : e - 2] = -np.inf                                        # two experts left
    v[8::50, ::2] = np.finfo(np.float32).min if dtype != "f16" else -65504
    v[9::50, ::3] = np.nan
    v[10::50, 1::4] = np.inf
    v[11::50] = np.linspace(-8, 8, e)[rng.permutation(e)]
    v[12::50] = 1 + rng.permutation(e) * np.float32(2.0 ** -23)        # scores closer than float32 resolves
    return v


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,topk", [(8, 2), (60, 4), (64, 6), (65, 16), (128, 8), (200, 8), (256, 8), (320, 8), (33, 17)])
def test_odd_rows_of_large_batches(e, topk, scoring, dtype):
    v = _odd_rows(e, dtype, e)
    bias = np.random.default_rng(e).standard_normal(e) * 0.05
    for t in (550, 4101):                       # a wave per token, and four tokens per wave
        _check(v, dtype, scoring, topk, renorm=True, pad=3, total=t)
        _check(v, dtype, scoring, topk, total=t)
        _check(v, dtype, scoring, topk, bias=bias, scale=2.5, total=t)
        odd = bias.copy()
        odd[[0, e - 1]] = [-np.inf, np.inf]
        odd[1] = np.nan
        _check(v, dtype, scoring, topk, bias=odd, renorm=True, total=t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups,kept,topk", [(256, 8, 4, 8), (160, 8, 3, 6), (128, 16, 5, 7), (128, 2, 1, 16),
                                                (30, 3, 2, 7), (36, 6, 6, 4), (8, 4, 1, 2), (512, 32, 4, 8), (480, 5, 2, 8)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_odd_rows_of_large_batches_with_groups(e, groups, kept, topk, group_top, scoring, dtype):
    v = _odd_rows(e, dtype, e + groups)
    kw = dict(groups=groups, topk_groups=kept, group_top=group_top)
    bias = np.random.default_rng(e).standard_normal(e) * 0.05
    for t in (550, 4102):
        _check(v, dtype, scoring, topk, renorm=scoring == "sigmoid", total=t, **kw)
        _check(v, dtype, scoring, topk, bias=bias, renorm=True, scale=2.5, total=t, **kw)
        _check(v, dtype, scoring, topk, bias=bias, pad=3, total=t, **kw)          # rows at odd addresses


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_more_tokens_than_one_launch_takes(scoring):
    t = (1 << 24) + 37
    v = np.random.default_rng(0).standard_normal((1009, 4))
    _check(v, "bf16", scoring, 1, total=t)
    _check(v, "f32", scoring, 2, bias=np.array([0.1, 0, -0.1, 0.3]), renorm=True, total=t)


def test_logits_past_2_31_elements():
    t, e = 8_400_000, 256                                                 # 2.15e9 logits
    v = np.random.default_rng(5).standard_normal((1000, e)).astype(np.float32)
    bits = synth.f32_to_bf16_bits(v)
    dev = torch.from_numpy(bits.view(np.int16)).cuda().repeat(t // 1000, 1)
    d = qg.make_route_desc(qg.R_SOFTMAX, e, 8, renormalize=True)
    ids = torch.empty((t, 8), dtype=torch.int32, device="cuda")
    w = torch.empty((t, 8), device="cuda")
    qg.moe_route(d, dev, qg.L_BF16, t, ids, w)
    torch.cuda.synchronize()
    rid, rw = RT.route(F.decode_bf16(bits), "softmax", 8, renorm=True)
    for first in (0, 8_388_000, t - 1000):                                # 8388608 * e = 2^31
        assert np.array_equal(ids[first:first + 1000].cpu().numpy(), rid)
        assert np.all(np.abs(w[first:first + 1000].cpu().numpy() - rw) <= 2.0 ** -24 * (1 + 2.0 ** -16) * rw + 2.0 ** -149)


@pytest.mark.parametrize("t", [70, 4100])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_addresses_of_single_elements(dtype, t):
    # logits and bias that start one element past a 16-byte boundary, rows of 64 without a gap
    rng = np.random.default_rng(t)
    v = rng.standard_normal((t, 64)).astype(np.float32)
    dev, held = _logits(v, dtype)
    shifted = torch.empty(t * 64 + 1, dtype=dev.dtype, device="cuda")
    shifted[1:] = dev.view(-1)
    b = torch.empty(65, device="cuda")
    bias = (rng.standard_normal(64) * 0.05).astype(np.float32)
    b[1:] = torch.from_numpy(bias).cuda()
    d = qg.make_route_desc(qg.R_SIGMOID, 64, 6, 8, 3, 2, True)
    ids = torch.empty((t, 6), dtype=torch.int32, device="cuda")
    w = torch.empty((t, 6), device="cuda")
    for lg, bs in ((shifted[1:], b[1:]), (dev, b[1:]), (shifted[1:], b[1:].clone())):
        qg.moe_route(d, lg, TYPE[dtype], t, ids, w, bs)
        torch.cuda.synchronize()
        rid, rw = RT.route(held, "sigmoid", 6, bias=bias, groups=8, topk_groups=3, group_top=2, renorm=True)
        assert np.array_equal(ids.cpu().numpy(), rid)
        assert np.all(np.abs(w.cpu().numpy() - rw) <= 2.0 ** -24 * (1 + 2.0 ** -16) * rw + 2.0 ** -149)


def test_another_stream_and_no_tokens():
    v = np.random.default_rng(0).standard_normal((77, 64))
    s = torch.cuda.Stream()
    _check(v, "f32", "softmax", 6, stream=s)
    d = qg.make_route_desc(qg.R_SOFTMAX, 64, 6)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    qg.moe_route(d, torch.empty((0, 64), device="cuda"), qg.L_F32, 0, e, e.float())
