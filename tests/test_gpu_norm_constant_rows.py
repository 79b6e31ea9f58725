"""Layer norms of rows whose values are all alike: v - mean(v) is zero whatever the value, so that the bias is left.

Nothing is rounded on the way, so the outputs are compared exactly.
"""
import pytest
import torch

import quantized_gemm_amd as qg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
O = {"bf16": qg.O_BF16, "f16": qg.O_F16}
L = {"bf16": qg.L_BF16, "f16": qg.L_F16, "f32": qg.L_F32}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qg.lib()
    yield


def _run(k, values, dtype, res, code=0, post=False):
    """Rows of one value each, as the residual or (post) as a block's output with its own norm; the normed rows."""
    n = len(values)
    rows = torch.tensor(values, dtype=torch.float64, device="cuda")[:, None].expand(n, k).to(DT[dtype if post else res]).contiguous()
    w = torch.linspace(-2, 2, k, device="cuda").to(DT[dtype])
    b = None if post else torch.linspace(-1, 3, k, device="cuda").to(DT[dtype])
    out = torch.full((n, k), float("nan"), dtype=DT[dtype], device="cuda")
    codes = torch.full((n, k), 0xA5, dtype=torch.uint8, device="cuda") if code else None
    scale = torch.full((n,), float("nan"), device="cuda") if code else None
    d = qg.make_norm_desc(0 if post else qg.N_LAYER, O[dtype], k, 1e-6, post_norm=qg.N_LAYER if post else 0,
                          res_type=L[dtype if post else res], code_type=code)
    if post:
        qg.norm_rows(d, n, rows, None, out, post_weight=w)
    else:
        qg.norm_rows(d, n, None, rows, None, out, codes, scale, weight=w, bias=b if not code else None)
    torch.cuda.synchronize()
    return out, (torch.zeros(k, device="cuda", dtype=DT[dtype]) if b is None or code else b), codes, scale


@pytest.mark.parametrize("k", [8, 128, 512, 1024, 2048, 4096, 8192, 16384, 32768])
@pytest.mark.parametrize("post", [False, True])
def test_constants_beyond_the_range_of_squares(k, post):
    # powers of two, whose sums and means are exact, so far up that eps over their square leaves float32
    values = [2.0 ** 57, 2.0 ** 64, -2.0 ** 100, 2.0 ** 127]
    for dtype, res in (("bf16", "bf16"), ("bf16", "f32")):
        out, want, _, _ = _run(k, values, dtype, res, post=post)
        assert torch.equal(out.float(), want.float().expand_as(out))


KS = [8, 40, 128, 136, 512, 1000, 1416, 4096, 5120, 8192, 8200, 20000, 32768]
VALUES = [1.0, -600.0, 1e-3, 12345.0, 0.1, 3e4]


@pytest.mark.parametrize("k", KS)
@pytest.mark.parametrize("dtype,res", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
def test_any_constant(k, dtype, res):
    values = VALUES + ([1e30, -3e38, 1e-30] if res != "f16" else [])
    out, want, _, _ = _run(k, values, dtype, res)
    assert torch.equal(out.float(), want.float().expand_as(out))
    out, _, _, _ = _run(k, VALUES, dtype, res, post=True)
    assert not out.any()
    for code in (qg.A_FP8_E4M3, qg.A_INT8):
        _, _, codes, scale = _run(k, values, dtype, res, code)
        assert not (codes & (0x7F if code == qg.A_FP8_E4M3 else 0xFF)).any() and (scale == 1).all()   # (e4m3 has a zero below 0)


@pytest.mark.parametrize("k", [40, 1416, 5120, 20000])
def test_rows_of_one_value_but_one(k):
    # one value beside the others, its place first, last or between: the mean is the others', but for its share
    for at in (0, k // 2, k - 1):
        x = torch.full((3, k), 50.0, device="cuda")
        x[:, at] += torch.tensor([1.0, 1000.0, -7.0], device="cuda")
        out = torch.full((3, k), float("nan"), dtype=torch.bfloat16, device="cuda")
        qg.norm_rows(qg.make_norm_desc(qg.N_LAYER, qg.O_BF16, k, 1e-6, res_type=qg.L_F32), 3, None, x, None, out)
        d = x.double() - x.double().mean(1, keepdim=True)
        z = d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-6)
        # of z, half a step of bf16 and a few roundings; of the mean, 64 roundings of 2^-24 of its terms, over the deviation
        noise = 2.0 ** -18 * x.double().abs().mean(1, keepdim=True) / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-6)
        assert ((out.double() - z).abs() <= (2.0 ** -8 + 2.0 ** -16) * z.abs() + noise).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("k", [40, 520, 1416, 9000])
def test_constants_beside_values_that_are_not_finite(value, k):
    for at in (0, k - 1):
        x = torch.full((3, k), 5.0, dtype=torch.bfloat16, device="cuda")
        x[1, at] = value
        out = torch.zeros((3, k), dtype=torch.bfloat16, device="cuda")
        qg.norm_rows(qg.make_norm_desc(qg.N_LAYER, qg.O_BF16, k, 1e-6), 3, None, x, None, out)
        assert torch.isnan(out[1]).all() and not out[[0, 2]].any()
