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
