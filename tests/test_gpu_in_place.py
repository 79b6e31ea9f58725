"""Outputs in an input's place give the same bits as beside it, for rows that a workgroup takes in turn too."""
import pytest
import torch

import quantized_gemm_amd as qg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qg.lib()
    yield


def _wide(rows, k, pad, dtype):
    return torch.randn((rows, k + pad), device="cuda").to(dtype)


@pytest.mark.parametrize("rows,k", [(5, 64), (3100, 1416), (2100, 4096), (700, 8192), (40, 16384)])
@pytest.mark.parametrize("pad", [0, 24])
def test_norm(rows, k, pad):
    torch.manual_seed(rows)
    y, r, r32 = _wide(rows, k, pad, torch.bfloat16), _wide(rows, k, pad, torch.bfloat16), _wide(rows, k, pad, torch.float32)
    w = torch.randn(k, device="cuda").to(torch.bfloat16)
    one = dict(y_stride=k + pad, res_stride=k + pad, out_stride=k + pad)

    def both(res, res_type, y, where):
        d = qg.make_norm_desc(qg.N_RMS, qg.O_BF16, k, 1e-6, res_type=res_type, **one)
        beside = torch.full_like(res, float("nan")), torch.full_like(r, float("nan"))
        qg.norm_rows(d, rows, y, res, beside[0] if "res" in where or y is not None else None, beside[1], weight=w)
        y2, res2 = None if y is None else y.clone(), res.clone()
        inside = res2 if "res" in where else None, {"y": y2, "residual": res2, "": torch.empty_like(r)}[where["out"]]
        qg.norm_rows(d, rows, y2, res2, inside[0], inside[1], weight=w)
        torch.cuda.synchronize()
        if inside[0] is not None:
            assert torch.equal(inside[0][:, :k], beside[0][:, :k]) and torch.equal(inside[0][:, k:], res[:, k:])
        assert torch.equal(inside[1][:, :k], beside[1][:, :k])

    both(r, qg.L_BF16, y, dict(res=1, out="y"))
    both(r32, qg.L_F32, y, dict(res=1, out="y"))
    both(r, qg.L_BF16, y, dict(out="y"))
    both(r, qg.L_BF16, None, dict(out="residual"))


@pytest.mark.parametrize("tokens,n,block", [(50, 136, 16), (300, 1864, 64), (700, 4096, 128), (3000, 5632, 128)])
@pytest.mark.parametrize("rank", [16, 64, 128])
def test_adapters(tokens, n, block, rank):
    torch.manual_seed(tokens)
    k, e, pad = 264, 3, 8
    x, base = _wide(tokens, k, 0, torch.bfloat16), _wide(tokens, n, pad, torch.bfloat16)
    a, b = torch.randn((e, 1, rank, k), device="cuda").to(torch.bfloat16), torch.randn((e, n, rank), device="cuda").to(torch.bfloat16)
    ids = torch.randint(-1, e, (tokens,), dtype=torch.int32, device="cuda")
    rows, blocks = qg.moe_capacity(tokens, 1, e, block)
    at = [torch.empty(z, dtype=torch.int32, device="cuda") for z in (rows, blocks, 1)]
    qg.moe_align(ids, tokens, 1, e, block, *at)
    d = qg.make_lora_desc(qg.O_BF16, e, rank, k, [n], base_stride=n + pad, y_stride=n + pad)
    ws = torch.empty(qg.lora_workspace_bytes(d, tokens, block), dtype=torch.uint8, device="cuda")
    beside, inside = base.clone(), base.clone()
    qg.lora(d, x, a, b, *at, tokens, block, base, beside, ws)
    qg.lora(d, x, a, b, *at, tokens, block, inside, inside, ws)
    torch.cuda.synchronize()
    assert torch.equal(beside, inside) and torch.equal(inside[:, n:], base[:, n:])
    assert torch.equal(inside[ids < 0], base[ids < 0]) and not torch.equal(inside[ids >= 0], base[ids >= 0])


def test_one_row_has_no_stride():
    torch.manual_seed(1)
    k = 4096
    y, r = (torch.randn((1, k), device="cuda").to(torch.bfloat16) for _ in "yr")
    w = torch.randn(k, device="cuda").to(torch.bfloat16)
    beside, inside = torch.empty_like(y), y.clone()
    for out, src in ((beside, y), (inside, inside)):
        qg.norm_rows(qg.make_norm_desc(qg.N_RMS, qg.O_BF16, k, 1e-6, y_stride=8 * k), 1, src, r, None, out, weight=w)
    a, b = torch.randn((1, 1, 16, k), device="cuda").to(torch.bfloat16), torch.randn((1, k, 16), device="cuda").to(torch.bfloat16)
    rows, blocks = qg.moe_capacity(1, 1, 1, 16)
    at = [torch.empty(z, dtype=torch.int32, device="cuda") for z in (rows, blocks, 1)]
    qg.moe_align(torch.zeros(1, dtype=torch.int32, device="cuda"), 1, 1, 1, 16, *at)
    d = qg.make_lora_desc(qg.O_BF16, 1, 16, k, [k], base_stride=8 * k)
    ws = torch.empty(qg.lora_workspace_bytes(d, 1, 16), dtype=torch.uint8, device="cuda")
    far, near = torch.empty_like(y), r.clone()
    qg.lora(d, y, a, b, *at, 1, 16, r, far, ws)
    qg.lora(d, y, a, b, *at, 1, 16, near, near, ws)
    torch.cuda.synchronize()
    assert torch.equal(beside, inside) and torch.equal(far, near) and not torch.equal(near, r)
