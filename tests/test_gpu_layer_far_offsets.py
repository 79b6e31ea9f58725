"""Adapters and attention whose rows lie beyond 2^31 elements, and the widest groups of query heads."""
import numpy as np
import pytest
import torch

import quantized_gemm_amd as qg
from oracle import layer_ops as LO
from test_gpu_attention import Case, _rows
from test_gpu_attention_paths import check, inside

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qg.lib()
    yield


def _d(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("block", [16, 64, 128])
def test_adapters(block):
    tokens, k, n, rank, e = 300001, 8192, 8192, 16, 3
    gen = torch.Generator(device="cuda").manual_seed(block)
    x, y = (torch.empty((tokens, k), dtype=torch.bfloat16, device="cuda").normal_(generator=gen) for _ in "xy")
    a = (torch.randn((e, 1, rank, k), generator=gen, device="cuda") / k ** 0.5).to(torch.bfloat16)
    b = (torch.randn((e, n, rank), generator=gen, device="cuda") / rank ** 0.5).to(torch.bfloat16)
    ids = torch.randint(-1, e, (tokens,), generator=gen, device="cuda").to(torch.int32)
    assert x.numel() > 1 << 31
    rows, blocks = qg.moe_capacity(tokens, 1, e, block)
    at = [torch.empty(z, dtype=torch.int32, device="cuda") for z in (rows, blocks, 1)]
    qg.moe_align(ids, tokens, 1, e, block, *at)
    d = qg.make_lora_desc(qg.O_BF16, e, rank, k, [n])
    ws = torch.empty(qg.lora_workspace_bytes(d, tokens, block), dtype=torch.uint8, device="cuda")
    some = torch.tensor([0, 1, 2, 262143, 262144, 262145, tokens - 70, tokens - 2, tokens - 1], device="cuda")
    base = _d(y[some])
    qg.lora(d, x, a, b, *at, tokens, block, y, y, ws)
    torch.cuda.synchronize()
    ref, mag = LO.lora(_d(x[some]), _d(a), _d(b), ids[some].cpu().numpy(), [rank] * e, np.ones(e), base, [n])
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -16 + (k / 8 + 64 + 512) * 2.0 ** -24) * mag
    assert (np.abs(_d(y[some]) - ref) <= tol).all()


def test_attention_rows():
    # as many sequences as a call takes, all on the same pages, rows of 32768 values and more
    batch, heads, kv, dim, page, pad = 65535, 128, 8, 256, 16, 512
    d = qg.make_kv_desc(qg.O_BF16, kv, dim, page, 3)
    cache = torch.full((qg.kv_cache_bytes(d),), 0xFF, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(3)
    k, v = _rows(rng, 48, kv * dim, "bf16"), _rows(rng, 48, kv * dim, "bf16")
    qg.kv_append(d, k, v, torch.arange(48, dtype=torch.int32, device="cuda"), 48, cache)
    q = torch.empty((batch, heads * dim + pad), dtype=torch.bfloat16, device="cuda").normal_()
    assert q.numel() > 1 << 31
    out = torch.full_like(q, float("nan"))
    lens = torch.arange(batch, dtype=torch.int32, device="cuda") % 49
    table = torch.arange(3, dtype=torch.int32, device="cuda").repeat(batch, 1)
    assert qg.attention_workspace_bytes(d, heads, batch, 1, batch, 48) == 0
    qg.attention(d, q, heads, cache, table, lens, batch, 48, dim ** -0.5, out, q_stride=heads * dim + pad, out_stride=heads * dim + pad)
    torch.cuda.synchronize()
    vals = [LO.mxfp4_values(_d(x)).reshape(48, kv, dim) for x in (k, v)]
    for b in (0, 1, 48, 32767, 65000, 65533, 65534):
        n = b % 49
        got = _d(out[b])
        assert np.isnan(got[heads * dim:]).all()
        r = LO.attention_terms(_d(q[b, :heads * dim]).reshape(1, heads, dim), [vals[0][:n]], [vals[1][:n]], [n], [1], dim ** -0.5)
        inside(got[:heads * dim].reshape(1, heads, dim), r, dim, "bf16")
    assert not torch.isnan(out[:, 0]).any()


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 256)])
@pytest.mark.parametrize("counts", [None, [3, 40, 1]])
def test_256_query_heads_of_a_key_head(dtype, dim, counts):
    check(Case([70, 600, 3], 256, 1, dim, 32, counts=counts, dtype=dtype).run())
    check(Case([70, 40, 3], 510, 2, dim, 128, counts=counts, dtype=dtype).run())


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_pages_of_128(dim):
    check(Case([70, 600, 129, 128], 6, 3, dim, 128, counts=[3, 140, 1, 5]).run())
    check(Case([70, 600, 129, 128], 6, 3, dim, 128, dtype="f16").run())
