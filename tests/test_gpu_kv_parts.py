"""The cache's rows beyond what one launch takes (2^31 words of eight values)."""
import numpy as np
import pytest
import torch

import quantized_gemm_amd as qg
from oracle import layer_ops as LO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qg.lib()
    yield


def test_append_and_read_in_two_launches():
    # 1024 heads of 256: 32768 tokens are a launch.  All but a few tokens are skipped: those at both sides of its end are not.
    heads, dim, page = 1024, 256, 16
    width, per = heads * dim, (1 << 31) // (2 * heads * dim // 8)
    tokens = per + 5
    d = qg.make_kv_desc(qg.O_BF16, heads, dim, page, 2)
    cache = torch.full((qg.kv_cache_bytes(d),), 0xFF, dtype=torch.uint8, device="cuda")
    at = [0, 7, per - 1, per, per + 1, tokens - 1]
    slots = torch.full((tokens,), -1, dtype=torch.int32, device="cuda")
    slots[torch.tensor(at, device="cuda")] = torch.tensor([31, 2, 0, 17, 30, 1], dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(1)
    k = torch.zeros((tokens, width), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros((tokens, width), dtype=torch.bfloat16, device="cuda")
    for x in (k, v):
        for t in at:
            x[t] = torch.from_numpy(rng.standard_normal(width).astype(np.float32)).cuda()
    qg.kv_append(d, k, v, slots, tokens, cache)
    want = [LO.mxfp4_values(x[torch.tensor(at, device="cuda")].double().cpu().numpy()) for x in (k, v)]
    for x in (k, v):
        x.fill_(float("nan"))
    qg.kv_read(d, cache, slots, tokens, k, v)
    torch.cuda.synchronize()
    for x, w in zip((k, v), want):
        assert np.array_equal(x[torch.tensor(at, device="cuda")].double().cpu().numpy(), w)
        x[torch.tensor(at, device="cuda")] = 0
        for i in range(0, tokens, 4096):
            assert not x[i:i + 4096].any(), i                     # zeros where there is no slot
