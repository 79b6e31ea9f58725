"""GPU runs of calls of qg_attention that a server makes: tables cut from wider ones, malformed offsets, mixed batches.

Bars and cases are those of test_gpu_attention.
"""
import numpy as np
import pytest
import torch

import quantized_gemm_amd as qg
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qg.lib()
    yield


@pytest.mark.parametrize("counts", [None, [20, 90, 31]])
def test_a_table_cut_from_a_wider_one(counts):
    c = Case([100, 700, 31], 8, 2, 128, 16, counts=counts)
    table = c.table
    wide = torch.full((5, table.shape[1] + 9), 1 << 30, dtype=torch.int32, device="cuda")   # pages outside the cache
    c.table = wide[1:4, 3:3 + table.shape[1]]
    c.table.copy_(table)
    c.run().check()
    c.table = torch.cat([table, torch.full_like(table, -1)], 0)[:3]
    c.run().check()


@pytest.mark.parametrize("many", [False, True])
def test_malformed_offsets_take_rows_that_there_are(many):
    # offsets outside the rows, descending, and far enough apart that their difference leaves 32 bits: the rows between them
    # that exist, max_q at most (below zero is the first row), and no others
    n = 90 if many else 3
    c = Case([100, 700, 31, 9], 8, 2, 128, 16, counts=[n, 2, 0, 0])
    low, high = -2 ** 31, 2 ** 31 - 1
    used = c.used
    for offsets in ([high, low, 0, 0, 0], [used + 3, 1 << 24, high, high, high], [low, -7, low, -1, 0], [used, high, low, high, low]):
        c.offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
        c.out.fill_(float("nan"))
        c.run()
        torch.cuda.synchronize()
        taken = {row for b, e in zip(offsets, offsets[1:]) for row in list(range(max(0, b), min(e, used)))[:c.max_q]}
        written = [row for row in range(used) if not torch.isnan(c.out[row]).any()]
        assert written == sorted(taken), offsets
        assert torch.isnan(c.out).any(1).sum() == torch.isnan(c.out).all(1).sum()
    c.offsets.copy_(torch.tensor([0, n, used, high, low], dtype=torch.int32))          # the first two as they should be
    c.run().check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("counts,lens", [([1, 1, 1], [40, 700, 3000]), ([12, 60, 200], [40, 90, 200]), ([3, 150, 2], [3000, 900, 33])])
def test_weights_add_up_to_one(dtype, dim, counts, lens):
    # values of one everywhere: the outputs are one, whatever the weights; scores up to ten powers of two apart, one token's
    # weight above the others'.  Sums of float32 are off by 2^-13 at most, a quarter of the smallest step beside one and less.
    c = Case(lens, 8, 2, dim, 16, counts=counts, dtype=dtype, sigma=2.0)
    rng = np.random.default_rng(5)
    width = 2 * dim
    for i, n in enumerate(lens):
        k = torch.from_numpy(rng.standard_normal((n, width)).astype(np.float32) * 2).to(c.q.dtype).cuda()
        t = np.arange(n)
        slots = c.table[i].cpu().numpy()[t // 16] * 16 + t % 16
        qg.kv_append(c.desc, k, torch.ones_like(k), torch.from_numpy(slots.astype(np.int32)).cuda(), n, c.cache)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out, torch.ones_like(c.out))
