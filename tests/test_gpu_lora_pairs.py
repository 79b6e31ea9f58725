"""Adapters where a wave has two pairs of column tiles (tiles of tokens x n / 256 >= 1024): the second pair's operands are
loaded during the first one's products, in a ring of LDS.  Bars are those of test_gpu_lora; the reference is by adapter.
"""
import numpy as np
import pytest
import torch

import quantized_gemm_amd as qg
import test_gpu_lora as TL
from test_gpu_lora import Case, _ids

pytestmark = pytest.mark.gpu
PLAIN = TL.LO.lora


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qg.lib()
    yield


def by_adapter(x, a, b, ids, ranks, scales, base, slice_ends):
    """oracle.layer_ops.lora with one product per adapter and slice: the same sums, for many tokens."""
    out = base.astype(np.float64).copy()
    mag = np.abs(out)
    for e in range(a.shape[0]):
        at = np.flatnonzero(ids == e)
        r = min(max(int(ranks[e]), 0), a.shape[2])
        begin = 0
        for s, end in enumerate(slice_ends):
            out[at, begin:end] += scales[e] * (x[at] @ a[e, s, :r].T) @ b[e, begin:end, :r].T
            mag[at, begin:end] += abs(scales[e]) * (np.abs(x[at]) @ np.abs(a[e, s, :r]).T) @ np.abs(b[e, begin:end, :r]).T
            begin = end
    return out, mag


@pytest.fixture(autouse=True)
def reference(monkeypatch):
    monkeypatch.setattr(TL.LO, "lora", by_adapter)


def test_reference():
    rng = np.random.default_rng(0)
    x, a, b = rng.standard_normal((9, 8)), rng.standard_normal((2, 2, 4, 8)), rng.standard_normal((2, 12, 4))
    args = (x, a, b, np.array([0, 1, -1, 1, 0, 5, 1, 1, 0]), [3, 4], [0.5, -2.0], rng.standard_normal((9, 12)), [5, 12])
    for got, want in zip(by_adapter(*args), PLAIN(*args)):
        assert np.allclose(got, want, rtol=1e-12, atol=1e-12)


def pairs(c):
    """Column pairs of a wave: two from 1024 tiles of tokens (16, or 64 of the map's block) x n / 256 on."""
    _, blocks = qg.moe_capacity(c.tokens, 1, c.desc.num_adapters, c.block)
    return 2 if blocks * max(1, c.block // 64) * (c.n // 256) >= 1024 else 1


RANKS = [16, 32, 40, 64, 128, 136, 256]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rank", RANKS)
def test_blocks_of_16(rank, dtype):
    # columns that end in the first pair, in the second, and between a wave's two
    for ends in ([8192], [4128, 8232], [96, 4448, 8200]):
        c = Case(400, 72, ends, rank, _ids(400, 12), dtype, adapters=12, block=16, ranks=[rank, rank - 3, 5, 0] * 3, pad=8)
        assert pairs(c) == 2
        c.run().check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rank", RANKS)
@pytest.mark.parametrize("block", [64, 128])
def test_blocks_of_many(rank, block, dtype):
    for tokens, ends in ((2000, [8192]), (2003, [96, 4448, 8200])):
        c = Case(tokens, 72, ends, rank, _ids(tokens, 3), dtype, adapters=3, block=block, ranks=[rank, rank - 3, 5], pad=8)
        assert pairs(c) == 2
        c.run().check()


@pytest.mark.parametrize("rank", [16, 64, 128, 256])
@pytest.mark.parametrize("block", [16, 128])
def test_in_place(rank, block):
    tokens = 400 if block == 16 else 2003
    c = Case(tokens, 136, [64, 8200], rank, _ids(tokens, 12), adapters=12, block=block, inplace=True)
    assert pairs(c) == 2
    c.run().check()


@pytest.mark.parametrize("rank", [16, 128])
def test_parts_of_k_for_many_tokens(rank):
    # K in as many parts as there are, steps that are not a whole number of parts, and tiles of tokens beside the block's end
    for k in (1000, 4104):
        c = Case(1100, k, [4096, 8192], rank, _ids(1100, 2), adapters=2, block=128, ranks=[rank, rank - 7])
        c.run().check()
