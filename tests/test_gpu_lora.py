"""GPU parity of low-rank adapters beside a shared product (qg_lora).

Bars, from the arithmetic: t is a float32 sum of k products (exact in float32 for 16-bit factors), off by at most k / 8 + 64
roundings of 2^-24 of its terms' magnitudes (an MFMA adds 8 products of a lane's chunk and more at a time); it
enters the second product as two 16-bit numbers that are off by 2^-16 (bf16) or 2^-22 (f16) of it, or of the largest t
of the token (f16 below its normal range); sums of rank products, two more roundings, and half a step of the output
(2^-8, 2^-11 of the value, 2^-25 below f16's normal range).
"""
import numpy as np
import pytest
import torch

import quantized_gemm_amd as qg
from oracle import layer_ops as LO

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SPLIT = {"bf16": 2.0 ** -16, "f16": 2.0 ** -20}
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
O = {"bf16": qg.O_BF16, "f16": qg.O_F16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qg.lib()
    yield


def _d(t):
    return t.double().cpu().numpy()


class Case:
    def __init__(self, tokens, k, ends, rank, ids, dtype="bf16", ranks=None, scales=None, adapters=None, block=None, pad=0, seed=0,
                 inplace=False):
        rng = np.random.default_rng(seed + tokens + 7 * k + rank)
        n, s = ends[-1], len(ends)
        e = adapters or int(max(ids)) + 1
        mk = lambda *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float32))  # noqa: E731
        self.tokens, self.n, self.dtype, self.ends, self.ids = tokens, n, dtype, ends, np.asarray(ids, np.int32)
        self.x = mk(tokens, k + pad).to(DT[dtype]).cuda()
        self.a = (mk(e, s, rank, k) / k ** 0.5).to(DT[dtype]).cuda()
        self.b = (mk(e, n, rank) / rank ** 0.5).to(DT[dtype]).cuda()
        self.base = mk(tokens, n + pad).to(DT[dtype]).cuda()
        self.ranks = None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device="cuda")
        self.scales = None if scales is None else torch.tensor(scales, dtype=torch.float32, device="cuda")
        self.rank_of = [rank] * e if ranks is None else ranks
        self.scale_of = np.ones(e) if scales is None else np.float32(scales).astype(np.float64)
        self.k = k
        for i, r in enumerate(self.rank_of):              # what lies behind an adapter's rank is not read
            self.a[i, :, max(0, r):] = float("nan")
            self.b[i, :, max(0, r):] = float("nan")
        self.desc = qg.make_lora_desc(O[dtype], e, rank, k, ends, x_stride=k + pad, base_stride=n + pad, y_stride=n + pad)
        self.block = block or qg.lora_block_m(tokens, e)
        rows, blocks = qg.moe_capacity(tokens, 1, e, self.block)
        self.map = [torch.full((z,), -7, dtype=torch.int32, device="cuda") for z in (rows, blocks, 1)]
        self.dev_ids = torch.from_numpy(self.ids).cuda()
        qg.moe_align(self.dev_ids, tokens, 1, e, self.block, *self.map)
        self.ws = torch.full((qg.lora_workspace_bytes(self.desc, tokens, self.block),), 0xA5, dtype=torch.uint8, device="cuda")
        self.want = LO.lora(_d(self.x)[:, :k], _d(self.a), _d(self.b), self.ids, self.rank_of, self.scale_of,
                            _d(self.base)[:, :n], ends)
        self.y = self.base if inplace else torch.full_like(self.base, float("nan"))
        self.inplace = inplace

    def run(self, stream=None):
        qg.lora(self.desc, self.x, self.a, self.b, *self.map, self.tokens, self.block, self.base, self.y, self.ws,
                ranks=self.ranks, scales=self.scales, stream=stream)
        return self

    def check(self):
        torch.cuda.synchronize()
        got = _d(self.y)
        ref, mag = self.want
        has = (self.ids >= 0) & (self.ids < self.desc.num_adapters)
        tol = U[self.dtype] * np.abs(ref) + (SPLIT[self.dtype] + (self.k / 8 + 64 + 512) * 2.0 ** -24) * mag + 2.0 ** -25
        # (f16: a token's smaller t may be off by 2^-25 of its largest)
        assert (np.abs(got[has][:, :self.n] - ref[has]) <= tol[has]).all()
        if not self.inplace:
            assert np.isnan(got[~has]).all() and np.isnan(got[:, self.n:]).all()      # left as they were
        else:
            assert np.array_equal(got[~has][:, :self.n], ref[~has])
        return self


def _ids(tokens, e, seed=0, none=0.2):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, e, tokens)
    return np.where(rng.random(tokens) < none, rng.choice([-1, e, 1000], tokens), ids)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rank", [8, 16, 24, 32, 48, 64, 128, 256])
@pytest.mark.parametrize("block", [16, 64, 128])
def test_ranks(dtype, rank, block):
    Case(37, 200, [104], rank, _ids(37, 3), dtype, adapters=3, block=block).run().check()
    Case(70, 1416, [64, 160, 296], rank, _ids(70, 2, none=0.0), dtype, adapters=2, block=block, scales=[0.5, -2.0]).run().check()


@pytest.mark.parametrize("tokens", [1, 2, 15, 16, 17, 64, 65, 129, 500])
def test_token_counts(tokens):
    for block in (16, 64, 128):
        Case(tokens, 264, [136], 16, _ids(tokens, 5), adapters=5, block=block).run().check()
    Case(tokens, 264, [32, 136], 40, _ids(tokens, 5), adapters=5, pad=8).run().check()


@pytest.mark.parametrize("k", [8, 56, 64, 72, 512, 1000, 4096, 7168])
@pytest.mark.parametrize("n", [8, 40, 128, 264, 1864])
def test_sizes(k, n):
    Case(5, k, [n], 16, [0, 1, 0, 1, 1], scales=[1.5, 0.25]).run().check()
    Case(90, k, [n], 32, _ids(90, 2), "f16", adapters=2, block=64).run().check()


@pytest.mark.parametrize("k", [64, 128, 192, 256, 320, 1088, 4096])
@pytest.mark.parametrize("rank,slices", [(72, [136]), (128, [64]), (64, [32, 64, 136]), (256, [64]), (136, [64, 128, 192])])
def test_many_ranks_for_many_tokens(k, rank, slices):
    # the first product's steps of 64, from one on; rank rows that end inside a wave's and a workgroup's share
    for dtype, block in (("bf16", 64), ("f16", 64), ("bf16", 128), ("f16", 128)):
        Case(150, k, slices, rank, _ids(150, 3), dtype, adapters=3, block=block, ranks=[rank, rank - 7, 3], pad=8).run().check()


@pytest.mark.parametrize("ranks", [[0, 1, 5, 8], [16, 15, 9, 7], [-3, 100, 16, 2]])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_adapters_of_smaller_rank(ranks, dtype):
    clipped = [min(max(r, 0), 16) for r in ranks]
    for slices in ([72], [32, 64, 128]):
        c = Case(40, 136, slices, 16, _ids(40, 4), dtype, ranks=clipped, adapters=4, scales=[1, 2, 3, 4])
        c.ranks = torch.tensor(ranks, dtype=torch.int32, device="cuda")     # taken into the range
        c.run().check()
    c = Case(80, 136, [264], 72, _ids(80, 4), dtype, ranks=[1, 33, 72, 64], adapters=4, block=64)
    c.run().check()


def test_in_place_and_beside():
    Case(50, 264, [136], 16, _ids(50, 3), adapters=3, inplace=True).run().check()
    Case(200, 264, [32, 136], 32, _ids(200, 3), "f16", adapters=3, block=64, pad=16, inplace=True).run().check()


def test_no_token_has_an_adapter():
    c = Case(20, 136, [72], 16, [-1] * 20, adapters=4).run()
    torch.cuda.synchronize()
    assert torch.isnan(c.y).all()
    qg.lora(c.desc, c.x, c.a, c.b, *c.map, 0, c.block, c.base, c.y, c.ws)       # no tokens: no-op


def test_many_adapters_and_slices():
    Case(512, 136, [32, 64, 96, 128, 160, 192, 224, 264], 8, np.random.default_rng(3).integers(0, 512, 512), adapters=512).run().check()


def test_f16_sums_beyond_the_type():
    # t of a hundred thousand and more: beyond f16, but not the result; and tiny t beside them
    c = Case(16, 512, [64], 16, [0] * 16, "f16")
    c.x.mul_(3000.0)
    c.a.mul_(60.0)
    c.a[0, 0, 1:].mul_(1e-3)
    c.b.mul_(1e-5)
    c.want = LO.lora(_d(c.x), _d(c.a), _d(c.b), c.ids, [16], np.ones(1), _d(c.base), [64])
    c.run().check()


def test_values_that_are_not_finite_stay_with_their_tokens():
    c = Case(40, 264, [136], 16, _ids(40, 3, none=0.0), adapters=3)
    c.x[7, 100] = float("nan")
    c.x[21, 3] = float("inf")
    c.base[30, 5] = float("inf")
    c.run()
    torch.cuda.synchronize()
    got = _d(c.y)
    rest = [i for i in range(40) if i not in (7, 21, 30)]
    ref, mag = c.want
    assert (np.abs(got - ref)[rest] <= (U["bf16"] * np.abs(ref) + 2.0 ** -14 * mag)[rest]).all()
    assert np.isnan(got[7]).all() and not np.isfinite(got[21]).any() and got[30, 5] == np.inf and np.isfinite(got[30, :5]).all()


def test_a_token_does_not_depend_on_its_place():
    # the same rows twice in a batch, at other places of other blocks
    c = Case(64, 264, [136], 16, [0] * 20 + [1] * 20 + [0] * 24, adapters=2, block=16)
    c.x[50:60] = c.x[0:10]
    c.base[50:60] = c.base[0:10]
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.y[50:60], c.y[0:10])


def test_other_stream_graph_and_shared_map():
    c = Case(130, 520, [264], 16, _ids(130, 6), adapters=6)
    d = Case(130, 264, [32, 136], 24, _ids(130, 6), adapters=6)     # another product of the same batch
    d.map, d.block = c.map, c.block
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run()
        d.run()
    side.synchronize()
    c.check()
    d.check()
    first = c.y.clone(), d.y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qg.moe_align(c.dev_ids, c.tokens, 1, 6, c.block, *c.map)
        c.run()
        d.run()
    for _ in range(3):
        for t in (c.y, d.y):
            t.fill_(float("nan"))
        c.ws.fill_(0x5A)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first[0].view(torch.int16), c.y.view(torch.int16))
        assert torch.equal(first[1].view(torch.int16), d.y.view(torch.int16))
