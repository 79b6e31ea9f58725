"""GPU parity of the 4-bit cache (qg_kv_append, qg_kv_read) and of the attention that reads it (qg_attention).

Bars: the cache is exact (each step of the quantization is).  Attention, from the arithmetic: scores are float32 sums of
exact products (16-bit query times a code with a power of two), off by D / 4 roundings of 2^-24 of their terms at most,
then one rounding by the scale; a weight is off by that, absolutely, times itself, and by 2^-21 of itself for the
exponential; sums of weights and of products over the tokens are float32 and, being split over lanes, waves and workgroups,
take less than 2^11 roundings of 2^-24 in turn at these lengths.  bf16 weights enter the second product rounded, 2^-8
of themselves at most, f16 ones as two bf16 numbers, 2^-16.  Then half a step of the output.  With M the reference's
magnitude (sum of w |V| (1 + scale sum |q k|) and its like for the sum of weights):
|out - ref| <= u |ref| + (2^-8 or 2^-16 + (D / 4 + 2) 2^-24 + 2^-20 + 2^-13) M, the last term the sums'.
"""
import numpy as np
import pytest
import torch

import quantized_gemm_amd as qg
from oracle import layer_ops as LO

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
O = {"bf16": qg.O_BF16, "f16": qg.O_F16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qg.lib()
    yield


def _d(t):
    return t.double().cpu().numpy()


def _rows(rng, n, width, dtype, sigma=1.0):
    return torch.from_numpy(rng.standard_normal((n, width)).astype(np.float32) * sigma).to(DT[dtype]).cuda()


# ---- the cache -------------------------------------------------------------------------------

@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_append_and_read_back_are_exact(dim, page, dtype):
    rng = np.random.default_rng(dim + page)
    heads, pages, n, pad = 3, 4, 2 * page + 5, 8
    d = qg.make_kv_desc(O[dtype], heads, dim, page, pages)
    cache = torch.full((qg.kv_cache_bytes(d),), 0xA5, dtype=torch.uint8, device="cuda")
    width = heads * dim
    k, v = (_rows(rng, n, width + pad, dtype, 10.0 ** rng.uniform(-3, 3)) for _ in "kv")
    k[1] = 0
    v[2, :40] = 0
    slots = rng.permutation(pages * page)[:n].astype(np.int32)
    slots[3], slots[4] = -1, pages * page                          # skipped
    dev = torch.from_numpy(slots).cuda()
    qg.kv_append(d, k, v, dev, n, cache, k_stride=width + pad, v_stride=width + pad)
    back = [torch.full((n, width), float("nan"), dtype=DT[dtype], device="cuda") for _ in "kv"]
    qg.kv_read(d, cache, dev, n, *back)
    torch.cuda.synchronize()
    for x, b in zip((k, v), back):
        want = LO.mxfp4_values(_d(x)[:, :width])
        want[3:5] = 0.0
        want = torch.from_numpy(want).to(DT[dtype]).double().numpy()    # (f16 below its range)
        assert np.array_equal(_d(b), want)
    # nothing else was written: a second append of the same rows to slots outside changes no byte
    before = cache.clone()
    qg.kv_append(d, k, v, torch.full_like(dev, -5), n, cache, k_stride=width + pad, v_stride=width + pad)
    torch.cuda.synchronize()
    assert torch.equal(before, cache)


def test_powers_of_two_at_the_ends_of_the_range():
    # bf16 blocks of every exponent it has, subnormal ones too, and rounding at every border of every code
    d = qg.make_kv_desc(qg.O_BF16, 1, 64, 256, 2)
    cache = torch.zeros(qg.kv_cache_bytes(d), dtype=torch.uint8, device="cuda")
    n = 280
    m = np.array([4.0, 7.96875, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.251, 0.749, 1.251, 1.749, 2.51, 3.49, 5.03])
    row = np.concatenate([m, -m, m[::-1], -m])
    x = torch.from_numpy(row[None, :] * np.exp2(np.arange(n)[:, None] - 150.0)).to(torch.bfloat16).cuda()   # (the largest: infinite)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    qg.kv_append(d, x, x, slots, n, cache)
    back = [torch.empty((n, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    qg.kv_read(d, cache, slots, n, *back)
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        want = LO.mxfp4_values(_d(x))
    finite = np.isfinite(_d(x)).all(axis=1)
    assert finite.sum() > 270
    # (a code of 2^-127 may be half of bf16's smallest number: compared as bf16 rounds it)
    want = torch.from_numpy(want).to(torch.bfloat16).double().numpy()
    for b in back:
        assert np.array_equal(_d(b)[finite], want[finite])


def test_append_writes_its_slots_only():
    d = qg.make_kv_desc(qg.O_BF16, 2, 64, 16, 5)
    rng = np.random.default_rng(1)
    cache = torch.zeros(qg.kv_cache_bytes(d), dtype=torch.uint8, device="cuda")
    every = torch.arange(80, dtype=torch.int32, device="cuda")
    k, v = _rows(rng, 80, 128, "bf16"), _rows(rng, 80, 128, "bf16")
    qg.kv_append(d, k, v, every, 80, cache)
    k2, v2 = _rows(rng, 3, 128, "bf16"), _rows(rng, 3, 128, "bf16")
    some = torch.tensor([17, 79, 4], dtype=torch.int32, device="cuda")
    qg.kv_append(d, k2, v2, some, 3, cache)
    back = [torch.empty((80, 128), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    qg.kv_read(d, cache, every, 80, *back)
    torch.cuda.synchronize()
    for x, x2, b in zip((k, v), (k2, v2), back):
        want = LO.mxfp4_values(_d(x))
        want[[17, 79, 4]] = LO.mxfp4_values(_d(x2))
        assert np.array_equal(_d(b), want)


def test_blocks_that_are_not_finite_are_nan():
    d = qg.make_kv_desc(qg.O_BF16, 1, 64, 16, 1)
    cache = torch.zeros(qg.kv_cache_bytes(d), dtype=torch.uint8, device="cuda")
    x = torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")
    x[0, 5], x[1, 40], x[2, 63] = float("nan"), float("inf"), -float("inf")
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    qg.kv_append(d, x, x, slots, 3, cache)
    back = [torch.empty((3, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    qg.kv_read(d, cache, slots, 3, *back)
    torch.cuda.synchronize()
    for b in back:
        assert torch.isnan(b[0, :32]).all() and torch.isnan(b[1:, 32:]).all()
        assert (b[0, 32:] == 1).all() and (b[1:, :32] == 1).all()


# ---- attention -------------------------------------------------------------------------------

class Case:
    def __init__(self, lens, heads, kv_heads, dim, page, counts=None, dtype="bf16", max_len=None, max_q=None, pad=0, sigma=1.0,
                 seed=0, extra_rows=0, bad_pages=()):
        rng = np.random.default_rng(seed + 17 * dim + page + len(lens))
        b = len(lens)
        self.lens, self.counts = list(lens), list(counts) if counts is not None else [1] * b
        self.dtype, self.heads, self.dim, self.batch = dtype, heads, dim, b
        self.max_len = max_len or max(1, max(lens))
        self.max_q = max_q or max(1, max(self.counts))
        held = [-(-n // page) for n in lens]
        pages = sum(held) + 2                                       # two that hold NaN: never to be read to any effect
        order = rng.permutation(pages)
        self.desc = qg.make_kv_desc(O[dtype], kv_heads, dim, page, pages)
        self.cache = torch.full((qg.kv_cache_bytes(self.desc),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN all over
        table = np.full((b, -(-self.max_len // page)), order[-1], np.int64)
        self.k, self.v, self.seen = [], [], []
        at = 0
        width = kv_heads * dim
        for i, n in enumerate(lens):
            table[i, :held[i]] = order[at:at + held[i]]
            at += held[i]
            rows = [_rows(rng, n, width, dtype, sigma) for _ in "kv"]
            if n:
                t = np.arange(n)
                slots = torch.from_numpy((table[i][t // page] * page + t % page).astype(np.int32)).cuda()
                qg.kv_append(self.desc, *rows, slots, n, self.cache)
            vals = [LO.mxfp4_values(_d(r)).reshape(n, kv_heads, dim) if n else np.zeros((0, kv_heads, dim)) for r in rows]
            self.k.append(vals[0])
            self.v.append(vals[1])
            seen = np.ones(n, bool)
            for p in [p for s, p in bad_pages if s == i]:
                table[i, p] = rng.choice([-1, pages, 1 << 30])
                seen[p * page:(p + 1) * page] = False
            self.seen.append(seen)
        self.table = torch.from_numpy(table.astype(np.int32)).cuda()
        self.dlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(self.counts)]).astype(np.int32)).cuda()
        self.tokens = sum(self.counts) + extra_rows
        self.q = _rows(rng, self.tokens, heads * dim + pad, dtype, 1.5)
        self.out = torch.full_like(self.q, float("nan"))
        self.scale = dim ** -0.5
        need = qg.attention_workspace_bytes(self.desc, heads, b, self.max_q, self.tokens, self.max_len)
        self.ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if need else None
        self.used = sum(self.counts)
        self.stride = heads * dim + pad

    def run(self, stream=None):
        plain = self.max_q == 1 and self.counts == [1] * self.batch and self.tokens == self.batch
        qg.attention(self.desc, self.q, self.heads, self.cache, self.table, self.dlens, self.batch, self.max_len, self.scale,
                     self.out, self.ws, q_offsets=None if plain else self.offsets, max_q=self.max_q, tokens=self.tokens,
                     q_stride=self.stride, out_stride=self.stride, stream=stream)
        return self

    def check(self):
        torch.cuda.synchronize()
        w = self.heads * self.dim
        got = _d(self.out)
        assert np.isnan(got[self.used:]).all() and np.isnan(got[:, w:]).all()          # left as they were
        q = _d(self.q)[:self.used, :w].reshape(self.used, self.heads, self.dim)
        ref, mag = LO.attention(q, self.k, self.v, self.lens, self.counts, self.scale, self.seen)
        got = got[:self.used, :w].reshape(ref.shape)
        rel = (2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -16) + (self.dim / 4 + 2) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -13
        tol = U[self.dtype] * np.abs(ref) + rel * mag + 2.0 ** -25
        assert (np.abs(got - ref) <= tol).all(), np.max(np.abs(got - ref) / tol)
        return self


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 256])
def test_decode(dtype, dim, page):
    Case([1, 15, 16, 17, 31, 32, 33, 63, 100, 257, 0], 6, 3, dim, page, dtype=dtype, pad=8).run().check()


@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 16, 17, 40])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_groups(group, dtype):
    Case([5, 130, 64], 2 * group, 2, 128, 16, dtype=dtype).run().check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 4, 16])
def test_several_queries(dtype, dim, group):
    # one to many per sequence, none, all of a sequence's tokens, more than it has (the first see nothing)
    Case([40, 7, 300, 64, 90, 3, 0], group, 1, dim, 16, counts=[3, 7, 1, 64, 0, 5, 2], dtype=dtype).run().check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_chunks(dtype, dim):
    Case([200, 333], 4, 2, dim, 32, counts=[200, 150], dtype=dtype, extra_rows=3, pad=8).run().check()


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64), ("bf16", 256)])
def test_split_over_long_sequences(dtype, dim):
    c = Case([3000, 1, 700, 0], 4, 2, dim, 64, dtype=dtype)
    assert c.ws is not None
    c.run().check()
    c = Case([2500, 40], 8, 2, dim, 16, counts=[20, 33], dtype=dtype)
    assert c.ws is not None
    c.run().check()


def test_lengths_below_the_maximum():
    # the table and the splits are made for longer sequences than there are
    Case([1, 70, 300], 8, 2, 128, 16, max_len=5000, max_q=9, counts=[1, 2, 9]).run().check()


def test_tokens_on_pages_outside_the_cache_are_not_seen():
    Case([100, 260], 8, 2, 128, 16, bad_pages=[(0, 0), (0, 6), (1, 3), (1, 4), (1, 16)]).run().check()
    Case([100, 260], 8, 2, 64, 64, bad_pages=[(0, 1), (1, 0), (1, 4)], counts=[9, 30], dtype="f16").run().check()
    Case([30], 4, 1, 128, 32, bad_pages=[(0, 0)]).run().check()      # nothing is seen: zeros


@pytest.mark.parametrize("counts", [[1, 1, 1], [9, 40, 3]])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-45, -0.25])
def test_scales_of_nothing_and_below(scale, counts):
    c = Case([33, 70, 517], 16, 2, 64, 16, counts=counts)
    c.scale = scale
    c.run().check()


def test_large_scores():
    # softmax close to a choice: scores of a hundred and more; weights that vanish
    c = Case([500, 33], 4, 2, 128, 16, sigma=6.0)
    c.scale = 1.0
    c.run().check()
    c = Case([500, 33], 4, 2, 128, 16, sigma=6.0, counts=[20, 33], dtype="f16")
    c.scale = -1.0
    c.run().check()


def _poison(c, seq, token, part, head, block, page, value=255):
    """Sets the exponent byte of a token's block in the cache."""
    d = c.desc
    p, dim = d.page_tokens, d.head_dim
    pid = int(c.table[seq, token // p])
    base = (pid * d.kv_heads + head) * p * (dim + dim // 16)
    t = token % p
    if part == "k":
        at = base + p * dim + t * (dim // 32) + block
    else:
        at = base + p * dim + p * (dim // 32) + ((t // 4) * (dim // 32) + block) * 4 + t % 4
    c.cache[at] = value
    x = (c.k if part == "k" else c.v)[seq]
    x[token, head, 32 * block:32 * block + 32] = np.nan


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts", [[1, 1], [12, 40]])
def test_nan_reaches_the_queries_that_see_it_only(dim, dtype, counts):
    c = Case([50, 90], 4, 2, dim, 16, counts=counts, dtype=dtype)
    _poison(c, 0, 49, "v", 1, dim // 32 - 1, 16)       # seen by the last query only
    _poison(c, 1, 70, "v", 0, 0, 16)
    _poison(c, 1, 88, "k", 1, 0, 16)
    c.run()
    torch.cuda.synchronize()
    got = _d(c.out).reshape(c.used, 4, dim)
    q = _d(c.q).reshape(got.shape)
    ref, mag = LO.attention(q, c.k, c.v, c.lens, c.counts, c.scale)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    tol = U[dtype] * np.abs(ref) + 2.0 ** -7 * mag + 2.0 ** -25
    assert (np.abs(got - ref)[ok] <= tol[ok]).all()
    assert np.isnan(got).any() and ok.any()


def test_a_query_alone_and_among_others():
    # the same query row against the same sequence, in a batch of other queries' tiles
    c = Case([200], 4, 1, 128, 16, counts=[33]).run()
    c.check()
    d = Case([200, 200], 4, 1, 128, 16, counts=[33, 33], seed=0)
    d.run().check()


def test_offsets_beyond_32_bits():
    # pages behind the first 2^32 bytes of the cache
    d = qg.make_kv_desc(qg.O_BF16, 8, 256, 256, 8000)
    assert qg.kv_cache_bytes(d) > (1 << 32)
    cache = torch.zeros(qg.kv_cache_bytes(d), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(2)
    n, width = 300, 8 * 256
    k, v = _rows(rng, n, width, "bf16"), _rows(rng, n, width, "bf16")
    table = torch.tensor([[7999, 7990]], dtype=torch.int32, device="cuda")
    t = np.arange(n)
    slots = torch.from_numpy((np.array([7999, 7990])[t // 256] * 256 + t % 256).astype(np.int32)).cuda()
    qg.kv_append(d, k, v, slots, n, cache)
    q = _rows(rng, 1, 8 * 256, "bf16")
    out = torch.empty_like(q)
    ws = torch.empty(max(16, qg.attention_workspace_bytes(d, 8, 1, 1, 1, 300)), dtype=torch.uint8, device="cuda")
    qg.attention(d, q, 8, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), 1, 300, 1 / 16, out, ws)
    torch.cuda.synchronize()
    vals = [LO.mxfp4_values(_d(x)).reshape(n, 8, 256) for x in (k, v)]
    ref, mag = LO.attention(_d(q).reshape(1, 8, 256), [vals[0]], [vals[1]], [n], [1], 1 / 16)
    assert (np.abs(_d(out).reshape(ref.shape) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7 * mag).all()
    back = [torch.empty((n, width), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    qg.kv_read(d, cache, slots, n, *back)
    torch.cuda.synchronize()
    assert np.array_equal(_d(back[1]).reshape(vals[1].shape), vals[1])


def test_other_stream_graph_and_growing_sequences():
    # one captured step: append of the new tokens, then attention, lengths read on the device
    c = Case([100, 700, 31], 8, 2, 128, 16, max_len=2048)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run()
    side.synchronize()
    c.check()
    rng = np.random.default_rng(9)
    k, v = (torch.zeros((3, 256), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qg.kv_append(c.desc, k, v, slots, 3, c.cache)
        c.run()
    for _ in range(3):
        new = [_rows(rng, 3, 256, "bf16") for _ in "kv"]
        k.copy_(new[0])
        v.copy_(new[1])
        at = []
        for i in range(3):
            n = c.lens[i]
            if n % 16 == 0:                                        # its last page is full: nothing new
                at.append(-1)
                continue
            at.append(int(c.table[i, n // 16]) * 16 + n % 16)
            for own, x in zip((c.k, c.v), new):
                own[i] = np.concatenate([own[i], LO.mxfp4_values(_d(x[i:i + 1])).reshape(1, 2, 128)])
            c.lens[i] = n + 1
            c.seen[i] = np.ones(n + 1, bool)
        slots.copy_(torch.tensor(at, dtype=torch.int32))
        c.dlens.copy_(torch.tensor(c.lens, dtype=torch.int32))
        c.out.fill_(float("nan"))
        c.ws.fill_(0xFF)
        graph.replay()
        c.check()
