"""GPU run of a decoder block's operators together, as a server uses them: norm and quantization, the quantized product
with the requests' adapters on it, the append to the 4-bit cache, attention over it, the product behind it, and the norm
with the residual for what follows, in one captured graph that is replayed with other tokens, lengths and adapters.

Each step is checked against float64 of what the step before left on the device, so that its own bar holds: those of
the operators' own tests, and for a product half a step of the output and k / 8 + 64 roundings of 2^-24 of its terms
(a scale more for each operand and the output).
"""
import numpy as np
import pytest
import torch

import quantized_gemm_amd as qg
from oracle import formats as F
from oracle import layer_ops as LO
from oracle import reference as R
from quantized_gemm_amd import layers, synth

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, DIM, PAGE = 512, 8, 2, 64, 16
QKV = (HEADS + 2 * KV) * DIM
ENDS = [HEADS * DIM, (HEADS + KV) * DIM, QKV]
ADAPTERS, RANK = 3, 16
U = 2.0 ** -8                                                      # half a step of bf16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qg.lib()
    yield


def _d(t):
    return t.double().cpu().numpy()


def _dev(rng, *shape, scale=1.0, mean=0.0):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * scale + mean).to(torch.bfloat16).cuda()


class Block:
    def __init__(self, counts, held, seed, ws=None):
        """counts: new tokens of each sequence; held: tokens that its cache holds already."""
        rng = np.random.default_rng(seed)
        self.rng, self.counts, self.held = rng, list(counts), list(held)
        self.t = t = sum(counts)
        b = len(counts)
        self.max_len = 160
        per = self.max_len // PAGE
        self.layers = [synth.dense_w8a8_fp8(t, QKV, HIDDEN, seed)[0], synth.dense_w8a8_fp8(t, HIDDEN, HEADS * DIM, seed + 1)[0]]
        self.p = [layers.prepare_layer(x) for x in self.layers]
        self.wide = [R.dequant_layer(x, 0) for x in self.layers]
        self.kv = qg.make_kv_desc(qg.O_BF16, KV, DIM, PAGE, b * per)
        self.cache = torch.full((qg.kv_cache_bytes(self.kv),), 0xFF, dtype=torch.uint8, device="cuda")
        self.pages = rng.permutation(b * per).reshape(b, per)
        self.table = torch.from_numpy(self.pages.astype(np.int32)).cuda()
        self.k, self.v = [], []
        for i, n in enumerate(held):
            rows = [_dev(rng, n, KV * DIM) for _ in "kv"]
            if n:
                qg.kv_append(self.kv, *rows, torch.tensor(self.slots(i, 0, n), dtype=torch.int32, device="cuda"), n, self.cache)
            self.k.append(LO.mxfp4_values(_d(rows[0])).reshape(n, KV, DIM) if n else np.zeros((0, KV, DIM)))
            self.v.append(LO.mxfp4_values(_d(rows[1])).reshape(n, KV, DIM) if n else np.zeros((0, KV, DIM)))
        norm = dict(code_type=qg.A_FP8_E4M3)
        self.first = qg.make_norm_desc(qg.N_RMS, qg.O_BF16, HIDDEN, 1e-6, **norm)
        self.last = qg.make_norm_desc(qg.N_RMS, qg.O_BF16, HIDDEN, 1e-6, post_norm=qg.N_RMS, **norm)
        self.lora = qg.make_lora_desc(qg.O_BF16, ADAPTERS, RANK, HIDDEN, ENDS)
        self.w = [_dev(rng, HIDDEN, scale=0.1, mean=1.0) for _ in range(3)]
        self.a = _dev(rng, ADAPTERS, 3, RANK, HIDDEN, scale=HIDDEN ** -0.5)
        self.b = _dev(rng, ADAPTERS, QKV, RANK, scale=RANK ** -0.5)
        bf = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        by = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.h, self.x, self.x8, self.xs = bf(t, HIDDEN), bf(t, HIDDEN), by(t, HIDDEN), torch.zeros(t, device="cuda")
        self.base, self.qkv = bf(t, QKV), bf(t, QKV)
        self.att, self.att8, self.atts = bf(t, HEADS * DIM), by(t, HEADS * DIM), torch.zeros(t, device="cuda")
        self.o, self.res = bf(t, HIDDEN), bf(t, HIDDEN)
        self.z, self.z8, self.zs = bf(t, HIDDEN), by(t, HIDDEN), torch.zeros(t, device="cuda")
        self.ids, self.slot, self.lens = i32(t), i32(t), i32(b)
        self.offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
        self.block = qg.lora_block_m(t, ADAPTERS)
        rows, blocks = qg.moe_capacity(t, 1, ADAPTERS, self.block)
        self.map = [i32(rows), i32(blocks), i32(1)]
        self.max_q = max(counts)
        need = max(qg.lora_workspace_bytes(self.lora, t, self.block),
                   qg.attention_workspace_bytes(self.kv, HEADS, b, self.max_q, t, self.max_len),
                   *(qg.workspace_bytes(p, t) for p, _ in self.p))
        self.ws = by(max(1, need)) if ws is None else ws           # one for all: they run in turn
        assert self.ws.numel() >= need

    def slots(self, i, begin, end):
        at = np.arange(begin, end)
        return list(self.pages[i][at // PAGE] * PAGE + at % PAGE)

    def fill(self, ids):
        """New hidden rows, adapters and lengths, in place."""
        self.h.copy_(_dev(self.rng, self.t, HIDDEN, scale=2.0))
        self.ids.copy_(torch.tensor(ids, dtype=torch.int32))
        slots = []
        for i, n in enumerate(self.counts):
            slots += self.slots(i, self.held[i], self.held[i] + n)
            self.held[i] += n
        self.slot.copy_(torch.tensor(slots, dtype=torch.int32))
        self.lens.copy_(torch.tensor(self.held, dtype=torch.int32))

    def run(self):
        t = self.t
        qg.norm_rows(self.first, t, None, self.h, None, self.x, self.x8, self.xs, weight=self.w[0])
        qg.gemm(self.p[0][0], self.x8, self.xs, self.base, t, self.ws)
        qg.moe_align(self.ids, t, 1, ADAPTERS, self.block, *self.map)
        self.qkv.copy_(self.base)
        qg.lora(self.lora, self.x, self.a, self.b, *self.map, t, self.block, self.qkv, self.qkv, self.ws)
        qg.kv_append(self.kv, self.qkv[:, ENDS[0]:], self.qkv[:, ENDS[1]:], self.slot, t, self.cache, k_stride=QKV, v_stride=QKV)
        qg.attention(self.kv, self.qkv, HEADS, self.cache, self.table, self.lens, len(self.counts), self.max_len, DIM ** -0.5,
                     self.att, self.ws, q_offsets=None if self.max_q == 1 else self.offsets, max_q=self.max_q, tokens=t, q_stride=QKV)
        qg.quantize_e4m3_rows(self.att, t, HEADS * DIM, qg.L_BF16, self.att8, self.atts)
        qg.gemm(self.p[1][0], self.att8, self.atts, self.o, t, self.ws)
        qg.norm_rows(self.last, t, self.o, self.h, self.res, self.z, self.z8, self.zs, weight=self.w[1], post_weight=self.w[2])

    def check(self):
        torch.cuda.synchronize()
        ids = self.ids.cpu().numpy()
        # the norm and its codes
        _, z, _, zmag = LO.norm_rows(res=_d(self.h), weight=_d(self.w[0]))
        self.normed(self.x, self.x8, self.xs, z, zmag)
        # the product, and the adapters on it
        self.product(self.base, self.x8, self.xs, self.wide[0])
        ref, mag = LO.lora(_d(self.x), _d(self.a), _d(self.b), ids, [RANK] * ADAPTERS, np.ones(ADAPTERS), _d(self.base), ENDS)
        has = (ids >= 0) & (ids < ADAPTERS)
        bar = U * np.abs(ref) + (2.0 ** -16 + (HIDDEN / 8 + 64 + 512) * 2.0 ** -24) * mag
        assert (np.abs(_d(self.qkv) - ref) <= np.where(has[:, None], bar, 0.0)).all()
        # what the cache has taken, and attention over it
        back = [torch.empty((self.t, KV * DIM), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        qg.kv_read(self.kv, self.cache, self.slot, self.t, *back)
        wide, at = _d(self.qkv), 0
        new = [LO.mxfp4_values(wide[:, b:e]) for b, e in zip(ENDS[:2], ENDS[1:])]
        for n, b in zip(new, back):
            assert np.array_equal(n, _d(b))
        for i, n in enumerate(self.counts):
            for own, x in zip((self.k, self.v), new):
                own[i] = np.concatenate([own[i], x[at:at + n].reshape(n, KV, DIM)])
            at += n
        ref, mag = LO.attention(wide[:, :ENDS[0]].reshape(self.t, HEADS, DIM), self.k, self.v, self.held, self.counts, DIM ** -0.5)
        bar = U * np.abs(ref) + (2.0 ** -8 + (DIM / 4 + 2) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -13) * mag
        assert (np.abs(_d(self.att).reshape(ref.shape) - ref) <= bar).all()
        # behind it
        self.product(self.o, self.att8, self.atts, self.wide[1])
        u, z, umag, zmag = LO.norm_rows(y=_d(self.o), res=_d(self.h), post="rms", weight=_d(self.w[1]), post_weight=_d(self.w[2]))
        assert (np.abs(_d(self.res) - u) <= U * np.abs(u) + 2.0 ** -18 * umag).all()
        self.normed(self.z, self.z8, self.zs, z, zmag)

    def normed(self, out, codes, scale, z, mag):
        noise = 2.0 ** -17 * mag
        assert (np.abs(_d(out) - z) <= U * np.abs(z) + noise).all()
        # e4m3: half a step of the code, 2^-4 of the value, or 2^-10 of the scale below its normal range
        s = _d(scale)[:, None]
        top = np.abs(z).max(axis=1, keepdims=True)
        assert (np.abs(s * 448.0 - top) <= 2.0 ** -16 * top + noise.max(axis=1, keepdims=True)).all()
        got = F.decode_e4m3(codes.cpu().numpy()).astype(np.float64) * s
        assert (np.abs(got - z) <= np.maximum(2.0 ** -4 * np.abs(z), 2.0 ** -10 * s) * (1 + 2.0 ** -16) + 2 * noise).all()

    def product(self, out, codes, scale, w):
        x = F.decode_e4m3(codes.cpu().numpy()).astype(np.float64) * _d(scale)[:, None]
        ref, mag = x @ w.T, np.abs(x) @ np.abs(w).T
        assert (np.abs(_d(out) - ref) <= U * np.abs(ref) + (x.shape[1] / 8 + 67) * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("counts, held", [
    ([1, 1, 1, 1, 1], [0, 15, 16, 40, 100]),                       # tokens one at a time, at and beside a page's end
    ([20, 1, 33, 2], [0, 31, 7, 16]),                              # chunks of prompts among them
])
def test_a_block(counts, held):
    c = Block(counts, held, seed=len(counts))
    ids = lambda turn: [(turn + i) % (ADAPTERS + 1) - 1 for i in range(c.t)]  # noqa: E731    (-1: no adapter)
    c.fill(ids(0))
    c.run()
    c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for turn in range(1, 4):
        c.fill(ids(turn))
        graph.replay()
        c.check()


IDS = [0, -1, 2, 1, 7]


def test_two_graphs_share_a_workspace():
    ws = torch.full((1 << 24,), 0xFF, dtype=torch.uint8, device="cuda")
    blocks = [Block([1, 1, 1], [90, 0, 47], 7, ws), Block([30, 1, 9], [2, 64, 15], 8, ws)]
    graphs = []
    for c in blocks:
        c.fill([IDS[i % 5] for i in range(c.t)])
        c.run()
        c.check()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run()
        graphs.append(graph)
    for turn in range(1, 4):
        for c in blocks:
            c.fill([IDS[(i + turn) % 5] for i in range(c.t)])
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        for c in blocks:
            c.check()


def test_two_streams_at_once():
    blocks = [Block([1, 1, 1, 1], [90, 0, 47, 15], 9), Block([30, 1, 9], [2, 64, 15], 10)]
    streams = [torch.cuda.Stream() for _ in blocks]
    for turn in range(3):
        for c in blocks:
            c.fill([IDS[(i + turn) % 5] for i in range(c.t)])
        torch.cuda.synchronize()
        for c, stream in zip(blocks, streams):
            with torch.cuda.stream(stream):
                c.run()
        for c in blocks:
            c.check()
