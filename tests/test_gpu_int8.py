"""GPU parity of the int8 W8A8 products, of the int8 row quantizers and of an int8 MoE layer from its router's logits.

Bars, from the arithmetic:
* product: the sum over K is an exact integer; y = out(float(sum) * scale[n] * x_scale[m]), three
  float32 roundings and the output's, all to nearest even, in a fixed order: bit for bit the same
  as the same four roundings in numpy, whatever the tile, the split over K or the other rows.
  Against float64: |y - ref| <= (u_out + 3 * 2^-24) * (1 + 2^-7) * |ref| + (K + 4) * 2^-53 * sum |terms| + 2^-25
  the second for the reference itself, which scales each term before it adds (where the integer sum
  is 0 its rounding is all there is), the last half a step of an f16 output below 2^-14;
* row quantizer: every step is a float32 operation with one rounding: codes and scales bit-exact;
* SwiGLU -> int8: bit-exact where silu(gate) is exact; else scales to 2^-20 relative (float32
  sigmoid with the hardware exponential, as for e4m3) and each value within half a code of the
  float64 activation plus that noise;
* the layer: the float64 layer with its two quantizations within 2e-2 of its largest output, see
  test_int8_layer_from_logits.
"""
import numpy as np
import pytest
import torch

import quantized_gemm_amd as qg
from quantized_gemm_amd import layers, synth
from oracle import formats as F
from oracle import layout as L
from oracle import moe_layer as ML
from oracle import quant as Q
from oracle import reference as R
from oracle import route as RT

pytestmark = pytest.mark.gpu

U_OUT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
T_DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16}
Q_OUT = {"bf16": qg.O_BF16, "f16": qg.O_F16}
Q_ACT = {"bf16": qg.A_BF16, "f16": qg.A_F16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qg.lib()
    yield


def _bits(v, out):
    return synth.f32_to_bf16_bits(v) if out == "bf16" else synth.f32_to_f16_bits(v)


def _want(x, xs, w, sw, out):
    """The product as its definition rounds it: 16-bit patterns [rows, N]."""
    p = (x.astype(np.float64) @ w.astype(np.float64).T)       # exact: integers below 2^53
    v = p.astype(np.float32) * sw.astype(np.float32)[None, :]
    v = v * xs.astype(np.float32)[:, None]
    return _bits(v, out)


def _got(y):
    return y.view(torch.int16).cpu().numpy().view(np.uint16)


def _run(p, x, xs, m, n, out, stream=None):
    y = torch.full((m, n), float("nan"), dtype=T_DTYPE[out], device="cuda")
    need = qg.workspace_bytes(p, m)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda") if need else None
    qg.gemm(p, x[:m], xs[:m], y, m, ws, stream=stream)
    torch.cuda.synchronize()
    return y


def test_prepare_and_read_back_are_exact():
    layer, _ = synth.moe_w8a8_int8(t=1, experts=3, topk=1, n=192, k=384, seed=1)
    layer.w[0, 0, :4] = [-128, 127, 0, -1]
    desc = layers.desc_for(layer)
    buf = torch.full((qg.prepared_bytes(desc),), 0xAB, dtype=torch.uint8, device="cuda")
    p = qg.prepare(desc, layers.to_dev(layer.w), layers.to_dev(layer.s), None, buf)
    torch.cuda.synchronize()
    assert np.array_equal(buf.cpu().numpy(), L.repack(layer))
    for e in range(3):
        out = torch.empty((192, 384), dtype=torch.float32, device="cuda")
        qg.dequant(p, e, out)
        want = layer.w[e].astype(np.float32) * layer.s[e, :, :1]
        assert np.array_equal(out.cpu().numpy(), want)


# rows around every tile height and the largest drawn, columns that end inside a tile, reductions of
# one step, of an odd number of steps and of many
@pytest.mark.parametrize("n,k,out", [(64, 128, "bf16"), (192, 768, "f16"), (320, 1408, "bf16"), (1856, 1408, "f16"),
                                     (256, 4096, "bf16"), (576, 8192, "bf16"), (6208, 896, "f16")])
def test_dense_is_exact_for_every_row_count(n, k, out):
    ms = [1, 2, 3, 4, 5, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 127, 128, 129, 200, 255, 257, 300, 513]
    layer, acts = synth.dense_w8a8_int8(m=max(ms), n=n, k=k, out=out, seed=n + k)
    p, buf = layers.prepare_layer(layer)
    x, xs = layers.acts_to_dev(acts)
    want = _want(acts.x, acts.x_scale, layer.w[0], layer.s[0, :, 0], out)
    ref = R.dense_reference(layer, acts)
    terms = (np.abs(acts.x.astype(np.float64)) @ np.abs(layer.w[0].astype(np.float64)).T) * layer.s[0, :, 0] * \
        acts.x_scale[:, None]
    for m in ms:
        y = _run(p, x, xs, m, n, out)
        assert np.array_equal(_got(y), want[:m]), f"m={m}: {np.count_nonzero(_got(y) != want[:m])} outputs differ"
        err = np.abs(y.double().cpu().numpy() - ref[:m])
        bound = (U_OUT[out] + 3 * 2.0 ** -24) * (1 + 2.0 ** -7) * np.abs(ref) + (k + 4) * 2.0 ** -53 * terms + 2.0 ** -25
        assert np.all(err <= bound[:m]), m


@pytest.mark.parametrize("m", [1, 24, 64, 512, 2500])
def test_dense_full_size_is_exact(m):
    layer, acts = synth.dense_w8a8_int8(m=m, n=7168, k=7168, seed=m)
    p, buf = layers.prepare_layer(layer)
    x, xs = layers.acts_to_dev(acts)
    y = _run(p, x, xs, m, 7168, "bf16")
    rows = np.unique(np.concatenate([[0, m - 1], np.random.default_rng(0).integers(0, m, 40)]))
    want = _want(acts.x[rows], acts.x_scale[rows], layer.w[0], layer.s[0, :, 0], "bf16")
    assert np.array_equal(_got(y)[rows], want)


# every tile height and width, K split and not, with 1, 2, 3 and no steps after the last whole turn of the stage ring
@pytest.mark.parametrize("out", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [(40, 8256, 640), (260, 8320, 1408), (257, 7168, 640), (200, 8256, 896), (513, 4160, 768),
                                   (1224, 1600, 512), (1000, 7168, 896), (2500, 1856, 1408), (1500, 10304, 896),
                                   (4000, 7168, 640), (668, 704, 23040), (300, 576, 4096), (65, 4160, 4096),
                                   (33, 1856, 8192), (300, 192, 2048), (777, 64, 1152), (200, 1856, 2176), (777, 1024, 4096),
                                   (130, 4160, 4224), (128, 8192, 8192), (500, 512, 8320)])
def test_every_tile_is_exact(m, n, k, out):
    layer, acts = synth.dense_w8a8_int8(m=m, n=n, k=k, out=out, seed=m + n + k)
    p, buf = layers.prepare_layer(layer)
    x, xs = layers.acts_to_dev(acts)
    y = torch.full((m + 1, n), float("nan"), dtype=T_DTYPE[out], device="cuda")
    need = qg.workspace_bytes(p, m)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    qg.gemm(p, x, xs, y, m, ws[:need] if need else None)
    torch.cuda.synchronize()
    assert torch.isnan(y[m]).all() and (ws[need:] == 0xA5).all()        # nothing behind the last row or the partials
    rows = np.unique(np.concatenate([[0, m - 1], np.random.default_rng(0).integers(0, m, 60)]))
    want = _want(acts.x[rows], acts.x_scale[rows], layer.w[0], layer.s[0, :, 0], out)
    assert np.array_equal(_got(y[:m])[rows], want)
    # the rows not sampled: the same bits as by the kernel or tile of 32 rows
    again = torch.full((m, n), float("nan"), dtype=T_DTYPE[out], device="cuda")
    for r in range(0, m, 32):                                         
        e = min(m, r + 32)
        z = qg.workspace_bytes(p, e - r)
        qg.gemm(p, x[r:e], xs[r:e].contiguous(), again[r:e], e - r,
                torch.empty(z, dtype=torch.uint8, device="cuda") if z else None)
    torch.cuda.synchronize()
    assert torch.equal(again.view(torch.int16), y[:m].view(torch.int16))


@pytest.mark.parametrize("m", [1, 20, 40, 200])
def test_sums_up_to_the_31st_bit(m):
    # K = 130944 of -128 x -128: 2145386496 < 2^31; then of -128 x 127, and rows of zeros
    n, k = 64, 131072 - 128
    w = np.full((1, n, k), -128, np.int8)
    w[0, 1::2] = 127
    x = np.full((m, k), -128, np.int8)
    if m > 2:
        x[2] = 0
    s = np.linspace(1e-9, 2e-9, n, dtype=np.float32).reshape(1, n, 1)
    xs = np.linspace(0.5, 1.5, m, dtype=np.float32)
    layer = synth.Layer("edge", "int8", "int8", "f32", "bf16", n, k, 0, 1, w, s, None)
    p, buf = layers.prepare_layer(layer)
    y = _run(p, torch.from_numpy(x).cuda(), torch.from_numpy(xs).cuda(), m, n, "bf16")
    assert np.array_equal(_got(y), _want(x, xs, w[0], s[0, :, 0], "bf16"))


def test_rows_do_not_depend_on_the_call():
    # batch-invariant without a flag, and with it: the same bits for a row alone and among others
    layer, acts = synth.dense_w8a8_int8(m=700, n=1024, k=1024, seed=3)
    p, buf = layers.prepare_layer(layer)
    pi, bufi = layers.prepare_layer(layer, compute_flags=qg.C_BATCH_INVARIANT)
    x, xs = layers.acts_to_dev(acts)
    whole = _got(_run(p, x, xs, 700, 1024, "bf16"))
    for m in (1, 7, 40, 130, 333):
        assert np.array_equal(_got(_run(p, x, xs, m, 1024, "bf16")), whole[:m])
        assert np.array_equal(_got(_run(pi, x, xs, m, 1024, "bf16")), whole[:m])


@pytest.mark.parametrize("m,k", [(16, 4096), (64, 4096), (200, 4096), (200, 8192)])
def test_noalloc_and_another_stream(m, k):
    layer, acts = synth.dense_w8a8_int8(m=m, n=1024, k=k, seed=m)
    p, buf = layers.prepare_layer(layer)
    x, xs = layers.acts_to_dev(acts)
    want = _want(acts.x, acts.x_scale, layer.w[0], layer.s[0, :, 0], "bf16")
    y = torch.full((m, 1024), float("nan"), dtype=torch.bfloat16, device="cuda")
    qg.gemm_noalloc(p, x, xs, y, m)
    torch.cuda.synchronize()
    assert np.array_equal(_got(y), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert np.array_equal(_got(_run(p, x, xs, m, 1024, "bf16", stream=s)), want)


def test_missing_or_small_workspace_is_refused():
    layer, acts = synth.dense_w8a8_int8(m=200, n=512, k=8192, seed=1)
    p, buf = layers.prepare_layer(layer)
    x, xs = layers.acts_to_dev(acts)
    need = qg.workspace_bytes(p, 200)
    assert need > 0
    y = torch.full((200, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    for ws in (None, torch.empty(need - 16, dtype=torch.uint8, device="cuda")):
        with pytest.raises(qg.QGError) as e:
            qg.gemm(p, x, xs, y, 200, ws)
        assert e.value.status == 5
    torch.cuda.synchronize()
    assert torch.isnan(y).all()


def test_no_rows():
    layer, acts = synth.dense_w8a8_int8(m=1, n=64, k=128, seed=1)
    p, buf = layers.prepare_layer(layer)
    x, xs = layers.acts_to_dev(acts)
    y = torch.full((1, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    qg.gemm(p, x, xs, y, 0)
    i = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    qg.moe_gemm(p, x, xs, i, i, i, 0, 1, 16, y)
    codes, scale = torch.full((1, 64), 7, dtype=torch.int8, device="cuda"), torch.full((1,), 7.0, device="cuda")
    qg.quantize_int8_rows(y, 0, 64, qg.A_BF16, codes, scale)
    qg.moe_swiglu(y, 0, 32, qg.O_BF16, qg.A_INT8, codes, scale)
    torch.cuda.synchronize()
    assert torch.isnan(y).all() and (codes == 7).all() and (scale == 7).all()


def test_two_streams_at_once():
    # two products in flight together, each with its own workspace and outputs
    layer, acts = synth.dense_w8a8_int8(m=200, n=1024, k=8192, seed=12)
    p, buf = layers.prepare_layer(layer)
    x, xs = layers.acts_to_dev(acts)
    want = _want(acts.x, acts.x_scale, layer.w[0], layer.s[0, :, 0], "bf16")
    need = max(qg.workspace_bytes(p, 64), qg.workspace_bytes(p, 200))
    assert need > 0
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    ys = [[torch.full((m, 1024), float("nan"), dtype=torch.bfloat16, device="cuda") for m in (64, 200)] for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s_, w_, y_ in zip(streams, ws, ys):
            for m, y in zip((64, 200), y_):
                qg.gemm(p, x, xs, y, m, w_, stream=s_)
    torch.cuda.synchronize()
    for y_ in ys:
        for m, y in zip((64, 200), y_):
            assert np.array_equal(_got(y), want[:m])


# ---- grouped ---------------------------------------------------------------------------------

def _align(ids, experts, bm, topk=None):
    t, k = ids.shape
    cs, cb = qg.moe_capacity(t, k, experts, bm)
    out = [torch.full((z,), -7, dtype=torch.int32, device="cuda") for z in (cs, cb, 1)]
    qg.moe_align(torch.from_numpy(np.ascontiguousarray(ids, np.int32)).cuda(), t, k, experts, bm, *out)
    return out


@pytest.mark.parametrize("bm", [4, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("t,n,k,out", [(1, 64, 128, "bf16"), (70, 320, 1408, "f16"), (600, 192, 640, "bf16")])
def test_grouped_is_exact_for_every_block(bm, t, n, k, out):
    experts, topk = 7, 3
    layer, acts = synth.moe_w8a8_int8(t=t, experts=experts, topk=topk, n=n, k=k, out=out, seed=t + bm)
    ids = acts.topk_ids.copy()
    ids[ids == 5] = 2                        # an expert without rows, another with the same token twice
    if t > 10:
        ids[3] = -1                          # a token routed nowhere
        ids[4, 1] = experts                  # a slot out of range
    p, buf = layers.prepare_layer(layer)
    x, xs = layers.acts_to_dev(acts)
    y = torch.full((t * topk, n), float("nan"), dtype=T_DTYPE[out], device="cuda")
    qg.moe_gemm(p, x, xs, *_align(ids, experts, bm), t, topk, bm, y)
    torch.cuda.synchronize()
    got = _got(y).reshape(t, topk, n)
    for e in range(experts):
        tt, jj = np.nonzero(ids == e)
        want = _want(acts.x[tt], acts.x_scale[tt], layer.w[e], layer.s[e, :, 0], out)
        assert np.array_equal(got[tt, jj], want), f"expert {e}"
    out_of = (ids < 0) | (ids >= experts)
    assert torch.isnan(y.view(t, topk, n)[torch.from_numpy(out_of)]).all()          # left as they were


@pytest.mark.parametrize("flag", [0, qg.C_BATCH_INVARIANT])
@pytest.mark.parametrize("t", [1, 9, 64, 500, 2000])
def test_grouped_with_the_chosen_block(t, flag):
    experts, topk, n, k = 16, 4, 256, 512
    layer, acts = synth.moe_w8a8_int8(t=t, experts=experts, topk=topk, n=n, k=k, seed=t)
    p, buf = layers.prepare_layer(layer, compute_flags=flag)
    bm = qg.moe_block_m(p, t, topk)
    x, xs = layers.acts_to_dev(acts)
    y = torch.full((t * topk, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    qg.moe_gemm(p, x, xs, *_align(acts.topk_ids, experts, bm), t, topk, bm, y)
    torch.cuda.synchronize()
    got = _got(y).reshape(t, topk, n)
    for e in range(experts):
        tt, jj = np.nonzero(acts.topk_ids == e)
        assert np.array_equal(got[tt, jj], _want(acts.x[tt], acts.x_scale[tt], layer.w[e], layer.s[e, :, 0], "bf16"))


@pytest.mark.parametrize("t,bm", [(1, 4), (9, 4), (100, 16), (100, 32), (1000, 32), (250, 64), (1000, 64), (1000, 128)])
def test_grouped_weights_beyond_the_caches(t, bm):
    # 115 MB of weights: loads past the caches and through them, 32 and 64 columns per workgroup
    experts, topk, n, k = 40, 4, 2816, 1024
    gen = torch.Generator(device="cuda").manual_seed(t + bm)
    w = torch.randint(-127, 128, (experts, n, k), generator=gen, device="cuda", dtype=torch.int8)
    sw = torch.rand((experts, n, 1), generator=gen, device="cuda") * 1e-3
    desc = qg.make_desc(qg.W_INT8, qg.S_F32, 0, 0, qg.A_INT8, qg.C_NATIVE, qg.O_BF16, experts, n, k)
    img = torch.empty(qg.prepared_bytes(desc), dtype=torch.uint8, device="cuda")
    p = qg.prepare(desc, w, sw, None, img)
    x = torch.randint(-127, 128, (t, k), generator=gen, device="cuda", dtype=torch.int8)
    xs = torch.rand(t, generator=gen, device="cuda") + 0.5
    ids = np.stack([np.random.default_rng(i).permutation(experts)[:topk] for i in range(t)]).astype(np.int32)
    y = torch.full((t * topk, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    qg.moe_gemm(p, x, xs, *_align(ids, experts, bm), t, topk, bm, y)
    torch.cuda.synchronize()
    got = _got(y).reshape(t, topk, n)
    for e in (0, 7, 23, 39) if t > 1 else ids[0]:
        tt, jj = np.nonzero(ids == e)
        want = _want(x.cpu().numpy()[tt], xs.cpu().numpy()[tt], w[e].cpu().numpy(), sw[e, :, 0].cpu().numpy(), "bf16")
        assert np.array_equal(got[tt, jj], want), e
    assert not torch.isnan(y).any()


def test_grouped_with_more_blocks_than_a_grid_axis():
    # 4.2 million rows of narrow experts: the chosen block is one that fits, a smaller one is refused
    experts, topk, n, k, t = 8, 8, 64, 4096, 524_200
    layer, _ = synth.moe_w8a8_int8(t=1, experts=experts, topk=topk, n=n, k=k, seed=3)
    p, buf = layers.prepare_layer(layer)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(-127, 128, (t, k), generator=gen, device="cuda", dtype=torch.int8)
    xs = torch.rand(t, generator=gen, device="cuda") + 0.5
    ids = np.tile(np.arange(experts, dtype=np.int32), (t, 1))
    y = torch.full((t * topk, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    bm = qg.moe_block_m(p, t, topk)
    qg.moe_gemm(p, x, xs, *_align(ids, experts, bm), t, topk, bm, y)
    torch.cuda.synchronize()
    rows = torch.tensor([0, 1, t // 2, t - 1], device="cuda")
    got = _got(y.view(t, topk, n)[rows])
    for e in range(experts):
        want = _want(x[rows].cpu().numpy(), xs[rows].cpu().numpy(), layer.w[e], layer.s[e, :, 0], "bf16")
        assert np.array_equal(got[:, e], want)
    few = torch.empty(16, dtype=torch.int32, device="cuda")
    with pytest.raises(qg.QGError) as err:
        qg.moe_gemm(p, x, xs, few, few, few, t, topk, 16, y)
    assert err.value.status == 2


def test_grouped_contiguous_rows():
    experts, n, k, rows = 4, 128, 256, 150
    layer, acts = synth.moe_w8a8_int8(t=rows, experts=experts, topk=1, n=n, k=k, seed=8)
    offs = np.array([0, 40, 40, 131, 140], np.int32)                    # rows 140.. belong to no expert
    p, buf = layers.prepare_layer(layer)
    cs, cb = qg.moe_capacity(rows, 1, experts, 32)
    m = [torch.empty(z, dtype=torch.int32, device="cuda") for z in (cs, cb, 1)]
    qg.moe_grouped_map(qg.MOE_CONTIGUOUS, torch.from_numpy(offs).cuda(), experts, rows, 0, 32, *m)
    x, xs = layers.acts_to_dev(acts)
    y = torch.full((rows, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    qg.moe_gemm(p, x, xs, *m, rows, 1, 32, y)
    torch.cuda.synchronize()
    for e in range(experts):
        r = slice(offs[e], offs[e + 1])
        assert np.array_equal(_got(y)[r], _want(acts.x[r], acts.x_scale[r], layer.w[e], layer.s[e, :, 0], "bf16"))
    assert torch.isnan(y[140:]).all()


# ---- quantizers ------------------------------------------------------------------------------

def _dev16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda()


def _quant_gpu(x, rows, k, call):
    codes = torch.full((rows + 1, k), 77, dtype=torch.int8, device="cuda")
    scale = torch.full((rows + 1,), 77.0, dtype=torch.float32, device="cuda")
    call(x, codes, scale)
    torch.cuda.synchronize()
    assert (codes[rows] == 77).all() and scale[rows] == 77.0               # nothing behind the last row
    return codes[:rows].cpu().numpy(), scale[:rows].cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,k", [(1, 8), (3, 504), (37, 1408), (5, 2048), (6, 2056), (9, 4096), (3, 7168), (4, 8192),
                                    (3, 8200), (2, 28672), (2, 32768), (1030, 64)])
def test_quantize_int8_rows_is_bit_exact(rows, k, dtype):
    bits, _ = synth.act_rows(rows, k, dtype, sigma=3.0, seed=rows + k)
    bits = bits.copy()
    to = synth.f32_to_bf16_bits if dtype == "bf16" else synth.f32_to_f16_bits
    if rows > 2:
        bits[1] = 0                                                         # an all-zero row
        bits[2] = to(np.resize(np.array([127, 0.5, 1.5, 2.5, -0.5, -126.5, 63.5, 1e-3], np.float32), k))   # halves
    if rows > 3:
        bits[3] = to(np.resize(np.array([2, 1, -1, 1.9921875, 6e-8, 0], np.float32), k))     # half of the largest
    if rows > 4:
        bits[4] = 1                                                         # the smallest subnormal number
    if rows > 5:
        bits[5, 0] = to(np.array([6e4], np.float32))[0]
    codes, scale = _quant_gpu(_dev16(bits), rows, k, lambda x, c, s: qg.quantize_int8_rows(x, rows, k, Q_ACT[dtype], c, s))
    rc, rs = Q.absmax_int8_rows(F.decode_act(bits, dtype).astype(np.float32))
    assert np.array_equal(scale.view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(codes, rc), f"{np.count_nonzero(codes != rc)} codes differ"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_int8_rows_over_the_whole_range(dtype):
    # every finite value up to a row's largest, for largest values over the whole range: subnormal, ordinary,
    # near the type's largest, with scales that float32 rounds either way
    rng = np.random.default_rng(7)
    top = 0x7F80 if dtype == "bf16" else 0x7C00                             # first bits that are not finite
    tops = np.concatenate([rng.integers(1, top, 90), [1, 2, 126, 127, 128, top - 1, top - 2, top // 2]])
    k = 32768
    rows = len(tops)
    bits = np.empty((rows, k), np.uint16)
    for r, t in enumerate(tops):
        near = rng.integers(max(0, int(t) - 9 * 128), int(t) + 1, k)         # the last few octaves: codes that are not 0
        bits[r] = np.where(rng.random(k) < 0.7, near, rng.integers(0, int(t) + 1, k)) | (rng.integers(0, 2, k) << 15)
        bits[r, int(t) % k] = t
    codes, scale = _quant_gpu(_dev16(bits), rows, k, lambda x, c, s: qg.quantize_int8_rows(x, rows, k, Q_ACT[dtype], c, s))
    rc, rs = Q.absmax_int8_rows(F.decode_act(bits, dtype).astype(np.float32))
    assert np.array_equal(scale.view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(codes, rc), f"{np.count_nonzero(codes != rc)} codes differ, rows {np.unique(np.nonzero(codes != rc)[0])}"


@pytest.mark.parametrize("rows,inter,dtype", [(6, 64, "bf16"), (11, 1408, "bf16"), (3, 8192, "f16"), (2, 16384, "bf16")])
def test_swiglu_int8_is_bit_exact_on_exact_activations(rows, inter, dtype):
    # gate = 32: silu(32) rounds to 32 in float32 and from float64, so act = 32 * up on both sides
    v = synth.gate_up_values(rows, inter, dtype, seed=inter).copy()
    v[:, :inter] = 0x4200 if dtype == "bf16" else 0x5000
    v[1, inter:] = 0
    codes, scale = _quant_gpu(_dev16(v), rows, inter,
                              lambda x, c, s: qg.moe_swiglu(x, rows, inter, Q_OUT[dtype], qg.A_INT8, c, s))
    _, rc, rs = ML.swiglu_int8(F.decode_act(v, dtype))
    assert np.array_equal(scale.view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(codes, rc)


@pytest.mark.parametrize("rows,inter,dtype", [(1, 8, "bf16"), (64, 1408, "bf16"), (33, 2056, "f16"), (2, 32768, "bf16")])
def test_swiglu_int8(rows, inter, dtype):
    v = synth.gate_up_values(rows, inter, dtype, seed=rows + inter)
    codes, scale = _quant_gpu(_dev16(v), rows, inter,
                              lambda x, c, s: qg.moe_swiglu(x, rows, inter, Q_OUT[dtype], qg.A_INT8, c, s))
    act, _, rs = ML.swiglu_int8(F.decode_act(v, dtype))
    assert np.all(np.abs(scale - rs) <= 2.0 ** -20 * rs)
    step = scale.astype(np.float64)[:, None]
    # half a code, the quotient's own rounding (127 * 2^-24 of a code) and the float32 activation
    bound = (0.5 + 2.0 ** -17) * step + 2.0 ** -16 * np.abs(act)
    assert np.all(np.abs(codes * step - act) <= bound)


def test_more_rows_than_one_launch_takes():
    # 2^21 rows a launch: the last rows of the first and the rows of the second against the first ones' results
    rows, k = (1 << 21) + 70, 16
    bits, _ = synth.act_rows(1000, k, "bf16", sigma=3.0, seed=1)
    x = _dev16(bits).repeat((rows + 999) // 1000, 1)[:rows].contiguous()
    rc, rs = Q.absmax_int8_rows(F.decode_act(bits, "bf16").astype(np.float32))
    codes = torch.full((rows + 1, k), 77, dtype=torch.int8, device="cuda")
    scale = torch.full((rows + 1,), 77.0, device="cuda")
    qg.quantize_int8_rows(x, rows, k, qg.A_BF16, codes, scale)
    torch.cuda.synchronize()
    reps = (rows + 999) // 1000
    assert torch.equal(codes[:rows], torch.from_numpy(rc).cuda().repeat(reps, 1)[:rows]) and (codes[rows] == 77).all()
    assert torch.equal(scale[:rows], torch.from_numpy(rs).cuda().repeat(reps)[:rows]) and scale[rows] == 77
    act = torch.full((rows + 1, 8), 77, dtype=torch.int8, device="cuda")
    first = torch.empty((1000, 8), dtype=torch.int8, device="cuda")
    qg.moe_swiglu(x, 1000, 8, qg.O_BF16, qg.A_INT8, first, torch.empty(1000, device="cuda"))
    qg.moe_swiglu(x, rows, 8, qg.O_BF16, qg.A_INT8, act, scale)
    torch.cuda.synchronize()
    assert torch.equal(act[:rows], first.repeat(reps, 1)[:rows]) and (act[rows] == 77).all()


# ---- sizes past 32 bits ------------------------------------------------------------------------

def test_outputs_past_2_31_elements():
    m, n, k = 1_060_000, 2048, 256                                       # 2.17e9 outputs
    layer, _ = synth.dense_w8a8_int8(m=1, n=n, k=k, seed=4)
    p, buf = layers.prepare_layer(layer)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-127, 128, (m, k), generator=gen, device="cuda", dtype=torch.int8)
    xs = torch.rand(m, generator=gen, device="cuda") + 0.5
    y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    qg.gemm(p, x, xs, y, m)
    torch.cuda.synchronize()
    rows = torch.tensor([0, 1, 524_287, 1_048_575, 1_048_576, 1_048_577, m - 257, m - 1])
    want = _want(x[rows.cuda()].cpu().numpy(), xs[rows.cuda()].cpu().numpy(), layer.w[0], layer.s[0, :, 0], "bf16")
    assert np.array_equal(_got(y[rows.cuda()]), want)


@pytest.mark.parametrize("bm", [16, 128])
def test_expert_weights_past_2_32_bytes(bm):
    experts, n, k, t = 40, 7168, 16384, 40                                # 4.7e9 bytes
    gen = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randint(-127, 128, (experts, n, k), generator=gen, device="cuda", dtype=torch.int8)
    sw = torch.rand((experts, n, 1), generator=gen, device="cuda") * 1e-4
    desc = qg.make_desc(qg.W_INT8, qg.S_F32, 0, 0, qg.A_INT8, qg.C_NATIVE, qg.O_BF16, experts, n, k)
    img = torch.empty(qg.prepared_bytes(desc), dtype=torch.uint8, device="cuda")
    p = qg.prepare(desc, w, sw, None, img)
    x = torch.randint(-127, 128, (t, k), generator=gen, device="cuda", dtype=torch.int8)
    xs = torch.rand(t, generator=gen, device="cuda") + 0.5
    ids = np.arange(t, dtype=np.int32).reshape(t, 1) % experts
    y = torch.empty((t, n), dtype=torch.bfloat16, device="cuda")
    qg.moe_gemm(p, x, xs, *_align(ids, experts, bm), t, 1, bm, y)
    torch.cuda.synchronize()
    for e in (0, 18, 36, 37, 39):                                         # 36 * n * k < 2^32 < 37 * n * k
        want = _want(x[e:e + 1].cpu().numpy(), xs[e:e + 1].cpu().numpy(), w[e].cpu().numpy(), sw[e, :, 0].cpu().numpy(), "bf16")
        assert np.array_equal(_got(y[e:e + 1]), want), e


def test_quantized_rows_past_2_31_elements():
    rows, k = 66_000, 32768                                               # 2.16e9 values
    bits, _ = synth.act_rows(500, k, "bf16", sigma=3.0, seed=9)
    x = _dev16(bits).repeat(rows // 500, 1)
    codes = torch.empty((rows, k), dtype=torch.int8, device="cuda")
    scale = torch.empty(rows, device="cuda")
    qg.quantize_int8_rows(x, rows, k, qg.A_BF16, codes, scale)
    torch.cuda.synchronize()
    rc, rs = Q.absmax_int8_rows(F.decode_bf16(bits).astype(np.float32))
    for first in (0, 65_000, 65_500):                                     # 65536 * k = 2^31
        assert np.array_equal(codes[first:first + 500].cpu().numpy(), rc)
        assert np.array_equal(scale[first:first + 500].cpu().numpy(), rs)


# ---- a whole layer -----------------------------------------------------------------------------

def _layer_buffers(t, topk, experts, up, down, pu, pd):
    rows, inter = t * topk, down.k
    bm, bd = qg.moe_block_m(pu, t, topk), qg.moe_block_m(pd, rows, 1)
    e = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device="cuda")    # noqa: E731
    b = dict(bm=bm, bd=bd, ids=e(t, topk), w=e(t, topk, dtype=torch.float32), xq=e(t, up.k, dtype=torch.int8),
             xs=e(t, dtype=torch.float32), y1=e(rows, 2 * inter, dtype=torch.bfloat16), aq=e(rows, inter, dtype=torch.int8),
             asc=e(rows, dtype=torch.float32), y2=e(rows, down.n, dtype=torch.bfloat16),
             out=e(t, down.n, dtype=torch.bfloat16))
    b["map"] = [e(z) for z in (*qg.moe_capacity(t, topk, experts, bm), 1)]
    b["map2"] = b["map"] if bd == bm else [e(z) for z in (*qg.moe_capacity(t, topk, experts, bd), 1)]
    return b


def _layer(desc, logits, bias, x16, up, down, pu, pd, b, t, topk, experts, stream=None):
    """Router -> sort -> int8 rows -> gate/up -> SwiGLU to int8 -> down -> weighted sum."""
    rows, inter = t * topk, down.k
    qg.moe_route(desc, logits, qg.L_F32, t, b["ids"], b["w"], bias, stream=stream)
    qg.moe_align(b["ids"], t, topk, experts, b["bm"], *b["map"], stream=stream)
    if b["bd"] != b["bm"]:
        qg.moe_align(b["ids"], t, topk, experts, b["bd"], *b["map2"], stream=stream)
    qg.quantize_int8_rows(x16, t, up.k, qg.A_BF16, b["xq"], b["xs"], stream=stream)
    qg.moe_gemm(pu, b["xq"], b["xs"], *b["map"], t, topk, b["bm"], b["y1"], stream=stream)
    qg.moe_swiglu(b["y1"], rows, inter, qg.O_BF16, qg.A_INT8, b["aq"], b["asc"], stream=stream)
    qg.moe_gemm(pd, b["aq"], b["asc"], *b["map2"], rows, 1, b["bd"], b["y2"], stream=stream)
    qg.moe_combine(b["y2"], b["w"], b["ids"], t, topk, experts, down.n, qg.O_BF16, b["out"], stream=stream)


def _layer_inputs(t, experts, topk, hidden, inter, seed):
    up, acts = synth.moe_w8a8_int8(t=t, experts=experts, topk=topk, n=2 * inter, k=hidden, seed=seed)
    down, _ = synth.moe_w8a8_int8(t=1, experts=experts, topk=1, n=hidden, k=inter, seed=seed + 100)
    x16, _ = synth.act_rows(t, hidden, "bf16", sigma=1.0, seed=seed)
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((t, experts)).astype(np.float32)
    bias = (rng.standard_normal(experts) * 0.1).astype(np.float32)
    return up, down, x16, logits, bias


def _layer_reference(up, down, x16, logits, bias, topk, kw):
    """The layer in float64 with the two int8 quantizations and the bfloat16 gate/up rows as stored."""
    ids, w = RT.route(logits, "sigmoid", topk, bias=bias, **kw)
    xq, xs = Q.absmax_int8_rows(F.decode_bf16(x16).astype(np.float32))
    y1 = Q.round_to_bf16(np.nan_to_num(R.moe_reference(up, synth.Acts(xq, xs, ids))))
    t = ids.shape[0]
    _, aq, asc = ML.swiglu_int8(y1.reshape(t * topk, -1))
    y2 = ML.down_reference(down, aq.astype(np.float64).reshape(t, topk, -1), ids, asc)
    return ids, ML.combine(np.nan_to_num(y2), w, ids, up.experts)


ROUTE = dict(groups=4, topk_groups=2, group_top=2, renorm=True, scale=1.5)


@pytest.mark.parametrize("t", [1, 33, 300, 1100])
def test_int8_layer_from_logits(t):
    # What the reference leaves out: y2 rounded to bfloat16 before the weighted sum (2^-8 of each
    # term), the output's rounding (2^-8), and codes of SwiGLU that the float32 sigmoid moves across
    # a half: rare, one code (1/127 of a row's largest activation) of one of `inter` terms each.
    # The first two are below 2^-8 * (1 + sum of |terms| / |out|); rows sum topk = 4 terms, so 2e-2 of the
    # largest output holds them with the third.
    experts, topk, hidden, inter = 16, 4, 512, 256
    up, down, x16, logits, bias = _layer_inputs(t, experts, topk, hidden, inter, t)
    logits[0, 3] = -np.inf
    if t > 5:
        logits[4] = np.nan                                       # a token that no expert takes
        logits[5, 4:] = -np.inf                                  # one with four experts left, of one group
    pu, b1 = layers.prepare_layer(up)
    pd, b2 = layers.prepare_layer(down)
    desc = qg.make_route_desc(qg.R_SIGMOID, experts, topk, 4, 2, 2, True, 1.5)
    b = _layer_buffers(t, topk, experts, up, down, pu, pd)
    _layer(desc, torch.from_numpy(logits).cuda(), torch.from_numpy(bias).cuda(), _dev16(x16), up, down, pu, pd, b, t, topk,
           experts)
    torch.cuda.synchronize()
    ids, ref = _layer_reference(up, down, x16, logits, bias, topk, ROUTE)
    assert np.array_equal(b["ids"].cpu().numpy(), ids)
    got = layers.out_bits_to_f64(b["out"])
    assert R.relative_error(got, ref) <= 2e-2
    if t > 5:
        assert np.all(got[4] == 0)


def test_int8_layer_captured_and_replayed():
    t, experts, topk, hidden, inter = 40, 16, 4, 512, 256
    up, down, x16, logits, bias = _layer_inputs(t, experts, topk, hidden, inter, 5)
    pu, b1 = layers.prepare_layer(up)
    pd, b2 = layers.prepare_layer(down)
    desc = qg.make_route_desc(qg.R_SIGMOID, experts, topk, 4, 2, 2, True, 1.5)
    b = _layer_buffers(t, topk, experts, up, down, pu, pd)
    eager = _layer_buffers(t, topk, experts, up, down, pu, pd)
    lg, bs, xd = torch.from_numpy(logits).cuda(), torch.from_numpy(bias).cuda(), _dev16(x16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _layer(desc, lg, bs, xd, up, down, pu, pd, b, t, topk, experts, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        _layer(desc, lg, bs, xd, up, down, pu, pd, b, t, topk, experts, stream=s)
    for k in range(4):
        lg.copy_(torch.from_numpy(np.roll(logits, k, axis=1).copy()))
        xd.copy_(_dev16(np.roll(x16, k, axis=0)))
        _layer(desc, lg, bs, xd, up, down, pu, pd, eager, t, topk, experts)
        b["out"].fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for name in ("ids", "w", "out"):
            assert torch.equal(b[name], eager[name]), (k, name)


@pytest.mark.parametrize("m,k", [(64, 4096), (200, 4096), (200, 8192)])
def test_two_captured_products_replayed_with_their_own_workspaces(m, k):
    layer, acts = synth.dense_w8a8_int8(m=m, n=1024, k=k, seed=9)
    p, buf = layers.prepare_layer(layer)
    x, xs = layers.acts_to_dev(acts)
    need = qg.workspace_bytes(p, m)
    graphs, s = [], torch.cuda.Stream()
    for i in range(2):
        xi = torch.roll(x, i, 0).contiguous()
        xsi = torch.roll(xs, i, 0).contiguous()
        y = torch.empty((m, 1024), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        qg.gemm(p, xi, xsi, y, m, ws, stream=s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            qg.gemm(p, xi, xsi, y, m, ws, stream=s)
        graphs.append((g, y, xi, xsi, ws))
    want = _want(acts.x, acts.x_scale, layer.w[0], layer.s[0, :, 0], "bf16")
    for _ in range(3):
        for g, y, *_ in graphs:
            y.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, *_ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i, (_, y, *_) in enumerate(graphs):
            assert np.array_equal(_got(y), np.roll(want, i, axis=0))
