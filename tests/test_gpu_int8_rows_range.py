"""Rows quantized to int8, SwiGLU among them, over the whole range of their inputs and outside it.

Bars, from the arithmetic.  Gates below -86 take exp(g / 4) four times as a factor.  One such factor is 2^x with
x = fl(fl(g / 4) log2 e): a half step of x, the 2^-26 by which the float32 constant is off times x (each times ln 2), and a
unit of the hardware's 2^x.  For |g| <= 88.7, x < 32: 0.69 (2^-20 + 32 * 2^-26) + 2^-23 = 1.12e-6; four of them
and five products (2^-24 each) 4.8e-6 < 2^-17.  For |g| <= 348, x < 126: 4 * (0.69 (2^-18 + 126 * 2^-26) + 2^-23) + 5 * 2^-24
= 1.65e-5 < 2^-15.  Gates from -86 up take exp(-g) once, x < 125: 0.69 (2^-18 + 125 * 2^-26) + 2^-23, and a reciprocal and
three roundings more: 4.4e-6 < 2^-17.  A result below 2^-126 is off by half a step of 2^-149 more.  Scales carry
the largest activation's error, a rounding (2^-24, below 2^-126 half a step) and the oracle's own of its input.
"""
import numpy as np
import pytest
import torch

import quantized_gemm_amd as qg
from quantized_gemm_amd import layers, synth
from oracle import formats as F
from oracle import moe_layer as ML
from oracle import quant as Q

pytestmark = pytest.mark.gpu

Q_OUT = {"bf16": qg.O_BF16, "f16": qg.O_F16}
TO = {"bf16": synth.f32_to_bf16_bits, "f16": synth.f32_to_f16_bits}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    qg.lib()
    yield


def _swiglu(bits, inter, dtype):
    rows = bits.shape[0]
    codes = torch.full((rows, inter), 77, dtype=torch.int8, device="cuda")
    scale = torch.full((rows,), 77.0, dtype=torch.float32, device="cuda")
    x = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda()
    qg.moe_swiglu(x, rows, inter, Q_OUT[dtype], qg.A_INT8, codes, scale)
    torch.cuda.synchronize()
    return codes.cpu().numpy(), scale.cpu().numpy()


def _check(gate, up, dtype, u):
    """u: the activations' relative error."""
    inter = gate.shape[1]
    bits = np.concatenate([TO[dtype](gate.astype(np.float32)), TO[dtype](up.astype(np.float32))], axis=1)
    codes, scale = _swiglu(bits, inter, dtype)
    act, _, rs = ML.swiglu_int8(F.decode_act(bits, dtype))
    assert np.all(np.abs(scale.astype(np.float64) - rs) <= (u + 2 * 2.0 ** -24) * rs + 2 * 2.0 ** -149)
    step = scale.astype(np.float64)[:, None]
    # half a code, the quotient's own rounding (127 * 2^-24 of a code), and the activation's error
    assert np.all(np.abs(codes * step - act) <= (0.5 + 2.0 ** -17) * step + u * np.abs(act) + 2.0 ** -149)
    # a row with an activation to represent uses the whole range of codes
    some = np.abs(act).max(1) > 2.0 ** -118
    assert some.any() and np.all(np.abs(codes[some]).max(1) == 127)


# a wave, 256 and 1024 threads per row
@pytest.mark.parametrize("inter", [64, 1408, 4096, 16384])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("low,high", [(-88.5, -87.5), (-87.25, -86.0), (-88.0, -80.0), (-86.0, 20.0)])
def test_rows_of_very_negative_gates(low, high, dtype, inter):
    rng = np.random.default_rng(inter)
    gate = rng.uniform(low, high, (5, inter))
    _check(gate, rng.standard_normal((5, inter)) * 3, dtype, 2.0 ** -17)


@pytest.mark.parametrize("low,high", [(-104.0, -88.0), (-150.0, -100.0), (-170.0, -86.0)])
def test_gates_below_float32_sigmoids_with_large_ups(low, high):
    # sigmoid(-150) is 2^-216, below every float32, and the activation with an up of 2^120 is 2^-89
    rng = np.random.default_rng(1)
    gate = rng.uniform(low, high, (6, 1408))
    up = np.ldexp(rng.uniform(0.5, 1, gate.shape), 120) * rng.choice([-1, 1], gate.shape)
    _check(gate, up, "bf16", 2.0 ** -15)


def test_the_most_negative_gates_give_zeros():
    # one ordinary activation per row; beside it gates whose activation is below every code
    gate = np.full((4, 256), -3e38)
    gate[1], gate[2], gate[3] = -360.0, -1000.0, -89.0
    up = np.full((4, 256), 2.0)
    gate[:, 7], up[:, 7] = 3.0, -5.0
    inter = 256
    bits = np.concatenate([TO["bf16"](gate.astype(np.float32)), TO["bf16"](up.astype(np.float32))], axis=1)
    codes, scale = _swiglu(bits, inter, "bf16")
    want = np.zeros((4, 256), np.int8)
    want[:, 7] = -127
    assert np.array_equal(codes, want) and np.all(np.isfinite(scale)) and np.all(scale > 0)


# ---- rows that hold something that is not finite -----------------------------------------------
# They have no scale: it is NaN and the codes are 0, so that every output of such a row's product is NaN.

BAD = [float("nan"), float("inf"), -float("inf")]


def _finite_but(rows, k, seed, at):
    """Normal rows; at: {row: (column, value)}."""
    v = (np.random.default_rng(seed).standard_normal((rows, k)) * 3).astype(np.float32)
    for r, (c, x) in at.items():
        v[r, c] = x
    return v


def _same(codes, scale, rc, rs, bad):
    assert np.isnan(scale[bad]).all() and (codes[bad] == 0).all()
    good = np.setdiff1d(np.arange(len(scale)), bad)
    assert np.array_equal(scale[good].view(np.uint32), rs[good].view(np.uint32)) and np.array_equal(codes[good], rc[good])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("k", [8, 504, 2048, 2056, 7168, 8200, 32768])
def test_quantized_rows_that_are_not_finite(k, dtype):
    # every position of a row lies on some thread's first or last piece
    at = {1: (0, BAD[0]), 2: (k - 1, BAD[0]), 3: (k // 2, BAD[1]), 4: (k - 1, BAD[2]), 6: (5, -float("nan")), 9: (k // 3, BAD[1])}
    v = _finite_but(11, k, k, at)
    v[8] = 0
    v[8, 3] = np.inf                                                       # nothing else in the row
    v[7] = np.nan
    bits = TO[dtype](v)
    x = torch.from_numpy(bits.view(np.int16)).cuda()
    codes = torch.full((11, k), 77, dtype=torch.int8, device="cuda")
    scale = torch.full((11,), 77.0, device="cuda")
    qg.quantize_int8_rows(x, 11, k, {"bf16": qg.A_BF16, "f16": qg.A_F16}[dtype], codes, scale)
    torch.cuda.synchronize()
    rc, rs = Q.absmax_int8_rows(F.decode_act(bits, dtype).astype(np.float32))
    bad = np.array([1, 2, 3, 4, 6, 7, 8, 9])
    assert np.array_equal(np.nonzero(np.isnan(rs))[0], bad)
    _same(codes.cpu().numpy(), scale.cpu().numpy(), rc, rs, bad)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("inter", [64, 1408, 4096, 16384])
def test_swiglu_rows_that_are_not_finite(inter, dtype):
    # in a gate, in an up, an up of infinity beside a gate that gives 0, a product past float32 (bf16 only)
    gate, up = np.full((10, inter), 32.0, np.float32), _finite_but(10, inter, inter, {})
    gate[1, 0], gate[2, inter - 1], gate[3, 7] = BAD
    up[4, 1], up[5, inter // 2], up[6, inter - 2] = BAD
    gate[7, 9], up[7, 9] = -60000.0, np.inf
    bad = [1, 2, 3, 4, 5, 6, 7]
    if dtype == "bf16":
        gate[8, 3], up[8, 3] = 1e30, 1e30
        bad.append(8)
    bits = np.concatenate([TO[dtype](gate), TO[dtype](up)], axis=1)
    codes, scale = _swiglu(bits, inter, dtype)
    with np.errstate(all="ignore"):
        _, rc, rs = ML.swiglu_int8(F.decode_act(bits, dtype))
    _same(codes, scale, rc, rs, np.array(bad))


@pytest.mark.parametrize("out", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [(5, 192, 512), (40, 192, 512), (700, 512, 640), (200, 512, 8192), (300, 4160, 2048)])
def test_a_product_of_such_rows_is_nan_in_them_alone(m, n, k, out):
    layer, acts = synth.dense_w8a8_int8(m=1, n=n, k=k, out=out, seed=m)
    p, buf = layers.prepare_layer(layer)
    bad = np.unique([1, m // 2, m - 1])
    v = _finite_but(m, k, m, {int(r): (int(r) % k, BAD[i % 3]) for i, r in enumerate(bad)})
    x = torch.from_numpy(TO["bf16"](v).view(np.int16)).cuda()
    codes, scale = torch.empty((m, k), dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    qg.quantize_int8_rows(x, m, k, qg.A_BF16, codes, scale)
    y = torch.full((m, n), 7.0, dtype={"bf16": torch.bfloat16, "f16": torch.float16}[out], device="cuda")
    need = qg.workspace_bytes(p, m)
    qg.gemm(p, codes, scale, y, m, torch.empty(need, dtype=torch.uint8, device="cuda") if need else None)
    torch.cuda.synchronize()
    nan = torch.isnan(y).cpu().numpy()
    assert nan[bad].all() and not np.delete(nan, bad, axis=0).any()
