"""SwiGLU to int8 over the whole range of its inputs.

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
from quantized_gemm_amd import synth
from oracle import formats as F
from oracle import moe_layer as ML

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
