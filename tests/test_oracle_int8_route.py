"""Pins of the int8 and routing references, and the host-side refusals of their entry points (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import quantized_gemm_amd as qg
from quantized_gemm_amd import layers, synth
from oracle import layout as L
from oracle import quant as Q
from oracle import reference as R
from oracle import route as RT


# ---- references ----------------------------------------------------------------------------

def test_absmax_int8_rows_worked_example():
    # 127 / 127 = 1: the codes are the values, halves go to the even integer
    x = np.array([[127.0, 0.5, 1.5, -2.5, -126.5, 63.5], [0.0] * 6, [-2.0, 1.0, 0, 0, 0, 0]], np.float32)
    codes, scale = Q.absmax_int8_rows(x)
    assert codes[0].tolist() == [127, 0, 2, -2, -126, 64] and scale[0] == 1.0
    assert codes[1].tolist() == [0] * 6 and scale[1] == 1.0
    assert codes[2, 0] == -127 and scale[2] == np.float32(2.0) / np.float32(127.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_absmax_int8_rows_decides_as_exact_arithmetic(dtype):
    # away from exact halves (2 * 127 * x an odd multiple of the largest value) the float32 quotient
    # rounds to the code that integer arithmetic gives: the nearest other quotient is at least
    # 1 / (2 * 2^11) of a code away from a half, float32 is 127 * 2^-23 off at most
    t = torch.bfloat16 if dtype == "bf16" else torch.float16
    x = torch.from_numpy(np.random.default_rng(3).standard_normal((200, 512)).astype(np.float32)).to(t)
    codes, _ = Q.absmax_int8_rows(x.float().numpy())
    unit = 2.0 ** -24 if dtype == "f16" else 2.0 ** -40
    v = np.round(x.double().numpy() / unit).astype(object)          # exact integers
    v = np.vectorize(int, otypes=[object])(v)
    amax = np.abs(v).max(axis=1)[:, None]
    num = 254 * v                                                    # code = v * 127 / amax = num / (2 amax)
    half = np.vectorize(lambda a, b: a % (2 * b) == b, otypes=[bool])(num, amax + 0 * v)
    want = np.vectorize(lambda a, b: (a + b) // (2 * b), otypes=[int])(num, amax + 0 * v)
    assert np.array_equal(codes[~half], want[~half]) and (~half).mean() > 0.99


def test_layout_round_trip_int8():
    layer, _ = synth.moe_w8a8_int8(t=2, experts=3, topk=2, n=64, k=256, seed=1)
    w, s, z = L.unpack(L.repack(layer), "int8", "int8", "f32", 64, 256, 0, 3, False)
    assert w.dtype == np.int8 and np.array_equal(w, layer.w) and np.array_equal(s, layer.s) and z is None
    sz = L.sizes("int8", "f32", 64, 256, 0, 3, False)
    assert qg.prepared_bytes(layers.desc_for(layer)) == sz["total"]


def test_dense_reference_int8_is_the_scaled_integer_product():
    layer, acts = synth.dense_w8a8_int8(m=5, n=64, k=256, seed=2)
    y = R.dense_reference(layer, acts)
    p = acts.x.astype(np.int64) @ layer.w[0].astype(np.int64).T
    want = p * layer.s[0, :, 0].astype(np.float64)[None, :] * acts.x_scale.astype(np.float64)[:, None]
    # the reference scales before it multiplies: two products rounded per term, K additions
    assert np.all(np.abs(y - want) <= (256 + 4) * 2.0 ** -53 * (np.abs(acts.x.astype(np.float64)) @
                  np.abs(layer.w[0].astype(np.float64)).T) * layer.s[0, :, 0][None, :] * acts.x_scale[:, None])


def test_route_worked_example():
    l = np.array([0.0, 2.0, 2.0, -1.0, 1.0, -np.inf, np.nan, 3.0])
    ids, w = RT.route_token(l, "softmax", 4)
    assert ids.tolist() == [7, 1, 2, 4]
    p = np.exp([0, 2, 2, -1, 1, 3.0])
    assert np.allclose(w, np.exp([3, 2, 2, 1.0]) / p.sum(), rtol=1e-14)
    ids, w = RT.route_token(l, "softmax", 8, renorm=True, scale=2.0)
    assert ids.tolist() == [7, 1, 2, 4, 0, 3, -1, -1] and abs(w.sum() - 2.0) < 1e-14 and w[6] == w[7] == 0
    # a bias decides the choice and leaves the weights alone
    b = np.zeros(8)
    b[3] = 10.0
    ids, w = RT.route_token(l, "sigmoid", 2, bias=b)
    assert ids.tolist() == [3, 7] and np.allclose(w, 1 / (1 + np.exp([1.0, -3.0])), rtol=1e-14)
    # groups {0,1} {2,3} {4,5} {6,7}: best values 2, 2, 1, 3 keep the last and (a tie) the first
    assert RT.route_token(l, "softmax", 3, groups=4, topk_groups=2)[0].tolist() == [7, 1, 0]
    # nothing eligible
    ids, w = RT.route_token(np.full(4, -np.inf), "softmax", 2, renorm=True)
    assert ids.tolist() == [-1, -1] and w.tolist() == [0, 0]
    # +inf is the largest finite value: a tie between two of them
    ids, w = RT.route_token(np.array([0, np.inf, np.inf, 1.0]), "softmax", 2)
    assert ids.tolist() == [1, 2] and w.tolist() == [0.5, 0.5]


def test_route_group_sums_of_two():
    # group 0 has the best single choice, group 1 the best two together
    l = np.log(np.array([9.0, 0.25, 4.0, 4.0]))                # sigmoid: 0.9, 0.2, 0.8, 0.8
    assert RT.route_token(l, "sigmoid", 1, groups=2, topk_groups=1, group_top=1)[0].tolist() == [0]
    assert RT.route_token(l, "sigmoid", 1, groups=2, topk_groups=1, group_top=2)[0].tolist() == [2]


def test_route_agrees_with_torch_where_it_can():
    l = np.random.default_rng(0).standard_normal((50, 40))
    ids, w = RT.route(l, "softmax", 6, renorm=True)
    p, i = torch.topk(torch.softmax(torch.from_numpy(l), 1), 6, dim=1)
    assert np.array_equal(ids, i.numpy().astype(np.int32))
    assert np.allclose(w, (p / p.sum(1, keepdim=True)).numpy(), rtol=1e-13)


# ---- refusals on the host --------------------------------------------------------------------

def _desc(**kw):
    base = dict(w_type=qg.W_INT8, s_type=qg.S_F32, group_k=0, has_zero=0, a_type=qg.A_INT8, compute=qg.C_NATIVE,
                out_type=qg.O_BF16, num_experts=1, n=512, k=1024)
    base.update(kw)
    return qg.make_desc(**base)


def test_int8_descriptions():
    assert qg.prepared_bytes(_desc()) == 512 * 1024 + 512 * 4
    assert qg.prepared_bytes(_desc(out_type=qg.O_F16)) > 0
    assert qg.prepared_bytes(_desc(compute=qg.C_BATCH_INVARIANT)) == qg.prepared_bytes(_desc())
    assert qg.prepared_bytes(_desc(k=131072 - 128)) > 0          # sums below 2^31
    for kw in (dict(k=131072), dict(s_type=qg.S_BF16), dict(group_k=128), dict(has_zero=1), dict(a_type=qg.A_FP8_E4M3),
               dict(a_type=qg.A_BF16), dict(compute=qg.C_W_TO_FP8), dict(n=100), dict(k=1000), dict(w_type=6),
               dict(a_type=6), dict(w_type=qg.W_FP8_E4M3), dict(w_type=qg.W_FP4_E2M1, s_type=qg.S_UE8M0, group_k=32),
               dict(w_type=qg.W_INT4, s_type=qg.S_BF16, group_k=128)):
        assert qg.prepared_bytes(_desc(**kw)) == 0, kw


def test_int8_products_reject_on_the_host():
    lib = qg.lib()
    fake = ctypes.c_void_p(4096)
    p = qg.Prepared()
    p.magic, p.layout_version, p.gfx_arch, p.desc, p.dev = 0x31504751, 1, 950, _desc(), 4096
    p.bytes = qg.prepared_bytes(p.desc)
    assert lib.qg_gemm(ctypes.byref(p), fake, None, fake, 4, None, 0, None) == 1         # token scales missing
    assert lib.qg_gemm(ctypes.byref(p), fake, fake, fake, 1 << 21, None, 0, None) == 2   # 2^31 activation bytes
    assert lib.qg_gemm(ctypes.byref(p), fake, fake, fake, 0, None, 0, None) == 0
    assert lib.qg_moe_gemm(ctypes.byref(p), fake, None, fake, fake, fake, 4, 2, 16, fake, None, 0, None) == 1
    assert lib.qg_moe_gemm(ctypes.byref(p), fake, fake, fake, fake, fake, 4, 2, 48, fake, None, 0, None) == 2


def test_int8_quantizers_reject_on_the_host():
    lib = qg.lib()
    fake = ctypes.c_void_p(4096)
    q = lib.qg_quantize_int8_rows
    assert q(fake, 0, 64, qg.A_BF16, fake, fake, None) == 0
    assert q(fake, -1, 64, qg.A_BF16, fake, fake, None) == 1
    assert q(fake, 4, 64, qg.A_INT8, fake, fake, None) == 1
    assert q(fake, 4, 60, qg.A_BF16, fake, fake, None) == 2
    assert q(fake, 4, 32776, qg.A_BF16, fake, fake, None) == 2
    assert q(fake, 4, 64, qg.A_BF16, None, fake, None) == 1
    assert q(fake, 4, 64, qg.A_BF16, fake, None, None) == 1
    assert q(ctypes.c_void_p(4100), 4, 64, qg.A_BF16, fake, fake, None) == 1
    assert q(fake, 4, 64, qg.A_BF16, ctypes.c_void_p(4100), fake, None) == 1             # codes 8-byte aligned
    assert q(fake, 4, 64, qg.A_BF16, fake, ctypes.c_void_p(4098), None) == 1
    s = lib.qg_moe_swiglu
    assert s(fake, 4, 64, qg.O_BF16, qg.A_INT8, fake, None, None) == 1                   # scales missing
    assert s(fake, 4, 64, qg.O_BF16, qg.A_INT8, fake, ctypes.c_void_p(4098), None) == 1
    assert s(fake, 4, 32776, qg.O_BF16, qg.A_INT8, fake, fake, None) == 2


def _route(tokens=4, stride=None, logits=4096, bias=None, ids=4096, weights=4096, in_type=qg.L_F32, **kw):
    d = dict(scoring=qg.R_SOFTMAX, num_experts=64, topk=4)
    d.update(kw)
    desc = qg.make_route_desc(**d)
    return qg.lib().qg_moe_route(ctypes.byref(desc), logits, in_type, desc.num_experts if stride is None else stride, bias,
                                 tokens, ids, weights, None)


def test_route_rejects_on_the_host():
    assert _route(tokens=0) == 0
    assert _route(tokens=0, logits=None, ids=None, weights=None) == 0
    assert qg.lib().qg_moe_route(None, 4096, qg.L_F32, 64, None, 4, 4096, 4096, None) == 1
    for kw in (dict(tokens=-1), dict(scoring=0), dict(scoring=3), dict(in_type=0), dict(in_type=4), dict(num_experts=0),
               dict(topk=0), dict(topk=65), dict(num_groups=0), dict(num_groups=3), dict(num_groups=4, topk_groups=5),
               dict(topk_groups=0), dict(topk_groups=2), dict(num_groups=32, topk_groups=1), dict(group_top=0),
               dict(group_top=3), dict(renormalize=2), dict(stride=63), dict(stride=-64), dict(logits=None), dict(ids=None),
               dict(weights=None), dict(logits=4098), dict(ids=4098), dict(weights=4098), dict(bias=4098),
               dict(logits=4097, in_type=qg.L_BF16)):
        assert _route(**kw) == 1, kw
    for kw in (dict(num_experts=513), dict(num_experts=512, topk=65),
               dict(num_experts=130, num_groups=65, topk_groups=65), dict(tokens=1 << 29), dict(stride=1 << 31)):
        assert _route(**kw) == 2, kw
