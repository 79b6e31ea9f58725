"""Pins of the references of norms, adapters, the 4-bit cache and attention, and the host-side refusals of their entry
points (no GPU)."""
import ctypes

import numpy as np
import pytest

import quantized_gemm_amd as qg
from oracle import layer_ops as LO

FAKE = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4104)       # not 16-byte aligned


# ---- references ----------------------------------------------------------------------------

def test_norm_worked_example():
    # mean square of (1, 1, 1, 7) is 13, of u - mean (-1.5, -1.5, -1.5, 4.5) 6.75
    v = np.array([[1.0, 1.0, 1.0, 7.0]])
    u, z, _, _ = LO.norm_rows(res=v, kind="rms", eps=3.0)
    assert np.allclose(z, v / 4.0) and np.array_equal(u, v)
    _, z, _, _ = LO.norm_rows(res=v, kind="layer", eps=2.25, weight=np.array([1.0, 1, 1, 2]), bias=np.array([0.0, 0, 1, 0]),
                              offset=1.0)
    assert np.allclose(z, [[-1.0, -1.0, 0.0, 4.5]])
    u, z, _, _ = LO.norm_rows(y=v, res=np.full((1, 4), 2.0), kind="", post="rms", eps=3.0, gate=np.array([0.0, 4, 4, 4]),
                              res_scale=0.5)
    assert z is None and np.allclose(u, [[2.0, 2.5, 2.5, 5.5]])


def test_lora_worked_example():
    x = np.array([[1.0, 2.0], [3.0, 1.0], [1.0, 1.0]])
    a = np.array([[[[1.0, 1.0], [9.0, 9.0]]], [[[0.0, 1.0], [1.0, 0.0]]]])     # [2 adapters][1][2][2]
    b = np.array([[[1.0, 9.0], [2.0, 9.0]], [[1.0, 0.0], [1.0, 1.0]]])         # [2][2 columns][2]
    out, mag = LO.lora(x, a, b, [0, 1, -1], [1, 2], [2.0, 1.0], np.zeros((3, 2)), [2])
    # adapter 0 has rank 1: t = 3; adapter 1: t = (1, 3)
    assert out.tolist() == [[6.0, 12.0], [1.0, 4.0], [0.0, 0.0]] and (mag >= np.abs(out)).all()


def test_attention_worked_example():
    k = [np.zeros((3, 1, 2))]
    v = [np.array([[[1.0, 0.0]], [[3.0, 0.0]], [[5.0, 6.0]]])]
    out, _ = LO.attention(np.ones((2, 1, 2)), k, v, [3], [2], 1.0)
    assert np.allclose(out[:, 0], [[2.0, 0.0], [3.0, 2.0]])                    # the first of the two sees two tokens
    out, _ = LO.attention(np.ones((2, 1, 2)), [k[0][:1]], [v[0][:1]], [1], [2], 1.0)
    assert np.allclose(out[:, 0], [[0.0, 0.0], [1.0, 0.0]])                    # the first sees none
    out, _ = LO.attention(np.ones((2, 1, 2)), k, v, [3], [2], 1.0, seen=[np.array([True, False, True])])
    assert np.allclose(out[:, 0], [[1.0, 0.0], [3.0, 3.0]])


def test_mxfp4_values_worked_example():
    x = np.zeros((1, 64))
    x[0, :3] = 7.0, -2.6, 0.2          # exponent 0: 6 (the largest code), -3, 0
    x[0, 40] = np.inf
    v = LO.mxfp4_values(x)
    assert v[0, :3].tolist() == [6.0, -3.0, 0.0] and np.isnan(v[0, 32:]).all() and not v[0, 3:32].any()


# ---- refusals --------------------------------------------------------------------------------

def _norm(desc=None, rows=4, y=FAKE, res=FAKE, res_out=FAKE, gate=None, post_weight=None, weight=FAKE, bias=None, out=FAKE,
          codes=None, scale=None, **kw):
    d = dict(norm=qg.N_RMS, type=qg.O_BF16, k=64, eps=1e-6)
    d.update(kw)
    return qg.lib().qg_norm_rows(ctypes.byref(qg.make_norm_desc(**d)) if desc is None else desc, rows, y, res, res_out, gate,
                                 post_weight, weight, bias, out, codes, scale, None)


def test_norm_rows_rejects_on_the_host():
    assert _norm(rows=0) == 0                                                   # no rows: no-op
    assert qg.lib().qg_norm_rows(None, 1, *[FAKE] * 10, None) == 1
    for kw in (dict(rows=-1), dict(norm=3), dict(norm=-1), dict(post_norm=3), dict(type=7), dict(res_type=9), dict(code_type=1),
               dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(weight_offset=float("nan")),
               dict(res_scale=float("inf")), dict(k=0), dict(y_stride=56), dict(y_stride=68), dict(res_stride=60),
               dict(out_stride=32), dict(gate_stride=32),
               dict(y=None, res=None), dict(res_out=None, out=None), dict(y=None, gate=FAKE), dict(y=None, post_norm=1),
               dict(y=None, post_weight=FAKE), dict(post_weight=FAKE), dict(norm=0), dict(norm=0, weight=None),
               dict(norm=0, weight=None, out=None, bias=FAKE), dict(codes=FAKE, scale=FAKE), dict(code_type=qg.A_INT8),
               dict(code_type=qg.A_INT8, codes=FAKE), dict(code_type=qg.A_INT8, codes=FAKE, scale=ctypes.c_void_p(4098)),
               dict(y=ODD), dict(res=ODD), dict(res_out=ODD), dict(gate=ODD), dict(weight=ODD), dict(bias=ODD), dict(out=ODD),
               dict(post_norm=1, post_weight=ODD), dict(code_type=qg.A_INT8, codes=ODD, scale=FAKE)):
        assert _norm(**kw) == 1, kw
    for kw in (dict(k=60), dict(k=32776), dict(k=40, code_type=qg.A_FP4_E2M1, codes=FAKE, scale=FAKE),
               dict(res_type=qg.L_F16), dict(type=qg.O_F16, res_type=qg.L_BF16), dict(rows=2 ** 31)):
        assert _norm(**kw) == 2, kw


def _lora(tokens=4, block=16, ptrs=None, ws_bytes=1 << 30, **kw):
    d = dict(type=qg.O_BF16, num_adapters=3, max_rank=16, k=64, slice_ends=[64])
    d.update(kw)
    p = dict(x=FAKE, a=FAKE, b=FAKE, ranks=None, scales=None, sorted=FAKE, experts=FAKE, pad=FAKE, base=FAKE, y=FAKE, ws=FAKE)
    p.update(ptrs or {})
    return qg.lib().qg_lora(ctypes.byref(qg.make_lora_desc(**d)), p["x"], p["a"], p["b"], p["ranks"], p["scales"], p["sorted"],
                            p["experts"], p["pad"], tokens, block, p["base"], p["y"], p["ws"], ws_bytes, None)


def test_lora_rejects_on_the_host():
    assert _lora(tokens=0) == 0
    assert qg.lib().qg_lora(None, *[FAKE] * 8, 4, 16, FAKE, FAKE, FAKE, 1 << 20, None) == 1
    for kw in (dict(tokens=-1), dict(type=9), dict(num_adapters=0), dict(max_rank=0), dict(k=0), dict(slice_ends=[]),
               dict(slice_ends=[0]), dict(slice_ends=[64, 64]), dict(slice_ends=[96, 64]), dict(x_stride=56), dict(y_stride=60),
               dict(base_stride=100)):
        assert _lora(**kw) == 1, kw
    d = qg.make_lora_desc(qg.O_BF16, 3, 16, 64, [64, 128])
    d.slice_end[1] = 120                                                        # the last slice ends at n
    assert qg.lora_workspace_bytes(d, 4, 16) == 0
    for name in ("x", "a", "b", "sorted", "experts", "pad", "base", "y"):
        assert _lora(ptrs={name: None}) == 1, name
    for name in ("x", "a", "b", "base", "y"):
        assert _lora(ptrs={name: ODD}) == 1, name
    for name in ("ranks", "scales", "sorted", "experts", "pad"):
        assert _lora(ptrs={name: ctypes.c_void_p(4098)}) == 1, name
    for kw in (dict(block=32), dict(num_adapters=513), dict(max_rank=264), dict(max_rank=12), dict(k=60), dict(slice_ends=[60]),
               dict(slice_ends=[40, 64]), dict(slice_ends=list(range(32, 320, 32))), dict(tokens=(1 << 24) + 1)):
        assert _lora(**kw) == 2, kw
    need = qg.lora_workspace_bytes(qg.make_lora_desc(qg.O_BF16, 3, 16, 64, [64]), 4, 16)
    assert need > 0 and _lora(ws_bytes=need - 1) == 5 and _lora(ptrs={"ws": None}) == 5 and _lora(ptrs={"ws": ODD}) == 5
    assert qg.lora_block_m(1, 8) == 16 and qg.lora_block_m(1024, 8) == 64 and qg.lora_block_m(4096, 8) == 128 and qg.lora_block_m(-1, 8) == 0
    assert qg.lora_block_m(4, 0) == 0


def test_kv_and_attention_reject_on_the_host():
    good = dict(type=qg.O_BF16, kv_heads=2, head_dim=64, page_tokens=16, num_pages=3)

    def desc(**kw):
        return ctypes.byref(qg.make_kv_desc(**dict(good, **kw)))

    # codes and exponents of keys and values: head_dim + head_dim / 16 bytes per token and head
    assert qg.kv_cache_bytes(qg.make_kv_desc(**good)) == 3 * 2 * 16 * (64 + 4)
    bad1 = (dict(type=5), dict(kv_heads=0), dict(num_pages=0), dict(page_tokens=0))
    bad2 = (dict(head_dim=96), dict(page_tokens=8), dict(page_tokens=48), dict(page_tokens=512), dict(kv_heads=1025),
            dict(num_pages=1 << 27))
    lib = qg.lib()
    for status, kws in ((1, bad1), (2, bad2)):
        for kw in kws:
            assert lib.qg_kv_append(desc(**kw), FAKE, 0, FAKE, 0, FAKE, 4, FAKE, None) == status, kw
            assert lib.qg_kv_read(desc(**kw), FAKE, FAKE, 4, FAKE, FAKE, None) == status, kw
            assert lib.qg_attention(desc(**kw), FAKE, 0, 4, FAKE, FAKE, 4, FAKE, None, 1, 1, 1, 64, 1.0, FAKE, 0, FAKE, 1 << 30,
                                    None) == status, kw
            assert qg.kv_cache_bytes(qg.make_kv_desc(**dict(good, **kw))) == 0
    assert lib.qg_kv_append(desc(), FAKE, 0, FAKE, 0, FAKE, 0, FAKE, None) == 0
    assert lib.qg_kv_read(desc(), FAKE, FAKE, 0, FAKE, FAKE, None) == 0
    for args in ((FAKE, 120, FAKE, 0, FAKE, 4, FAKE), (FAKE, 0, FAKE, 132, FAKE, 4, FAKE), (FAKE, 0, FAKE, 0, FAKE, -1, FAKE),
                 (None, 0, FAKE, 0, FAKE, 4, FAKE), (FAKE, 0, None, 0, FAKE, 4, FAKE), (FAKE, 0, FAKE, 0, None, 4, FAKE),
                 (FAKE, 0, FAKE, 0, FAKE, 4, None), (ODD, 0, FAKE, 0, FAKE, 4, FAKE), (FAKE, 0, ODD, 0, FAKE, 4, FAKE),
                 (FAKE, 0, FAKE, 0, FAKE, 4, ODD), (FAKE, 0, FAKE, 0, ctypes.c_void_p(4098), 4, FAKE)):
        assert lib.qg_kv_append(desc(), *args, None) == 1, args
    for args in ((FAKE, FAKE, -1, FAKE, FAKE), (None, FAKE, 4, FAKE, FAKE), (FAKE, None, 4, FAKE, FAKE), (FAKE, FAKE, 4, None, FAKE),
                 (FAKE, FAKE, 4, FAKE, ODD)):
        assert lib.qg_kv_read(desc(), *args, None) == 1, args

    def attn(**kw):
        p = dict(d=desc(), q=FAKE, q_stride=0, heads=4, cache=FAKE, table=FAKE, table_stride=4, lens=FAKE, offs=None, batch=2,
                 max_q=1, tokens=2, max_len=64, scale=0.125, out=FAKE, out_stride=0, ws=FAKE, ws_bytes=1 << 30)
        p.update(kw)
        return lib.qg_attention(p["d"], p["q"], p["q_stride"], p["heads"], p["cache"], p["table"], p["table_stride"], p["lens"],
                                p["offs"], p["batch"], p["max_q"], p["tokens"], p["max_len"], p["scale"], p["out"],
                                p["out_stride"], p["ws"], p["ws_bytes"], None)

    assert attn(batch=0, tokens=0) == 0 and attn(offs=FAKE, tokens=0) == 0
    for kw in (dict(heads=3), dict(heads=0), dict(batch=-1), dict(max_q=0), dict(tokens=-1), dict(max_len=-1), dict(q_stride=248),
               dict(out_stride=260), dict(scale=float("nan")), dict(scale=float("inf")), dict(table_stride=3), dict(max_q=2),
               dict(tokens=3), dict(q=None), dict(out=None), dict(cache=None), dict(lens=None), dict(table=None), dict(q=ODD),
               dict(out=ODD), dict(cache=ODD), dict(table=ctypes.c_void_p(4098)), dict(lens=ctypes.c_void_p(4098)),
               dict(offs=ctypes.c_void_p(4098)), dict(d=None)):
        assert attn(**kw) == 1, kw
    for kw in (dict(heads=2 * 257), dict(batch=65536, tokens=65536), dict(offs=FAKE, tokens=(1 << 24) + 1)):
        assert attn(**kw) == 2, kw
    long = dict(max_len=4096, table_stride=256)
    need = qg.attention_workspace_bytes(qg.make_kv_desc(**dict(good)), 4, 2, 1, 2, 4096)
    assert need > 0
    assert attn(ws_bytes=need - 1, **long) == 5 and attn(ws=None, **long) == 5 and attn(ws=ODD, **long) == 5
    assert qg.attention_workspace_bytes(qg.make_kv_desc(**good), 3, 2, 1, 2, 4096) == 0


@pytest.mark.parametrize("batch,max_q,max_len", [(1, 1, 32768), (64, 1, 8192), (4, 512, 4608), (300, 1, 100)])
def test_attention_workspace_holds_whole_splits(batch, max_q, max_len):
    for dim in (64, 128, 256):
        d = qg.make_kv_desc(qg.O_F16, 2, dim, 16, 1 << 20)
        need = qg.attention_workspace_bytes(d, 8, batch, max_q, batch * max_q, max_len)
        one = batch * max_q * 8 * (dim + 2) * 4
        assert need % one == 0 and need // one != 1


def test_sizes_beyond_64_bits_are_refused():
    lib = qg.lib()
    far = qg.make_kv_desc(qg.O_BF16, 1, 64, 256, 1 << 60)
    assert qg.kv_cache_bytes(far) == 0
    assert lib.qg_kv_append(ctypes.byref(far), FAKE, 0, FAKE, 0, FAKE, 4, FAKE, None) == 2
    d = qg.make_kv_desc(qg.O_BF16, 1, 64, 16, 4)

    def attn(table_stride, scale):
        return lib.qg_attention(ctypes.byref(d), FAKE, 0, 1, FAKE, FAKE, table_stride, FAKE, None, 1, 1, 1, 64, scale, FAKE, 0, FAKE,
                                1 << 30, None)

    assert attn((1 << 60) + 4, 1.0) == 1                            # rows of the table that 64 bits of bytes do not hold
    assert attn(4, 3e38) == 1 and attn(4, -3e38) == 1               # (infinite in powers of two)
    lora = qg.make_lora_desc(qg.O_BF16, 2, 16, 64, [64])
    assert qg.lora_workspace_bytes(lora, 1 << 24, 16) > 0
    assert qg.lora_workspace_bytes(lora, (1 << 24) + 1, 16) == 0 and qg.lora_workspace_bytes(lora, 1 << 62, 64) == 0
    assert lib.qg_lora(ctypes.byref(lora), FAKE, FAKE, FAKE, None, None, FAKE, FAKE, FAKE, 1 << 62, 16, FAKE, FAKE, FAKE, 1 << 62,
                       None) == 2
