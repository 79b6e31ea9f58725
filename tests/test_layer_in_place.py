"""Outputs in an input's place whose rows lie elsewhere are refused on the host (no GPU): a row would be overwritten before
it is read."""
import ctypes

import quantized_gemm_amd as qg

A, B, C = (ctypes.c_void_p(4096 * i) for i in (1, 2, 3))


def _norm(y, res, res_out, out, **kw):
    d = qg.make_norm_desc(qg.N_RMS, kw.pop("type", qg.O_BF16), 64, 1e-6, **kw)
    return qg.lib().qg_norm_rows(ctypes.byref(d), 4, y, res, res_out, None, None, None, None, out, None, None, None)


def test_norm_in_place_has_the_inputs_rows():
    for args, kw in (((A, B, B, A), dict(y_stride=128)), ((A, B, C, A), dict(out_stride=72)), ((None, B, None, B), dict(res_stride=72)),
                     ((None, B, None, B), dict(out_stride=128)), ((None, B, None, B), dict(res_type=qg.L_F32)),
                     ((A, B, A, None), dict(res_type=qg.L_F32)), ((A, B, A, None), dict(y_stride=128)), ((A, B, C, C), {})):
        assert _norm(*args, **kw) == 1, (args, kw)


def test_adapters_in_place_have_the_bases_rows():
    for kw in (dict(base_stride=72), dict(y_stride=72), dict(base_stride=128, y_stride=72)):
        d = qg.make_lora_desc(qg.O_BF16, 3, 16, 64, [64], **kw)
        for block in (16, 64):
            assert qg.lib().qg_lora(ctypes.byref(d), A, A, A, None, None, A, A, A, 4, block, B, B, C, 1 << 30, None) == 1
