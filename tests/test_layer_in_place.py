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
