"""Python binding of libqg.so, the MI355X (gfx950) quantized GEMM library.

Argument marshalling only: torch tensors supply device pointers, torch's current
stream supplies the hipStream_t, and every step of the computation runs in the
library's HIP kernels.  The entry points mirror include/qg.h one to one:
``prepared_bytes``, ``prepare``, ``workspace_bytes``, ``gemm``, ``moe_block_m``,
``moe_capacity``, ``moe_align``, ``moe_grouped_map``, ``moe_gemm``, ``moe_swiglu``,
``moe_combine``, ``moe_route``, ``quantize_e4m3_rows``, ``quantize_int8_rows``,
``quantize_e2m1_rows``, ``norm_rows``, ``lora_block_m``, ``lora_workspace_bytes``, ``lora``, ``kv_cache_bytes``,
``kv_append``, ``kv_read``, ``attention_workspace_bytes``, ``attention``, ``dequant``, ``status_str``, ``version`` and the measurement helpers
``ceiling_read`` and ``ceiling_mfma``.

There is no fallback: if libqg.so is missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqg.so")

# Enumerations (values as in include/qg.h).
W_INT4, W_UINT4, W_FP4_E2M1, W_FP8_E4M3, W_INT8 = 1, 2, 3, 4, 5
S_F16, S_BF16, S_F32, S_UE8M0 = 1, 2, 3, 4
A_F16, A_BF16, A_FP8_E4M3, A_FP4_E2M1, A_INT8 = 1, 2, 3, 4, 5
O_F16, O_BF16 = 1, 2
C_NATIVE, C_W_TO_FP8, C_BATCH_INVARIANT = 0, 1, 4
MOE_CONTIGUOUS, MOE_MASKED = 1, 2
R_SOFTMAX, R_SIGMOID = 1, 2
L_F16, L_BF16, L_F32 = 1, 2, 3
N_RMS, N_LAYER = 1, 2

STATUS = {0: "QG_OK", 1: "QG_ERR_INVALID_ARG", 2: "QG_ERR_UNSUPPORTED", 3: "QG_ERR_ARCH_MISMATCH",
          4: "QG_ERR_NOT_PREPARED", 5: "QG_ERR_WORKSPACE", 6: "QG_ERR_CAPACITY", 7: "QG_ERR_HIP"}
EXPORTS = ["qg_prepared_bytes", "qg_prepare", "qg_workspace_bytes", "qg_gemm", "qg_moe_block_m", "qg_moe_capacity",
           "qg_moe_align", "qg_moe_grouped_map", "qg_moe_gemm", "qg_moe_swiglu", "qg_moe_combine",
           "qg_quantize_e4m3_rows", "qg_quantize_int8_rows", "qg_quantize_e2m1_rows", "qg_moe_route", "qg_norm_rows",
           "qg_lora_block_m", "qg_lora_workspace_bytes", "qg_lora", "qg_kv_cache_bytes", "qg_kv_append", "qg_kv_read",
           "qg_attention_workspace_bytes", "qg_attention", "qg_dequant",
           "qg_ceiling_read", "qg_ceiling_mfma", "qg_ceiling_lds",
           "qg_gemm_noalloc", "qg_noalloc_scratch_bytes",
           "qg_status_str", "qg_version"]


class QGError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({_status_text(status)})")


class LayerDesc(ctypes.Structure):
    _fields_ = [("w_type", ctypes.c_int32), ("s_type", ctypes.c_int32), ("group_k", ctypes.c_int32),
                ("has_zero", ctypes.c_int32), ("a_type", ctypes.c_int32), ("compute", ctypes.c_int32),
                ("out_type", ctypes.c_int32), ("num_experts", ctypes.c_int32), ("n", ctypes.c_int64),
                ("k", ctypes.c_int64)]


class RouteDesc(ctypes.Structure):
    _fields_ = [("scoring", ctypes.c_int32), ("num_experts", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("num_groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("weight_scale", ctypes.c_float)]


class NormDesc(ctypes.Structure):
    _fields_ = [("norm", ctypes.c_int32), ("post_norm", ctypes.c_int32), ("type", ctypes.c_int32),
                ("res_type", ctypes.c_int32), ("code_type", ctypes.c_int32), ("eps", ctypes.c_float),
                ("weight_offset", ctypes.c_float), ("res_scale", ctypes.c_float), ("k", ctypes.c_int64),
                ("y_stride", ctypes.c_int64), ("res_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
                ("gate_stride", ctypes.c_int64)]


class LoraDesc(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("num_adapters", ctypes.c_int32), ("max_rank", ctypes.c_int32),
                ("num_slices", ctypes.c_int32), ("n", ctypes.c_int64), ("k", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("base_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64), ("slice_end", ctypes.c_int64 * 8)]


class KvDesc(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("num_pages", ctypes.c_int64)]


class Prepared(ctypes.Structure):
    _fields_ = [("magic", ctypes.c_uint32), ("layout_version", ctypes.c_uint32), ("gfx_arch", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32), ("desc", LayerDesc), ("dev", ctypes.c_void_p),
                ("bytes", ctypes.c_uint64), ("off_w", ctypes.c_uint64), ("off_s", ctypes.c_uint64),
                ("off_z", ctypes.c_uint64), ("w_expert_bytes", ctypes.c_uint64), ("s_expert_bytes", ctypes.c_uint64),
                ("z_expert_bytes", ctypes.c_uint64)]


_lib = None


def lib():
    """Load libqg.so (built in-tree by quantized_gemm_amd.build); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} not found: build it with `python -m quantized_gemm_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        pd, pp = ctypes.POINTER(LayerDesc), ctypes.POINTER(Prepared)
        L.qg_prepared_bytes.argtypes, L.qg_prepared_bytes.restype = [pd], sz
        L.qg_prepare.argtypes, L.qg_prepare.restype = [pd, vp, vp, vp, vp, sz, pp, vp], i32
        L.qg_workspace_bytes.argtypes, L.qg_workspace_bytes.restype = [pp, i64, i32], sz
        L.qg_gemm.argtypes, L.qg_gemm.restype = [pp, vp, vp, vp, i64, vp, sz, vp], i32
        L.qg_moe_block_m.argtypes, L.qg_moe_block_m.restype = [pp, i64, i32], i32
        L.qg_moe_capacity.argtypes = [i64, i32, i32, i32, ctypes.POINTER(i64), ctypes.POINTER(i64)]
        L.qg_moe_capacity.restype = i32
        L.qg_moe_align.argtypes = [vp, i64, i32, i32, i32, vp, i64, vp, i64, vp, vp]
        L.qg_moe_align.restype = i32
        L.qg_moe_grouped_map.argtypes = [i32, vp, i32, i64, i64, i32, vp, i64, vp, i64, vp, vp]
        L.qg_moe_grouped_map.restype = i32
        L.qg_moe_gemm.argtypes = [pp, vp, vp, vp, vp, vp, i64, i32, i32, vp, vp, sz, vp]
        L.qg_moe_gemm.restype = i32
        L.qg_moe_swiglu.argtypes, L.qg_moe_swiglu.restype = [vp, i64, i64, i32, i32, vp, vp, vp], i32
        L.qg_moe_combine.argtypes = [vp, vp, vp, i64, i32, i32, i64, i32, vp, vp]
        L.qg_moe_combine.restype = i32
        L.qg_quantize_e4m3_rows.argtypes = [vp, i64, i64, i32, vp, vp, vp]
        L.qg_quantize_e2m1_rows.argtypes, L.qg_quantize_e2m1_rows.restype = [vp, i64, i64, i32, vp, vp, vp], i32
        L.qg_quantize_e4m3_rows.restype = i32
        L.qg_quantize_int8_rows.argtypes, L.qg_quantize_int8_rows.restype = [vp, i64, i64, i32, vp, vp, vp], i32
        L.qg_moe_route.argtypes = [ctypes.POINTER(RouteDesc), vp, i32, i64, vp, i64, vp, vp, vp]
        L.qg_moe_route.restype = i32
        f32 = ctypes.c_float
        pn, pl, pk = ctypes.POINTER(NormDesc), ctypes.POINTER(LoraDesc), ctypes.POINTER(KvDesc)
        L.qg_norm_rows.argtypes, L.qg_norm_rows.restype = [pn, i64] + [vp] * 11, i32
        L.qg_lora_block_m.argtypes, L.qg_lora_block_m.restype = [i64, i32], i32
        L.qg_lora_workspace_bytes.argtypes, L.qg_lora_workspace_bytes.restype = [pl, i64, i32], sz
        L.qg_lora.argtypes = [pl] + [vp] * 8 + [i64, i32, vp, vp, vp, sz, vp]
        L.qg_lora.restype = i32
        L.qg_kv_cache_bytes.argtypes, L.qg_kv_cache_bytes.restype = [pk], sz
        L.qg_kv_append.argtypes, L.qg_kv_append.restype = [pk, vp, i64, vp, i64, vp, i64, vp, vp], i32
        L.qg_kv_read.argtypes, L.qg_kv_read.restype = [pk, vp, vp, i64, vp, vp, vp], i32
        L.qg_attention_workspace_bytes.argtypes = [pk, i32, i64, i64, i64, i64]
        L.qg_attention_workspace_bytes.restype = sz
        L.qg_attention.argtypes = [pk, vp, i64, i32, vp, vp, i64, vp, vp, i64, i64, i64, i64, f32, vp, i64, vp, sz, vp]
        L.qg_attention.restype = i32
        L.qg_dequant.argtypes, L.qg_dequant.restype = [pp, i32, vp, vp], i32
        u64 = ctypes.c_uint64
        L.qg_gemm_noalloc.argtypes, L.qg_gemm_noalloc.restype = [pp, vp, vp, vp, i64, vp], i32
        L.qg_noalloc_scratch_bytes.argtypes, L.qg_noalloc_scratch_bytes.restype = [], sz
        L.qg_ceiling_read.argtypes, L.qg_ceiling_read.restype = [vp, u64, i32, vp, u64, vp], i32
        L.qg_ceiling_mfma.argtypes, L.qg_ceiling_mfma.restype = [i32, i64, i32, vp, u64, vp], i32
        L.qg_ceiling_lds.argtypes, L.qg_ceiling_lds.restype = [i64, i32, vp, u64, vp], i32
        L.qg_status_str.argtypes, L.qg_status_str.restype = [i32], ctypes.c_char_p
        L.qg_version.argtypes, L.qg_version.restype = [], i32
        _lib = L
    return _lib


def _status_text(s: int) -> str:
    try:
        return lib().qg_status_str(s).decode()
    except Exception:  # library unavailable while formatting an error
        return "?"


def status_str(s: int) -> str:
    return lib().qg_status_str(s).decode()


def version() -> int:
    return lib().qg_version()


def _ptr(t):
    return None if t is None else t.data_ptr()


_torch_c = None


def _stream(stream):
    """The hipStream_t of a torch stream or of an address; None: torch's current stream of the current device."""
    global _torch_c
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if _torch_c is None:
        import torch
        torch.cuda.current_stream()      # initialises torch's side once; the raw lookups below need it
        _torch_c = torch._C
    # the address alone: a torch.cuda.Stream object costs more than the launch of a small kernel
    return _torch_c._cuda_getCurrentRawStream(_torch_c._cuda_getDevice())


def _check(status: int, where: str):
    if status != 0:
        raise QGError(status, where)


def make_desc(w_type, s_type, group_k, has_zero, a_type, compute, out_type, num_experts, n, k) -> LayerDesc:
    return LayerDesc(w_type, s_type, group_k, int(has_zero), a_type, compute, out_type, num_experts, n, k)


def prepared_bytes(desc: LayerDesc) -> int:
    return lib().qg_prepared_bytes(ctypes.byref(desc))


def prepare(desc: LayerDesc, w, scales, zeros, out, stream=None) -> Prepared:
    """Repack logical device tensors into ``out`` (a uint8 device tensor) and return the handle."""
    p = Prepared()
    st = lib().qg_prepare(ctypes.byref(desc), _ptr(w), _ptr(scales), _ptr(zeros), _ptr(out),
                          out.numel() * out.element_size(), ctypes.byref(p), _stream(stream))
    _check(st, "qg_prepare")
    return p


def workspace_bytes(p: Prepared, m_or_tokens: int, topk: int = 0) -> int:
    return lib().qg_workspace_bytes(ctypes.byref(p), m_or_tokens, topk)


def gemm(p: Prepared, x, x_scale, y, m: int, ws=None, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    st = lib().qg_gemm(ctypes.byref(p), _ptr(x), _ptr(x_scale), _ptr(y), m, _ptr(ws), ws_bytes, _stream(stream))
    _check(st, "qg_gemm")


def gemm_call(p: Prepared, x, x_scale, y, m: int, ws=None, stream=None):
    """qg_gemm with every argument converted once: returns a no-argument callable that enqueues
    the same launch again (for timing loops, where per-call tensor slicing and stream lookup
    would cost more host time than a small kernel takes on the GPU)."""
    fn = lib().qg_gemm
    args = (ctypes.byref(p), _ptr(x), _ptr(x_scale), _ptr(y), m, _ptr(ws),
            0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))

    def call():
        st = fn(*args)
        if st != 0:
            raise QGError(st, "qg_gemm")
    return call


def gemm_noalloc(p: Prepared, x, x_scale, y, m: int, stream=None):
    """qg_gemm with the library's own per-GPU scratch array as the workspace (no allocation)."""
    st = lib().qg_gemm_noalloc(ctypes.byref(p), _ptr(x), _ptr(x_scale), _ptr(y), m, _stream(stream))
    _check(st, "qg_gemm_noalloc")


def noalloc_scratch_bytes() -> int:
    return lib().qg_noalloc_scratch_bytes()


def moe_block_m(p: Prepared, tokens: int, topk: int) -> int:
    return lib().qg_moe_block_m(ctypes.byref(p), tokens, topk)


def moe_capacity(tokens: int, topk: int, num_experts: int, block_m: int):
    cs, cb = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().qg_moe_capacity(tokens, topk, num_experts, block_m, ctypes.byref(cs), ctypes.byref(cb)),
           "qg_moe_capacity")
    return cs.value, cb.value


def moe_align(topk_ids, tokens: int, topk: int, num_experts: int, block_m: int, sorted_ids, expert_ids,
              num_post_pad, stream=None):
    st = lib().qg_moe_align(_ptr(topk_ids), tokens, topk, num_experts, block_m, _ptr(sorted_ids), sorted_ids.numel(),
                            _ptr(expert_ids), expert_ids.numel(), _ptr(num_post_pad), _stream(stream))
    _check(st, "qg_moe_align")


def moe_grouped_map(layout: int, offsets_or_counts, num_experts: int, rows_total: int, rows_per_expert: int,
                    block_m: int, sorted_ids, expert_ids, num_post_pad, stream=None):
    """Block map of a grouped-contiguous (offsets [E+1]) or grouped-masked (counts [E]) MoE input."""
    st = lib().qg_moe_grouped_map(layout, _ptr(offsets_or_counts), num_experts, rows_total, rows_per_expert, block_m,
                                  _ptr(sorted_ids), sorted_ids.numel(), _ptr(expert_ids), expert_ids.numel(),
                                  _ptr(num_post_pad), _stream(stream))
    _check(st, "qg_moe_grouped_map")


def moe_gemm(p: Prepared, x, x_scale, sorted_ids, expert_ids, num_post_pad, tokens: int, topk: int, block_m: int,
             y, ws=None, stream=None):
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    st = lib().qg_moe_gemm(ctypes.byref(p), _ptr(x), _ptr(x_scale), _ptr(sorted_ids), _ptr(expert_ids),
                           _ptr(num_post_pad), tokens, topk, block_m, _ptr(y), _ptr(ws), ws_bytes, _stream(stream))
    _check(st, "qg_moe_gemm")


def moe_gemm_call(p: Prepared, x, x_scale, sorted_ids, expert_ids, num_post_pad, tokens: int, topk: int,
                  block_m: int, y, ws=None, stream=None):
    """qg_moe_gemm with every argument converted once (see gemm_call)."""
    fn = lib().qg_moe_gemm
    args = (ctypes.byref(p), _ptr(x), _ptr(x_scale), _ptr(sorted_ids), _ptr(expert_ids), _ptr(num_post_pad), tokens,
            topk, block_m, _ptr(y), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))

    def call():
        st = fn(*args)
        if st != 0:
            raise QGError(st, "qg_moe_gemm")
    return call


def moe_swiglu(gate_up, rows: int, inter: int, in_type: int, out_type: int, out, out_scale=None, stream=None):
    """act = silu(gate) * up per row (gate = first ``inter`` columns); f16/bf16, per-row e4m3 or int8, or MXFP4 output."""
    st = lib().qg_moe_swiglu(_ptr(gate_up), rows, inter, in_type, out_type, _ptr(out), _ptr(out_scale),
                             _stream(stream))
    _check(st, "qg_moe_swiglu")


def moe_combine(y, weights, topk_ids, tokens: int, topk: int, num_experts: int, n: int, dtype: int, out,
                stream=None):
    """out[t] = sum_j weights[t, j] * y[t*topk + j] over the slots routed inside [0, E)."""
    st = lib().qg_moe_combine(_ptr(y), _ptr(weights), _ptr(topk_ids), tokens, topk, num_experts, n, dtype, _ptr(out),
                              _stream(stream))
    _check(st, "qg_moe_combine")


def quantize_e4m3_rows(x, rows: int, k: int, in_type: int, codes, scale, stream=None):
    """Per-token absmax e4m3 quantization of 16-bit rows: codes [rows][k] uint8, scale [rows] float32."""
    st = lib().qg_quantize_e4m3_rows(_ptr(x), rows, k, in_type, _ptr(codes), _ptr(scale), _stream(stream))
    _check(st, "qg_quantize_e4m3_rows")


def quantize_int8_rows(x, rows: int, k: int, in_type: int, codes, scale, stream=None):
    """Per-token absmax int8 quantization of 16-bit rows: codes [rows][k] int8, scale [rows] float32 (NaN, with
    codes 0, for a row that holds a NaN or an infinity)."""
    st = lib().qg_quantize_int8_rows(_ptr(x), rows, k, in_type, _ptr(codes), _ptr(scale), _stream(stream))
    _check(st, "qg_quantize_int8_rows")


def make_route_desc(scoring, num_experts, topk, num_groups=1, topk_groups=1, group_top=1, renormalize=False,
                    weight_scale=1.0) -> RouteDesc:
    return RouteDesc(scoring, num_experts, topk, num_groups, topk_groups, group_top, int(renormalize), weight_scale)


def moe_route(desc: RouteDesc, logits, in_type: int, tokens: int, topk_ids, topk_weights, bias=None,
              row_stride: int | None = None, stream=None):
    """Router logits [tokens] rows of E (``row_stride`` elements apart, default E) -> topk_ids int32 and
    topk_weights float32, both [tokens][topk], for moe_align, moe_gemm and moe_combine."""
    st = lib().qg_moe_route(ctypes.byref(desc), _ptr(logits), in_type, desc.num_experts if row_stride is None else row_stride,
                            _ptr(bias), tokens, _ptr(topk_ids), _ptr(topk_weights), _stream(stream))
    _check(st, "qg_moe_route")


def quantize_e2m1_rows(x, rows: int, k: int, in_type: int, codes, scales, stream=None):
    """MXFP4 quantization of 16-bit rows: codes [rows][k/2] uint8 (packed e2m1), scales [rows][k/32] uint8."""
    st = lib().qg_quantize_e2m1_rows(_ptr(x), rows, k, in_type, _ptr(codes), _ptr(scales), _stream(stream))
    _check(st, "qg_quantize_e2m1_rows")


def make_norm_desc(norm, type, k, eps, post_norm=0, res_type=None, code_type=0, weight_offset=0.0, res_scale=1.0,
                   y_stride=0, res_stride=0, out_stride=0, gate_stride=0) -> NormDesc:
    """norm, post_norm: N_RMS, N_LAYER or 0; type: O_*; res_type: L_* (default: type's); code_type: A_* or 0."""
    res = (L_F16 if type == O_F16 else L_BF16) if res_type is None else res_type
    return NormDesc(norm, post_norm, type, res, code_type, eps, weight_offset, res_scale, k, y_stride, res_stride, out_stride,
                    gate_stride)


def norm_rows(desc: NormDesc, rows: int, y, residual, residual_out=None, out=None, codes=None, scale=None, *, weight=None,
              bias=None, gate=None, post_weight=None, stream=None):
    """u = residual + res_scale * gate * [N_post](y) -> residual_out; N(u) -> out (16 bits) and/or codes and scale."""
    st = lib().qg_norm_rows(ctypes.byref(desc), rows, _ptr(y), _ptr(residual), _ptr(residual_out), _ptr(gate),
                            _ptr(post_weight), _ptr(weight), _ptr(bias), _ptr(out), _ptr(codes), _ptr(scale), _stream(stream))
    _check(st, "qg_norm_rows")


def make_lora_desc(type, num_adapters, max_rank, k, slice_ends, x_stride=0, base_stride=0, y_stride=0) -> LoraDesc:
    """slice_ends: the columns behind each slice, the last one n ([n] for a single projection)."""
    ends = [int(e) for e in slice_ends]
    return LoraDesc(type, num_adapters, max_rank, len(ends), ends[-1] if ends else 0, k, x_stride, base_stride, y_stride,
                    (ctypes.c_int64 * 8)(*ends[:8]))


def lora_block_m(tokens: int, num_adapters: int) -> int:
    """Block size of the map (moe_align with topk 1) that lora takes for a batch."""
    return lib().qg_lora_block_m(tokens, num_adapters)


def lora_workspace_bytes(desc: LoraDesc, tokens: int, block_m: int) -> int:
    return lib().qg_lora_workspace_bytes(ctypes.byref(desc), tokens, block_m)


def lora(desc: LoraDesc, x, a, b, sorted_ids, expert_ids, num_post_pad, tokens: int, block_m: int, base, y, ws, ranks=None,
         scales=None, stream=None):
    """y = base + scales * (x A^T) B^T for the tokens of the block map, each with its own adapter's A and B."""
    st = lib().qg_lora(ctypes.byref(desc), _ptr(x), _ptr(a), _ptr(b), _ptr(ranks), _ptr(scales), _ptr(sorted_ids),
                       _ptr(expert_ids), _ptr(num_post_pad), tokens, block_m, _ptr(base), _ptr(y), _ptr(ws),
                       0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "qg_lora")


def make_kv_desc(type, kv_heads, head_dim, page_tokens, num_pages) -> KvDesc:
    return KvDesc(type, kv_heads, head_dim, page_tokens, num_pages)


def kv_cache_bytes(desc: KvDesc) -> int:
    return lib().qg_kv_cache_bytes(ctypes.byref(desc))


def kv_append(desc: KvDesc, k, v, slots, tokens: int, cache, k_stride: int = 0, v_stride: int = 0, stream=None):
    """Rows of keys and values into the MXFP4 cache, each token at its slot (int32; outside the cache: skipped)."""
    st = lib().qg_kv_append(ctypes.byref(desc), _ptr(k), k_stride, _ptr(v), v_stride, _ptr(slots), tokens, _ptr(cache),
                            _stream(stream))
    _check(st, "qg_kv_append")


def kv_read(desc: KvDesc, cache, slots, tokens: int, k, v, stream=None):
    """The keys and values at the slots, as contiguous 16-bit rows."""
    st = lib().qg_kv_read(ctypes.byref(desc), _ptr(cache), _ptr(slots), tokens, _ptr(k), _ptr(v), _stream(stream))
    _check(st, "qg_kv_read")


def attention_workspace_bytes(desc: KvDesc, q_heads: int, batch: int, max_q: int, tokens: int, max_len: int) -> int:
    return lib().qg_attention_workspace_bytes(ctypes.byref(desc), q_heads, batch, max_q, tokens, max_len)


def _table(table, page_tokens: int, max_len: int):
    """Address of a block table and the distance of its rows, as its tensor has them (a slice of a wider one, too)."""
    if table is None:
        return None, 0
    shape, stride = table.shape, table.stride()      # (each asked for once: the host's time of a small call)
    width = shape[-1]
    if width * page_tokens < max_len or (stride[-1] != 1 and width > 1) or (len(shape) > 2 and not table.is_contiguous()):
        raise QGError(1, "qg_attention")
    return table.data_ptr(), stride[0] if len(shape) == 2 and shape[0] > 1 else width


def attention(desc: KvDesc, q, q_heads: int, cache, block_table, seq_lens, batch: int, max_len: int, scale: float, out, ws=None,
              q_offsets=None, max_q: int = 1, tokens: int | None = None, q_stride: int = 0, out_stride: int = 0, stream=None):
    """Causal attention of each sequence's newest queries over its tokens in the MXFP4 cache; block_table [batch][pages]
    int32, its rows as far apart as its stride says (None: no sequence has tokens, max_len 0); tokens: rows of q (default:
    its first dimension)."""
    table, table_stride = _table(block_table, desc.page_tokens, max_len)
    st = lib().qg_attention(ctypes.byref(desc), _ptr(q), q_stride, q_heads, _ptr(cache), table, table_stride,
                            _ptr(seq_lens), _ptr(q_offsets), batch, max_q, q.shape[0] if tokens is None else tokens, max_len,
                            scale, _ptr(out), out_stride, _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                            _stream(stream))
    _check(st, "qg_attention")


def dequant(p: Prepared, expert: int, out, stream=None):
    _check(lib().qg_dequant(ctypes.byref(p), expert, _ptr(out), _stream(stream)), "qg_dequant")


def ceiling_read(buf, nbytes: int, loads_per_lane: int, sink, stream=None):
    """Measurement helper: one streaming read of ``nbytes`` of ``buf`` (see qg_ceiling_read)."""
    _check(lib().qg_ceiling_read(_ptr(buf), nbytes, loads_per_lane, _ptr(sink), sink.numel(), _stream(stream)),
           "qg_ceiling_read")


def ceiling_mfma(dtype: int, iters: int, workgroups: int, sink, stream=None):
    """Measurement helper: back-to-back MFMAs (dtype 0 bf16, 1 e4m3, 2 e2m1; see qg_ceiling_mfma)."""
    _check(lib().qg_ceiling_mfma(dtype, iters, workgroups, _ptr(sink), sink.numel(), _stream(stream)),
           "qg_ceiling_mfma")


def ceiling_lds(iters: int, workgroups: int, sink, stream=None):
    """Measurement helper: conflict-free 16-byte LDS reads by 8 waves per workgroup (see qg_ceiling_lds)."""
    _check(lib().qg_ceiling_lds(iters, workgroups, _ptr(sink), sink.numel(), _stream(stream)), "qg_ceiling_lds")
