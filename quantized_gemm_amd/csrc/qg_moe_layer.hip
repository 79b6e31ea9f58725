// The steps of an MoE layer around its two grouped products.  The pages time an MoE
// layer as its gate/up product plus its down product ("Humming: Fast, Flexible Kernels
// for Quantized Inference", benchmark paragraph; "Humming" wiki article, "Reported
// performance"); what joins them is this library's reading:
//
//  * SwiGLU on each (token, slot) row of the gate/up output [gate | up]:
//    act = silu(gate) * up, silu(g) = g / (1 + e^-g), in float32; written as f16/bf16, or
//    quantized per row to e4m3 (scale = max|row| / 448, 1 for an all-zero row; RNE after
//    clamping to +-448) when the down product takes FP8 activations.
//  * The down product is the grouped GEMM itself with one input row per slot.
//  * Combine: out[t] = sum_j w[t, j] * y[t * topk + j] over the slots routed inside
//    [0, E), float32 in slot order, one rounding at the end.
//  * Per-token e4m3 quantization of 16-bit activations (the input of a W4A8 product), the
//    same row quantizer without the SwiGLU.
//  * The same pair for int8 activations: scale = max|row| / 127 (1 where that is 0), code =
//    round to nearest even of row / scale.
//
// All three are HBM-bound streams: 16-byte loads and stores, 8 elements per thread-piece,
// consecutive lanes on consecutive pieces of a row.  The per-row e4m3 quantization reduces a
// row's absmax within one wave for rows up to 2048 wide, within a workgroup beyond.
#include "qg_device.h"
#include "qg_kernels.h"

namespace qg {

namespace {

template <int T>   // O_F16 / O_BF16
__device__ __forceinline__ float to_f32(uint32_t bits16) {
  if constexpr (T == O_BF16) return bf16_bits_to_f32(bits16);
  else return f16_bits_to_f32(bits16);
}

template <int T>
__device__ __forceinline__ void unpack8(const u32x4 v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = to_f32<T>(v[i] & 0xFFFFu);
    f[2 * i + 1] = to_f32<T>(v[i] >> 16);
  }
}

template <int T>
__device__ __forceinline__ u32x4 pack8(const float* f) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = (uint32_t)f32_to_out<T>(f[2 * i]) | ((uint32_t)f32_to_out<T>(f[2 * i + 1]) << 16);
  return o;
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + __expf(-g)); }

template <int IN>
__device__ __forceinline__ void swiglu8(const uint16_t* row, int64_t inter, int64_t c8, float* act) {
  float g[8], u[8];
  unpack8<IN>(ldg16(row + 8 * c8), g);
  unpack8<IN>(ldg16(row + inter + 8 * c8), u);
#pragma unroll
  for (int i = 0; i < 8; ++i) act[i] = silu(g[i]) * u[i];
}

// One thread per 8 outputs of a row.
template <int IN, int OUT>
__global__ __launch_bounds__(256) void swiglu_kernel(const uint16_t* __restrict__ gu, int64_t rows, int64_t inter,
                                                     uint16_t* __restrict__ out) {
  const int64_t per_row = inter >> 3;
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (p >= rows * per_row) return;
  const int64_t r = p / per_row, c8 = p - r * per_row;
  float act[8];
  swiglu8<IN>(gu + r * 2 * inter, inter, c8, act);
  *(u32x4*)(out + r * inter + 8 * c8) = pack8<OUT>(act);
}

// SwiGLU -> MXFP4, one thread per 32 outputs of a row: the activations are computed exactly as
// swiglu_kernel does, rounded to bfloat16 (the 16-bit SwiGLU output), then encoded, so the
// result equals swiglu_kernel followed by the MXFP4 row quantizer bit for bit.
template <int IN>
__global__ __launch_bounds__(256) void swiglu_e2m1_kernel(const uint16_t* __restrict__ gu, int64_t rows, int64_t inter,
                                                          uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int64_t per_row = inter >> 5;
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (p >= rows * per_row) return;
  const int64_t r = p / per_row, blk = p - r * per_row;
  float act[32];
#pragma unroll
  for (int q = 0; q < 4; ++q) swiglu8<IN>(gu + r * 2 * inter, inter, 4 * blk + q, act + 8 * q);
#pragma unroll
  for (int i = 0; i < 32; ++i) act[i] = bf16_bits_to_f32(f32_to_out<O_BF16>(act[i]));
  u32x4 packed;
  const uint32_t e8 = mxfp4_encode32(act, packed);
  *(u32x4*)(codes + r * (inter >> 1) + 16 * blk) = packed;
  scales[p] = (uint8_t)e8;
}

// One workgroup of 256 threads per row; each thread keeps up to kSwigluE4m3Pieces pieces of 8
// activations in registers while the row's absmax is reduced, then quantizes them.
constexpr int kSwigluE4m3Pieces = 4;   // inter <= 256 * 4 * 8 = 8192

template <int IN, bool SILU>
__global__ __launch_bounds__(256) void swiglu_e4m3_kernel(const uint16_t* __restrict__ gu, int64_t inter,
                                                          uint8_t* __restrict__ codes, float* __restrict__ scale) {
  __shared__ float s_wmax[4];
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x;
  const int64_t per_row = inter >> 3;
  const uint16_t* row = gu + r * (SILU ? 2 : 1) * inter;
  float act[kSwigluE4m3Pieces][8];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kSwigluE4m3Pieces; ++i) {
    const int64_t c8 = tid + 256 * i;
    if (c8 < per_row) {
      if constexpr (SILU) swiglu8<IN>(row, inter, c8, act[i]);
      else unpack8<IN>(ldg16(row + 8 * c8), act[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(act[i][e]));
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
  if ((tid & 63) == 0) s_wmax[tid >> 6] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(s_wmax[0], s_wmax[1]), fmaxf(s_wmax[2], s_wmax[3]));
  const float sc = amax == 0.0f ? 1.0f : amax / 448.0f;     // correctly rounded division
  if (tid == 0) scale[r] = sc;
#pragma unroll
  for (int i = 0; i < kSwigluE4m3Pieces; ++i) {
    const int64_t c8 = tid + 256 * i;
    if (c8 < per_row) {
      uint32_t w[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = fminf(fmaxf(act[i][4 * h + e] / sc, -448.0f), 448.0f);
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);   // bytes 0, 1
        v = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], v, true);        // bytes 2, 3
        w[h] = (uint32_t)v;
      }
      u32x2 o;
      o[0] = w[0];
      o[1] = w[1];
      *(u32x2*)(codes + r * inter + 8 * c8) = o;
    }
  }
}

// Rows up to kSwigluWaveRow wide: one wave per row (four rows per workgroup), the absmax
// reduced with wave shuffles only; every lane keeps up to four pieces in registers.
constexpr int kSwigluWaveRow = 64 * 4 * 8;

// SILU: the row is [gate | up] and its SwiGLU is quantized; else the row itself (per-token
// quantization of 16-bit activations).
template <int IN, bool SILU>
__global__ __launch_bounds__(256) void swiglu_e4m3_wave_kernel(const uint16_t* __restrict__ gu, int64_t rows,
                                                               int64_t inter, uint8_t* __restrict__ codes,
                                                               float* __restrict__ scale) {
  const int lane = threadIdx.x & 63;
  const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (r >= rows) return;                       // whole waves leave together
  const int64_t per_row = inter >> 3;
  const uint16_t* row = gu + r * (SILU ? 2 : 1) * inter;
  float act[4][8];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t c8 = lane + 64 * i;
    if (c8 < per_row) {
      if constexpr (SILU) swiglu8<IN>(row, inter, c8, act[i]);
      else unpack8<IN>(ldg16(row + 8 * c8), act[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(act[i][e]));
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
  const float sc = amax == 0.0f ? 1.0f : amax / 448.0f;     // correctly rounded division
  if (lane == 0) scale[r] = sc;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t c8 = lane + 64 * i;
    if (c8 < per_row) {
      u32x2 o;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) q[e] = fminf(fmaxf(act[i][4 * h + e] / sc, -448.0f), 448.0f);
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], v, true);
        o[h] = (uint32_t)v;
      }
      *(u32x2*)(codes + r * inter + 8 * c8) = o;
    }
  }
}

// int8 rows, as they are or as SwiGLU of [gate | up]: one row per NT threads (NT = 64: a wave per
// row, four rows per workgroup), each keeping up to P pieces of 8 values in registers between the
// maximum and the codes, so that the row is read once.  The quotient is rounded to float32 and
// then to an integer, as the definition says; for a row of 16-bit values it decides every code
// but those of exact halves as exact arithmetic does.
//
// The quotients of a row share their divisor, so its reciprocal is divided out once and each quotient
// takes two corrections by its exact remainder: the first leaves less than a unit in the last place, from
// where the second gives the correctly rounded quotient (Markstein, IBM J. Res. Dev. 34, 1990).  Divisors
// whose remainders could leave the range of float32 go through the division itself.
// Bound by bytes: 4096 rows of 7168 bf16 16.4-17.0 us (5.2-5.4 TB/s), 49152 SwiGLU rows of 1408 65.3-66 us (5.2-5.3);
// with a division per quotient and per sigmoid 21.9 and 87 us, bound by instruction issue.
//
// A row that holds a NaN or an infinity has no scale: it is set to NaN and the codes to 0, so that what is
// multiplied with the row is NaN.  The maximum keeps NaNs (one instruction for two values either way).
__device__ __forceinline__ uint32_t int8_codes(const float* v, float sc, float inv) {
  uint32_t b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float q = v[e] * inv;
    q = __builtin_fmaf(__builtin_fmaf(-q, sc, v[e]), inv, q);
    q = __builtin_fmaf(__builtin_fmaf(-q, sc, v[e]), inv, q);
    // |q| <= 127: the sum's last bit is 1, so it rounds to an integer, whose low byte is the code
    b[e] = __float_as_uint(q + 12582912.0f);
  }
  const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u);
  return lo | (hi << 16);
}
__device__ __forceinline__ uint32_t int8_codes_divided(const float* v, float sc) {
  if (sc != sc) return 0;
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float q = fminf(fmaxf(__builtin_rintf(v[e] / sc), -127.0f), 127.0f);
    w |= ((uint32_t)(int)q & 0xFFu) << (8 * e);
  }
  return w;
}

// SwiGLU in float32 with the hardware reciprocal: the activation is rounded to a code of seven bits next.
// Below a gate of -86 the reciprocal leaves the range in which the hardware gives it to a unit in the last
// place (it flushes what is below 2^-126), and exp(-g) that of float32; 1 / (1 + exp(-g)) is exp(g) to 2^-124
// there, taken as four factors exp(g / 4), none of which leaves the range before the activation does.  (49152 rows of 1408:
// 65.0 us without that branch, 65.3 with it.)
template <int IN>
__device__ __forceinline__ void swiglu8_rcp(const uint16_t* row, int64_t inter, int64_t c8, float* act) {
  float g[8], u[8];
  unpack8<IN>(ldg16(row + 8 * c8), g);
  unpack8<IN>(ldg16(row + inter + 8 * c8), u);
  float lowest = g[0];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    act[i] = g[i] * __builtin_amdgcn_rcpf(1.0f + __expf(-g[i])) * u[i];
    lowest = fminf(lowest, g[i]);
  }
  if (lowest < -86.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float e = __expf(0.25f * g[i]);
      act[i] = g[i] < -86.0f ? g[i] * e * (u[i] * e) * e * e : act[i];
    }
  }
}

template <int IN, bool SILU, int NT, int P>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void rows_int8_kernel(const uint16_t* __restrict__ x, int64_t rows,
                                                                       int64_t k, int8_t* __restrict__ codes,
                                                                       float* __restrict__ scale) {
  constexpr int RPB = NT < 256 ? 256 / NT : 1;             // rows per workgroup
  const int tid = threadIdx.x % NT;
  const int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / NT;
  if (r >= rows) return;                                   // NT = 64: whole waves leave together
  const int64_t per_row = k >> 3;
  const uint16_t* row = x + r * (SILU ? 2 : 1) * k;
  float v[P][8];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int64_t c8 = tid + NT * i;
    if (c8 < per_row) {
      if constexpr (SILU) swiglu8_rcp<IN>(row, k, c8, v[i]);
      else unpack8<IN>(ldg16(row + 8 * c8), v[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = __builtin_elementwise_maximum(amax, fabsf(v[i][e]));
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) amax = __builtin_elementwise_maximum(amax, __shfl_xor(amax, off, 64));
  if constexpr (NT > 64) {
    __shared__ float s_wmax[NT / 64];
    if ((tid & 63) == 0) s_wmax[tid >> 6] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) amax = __builtin_elementwise_maximum(amax, s_wmax[w]);
  }
  float sc = amax / 127.0f;                                // correctly rounded division
  if (sc == 0.0f) sc = 1.0f;
  if (!(amax < __builtin_inff())) sc = __builtin_nanf("");
  if (tid == 0) scale[r] = sc;
  const bool direct = !(sc >= 0x1p-100f && sc <= 0x1p100f);
  const float inv = 1.0f / sc;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int64_t c8 = tid + NT * i;
    if (c8 < per_row) {
      u32x2 o;
      if (direct) o = u32x2{int8_codes_divided(v[i], sc), int8_codes_divided(v[i] + 4, sc)};
      else o = u32x2{int8_codes(v[i], sc, inv), int8_codes(v[i] + 4, sc, inv)};
      *(u32x2*)(codes + r * k + 8 * c8) = o;
    }
  }
}

// One thread per 8 outputs of a token.  Slots go in groups of 8 with every row load of a
// group in flight at once: a dropped slot's row exists (it is only unwritten), so it is read
// like the others and discarded with a select, never multiplied (it may hold NaN).
template <int T>
__global__ __launch_bounds__(256) void combine_kernel(const uint16_t* __restrict__ y, const float* __restrict__ w,
                                                      const int32_t* __restrict__ ids, int64_t tokens, int topk,
                                                      int experts, int64_t n, uint16_t* __restrict__ out) {
  constexpr int G = 8;
  const int64_t per_row = n >> 3;
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (p >= tokens * per_row) return;
  const int64_t t = p / per_row, c8 = p - t * per_row;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < topk; j0 += G) {
    u32x4 v[G];
    bool ok[G];
    float wj[G];
#pragma unroll
    for (int u = 0; u < G; ++u) {
      const int j = j0 + u;
      const int64_t f = t * topk + (j < topk ? j : topk - 1);
      const int e = ids[f];
      ok[u] = j < topk && e >= 0 && e < experts;
      wj[u] = w[f];
      v[u] = ldg16(y + f * n + 8 * c8);
    }
#pragma unroll
    for (int u = 0; u < G; ++u) {
      float vv[8];
      unpack8<T>(v[u], vv);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = ok[u] ? __builtin_fmaf(wj[u], vv[i], acc[i]) : acc[i];
    }
  }
  *(u32x4*)(out + t * n + 8 * c8) = pack8<T>(acc);
}

}  // namespace

template <bool SILU>
static bool launch_rows_e4m3(const uint16_t* g, int64_t rows, int64_t inter, int in_t, void* out, float* out_scale,
                             hipStream_t st) {
  if (inter > 256 * kSwigluE4m3Pieces * 8) return false;
  if (inter <= kSwigluWaveRow) {
    const dim3 grid((unsigned)((rows + 3) / 4));
    if (in_t == O_BF16)
      hipLaunchKernelGGL((swiglu_e4m3_wave_kernel<O_BF16, SILU>), grid, dim3(256), 0, st, g, rows, inter, (uint8_t*)out,
                         out_scale);
    else
      hipLaunchKernelGGL((swiglu_e4m3_wave_kernel<O_F16, SILU>), grid, dim3(256), 0, st, g, rows, inter, (uint8_t*)out,
                         out_scale);
    return true;
  }
  const dim3 grid((unsigned)rows);
  if (in_t == O_BF16)
    hipLaunchKernelGGL((swiglu_e4m3_kernel<O_BF16, SILU>), grid, dim3(256), 0, st, g, inter, (uint8_t*)out, out_scale);
  else
    hipLaunchKernelGGL((swiglu_e4m3_kernel<O_F16, SILU>), grid, dim3(256), 0, st, g, inter, (uint8_t*)out, out_scale);
  return true;
}

// (a launch takes fewer than 2^32 threads)
constexpr int64_t kInt8RowsPerLaunch = 1 << 21;

template <int IN, bool SILU, int NT, int P>
static void launch_rows_int8_one(const uint16_t* x, int64_t rows, int64_t k, int8_t* codes, float* scale, hipStream_t st) {
  constexpr int RPB = NT < 256 ? 256 / NT : 1;
  for (int64_t r = 0; r < rows; r += kInt8RowsPerLaunch) {
    const int64_t n = rows - r < kInt8RowsPerLaunch ? rows - r : kInt8RowsPerLaunch;
    hipLaunchKernelGGL((rows_int8_kernel<IN, SILU, NT, P>), dim3((unsigned)((n + RPB - 1) / RPB)), dim3(NT * RPB), 0, st,
                       x + r * (SILU ? 2 : 1) * k, n, k, codes + r * k, scale + r);
  }
}

// A wave per row up to 2048 values, 256 threads up to 8192, 1024 up to kInt8RowMax.
template <int IN, bool SILU>
static bool launch_rows_int8(const uint16_t* x, int64_t rows, int64_t k, int8_t* codes, float* scale, hipStream_t st) {
  if (k <= 64 * 4 * 8) launch_rows_int8_one<IN, SILU, 64, 4>(x, rows, k, codes, scale, st);
  else if (k <= 256 * 4 * 8) launch_rows_int8_one<IN, SILU, 256, 4>(x, rows, k, codes, scale, st);
  else if (k <= kInt8RowMax) launch_rows_int8_one<IN, SILU, 1024, 4>(x, rows, k, codes, scale, st);
  else return false;
  return true;
}

bool launch_quant_rows_int8(const void* x, int64_t rows, int64_t k, int in_t, bool silu, int8_t* codes, float* scale,
                            hipStream_t st) {
  const uint16_t* g = (const uint16_t*)x;
  if (in_t == O_BF16) return silu ? launch_rows_int8<O_BF16, true>(g, rows, k, codes, scale, st)
                                  : launch_rows_int8<O_BF16, false>(g, rows, k, codes, scale, st);
  if (in_t == O_F16) return silu ? launch_rows_int8<O_F16, true>(g, rows, k, codes, scale, st)
                                 : launch_rows_int8<O_F16, false>(g, rows, k, codes, scale, st);
  return false;
}

bool launch_swiglu(const void* gu, int64_t rows, int64_t inter, int in_t, int out_t, void* out, void* out_scale,
                   hipStream_t st) {
  const uint16_t* g = (const uint16_t*)gu;
  if (out_t == A_INT8) return launch_quant_rows_int8(gu, rows, inter, in_t, true, (int8_t*)out, (float*)out_scale, st);
  if (out_t == A_FP8) return launch_rows_e4m3<true>(g, rows, inter, in_t, out, (float*)out_scale, st);
  if (out_t == A_FP4) {
    const dim3 grid4((unsigned)((rows * (inter >> 5) + 255) / 256));
    uint8_t* c = (uint8_t*)out;
    uint8_t* e = (uint8_t*)out_scale;
    if (in_t == O_BF16) hipLaunchKernelGGL((swiglu_e2m1_kernel<O_BF16>), grid4, dim3(256), 0, st, g, rows, inter, c, e);
    else if (in_t == O_F16) hipLaunchKernelGGL((swiglu_e2m1_kernel<O_F16>), grid4, dim3(256), 0, st, g, rows, inter, c, e);
    else return false;
    return true;
  }
  const int64_t pieces = rows * (inter >> 3);
  const dim3 grid((unsigned)((pieces + 255) / 256));
  uint16_t* o = (uint16_t*)out;
  if (in_t == O_BF16 && out_t == A_BF16) hipLaunchKernelGGL((swiglu_kernel<O_BF16, O_BF16>), grid, dim3(256), 0, st, g, rows, inter, o);
  else if (in_t == O_BF16 && out_t == A_F16) hipLaunchKernelGGL((swiglu_kernel<O_BF16, O_F16>), grid, dim3(256), 0, st, g, rows, inter, o);
  else if (in_t == O_F16 && out_t == A_BF16) hipLaunchKernelGGL((swiglu_kernel<O_F16, O_BF16>), grid, dim3(256), 0, st, g, rows, inter, o);
  else if (in_t == O_F16 && out_t == A_F16) hipLaunchKernelGGL((swiglu_kernel<O_F16, O_F16>), grid, dim3(256), 0, st, g, rows, inter, o);
  else return false;
  return true;
}

bool launch_quant_rows_e4m3(const void* x, int64_t rows, int64_t k, int in_t, void* codes, float* scale,
                            hipStream_t st) {
  return launch_rows_e4m3<false>((const uint16_t*)x, rows, k, in_t, codes, scale, st);
}

bool launch_combine(const void* y, const float* w, const int32_t* ids, int64_t tokens, int topk, int experts, int64_t n,
                    int dtype, void* out, hipStream_t st) {
  const int64_t pieces = tokens * (n >> 3);
  const dim3 grid((unsigned)((pieces + 255) / 256));
  const uint16_t* yy = (const uint16_t*)y;
  uint16_t* o = (uint16_t*)out;
  if (dtype == O_BF16) hipLaunchKernelGGL(combine_kernel<O_BF16>, grid, dim3(256), 0, st, yy, w, ids, tokens, topk, experts, n, o);
  else if (dtype == O_F16) hipLaunchKernelGGL(combine_kernel<O_F16>, grid, dim3(256), 0, st, yy, w, ids, tokens, topk, experts, n, o);
  else return false;
  return true;
}

}  // namespace qg
