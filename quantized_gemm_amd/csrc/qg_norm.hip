// The norms before and after a block, with its gate, its residual and the quantization of what the next product
// reads, in one pass over the rows:
//
//   h = y, or N_post(y);  u = res + res_scale * gate * h;  res_out = u;  z = N(u), in 16 bits and/or as codes
//   N(v) = (v - c) / sqrt(mean((v - c)^2) + eps) * (offset + weight) + bias, c = 0 (RMS) or mean(v) (layer norm)
//
// Everything between the loads and the stores is float32: u goes into the second norm, and z into the codes,
// without being rounded to 16 bits in between.  The mean square is taken from the values less their mean (a
// second sum over registers), which loses nothing where the mean is far from zero.
//
// Bound by bytes.  A row stays in registers between the sums (P pieces of 8 values per thread), so that each
// input is read once; NT threads share a row, and a sum over them is a wave's exchange plus one barrier.
#include "qg_device.h"
#include "qg_kernels.h"
#include "qg_rows.h"

namespace qg {

namespace {

// The value of the lane whose place in its four neighbours is this one's, XOR 1 (M = 0xB1) or XOR 2 (0x4E).
template <int M>
__device__ __forceinline__ float neighbour(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), M, 0xF, 0xF, true));
}

// A sum or a NaN-keeping maximum over the NT threads of a row; `slot`: NT / 64 words of LDS of its own.
template <int NT, bool MAX>
__device__ __forceinline__ float over_row(float v, float* slot) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const float o = __shfl_xor(v, off, 64);
    v = MAX ? __builtin_elementwise_maximum(v, o) : v + o;
  }
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slot[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) v = MAX ? __builtin_elementwise_maximum(v, slot[w]) : v + slot[w];
  }
  return v;
}

// Centres the row's values (layer norm) and returns what they are to be multiplied with.  Where the sums
// leave float32 while the values are finite, values and eps are first brought down by a power of two.
template <int NT, int P>
__device__ __forceinline__ float normalize(float (&v)[P][8], const bool (&in)[P], bool layer, float inv_k, float eps,
                                           float (*slots)[NT / 64]) {
  for (int pass = 0;; ++pass) {
    float (*slot)[NT / 64] = slots + 3 * pass;
    float mean = 0.f;
    if (layer) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[i][e];
      mean = over_row<NT, false>(s, slot[0]) * inv_k;
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = in[i] ? v[i][e] - mean : 0.f;
        ss = __builtin_fmaf(d, d, ss);
      }
    ss = over_row<NT, false>(ss, slot[1]);
    if (ss < __builtin_inff() || pass == 1) {
      if (layer) {
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] = in[i] ? v[i][e] - mean : 0.f;
      }
      return 1.0f / __builtin_sqrtf(__builtin_fmaf(ss, inv_k, eps));
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = __builtin_elementwise_maximum(amax, fabsf(v[i][e]));
    amax = over_row<NT, true>(amax, slot[2]);
    if (amax < __builtin_inff()) {
      const int down = -__builtin_amdgcn_frexp_expf(amax);
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = __builtin_ldexpf(v[i][e], down);
      eps = __builtin_ldexpf(eps, 2 * down);
    }
  }
}

template <int T, bool R32, int NT, int P>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void norm_rows_kernel(NormArgs a) {
  constexpr int RPB = NT < 256 ? 256 / NT : 1;                // rows per workgroup
  __shared__ float slots[13][NT / 64];
  const int tid = threadIdx.x % NT;
  const int64_t r = a.row0 + (int64_t)blockIdx.x * RPB + threadIdx.x / NT;
  if (r >= a.rows) return;                                    // NT = 64: whole waves leave together
  const int per_row = (int)(a.k >> 3);
  const float inv_k = 1.0f / (float)a.k;
  bool in[P];
#pragma unroll
  for (int i = 0; i < P; ++i) in[i] = tid + NT * i < per_row;

  float u[P][8];
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) u[i][e] = 0.f;
  if (a.y) {
    const uint16_t* row = (const uint16_t*)a.y + r * a.y_stride;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (in[i]) unpack8<T>(ldg16(row + 8 * (tid + NT * i)), u[i]);
  }
  float res[P][8];
  if (a.res) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int64_t at = r * a.res_stride + 8 * (tid + NT * i);
      if (!in[i]) continue;
      if constexpr (R32) {
        *(f32x4*)res[i] = *(const f32x4*)((const float*)a.res + at);
        *(f32x4*)(res[i] + 4) = *(const f32x4*)((const float*)a.res + at + 4);
      } else {
        unpack8<T>(ldg16((const uint16_t*)a.res + at), res[i]);
      }
    }
  }
  if (a.post != 0) {
    const float f = normalize<NT, P>(u, in, a.post == kNormLayer, inv_k, a.eps, slots);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (in[i]) {
        float w[8];
        if (a.post_weight) unpack8<T>(ldg16((const uint16_t*)a.post_weight + 8 * (tid + NT * i)), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] *= f * (a.post_weight ? a.weight_offset + w[e] : 1.0f);
      }
  }
  if (a.y) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (in[i]) {
        if (a.gate) {
          float g[8];
          unpack8<T>(ldg16((const uint16_t*)a.gate + r * a.gate_stride + 8 * (tid + NT * i)), g);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[i][e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] = a.res ? __builtin_fmaf(a.res_scale, u[i][e], res[i][e]) : a.res_scale * u[i][e];
      }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (in[i])
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] = res[i][e];
  }
  if (a.res_out) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int64_t at = r * a.res_stride + 8 * (tid + NT * i);
      if (!in[i]) continue;
      if constexpr (R32) {
        *(f32x4*)((float*)a.res_out + at) = *(const f32x4*)u[i];
        *(f32x4*)((float*)a.res_out + at + 4) = *(const f32x4*)(u[i] + 4);
      } else {
        *(u32x4*)((uint16_t*)a.res_out + at) = pack8<T>(u[i]);
      }
    }
  }
  if (a.norm == 0) return;
  const float f = normalize<NT, P>(u, in, a.norm == kNormLayer, inv_k, a.eps, slots + 6);
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (in[i]) {
      float w[8], b[8];
      if (a.weight) unpack8<T>(ldg16((const uint16_t*)a.weight + 8 * (tid + NT * i)), w);
      if (a.bias) unpack8<T>(ldg16((const uint16_t*)a.bias + 8 * (tid + NT * i)), b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = u[i][e] * f;
        u[i][e] = __builtin_fmaf(n, a.weight ? a.weight_offset + w[e] : 1.0f, a.bias ? b[e] : 0.0f);
      }
    }
  if (a.out) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (in[i]) *(u32x4*)((uint16_t*)a.out + r * a.out_stride + 8 * (tid + NT * i)) = pack8<T>(u[i]);
  }
  if (a.code == A_FP4) {
    // a block of 32 lies in four neighbouring threads
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = __builtin_elementwise_maximum(amax, fabsf(u[i][e]));
      amax = __builtin_elementwise_maximum(amax, neighbour<0xB1>(amax));
      amax = __builtin_elementwise_maximum(amax, neighbour<0x4E>(amax));
      uint32_t codes;
      const uint32_t e8 = mxfp4_encode8(u[i], amax, codes);
      if (in[i]) {
        const int c8 = tid + NT * i;
        *(uint32_t*)((uint8_t*)a.codes + r * (a.k >> 1) + 4 * c8) = codes;
        if ((c8 & 3) == 0) ((uint8_t*)a.scale)[r * (a.k >> 5) + (c8 >> 2)] = (uint8_t)e8;
      }
    }
  } else if (a.code != 0) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = __builtin_elementwise_maximum(amax, in[i] ? fabsf(u[i][e]) : 0.f);
    amax = over_row<NT, true>(amax, slots[12]);
    float sc = amax / (a.code == A_FP8 ? 448.0f : 127.0f);    // correctly rounded division
    if (sc == 0.0f) sc = 1.0f;
    if (!(amax < __builtin_inff())) sc = __builtin_nanf("");
    if (tid == 0) ((float*)a.scale)[r] = sc;
    const bool direct = !(sc >= 0x1p-100f && sc <= 0x1p100f);
    const float inv = 1.0f / sc;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (in[i]) {
        u32x2 o;
        if (a.code == A_FP8)
          o = direct ? u32x2{e4m3_codes_divided(u[i], sc), e4m3_codes_divided(u[i] + 4, sc)}
                     : u32x2{e4m3_codes(u[i], sc, inv), e4m3_codes(u[i] + 4, sc, inv)};
        else
          o = direct ? u32x2{int8_codes_divided(u[i], sc), int8_codes_divided(u[i] + 4, sc)}
                     : u32x2{int8_codes(u[i], sc, inv), int8_codes(u[i] + 4, sc, inv)};
        *(u32x2*)((uint8_t*)a.codes + r * a.k + 8 * (tid + NT * i)) = o;
      }
  }
}

constexpr int64_t kNormRowsPerLaunch = 1 << 21;   // a launch takes fewer than 2^32 threads

template <int T, bool R32, int NT, int P>
void launch_one(NormArgs a, hipStream_t st) {
  constexpr int RPB = NT < 256 ? 256 / NT : 1;
  const int64_t rows = a.rows;
  for (a.row0 = 0; a.row0 < rows; a.row0 += kNormRowsPerLaunch) {
    a.rows = rows - a.row0 < kNormRowsPerLaunch ? rows : a.row0 + kNormRowsPerLaunch;
    const unsigned grid = (unsigned)((a.rows - a.row0 + RPB - 1) / RPB);
    hipLaunchKernelGGL((norm_rows_kernel<T, R32, NT, P>), dim3(grid), dim3(NT * RPB), 0, st, a);
  }
}

template <int T, bool R32>
void launch_shape(const NormArgs& a, hipStream_t st) {
  const int64_t k = a.k;
  if (k <= 512) launch_one<T, R32, 64, 1>(a, st);
  else if (k <= 1024) launch_one<T, R32, 64, 2>(a, st);
  else if (k <= 2048) launch_one<T, R32, 256, 1>(a, st);
  else if (k <= 4096) launch_one<T, R32, 256, 2>(a, st);
  else if (k <= 8192) launch_one<T, R32, 256, 4>(a, st);
  else if (k <= 16384) launch_one<T, R32, 1024, 2>(a, st);
  else launch_one<T, R32, 1024, 4>(a, st);
}

}  // namespace

void launch_norm_rows(const NormArgs& a, int type, bool res32, hipStream_t st) {
  if (type == O_BF16) res32 ? launch_shape<O_BF16, true>(a, st) : launch_shape<O_BF16, false>(a, st);
  else res32 ? launch_shape<O_F16, true>(a, st) : launch_shape<O_F16, false>(a, st);
}

}  // namespace qg
