// The norms before and after a block, with its gate, its residual and the quantization of what the next product
// reads, in one pass over the rows:
//
//   h = y, or N_post(y);  u = res + res_scale * gate * h;  res_out = u;  z = N(u), in 16 bits and/or as codes
//   N(v) = (v - c) / sqrt(mean((v - c)^2) + eps) * (offset + weight) + bias, c = 0 (RMS) or mean(v) (layer norm)
//
// Everything between the loads and the stores is float32: u goes into the second norm, and z into the codes,
// without being rounded to 16 bits in between.  The mean square is taken from the values less their mean (a
// second sum over registers), which loses nothing where the mean is far from zero.  The mean is kept between the row's
// least and largest value: of a row whose values are all alike zeros are left, not a last bit of them over sqrt(eps).
//
// Bound by bytes.  A row stays in registers between the sums (P pieces of 8 values per thread; of rows above 16384 values
// 63 to 99 registers' worth goes through scratch memory: 2048 rows of 32768 225 us, 2.4 TB/s), so that each
// input is read once; NT threads share a row, and a sum over them is a wave's exchange plus one barrier.  Rows of 1025 to
// 8192 values are taken in turn by a workgroup (KEEP), the next one's loads on their way during one's sums, and weights and
// a shared gate stay in registers.  Longer rows lack the registers for it (2048 rows of 16384 values: 57 us, in turn 150),
// and shorter ones need no barrier to wait at (65536 rows of 512: 47 us, in turn 53); those are one to a workgroup or part
// of it, and read the weights again.  Workgroups that are no more than the GPU holds at once: 16384 rows of 4096 in 768
// workgroups 95 us, in 1024 115.  Measured: those (both norms, gate, residual, to e4m3) 95 us, 4.9 TB/s (155 with a
// workgroup per row, 137 with sums exchanged through LDS), to MXFP4 83; 4096 rows of 7168 to e4m3 45 us, to MXFP4 40; one
// 4.3 us; 65536 rows of 128 13 us (29 with a whole wave to a row).
#include "qg_device.h"
#include "qg_kernels.h"
#include "qg_rows.h"

namespace qg {

namespace {

// Words that the waves of a row leave their sums in.
template <int NT>
constexpr int kSlots = NT > 64 ? NT / 64 : 1;

// Sums or NaN-keeping maxima of N values over the NT threads of a row; `slots`: NT / 64 words of LDS for each.
template <int NT, bool MAX, int N>
__device__ __forceinline__ void over_row(float (&v)[N], float (*slots)[kSlots<NT>]) {
  auto with = [](float x, float y) __attribute__((always_inline)) { return MAX ? __builtin_elementwise_maximum(x, y) : x + y; };
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = over_lanes<(NT < 64 ? NT : 64)>(v[n], with);
  if constexpr (NT > 64) {
#pragma unroll
    for (int n = 0; n < N; ++n)
      if ((threadIdx.x & 63) == 0) slots[n][threadIdx.x >> 6] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = slots[n][0];
#pragma unroll
      for (int w = 1; w < NT / 64; ++w) v[n] = with(v[n], slots[n][w]);
    }
  }
}
template <int NT, bool MAX>
__device__ __forceinline__ float over_row(float v, float (*slots)[kSlots<NT>]) {
  float one[1] = {v};
  over_row<NT, MAX>(one, slots);
  return one[0];
}

// Sums of a row that one norm takes.
constexpr int kNormSums = 5;

// Centres the row's values (layer norm; those behind its end are zeros and stay so) and returns what they are to be
// multiplied with.  Where the sums leave float32 while the values are finite, values and eps are first brought down by a
// power of two.
template <int NT, int P>
__device__ __forceinline__ float normalize(float (&v)[P][8], const bool (&in)[P], bool layer, float inv_k, float eps,
                                           float (*slots)[kSlots<NT>]) {
  auto squares = [&]() __attribute__((always_inline)) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[i][e], v[i][e], ss);
    return ss;
  };
  if (!layer) {
    const float ss = over_row<NT, false>(squares(), slots);
    if (ss < __builtin_inff()) return 1.0f / __builtin_sqrtf(__builtin_fmaf(ss, inv_k, eps));
  }
  // layer norm, or squares beyond float32 (the values as they were)
  float ends[2] = {-__builtin_inff(), -__builtin_inff()};     // the largest value, and less the least
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (!in[i]) continue;
      ends[0] = __builtin_elementwise_maximum(ends[0], v[i][e]);
      ends[1] = __builtin_elementwise_maximum(ends[1], -v[i][e]);
    }
  over_row<NT, true>(ends, slots + 1);
  const float amax = __builtin_elementwise_maximum(ends[0], ends[1]);
  if (amax > 0x1p56f && amax < __builtin_inff()) {            // (2^15 squares of 2^56 stay inside)
    const int down = -__builtin_amdgcn_frexp_expf(amax);
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = __builtin_ldexpf(v[i][e], down);
    for (float& v : ends) v = __builtin_ldexpf(v, down);
    // (a row of one value has no variance left: not over zero, which would make its zeros NaN)
    eps = fmaxf(__builtin_ldexpf(eps, 2 * down), 0x1p-126f);
  }
  if (layer) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += v[i][e];
    // (values that are not finite make the squares NaN, whatever the mean)
    const float mean = fmaxf(fminf(over_row<NT, false>(sum, slots + 3) * inv_k, ends[0]), -ends[1]);
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = in[i] ? v[i][e] - mean : 0.f;
  }
  const float ss = over_row<NT, false>(squares(), slots + 4);
  return 1.0f / __builtin_sqrtf(__builtin_fmaf(ss, inv_k, eps));
}

// v *= f * (offset + weight), without a weight f alone.
template <int T>
__device__ __forceinline__ void scale_by(float (&v)[8], float f, bool weighted, float offset, const u32x4& raw) {
  if (!weighted) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= f;
    return;
  }
  float w[8];
  unpack8<T>(raw, w);
  if (offset != 0.0f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] += offset;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = v[e] * f * w[e];
}

// Takes the 16 bytes as new ones, so that what is made of them is not kept in (four times as many) registers over a loop.
__device__ __forceinline__ void opaque(u32x4& v) { asm volatile("" : "+v"(v)); }

// A thread's pieces of a row, as they lie in memory.
template <int P, bool R32>
struct RawRow {
  u32x4 y[P], gate[P], res[P][R32 ? 2 : 1];
};

// KEEP: rows in turn, see above; else one row, and the shared rows read where they are used.
template <int T, bool R32, int NT, int P, bool KEEP>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void norm_rows_kernel(NormArgs a) {
  constexpr int RPB = NT < 256 ? 256 / NT : 1;                // rows per workgroup
  __shared__ float slots[2][2 * kNormSums + 1][kSlots<NT>];   // one row's sums while another's are still read
  const int tid = threadIdx.x % NT;
  const int per_row = (int)(a.k >> 3);
  const float inv_k = 1.0f / (float)a.k;
  bool in[P];
#pragma unroll
  for (int i = 0; i < P; ++i) in[i] = tid + NT * i < per_row;
  auto piece = [&](const void* p, int i) __attribute__((always_inline)) {
    return ldg16((const uint16_t*)p + 8 * (tid + NT * i));
  };
  // what all rows share
  u32x4 wp[P], w[P], b[P], g[P];
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (in[i]) {
        if (a.post_weight) wp[i] = piece(a.post_weight, i);
        if (a.weight) w[i] = piece(a.weight, i);
        if (a.bias) b[i] = piece(a.bias, i);
        if (a.gate && a.gate_stride == 0) g[i] = piece(a.gate, i);
      }
  }
  RawRow<P, R32> raw;
  auto load = [&](int64_t r) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (in[i]) {
        if (a.y) raw.y[i] = piece((const uint16_t*)a.y + r * a.y_stride, i);
        if (a.res) {
          if constexpr (R32) {
            const float* const at = (const float*)a.res + r * a.res_stride + 8 * (tid + NT * i);
            raw.res[i][0] = ldg16(at);
            raw.res[i][1] = ldg16(at + 4);
          } else {
            raw.res[i][0] = piece((const uint16_t*)a.res + r * a.res_stride, i);
          }
        }
        if (KEEP && a.gate && a.gate_stride != 0) raw.gate[i] = piece((const uint16_t*)a.gate + r * a.gate_stride, i);
      }
  };

  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / NT;
  if (r >= a.rows) return;                                    // NT <= 64: a row's lanes leave together
  load(r);
  for (int turn = 0; r < a.rows; r += step, turn ^= 1) {
    if (!KEEP && r >= step) load(r);                          // (more rows than a launch has workgroups)
    float (*const slot)[kSlots<NT>] = slots[turn];
    float u[P][8], res[P][8];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if constexpr (KEEP) {
        opaque(wp[i]);
        opaque(w[i]);
        opaque(b[i]);
        opaque(g[i]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) u[i][e] = 0.f;
      if (!in[i]) continue;
      if (a.y) unpack8<T>(raw.y[i], u[i]);
      if (a.res) {
        if constexpr (R32) {
#pragma unroll
          for (int e = 0; e < 8; ++e) res[i][e] = __uint_as_float(raw.res[i][e >> 2][e & 3]);
        } else {
          unpack8<T>(raw.res[i][0], res[i]);
        }
      }
      if (KEEP && a.gate && a.gate_stride != 0) g[i] = raw.gate[i];
    }
    if (KEEP && r + step < a.rows) load(r + step);             // the next row's, on their way during this one's sums
    if (a.post != 0) {
      const float f = normalize<NT, P>(u, in, a.post == kNormLayer, inv_k, a.eps, slot);
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (in[i]) {
          if (!KEEP && a.post_weight) wp[i] = piece(a.post_weight, i);
          scale_by<T>(u[i], f, a.post_weight != nullptr, a.weight_offset, wp[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (!in[i]) continue;
      if (a.y) {
        if (a.gate) {
          if (!KEEP) g[i] = piece((const uint16_t*)a.gate + r * a.gate_stride, i);
          float v[8];
          unpack8<T>(g[i], v);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[i][e] *= v[e];
        }
        if (a.res) {
#pragma unroll
          for (int e = 0; e < 8; ++e) u[i][e] = __builtin_fmaf(a.res_scale, u[i][e], res[i][e]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) u[i][e] *= a.res_scale;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] = res[i][e];
      }
      if (a.res_out) {
        const int64_t at = r * a.res_stride + 8 * (tid + NT * i);
        if constexpr (R32) {
          *(f32x4*)((float*)a.res_out + at) = f32x4{u[i][0], u[i][1], u[i][2], u[i][3]};
          *(f32x4*)((float*)a.res_out + at + 4) = f32x4{u[i][4], u[i][5], u[i][6], u[i][7]};
        } else {
          *(u32x4*)((uint16_t*)a.res_out + at) = pack8<T>(u[i]);
        }
      }
    }
    if (a.norm == 0) continue;
    const float f = normalize<NT, P>(u, in, a.norm == kNormLayer, inv_k, a.eps, slot + kNormSums);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (in[i]) {
        if (!KEEP && a.weight) w[i] = piece(a.weight, i);
        scale_by<T>(u[i], f, a.weight != nullptr, a.weight_offset, w[i]);
        if (a.bias) {
          if (!KEEP) b[i] = piece(a.bias, i);
          float v[8];
          unpack8<T>(b[i], v);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[i][e] += v[e];
        }
        if (a.out) *(u32x4*)((uint16_t*)a.out + r * a.out_stride + 8 * (tid + NT * i)) = pack8<T>(u[i]);
      }
    if (a.code == A_FP4) {
      // a block of 32 lies in four neighbouring threads
#pragma unroll
      for (int i = 0; i < P; ++i) {
        float most = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) most = __builtin_elementwise_maximum(most, fabsf(u[i][e]));
        most = __builtin_elementwise_maximum(most, neighbour<0xB1>(most));
        most = __builtin_elementwise_maximum(most, neighbour<0x4E>(most));
        uint32_t codes;
        const uint32_t e8 = mxfp4_encode8(u[i], most, codes);
        if (in[i]) {
          const int c8 = tid + NT * i;
          *(uint32_t*)((uint8_t*)a.codes + r * (a.k >> 1) + 4 * c8) = codes;
          if ((c8 & 3) == 0) ((uint8_t*)a.scale)[r * (a.k >> 5) + (c8 >> 2)] = (uint8_t)e8;
        }
      }
    } else if (a.code != 0) {
      float amax = 0.f;                                       // (zeros behind the row's end)
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = __builtin_elementwise_maximum(amax, fabsf(u[i][e]));
      amax = over_row<NT, true>(amax, slot + 2 * kNormSums);
      float sc = amax / (a.code == A_FP8 ? 448.0f : 127.0f);  // correctly rounded division
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
}

// Workgroups: with KEEP as many as the GPU holds at once, each taking rows in turn (4 waves per SIMD with one piece per thread,
// 3 with two).
template <int T, bool R32, int NT, int P, bool KEEP>
void launch_one(const NormArgs& a, hipStream_t st) {
  constexpr int RPB = NT < 256 ? 256 / NT : 1, WAVES = P == 1 ? 16 : 12;
  const int64_t groups = (a.rows + RPB - 1) / RPB, most = KEEP ? 256 * (WAVES / (NT * RPB / 64)) : (int64_t)1 << 21;
  const dim3 grid((unsigned)(groups < most ? groups : most));
  hipLaunchKernelGGL((norm_rows_kernel<T, R32, NT, P, KEEP>), grid, dim3(NT * RPB), 0, st, a);
}

template <int T, bool R32>
void launch_shape(const NormArgs& a, hipStream_t st) {
  const int64_t k = a.k;
  if (k <= 128) launch_one<T, R32, 16, 1, false>(a, st);
  else if (k <= 512) launch_one<T, R32, 64, 1, false>(a, st);
  else if (k <= 1024) launch_one<T, R32, 64, 2, false>(a, st);
  else if (k <= 2048) launch_one<T, R32, 256, 1, true>(a, st);
  else if (k <= 4096) launch_one<T, R32, 256, 2, true>(a, st);
  else if (k <= 8192) launch_one<T, R32, 512, 2, true>(a, st);
  else if (k <= 16384) launch_one<T, R32, 1024, 2, false>(a, st);
  else launch_one<T, R32, 1024, 4, false>(a, st);
}

}  // namespace

void launch_norm_rows(const NormArgs& a, int type, bool res32, hipStream_t st) {
  if (type == O_BF16) res32 ? launch_shape<O_BF16, true>(a, st) : launch_shape<O_BF16, false>(a, st);
  else res32 ? launch_shape<O_F16, true>(a, st) : launch_shape<O_F16, false>(a, st);
}

}  // namespace qg
