// Attention over a paged cache of keys and values in MXFP4 (qg_kernels.h has its layout):
//
//   out[i] = softmax(scale q[i] K^T) V per query head over the tokens that query i sees: those up to its own place
//
// One pass over the cached tokens with the running maximum and sum of the softmax.  The rows of a tile are the
// queries of one key head: (token, head of the group), 16 or a multiple of them.  A wave takes 32 tokens a step:
//
//   S^T = K q^T    MFMA 16x16x32, first operand two tiles of 16 tokens: a lane's 16 (D = 128) bytes of a key are one
//                  block of 32 values and one scale, converted in registers; lane (row, c) gets the scores of
//                  tokens 4 c .. 4 c + 3 and 16 + 4 c .. 16 + 4 c + 3 of query `row`
//   O^T += V^T P^T the same lanes' weights are the second operand as they stand, in that order of tokens; the first
//                  is made from words of 8 codes of one token each: converted in pairs of values, then
//                  regrouped into pairs of tokens
//
// so that no score or weight leaves its lane.  Codes times their power of two are exact in bf16, whatever the
// queries' type.  bf16 queries multiply as they are and weights are rounded to bf16, an error of at most 2^-8 of each, of
// the size of the output's own rounding; their sum is of the rounded ones, so that they add up to one (a token that
// takes most of the weight would else be off by its own rounding: outputs of equal values were).  A low part of the
// weights beside it takes the whole error from 0.0023 to 0.0017 (32768 tokens), which is the output's rounding alone, and
// costs 5 to 13% for one query (64 sequences 59 -> 62 us) and half as much again for many (a prompt of 4608 tokens 208 ->
// 341).  f16 has three bits more, so f16 queries and weights are taken as a high and a low bf16 part, which hold all of them.
//
// The maximum only moves when a score is more than 2^8 times above it: weights stay below 2^8 and the exchange
// between lanes and the rescaling of O are rare.
#include <algorithm>
#include <type_traits>

#include "qg_attention_rows.h"
#include "qg_device.h"
#include "qg_kernels.h"
#include "qg_rows.h"

namespace qg {

namespace {

constexpr int kAttnWaves = 4;
constexpr int kMaxParts = 64;
constexpr float kLazy = 8.0f;
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ u32x4 bf16_low(const float* v, u32x4 hi) {
  float lo[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float h = bf16_bits_to_f32(e & 1 ? hi[e >> 1] >> 16 : hi[e >> 1] & 0xFFFFu);
    lo[e] = v[e] - h;
  }
  return u32x4{pack2<A_BF16>(lo[0], lo[1]), pack2<A_BF16>(lo[2], lo[3]), pack2<A_BF16>(lo[4], lo[5]), pack2<A_BF16>(lo[6], lo[7])};
}
__device__ __forceinline__ u32x4 bf16_high(const float* v) {
  return u32x4{pack2<A_BF16>(v[0], v[1]), pack2<A_BF16>(v[2], v[3]), pack2<A_BF16>(v[4], v[5]), pack2<A_BF16>(v[6], v[7])};
}
// c + the two bf16 numbers of a word (half the instructions of float32 additions, and these are of the rounded numbers)
__device__ __forceinline__ float add_pair(uint32_t w, float c) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, 0x3F803F80u), c, false);
}
template <int B>
__device__ __forceinline__ uint32_t cvt_pair(uint32_t w, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, B));
}
// UE8M0 byte b of a word -> the conversion's scale.  It takes the exponent field alone: 0 is 2^-127, 255 NaN.
__device__ __forceinline__ uint32_t power_bits(uint32_t word, int b) { return ((word >> (8 * b)) & 0xFFu) << 23; }
constexpr uint32_t kNanPower = 0x7F800000u;

// What a lane loads of a step: 32 tokens.
template <int D>
struct Step {
  static constexpr int KW = D / 32;                 // words of a key per lane
  static constexpr int VU = D == 256 ? 2 : 1;       // 16-byte units of four tokens per tile and lane
  uint32_t k[2][KW];
  uint32_t ks[2];                                   // exponent bytes of the keys' blocks
  u32x4 v[2][VU];
  uint32_t vs[2];                                   // exponent bytes of four tokens
  bool ok[2];                                       // the tile's page is in the cache
};

// row / group for rows below 2^24 and groups of at most 256: group_inv = ceil(2^32 / group)
__device__ __forceinline__ int over_group(int row, const AttnArgs& a) {
  return a.group == 1 ? row : (int)__umulhi((uint32_t)row, a.group_inv);
}

// A sequence's rows of queries and outputs.
__device__ __forceinline__ Queries queries_of(const AttnArgs& a, int b) {
  if (!a.q_offsets) return Queries{b, 1};
  return sequence_queries(a.q_offsets[b], a.q_offsets[b + 1], (int)a.tokens, a.max_q);   // (at most 2^24)
}

// The sequence of workgroup (., y, z).  Workgroups go to the eight dies and on each to its four shader engines in turn, whatever
// work they hold: were y the sequence itself, all of a sequence would go to one of them in batches of 4, 8, ... (4
// sequences of 1152 to 4608 tokens, 512 queries each: 202 us, and 155 turned; decoding of equal ones alike).
__device__ __forceinline__ int turned(uint32_t y, uint32_t z, uint32_t batch) { return (int)((y + z + (z >> 2)) % batch); }

// Values d .. d + N - 1 of a row (a query and its head), and with the first of them its sum of weights and maximum: the
// outputs, or one part's.
template <int T, int D, int N>
__device__ __forceinline__ void store_row(const AttnArgs& a, int hk, int split, int64_t q0, int row, int d, const float* v, float sum,
                                          float top, bool whole) {
  const int qi = over_group(row, a), head = hk * a.group + row - qi * a.group;
  if (!whole) {
    const int64_t at = (int64_t)split * a.rows + (q0 + qi) * a.q_heads + head;
#pragma unroll
    for (int e = 0; e < N; e += 4) *(f32x4*)(a.part + at * D + d + e) = *(const f32x4*)(v + e);
    if (d == 0) {
      float* const ml = a.part + (int64_t)a.nsplit * a.rows * D + at * 2;
      ml[0] = top;
      ml[1] = sum;
    }
  } else {
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;            // a row that sees nothing: zeros
    uint16_t* const o = (uint16_t*)a.out + (q0 + qi) * a.out_stride + head * D + d;
    uint32_t w[N / 2];
#pragma unroll
    for (int e = 0; e < N; e += 2) w[e / 2] = pack2<T == O_F16 ? A_F16 : A_BF16>(v[e] * inv, v[e + 1] * inv);
    if constexpr (N == 8) *(u32x4*)o = u32x4{w[0], w[1], w[2], w[3]};
    else *(u32x2*)o = u32x2{w[0], w[1]};
  }
}

// Up to 16 rows per key head (decoding): one row tile, whose tokens the workgroup's waves take in turn, each with a maximum
// and sums of its own until the end.  Bound by reading the codes, each once.
// (two waves per SIMD at least: with 256 registers or fewer the sums stay where the vector unit reads them)
template <int T, int D>
__global__ __launch_bounds__(64 * kAttnWaves) __attribute__((amdgpu_waves_per_eu(2))) void attention_kernel(AttnArgs a) {
  constexpr bool HILO = T == O_F16;
  constexpr int RT = 1;                             // row tiles (the same without the loops over them is 1 to 3% slower)
  constexpr int KW = D / 32, NJ = D / 16;           // MFMAs of a score tile; tiles of 16 output values
  constexpr int OP = D + 4;
  __shared__ __attribute__((aligned(16))) float so[kAttnWaves * 16 * OP];
  __shared__ float sm[kAttnWaves][16], sl[kAttnWaves][16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, c = lane >> 4;

  // ---- the tile: sequence, key head, rows, tokens -------------------------------------
  // (key heads and sequences fastest: tiles that read the same keys run on the same XCD where their number allows)
  const int hk = blockIdx.x, b = turned(blockIdx.y, blockIdx.z, gridDim.y);
  const int split = blockIdx.z;
  const Queries rows = queries_of(a, b);
  const int64_t q0 = rows.first;
  const int nq = rows.count;
  const int row_count = nq * a.group;
  constexpr int row0 = 0;                           // (all rows are in one tile)
  if (row_count <= 0) return;
  const int len = max(0, min(a.lens[b], a.max_len));
  int sees[RT], qrow[RT];                           // tokens that row 16 t + r sees; its query
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int row = min(row0 + 16 * t + r, row_count - 1);
    qrow[t] = over_group(row, a);
    sees[t] = max(0, len - nq + qrow[t] + 1);
  }
  const int last_row = min(row0 + 16 * RT, row_count) - 1;
  const int most = __builtin_amdgcn_readfirstlane(max(0, len - nq + over_group(last_row, a) + 1));
  const int least = __builtin_amdgcn_readfirstlane(max(0, len - nq + over_group(row0, a) + 1));
  const int steps = (most + 31) >> 5, begin = split * a.chunk, end = min(steps, begin + a.chunk);
  if (split > 0 && begin >= steps) return;          // (the same for all waves)
  const bool whole = steps <= a.chunk;              // one part: the outputs themselves

  // ---- queries ---------------------------------------------------------------------------
  u32x4 qf[RT][KW], ql[HILO ? RT : 1][HILO ? KW : 1];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int row = min(row0 + 16 * t + r, row_count - 1);
    const int head = hk * a.group + row - qrow[t] * a.group;
    const uint16_t* p = (const uint16_t*)a.q + (q0 + qrow[t]) * a.q_stride + head * D + c * (D / 4);
#pragma unroll
    for (int j = 0; j < KW; ++j) {
      qf[t][j] = ldg16(p + 8 * j) ^ a.q_sign;
      if constexpr (HILO) {
        float v[8];
        unpack8<O_F16>(qf[t][j], v);
        qf[t][j] = bf16_high(v);
        ql[t][j] = bf16_low(v, qf[t][j]);
      }
    }
  }

  const int page = 1 << a.page_shift;
  const int64_t half = (int64_t)page * (D / 2), tail = (int64_t)page * (D / 32), head_bytes = 2 * (half + tail);
  const int32_t* const table = a.table + (int64_t)b * a.table_stride;
  const int last_page = max(0, len - 1) >> a.page_shift;
  constexpr int STRIDE = kAttnWaves;
  const int first = begin + wave, count = first < end ? (end - first + STRIDE - 1) / STRIDE : 0;   // this wave's steps
  const uint32_t k_at = r * (D / 2) + c * (D / 8), ks_at = r * (D / 32) + (D == 256 ? 2 * c : D == 128 ? c : c >> 1);
  const uint32_t v_at = c * (2 * D) + 16 * (D == 256 ? 2 * r : D == 128 ? r : r >> 1);
  const uint32_t vs_at = 4 * (c * (D / 32) + (D == 256 ? r >> 1 : D == 128 ? r >> 2 : r >> 3));
  // page of half h of this wave's step n, in lane 2 (n - ids0) + h: the loads of a step wait for no other load
  int ids = 0, ids0 = 0;
  auto load_ids = [&](int n0) __attribute__((always_inline)) {
    ids0 = n0;
    const int t0 = 32 * (first + STRIDE * min(n0 + (lane >> 1), count - 1)) + 16 * (lane & 1);
    ids = table[min(t0 >> a.page_shift, last_page)];
  };
  auto load = [&](int n, Step<D>& s) __attribute__((always_inline)) {
    n = min(n, count - 1);                          // (past the end: the last once more)
    const int step = first + STRIDE * n;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t0 = 32 * step + 16 * h;
      const int id = __builtin_amdgcn_readlane(ids, 2 * (n - ids0) + h);
      s.ok[h] = id >= 0 && id < a.num_pages;
      // (wave-uniform addresses, and per lane the offsets that stay)
      const int t = t0 & (page - 1);
      const uint8_t* const base = a.cache + ((int64_t)(s.ok[h] ? id : 0) * a.kv_heads + hk) * head_bytes;
      const uint8_t* const kb = base + t * (D / 2);
      const uint8_t* const vb = base + half + t * (D / 2);
      const uint8_t* const ksb = base + 2 * half + t * (D / 32);
      const uint8_t* const vsb = base + 2 * half + tail + t * (D / 32);
      if constexpr (KW == 2) {
        const u32x2 w = *(const u32x2*)(kb + k_at);
        s.k[h][0] = w[0];
        s.k[h][1] = w[1];
      } else {
#pragma unroll
        for (int j = 0; j < KW; j += 4) {
          const u32x4 w = ldg16_stream(kb + k_at + 4 * j);
#pragma unroll
          for (int e = 0; e < 4; ++e) s.k[h][j + e] = w[e];
        }
      }
      if constexpr (D == 256) s.ks[h] = *(const uint16_t*)(ksb + ks_at);
      else s.ks[h] = ksb[ks_at];
      s.v[h][0] = ldg16_stream(vb + v_at);
      if constexpr (D == 256) s.v[h][1] = ldg16_stream(vb + v_at + 16);
      s.vs[h] = *(const uint32_t*)(vsb + vs_at);
    }
  };

  f32x4 acc[RT][NJ];
  float m[RT], l[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    m[t] = kNegInf;
    l[t] = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  auto compute = [&](int step, Step<D>& s) __attribute__((always_inline)) {
    // scores: lane (r, c) has tokens 4 c + i (h = 0) and 16 + 4 c + i (h = 1) of each row tile's row r
    f32x4 sc[RT][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 kf[KW];
#pragma unroll
      for (int j = 0; j < KW; ++j) {
        const float p = __uint_as_float(power_bits(s.ks[h], D == 256 ? j >> 2 : 0));
        kf[j] = u32x4{cvt_pair<0>(s.k[h][j], p), cvt_pair<1>(s.k[h][j], p), cvt_pair<2>(s.k[h][j], p), cvt_pair<3>(s.k[h][j], p)};
      }
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KW; ++j) {
          x = mfma16x16x32<A_BF16>(kf[j], qf[t][j], x);
          if constexpr (HILO) x = mfma16x16x32<A_BF16>(kf[j], ql[t][j], x);
        }
        sc[t][h] = x;
      }
    }
    const bool cut = 32 * step + 32 > least || !s.ok[0] || !s.ok[1];   // some row does not see some of the tokens
    if (cut) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!s.ok[h] || 32 * step + 16 * h + 4 * c + i >= sees[t]) sc[t][h][i] = kNegInf;
    }
    // weights
    u32x4 pf[RT], pl[HILO ? RT : 1];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      float top = sc[t][0][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, sc[t][e >> 2][e & 3]);
      top *= a.scale_log2;
      if (__any(top > m[t] + kLazy)) {              // (from -inf on, too)
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float up = fmaxf(m[t], top);
        const float f = up == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m[t] - up);
        m[t] = up;
        l[t] *= f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[t][j] *= f;
      }
      const float base = m[t] == kNegInf ? 0.f : m[t];
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][e >> 2][e & 3], a.scale_log2, -base));
        if constexpr (HILO) l[t] += p[e];
      }
      pf[t] = bf16_high(p);
      if constexpr (HILO) {
        pl[t] = bf16_low(p, pf[t]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) l[t] = add_pair(pf[t][e], l[t]);
      }
    }
    // values: tokens that some row does not see must not reach its sums, weight 0 or not
    uint32_t vp[2][4];
    bool bad[2][4];
    bool any_bad = false;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        vp[h][i] = power_bits(s.vs[h], i);
        bad[h][i] = false;
        if (cut) {
          const int tok = 32 * step + 16 * h + 4 * c + i;
          if (!s.ok[h] || tok >= most) vp[h][i] = 0;                    // seen by no row: what is there does not matter
          bad[h][i] = vp[h][i] == kNanPower;                            // seen by some: its NaN goes to those only
          if (bad[h][i]) vp[h][i] = 0;
          any_bad |= bad[h][i];
        }
      }
    auto values = [&](auto use) __attribute__((always_inline)) {
      constexpr int WORDS = D == 256 ? 2 : 1, PAIRS = D == 64 ? 2 : 4;
#pragma unroll
      for (int w = 0; w < WORDS; ++w) {
        uint32_t word[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) word[h][i] = D == 64 ? s.v[h][0][i] >> (16 * (r & 1)) : s.v[h][w][i];
        auto pair = [&](auto B_) __attribute__((always_inline)) {
          constexpr int B = decltype(B_)::value;
          uint32_t x[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[h][i] = cvt_pair<B>(word[h][i], __uint_as_float(vp[h][i]));
          u32x4 even, odd;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            even[e] = __builtin_amdgcn_perm(x[e >> 1][2 * (e & 1) + 1], x[e >> 1][2 * (e & 1)], 0x05040100u);
            odd[e] = __builtin_amdgcn_perm(x[e >> 1][2 * (e & 1) + 1], x[e >> 1][2 * (e & 1)], 0x07060302u);
          }
          use(8 * w + 2 * B, even);
          use(8 * w + 2 * B + 1, odd);
        };
        pair(std::integral_constant<int, 0>{});
        pair(std::integral_constant<int, 1>{});
        if constexpr (PAIRS == 4) {
          pair(std::integral_constant<int, 2>{});
          pair(std::integral_constant<int, 3>{});
        }
      }
    };
    values([&](int j, u32x4 vf) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        acc[t][j] = mfma16x16x32<A_BF16>(vf, pf[t], acc[t][j]);
        if constexpr (HILO) acc[t][j] = mfma16x16x32<A_BF16>(vf, pl[t], acc[t][j]);
      }
    });
    if (__any(any_bad)) {
      // rare: which sums have a NaN among the values their row sees
      u32x4 nan;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        nan[e] = (bad[e >> 1][2 * (e & 1)] ? 0x3F80u : 0u) | (bad[e >> 1][2 * (e & 1) + 1] ? 0x3F800000u : 0u);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        float seen[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) seen[e] = 32 * step + 16 * (e >> 2) + 4 * c + (e & 3) < sees[t] ? 1.f : 0.f;
        // the count's row rho stands for the values NJ rho .. NJ rho + NJ - 1, which share their blocks
        const f32x4 count = mfma16x16x32<A_BF16>(nan, bf16_high(seen), f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (count[i] > 0.f) acc[t][j][i] = __builtin_nanf("");
      }
    }
  };

  // ---- the tokens, one step's loads ahead (two take registers that a third wave per SIMD needs: 64 sequences of up
  // to 8192 tokens 75 against 66 us) --------------------------------------------------------
  if (count > 0) {
    Step<D> s0, s1;
    load_ids(0);
    load(0, s0);
    for (int n = 0; n < count; n += 2) {
      if (n - ids0 >= 29) load_ids(n);              // (32 steps' pages at a time, of which this turn takes three)
      load(n + 1, s1);
      compute(first + STRIDE * n, s0);
      load(n + 2, s0);
      if (n + 1 < count) compute(first + STRIDE * (n + 1), s1);
    }
  }
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    l[t] += __shfl_xor(l[t], 16, 64);
    l[t] += __shfl_xor(l[t], 32, 64);
  }

  // ---- out: lane (r, c) has values NJ (4 c + i) + j of row r -----------------------------
  // the waves' sums of the same rows, brought to one maximum, in the waves' order
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NJ; j += 4)
      *(f32x4*)&so[(wave * 16 + r) * OP + NJ * (4 * c + i) + j] = f32x4{acc[0][j][i], acc[0][j + 1][i], acc[0][j + 2][i], acc[0][j + 3][i]};
  if (c == 0) {
    sm[wave][r] = m[0];
    sl[wave][r] = l[0];
  }
  __syncthreads();
  constexpr int N = NJ < 8 ? NJ : 8, PIECES = D / N;
  for (int i = tid; i < 16 * PIECES; i += 64 * kAttnWaves) {
    const int row = i / PIECES, d = (i - row * PIECES) * N;
    if (row0 + row >= row_count) continue;
    float top = sm[0][row];
#pragma unroll
    for (int w = 1; w < kAttnWaves; ++w) top = fmaxf(top, sm[w][row]);
    float sum = 0.f, v[N];
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = 0.f;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      const float f = sm[w][row] == kNegInf ? 0.f : __builtin_amdgcn_exp2f(sm[w][row] - top);
      sum += sl[w][row] * f;
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = __builtin_fmaf(so[(w * 16 + row) * OP + d + e], f, v[e]);
    }
    store_row<T, D, N>(a, hk, split, q0, row0 + row, d, v, sum, top, whole);
  }
}

// Many rows per key head (prompts): every wave has 16 RT rows of its own, and the workgroup's waves share the work of making
// operands of 32 tokens' codes: each converts a quarter of them, once for all rows of the workgroup, into an LDS image in the
// order that lanes read (1 KiB per operand, 16 bytes per lane side by side), two images in turn, one barrier per 32
// tokens.  Converted by every wave for itself the operands cost as many instructions as the softmax of 64 rows (RT = 4, 2048
// rows, D = 128: 281 us).  RT is what leaves room for two waves per SIMD, one multiplying while the other
// takes exponentials: those bound it, about as much as the products do.  Products go before other waves' exponentials
// (s_setprio: 5%), and the scheduler mixes a step's conversion into the products of the step before (10 to 15%).  D = 128,
// bf16: a prompt of 4608 tokens (32 query heads over 8) 195 to 220 us from card to card, 790 to 890 TFLOP/s.
template <int T, int D, int RT>
__global__ __launch_bounds__(64 * kAttnWaves) __attribute__((amdgpu_waves_per_eu(2))) void attention_rows_kernel(AttnArgs a) {
  constexpr bool HILO = T == O_F16;
  constexpr int KW = D / 32, NJ = D / 16;
  constexpr int KQ = D == 64 ? 1 : KW / 4, VQ = D == 64 ? 1 : NJ / 8;   // words of a key, and pairs of output tiles, that a wave converts
  __shared__ __attribute__((aligned(16))) u32x4 image[2][2 * KW + NJ][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, c = lane >> 4;
  const int hk = blockIdx.x, b = turned(blockIdx.y, blockIdx.z, gridDim.y);
  // (the last queries first: they see the most tokens; and the first parts, which are whole)
  const int tiles = (int)gridDim.z / a.nsplit, split = (int)blockIdx.z / tiles, tile = tiles - 1 - ((int)blockIdx.z - split * tiles);
  const Queries rows = queries_of(a, b);
  const int64_t q0 = rows.first;
  const int nq = rows.count;
  constexpr int ROWS = 16 * RT * kAttnWaves;
  const int row_count = nq * a.group, tile0 = tile * ROWS, row0 = tile0 + wave * 16 * RT;
  if (tile0 >= row_count) return;
  const int len = max(0, min(a.lens[b], a.max_len));
  // tokens that rows see: all of the workgroup's (fewest, most), this wave's
  auto seen_by = [&](int row) __attribute__((always_inline)) {
    return __builtin_amdgcn_readfirstlane(max(0, len - nq + over_group(min(row, row_count - 1), a) + 1));
  };
  const int all_least = seen_by(tile0), all_most = seen_by(tile0 + ROWS - 1);
  const int least = seen_by(row0), most = row0 < row_count ? seen_by(row0 + 16 * RT - 1) : 0;
  const int steps = (all_most + 31) >> 5, begin = split * a.chunk, end = min(steps, begin + a.chunk);
  if (split > 0 && begin >= steps) return;
  const bool whole = steps <= a.chunk;
  int sees[RT];
  u32x4 qf[RT][KW], ql[HILO ? RT : 1][HILO ? KW : 1];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int row = min(row0 + 16 * t + r, row_count - 1), qi = over_group(row, a);
    sees[t] = max(0, len - nq + qi + 1);
    const int head = hk * a.group + row - qi * a.group;
    const uint16_t* p = (const uint16_t*)a.q + (q0 + qi) * a.q_stride + head * D + c * (D / 4);
#pragma unroll
    for (int j = 0; j < KW; ++j) {
      qf[t][j] = ldg16(p + 8 * j) ^ a.q_sign;
      if constexpr (HILO) {
        float v[8];
        unpack8<O_F16>(qf[t][j], v);
        qf[t][j] = bf16_high(v);
        ql[t][j] = bf16_low(v, qf[t][j]);
      }
    }
  }

  const int page = 1 << a.page_shift;
  const int64_t half = (int64_t)page * (D / 2), tail = (int64_t)page * (D / 32), head_bytes = 2 * (half + tail);
  const int32_t* const table = a.table + (int64_t)b * a.table_stride;
  const int last_page = max(0, len - 1) >> a.page_shift;
  // this wave's quarter: words KQ wave .. of each lane's part of a key (D = 64: of two, waves 0 and 1), pairs VQ wave .. of
  // the output tiles (D = 64: of two, likewise)
  const int part = D == 64 ? wave & 1 : wave;
  const uint32_t k_at = r * (D / 2) + c * (D / 8) + 4 * KQ * part, ks_at = r * (D / 32) + (D == 256 ? 2 * c : D == 128 ? c : c >> 1);
  const uint32_t v_at = c * (2 * D) + 16 * (D == 256 ? 2 * r + (part >> 1) : D == 128 ? r : r >> 1);
  const uint32_t vs_at = 4 * (c * (D / 32) + (D == 256 ? r >> 1 : D == 128 ? r >> 2 : r >> 3));
  struct Raw { uint32_t k[2][KQ], ks[2], vs[2]; u32x4 v[2]; bool ok[2]; };
  // (pages in lanes, as in attention_kernel)
  int ids = 0, ids0 = 0;
  auto load_ids = [&](int step) __attribute__((always_inline)) {
    ids0 = step;
    ids = table[min((32 * (step + (lane >> 1)) + 16 * (lane & 1)) >> a.page_shift, last_page)];
  };
  auto load = [&](int step, Raw& s) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t0 = 32 * step + 16 * h, id = __builtin_amdgcn_readlane(ids, 2 * (step - ids0) + h);
      s.ok[h] = id >= 0 && id < a.num_pages;
      const int t = t0 & (page - 1);
      const uint8_t* const base = a.cache + ((int64_t)(s.ok[h] ? id : 0) * a.kv_heads + hk) * head_bytes;
      const uint8_t* const kb = base + t * (D / 2);
      const uint8_t* const ksb = base + 2 * half + t * (D / 32);
#pragma unroll
      for (int i = 0; i < KQ; ++i) s.k[h][i] = *(const uint32_t*)(kb + k_at + 4 * i);
      if constexpr (D == 256) s.ks[h] = *(const uint16_t*)(ksb + ks_at);
      else s.ks[h] = ksb[ks_at];
      s.v[h] = ldg16(base + half + t * (D / 2) + v_at);
      s.vs[h] = *(const uint32_t*)(base + 2 * half + tail + t * (D / 32) + vs_at);
    }
  };
  // a step's exponent bytes of values, where NaN is among them that some row of the workgroup does not see: see attention_kernel
  struct Odd { uint32_t vs[2]; bool any, ok[2]; };
  auto odd_value = [&](int step, const Odd& o, int h, int i) __attribute__((always_inline)) {
    return ((o.vs[h] >> (8 * i)) & 0xFFu) == 0xFFu && o.ok[h] && 32 * step + 16 * h + 4 * c + i < all_most;
  };
  auto powers = [&](int step, const Raw& s, uint32_t (&vp)[2][4], Odd& odd) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      odd.vs[h] = s.vs[h];
      odd.ok[h] = s.ok[h];
#pragma unroll
      for (int i = 0; i < 4; ++i) vp[h][i] = power_bits(s.vs[h], i);
    }
    odd.any = false;
    if (32 * step + 32 > all_least || !s.ok[0] || !s.ok[1]) {
      bool bad = false;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool o = odd_value(step, odd, h, i);
          bad |= o;
          if (o || !s.ok[h] || 32 * step + 16 * h + 4 * c + i >= all_most) vp[h][i] = 0;
        }
      odd.any = __any(bad);
    }
  };
  auto emit = [&](const Raw& s, const uint32_t (&vp)[2][4], u32x4 (*to)[64]) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < KQ; ++i) {
        const int j = KQ * part + i;                // (D = 256: words 0-3 are of the first block)
        const float p = __uint_as_float(D == 256 ? ((s.ks[h] >> (part >= 2 ? 8 : 0)) & 0xFFu) << 23 : power_bits(s.ks[h], 0));
        if (D != 64 || wave < 2)
          to[h * KW + j][lane] = u32x4{cvt_pair<0>(s.k[h][i], p), cvt_pair<1>(s.k[h][i], p), cvt_pair<2>(s.k[h][i], p), cvt_pair<3>(s.k[h][i], p)};
      }
#pragma unroll
    for (int i = 0; i < VQ; ++i) {
      // pair `part` of the word (D = 64: of its half; D = 256: two pairs of the word that part / 2 names)
      const int pair = D == 256 ? 2 * (part & 1) + i : part, shift = 8 * pair + (D == 64 ? 16 * (r & 1) : 0);
      uint32_t x[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[h][e] = cvt_pair<0>(s.v[h][e] >> shift, __uint_as_float(vp[h][e]));
      u32x4 even, odd_v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        even[e] = __builtin_amdgcn_perm(x[e >> 1][2 * (e & 1) + 1], x[e >> 1][2 * (e & 1)], 0x05040100u);
        odd_v[e] = __builtin_amdgcn_perm(x[e >> 1][2 * (e & 1) + 1], x[e >> 1][2 * (e & 1)], 0x07060302u);
      }
      const int j = D == 256 ? 8 * (part >> 1) + 2 * pair : 2 * pair;
      if (D != 64 || wave >= 2) {
        to[2 * KW + j][lane] = even;
        to[2 * KW + j + 1][lane] = odd_v;
      }
    }
  };

  f32x4 acc[RT][NJ];
  float m[RT], l[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    m[t] = kNegInf;
    l[t] = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  auto compute = [&](int step, const u32x4 (*from)[64], const Odd& odd, auto&& beside) __attribute__((always_inline)) {
    // operands are read AHEAD of the products that take them
    constexpr int AHEAD = 3, NK = 2 * KW;
    u32x4 ring[AHEAD + 1];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) ring[i] = from[i][lane];
    f32x4 sc[RT][2];
    __builtin_amdgcn_s_setprio(1);
    beside();
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int h = i / KW, j = i % KW;
      ring[(i + AHEAD) % (AHEAD + 1)] = from[i + AHEAD][lane];     // (the first ones of the values at the end)
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        sc[t][h] = mfma16x16x32<A_BF16>(ring[i % (AHEAD + 1)], qf[t][j], j == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : sc[t][h]);
        if constexpr (HILO) sc[t][h] = mfma16x16x32<A_BF16>(ring[i % (AHEAD + 1)], ql[t][j], sc[t][h]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(0);
    if (32 * step + 32 > least || !odd.ok[0] || !odd.ok[1]) {
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!odd.ok[h] || 32 * step + 16 * h + 4 * c + i >= sees[t]) sc[t][h][i] = kNegInf;
    }
    float top[RT];
    bool up = false;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      top[t] = sc[t][0][0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top[t] = fmaxf(top[t], sc[t][e >> 2][e & 3]);
      top[t] *= a.scale_log2;
      up |= top[t] > m[t] + kLazy;
    }
    if (__any(up)) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        float x = fmaxf(top[t], __shfl_xor(top[t], 16, 64));
        x = fmaxf(m[t], fmaxf(x, __shfl_xor(x, 32, 64)));
        const float f = x == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m[t] - x);
        m[t] = x;
        l[t] *= f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[t][j] *= f;
      }
    }
    u32x4 pf[RT], pl[HILO ? RT : 1];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const float base = m[t] == kNegInf ? 0.f : m[t];
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][e >> 2][e & 3], a.scale_log2, -base));
      pf[t] = bf16_high(p);
      if constexpr (HILO) {
        l[t] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
        pl[t] = bf16_low(p, pf[t]);
      } else {
        l[t] = add_pair(pf[t][3], add_pair(pf[t][2], add_pair(pf[t][1], add_pair(pf[t][0], l[t]))));
      }
    }
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int i = NK + j;
      if (j + AHEAD < NJ) ring[(i + AHEAD) % (AHEAD + 1)] = from[i + AHEAD][lane];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        acc[t][j] = mfma16x16x32<A_BF16>(ring[i % (AHEAD + 1)], pf[t], acc[t][j]);
        if constexpr (HILO) acc[t][j] = mfma16x16x32<A_BF16>(ring[i % (AHEAD + 1)], pl[t], acc[t][j]);
      }
    }
    __builtin_amdgcn_s_setprio(0);
    if (odd.any) {
      u32x4 nan = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (odd_value(step, odd, e >> 2, e & 3)) nan[e >> 1] |= e & 1 ? 0x3F800000u : 0x3F80u;
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        float seen[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) seen[e] = 32 * step + 16 * (e >> 2) + 4 * c + (e & 3) < sees[t] ? 1.f : 0.f;
        const f32x4 count = mfma16x16x32<A_BF16>(nan, bf16_high(seen), f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (count[i] > 0.f) acc[t][j][i] = __builtin_nanf("");
      }
    }
  };
  // step n's image is made among step n - 1's first products, from codes loaded a step earlier still
  if (begin < end) {
    Raw raw;
    Odd odd, odd_next;
    uint32_t vp[2][4];
    load_ids(begin);
    load(begin, raw);
    powers(begin, raw, vp, odd);
    emit(raw, vp, image[0]);
    load(min(begin + 1, end - 1), raw);
    __syncthreads();
    for (int step = begin; step < end; ++step) {
      const int at = (step - begin) & 1;
      const int next = min(step + 1, end - 1), later = min(step + 2, end - 1);      // (the last ones are made again, for nothing)
      powers(next, raw, vp, odd_next);
      if (later - ids0 >= 32) load_ids(later);
      auto beside = [&]() __attribute__((always_inline)) {
        emit(raw, vp, image[at ^ 1]);
        load(later, raw);
      };
      if (32 * step < most) compute(step, image[at], odd, beside);
      else beside();
      odd = odd_next;
      __syncthreads();
    }
  }
  if (row0 >= row_count) return;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    l[t] += __shfl_xor(l[t], 16, 64);
    l[t] += __shfl_xor(l[t], 32, 64);
    const int row = row0 + 16 * t + r;
    if (row >= row_count) continue;
    constexpr int N = NJ < 8 ? NJ : 8;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < NJ; j += N) {
        float v[N];
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = acc[t][j + e][i];
        store_row<T, D, N>(a, hk, split, q0, row, NJ * (4 * c + i) + j, v, l[t], m[t], whole);
      }
  }
}

// Steps that a row's tile was taken in: its parts are those of a.chunk steps each.
__device__ __forceinline__ int steps_of(const AttnArgs& a, int b, int nq, int qi, int head) {
  const int row_count = nq * a.group, in_group = qi * a.group + head - over_group(head, a) * a.group;
  const int last_row = min(in_group - in_group % a.tile_rows + a.tile_rows, row_count) - 1;
  const int len = max(0, min(a.lens[b], a.max_len));
  return (max(0, len - nq + over_group(last_row, a) + 1) + 31) >> 5;
}

// A row's parts, brought to one maximum, in a fixed order.  One workgroup per row: D / 4 threads take four values
// each, 1024 / D groups of them every so many-th part, so that a long sequence's parts are read side by side.
template <int T, int D>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a) {
  constexpr int LPR = D / 4, GROUPS = 256 / LPR;
  __shared__ float weight[kMaxParts];
  __shared__ __attribute__((aligned(16))) float sums[GROUPS][D];
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
  const Queries rows = queries_of(a, b);
  const int64_t q0 = rows.first;
  const int nq = rows.count;
  const int head = blockIdx.x, qi = blockIdx.z;
  if (qi >= nq) return;
  const int steps = steps_of(a, b, nq, qi, head);
  if (steps <= a.chunk) return;                     // one part: written already
  const int64_t row = (q0 + qi) * a.q_heads + head;
  const float* ml = a.part + (int64_t)a.nsplit * a.rows * D + row * 2;
  // every wave: maximum and sum of all parts (64 or fewer, one per lane)
  const float ms = lane * a.chunk < steps ? ml[(int64_t)lane * a.rows * 2] : kNegInf;
  const float ls = lane * a.chunk < steps ? ml[(int64_t)lane * a.rows * 2 + 1] : 0.f;
  const float top = over_lanes<64>(ms, [](float x, float y) { return fmaxf(x, y); });
  const float f = ms == kNegInf ? 0.f : __builtin_amdgcn_exp2f(ms - top);
  const float sum = over_lanes<64>(ls * f, [](float x, float y) { return x + y; });
  if (tid < 64) weight[lane] = f;
  __syncthreads();
  const int g = tid / LPR, d = (tid % LPR) * 4;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = g; s * a.chunk < steps; s += GROUPS) v += *(const f32x4*)(a.part + ((int64_t)s * a.rows + row) * D + d) * weight[s];
  *(f32x4*)&sums[g][d] = v;
  __syncthreads();
  if (g != 0) return;
#pragma unroll
  for (int i = 1; i < GROUPS; ++i) v += *(const f32x4*)&sums[i][d];
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  constexpr int AF = T == O_F16 ? A_F16 : A_BF16;
  *(u32x2*)((uint16_t*)a.out + (q0 + qi) * a.out_stride + head * D + d) =
      u32x2{pack2<AF>(v[0] * inv, v[1] * inv), pack2<AF>(v[2] * inv, v[3] * inv)};
}

// The same for many rows of few parts: D / 4 lanes per row, 1024 / D rows per workgroup.
template <int T, int D>
__global__ __launch_bounds__(256) void attention_join_rows_kernel(AttnArgs a) {
  constexpr int LPR = D / 4, RPB = 256 / LPR;
  const int b = blockIdx.y, qi = blockIdx.z;
  const Queries rows = queries_of(a, b);
  const int64_t q0 = rows.first;
  const int nq = rows.count;
  const int head = (int)blockIdx.x * RPB + threadIdx.x / LPR, d = (threadIdx.x % LPR) * 4;
  if (qi >= nq || head >= a.q_heads) return;
  const int steps = steps_of(a, b, nq, qi, head);
  if (steps <= a.chunk) return;                     // one part: written already
  const int64_t row = (q0 + qi) * a.q_heads + head;
  const float* const ml = a.part + (int64_t)a.nsplit * a.rows * D + row * 2;
  float top = kNegInf, sum = 0.f;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s * a.chunk < steps; ++s) {
    const float ms = ml[(int64_t)s * a.rows * 2], ls = ml[(int64_t)s * a.rows * 2 + 1];
    const f32x4 o = *(const f32x4*)(a.part + ((int64_t)s * a.rows + row) * D + d);
    const float up = fmaxf(top, ms);
    const float f0 = top == kNegInf ? 0.f : __builtin_amdgcn_exp2f(top - up), f1 = ms == kNegInf ? 0.f : __builtin_amdgcn_exp2f(ms - up);
    sum = sum * f0 + ls * f1;
    v = v * f0 + o * f1;
    top = up;
  }
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  constexpr int AF = T == O_F16 ? A_F16 : A_BF16;
  *(u32x2*)((uint16_t*)a.out + (q0 + qi) * a.out_stride + head * D + d) =
      u32x2{pack2<AF>(v[0] * inv, v[1] * inv), pack2<AF>(v[2] * inv, v[3] * inv)};
}

// Row tiles of a wave of attention_rows_kernel.
constexpr int many_rows(int type, int dim) {
  return dim == 256 ? 1 : type == O_BF16 ? (dim == 64 ? 4 : 3) : (dim == 64 ? 3 : 2);
}
constexpr bool shares_rows(int64_t rows) { return rows <= 16; }
constexpr int tile_of(int type, int dim, bool share) { return share ? 16 : 16 * kAttnWaves * many_rows(type, dim); }   // rows of a workgroup

template <int T, int D>
void launch_one(AttnArgs a, hipStream_t st) {
  const int64_t rows = (int64_t)a.max_q * a.group;
  const bool share = shares_rows(rows);
  a.tile_rows = tile_of(T, D, share);
  const dim3 grid(a.kv_heads, a.batch, (unsigned)((rows + a.tile_rows - 1) / a.tile_rows * a.nsplit));
  if (share) hipLaunchKernelGGL((attention_kernel<T, D>), grid, dim3(64 * kAttnWaves), 0, st, a);
  else hipLaunchKernelGGL((attention_rows_kernel<T, D, many_rows(T, D)>), grid, dim3(64 * kAttnWaves), 0, st, a);
  if (a.nsplit == 1) return;
  // a workgroup per row while the rows are few
  constexpr int RPB = 1024 / D;
  if ((int64_t)a.batch * a.max_q * a.q_heads <= 4096)
    hipLaunchKernelGGL((attention_join_kernel<T, D>), dim3(a.q_heads, a.batch, a.max_q), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((attention_join_rows_kernel<T, D>), dim3((a.q_heads + RPB - 1) / RPB, a.batch, a.max_q), dim3(256), 0, st, a);
}

}  // namespace

// Parts of 32 * chunk tokens: of equal work whatever the sequences' lengths.  Decoding: as many as fill the GPU if all
// sequences had the maximum, none shorter than 512 tokens (what a part costs beside its tokens).  Many rows: only while a
// workgroup per tile leaves CUs without two (a prompt of 4608 tokens, 768 tiles: whole 210 us, in parts 222 and 15 to join
// them; 4 sequences of up to 4608 tokens with 512 new ones each, 352 tiles: whole 203 us, in three parts 158
// and 18, in two 160 and 12; one sequence of 8192 with 2048 new ones, 344 tiles: three 321 and 21, two 358 and 15: three
// cost the first 4 us and save the second 31).  Every sequence counts as if it had max_q queries: single tokens of long
// sequences beside a chunk are not split (one chunk of 512 among 63 single tokens of up to 32768, 64 heads over 8: 1272 us,
// in two calls 134 and 225), and more than 16 rows per key head go to the many rows' kernel (3 queries of 64 sequences of up
// to 8192, 24 rows: 324 us, one query 59 and 6).
AttnSplit attn_split(int64_t batch, int q_heads, int kv_heads, int64_t max_q, int64_t max_len, int dim, int type) {
  const int64_t rows = max_q * (q_heads / kv_heads);
  const bool share = shares_rows(rows);
  const int64_t per = tile_of(type, dim, share), row_tiles = (rows + per - 1) / per;
  const int64_t tiles = batch * kv_heads * row_tiles, steps = std::max<int64_t>(1, (max_len + 31) / 32);
  int64_t chunk = std::max({steps * tiles / (share ? 2048 : 1024), (int64_t)16, (steps + kMaxParts - 1) / kMaxParts});
  if (!share && tiles >= 512) chunk = steps;
  chunk = std::min((chunk + 3) / 4 * 4, (steps + 3) / 4 * 4);
  return AttnSplit{(int)((steps + chunk - 1) / chunk), (int)chunk, row_tiles};
}

bool launch_attention(const AttnArgs& a, int type, hipStream_t st) {
  if (a.dim == 64) type == O_BF16 ? launch_one<O_BF16, 64>(a, st) : launch_one<O_F16, 64>(a, st);
  else if (a.dim == 128) type == O_BF16 ? launch_one<O_BF16, 128>(a, st) : launch_one<O_F16, 128>(a, st);
  else if (a.dim == 256) type == O_BF16 ? launch_one<O_BF16, 256>(a, st) : launch_one<O_F16, 256>(a, st);
  else return false;
  return true;
}

}  // namespace qg
