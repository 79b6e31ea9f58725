// Low-rank adapters of many requests beside a projection that they share:
//
//   t[m][s] = x[m] A[a, s]^T over the adapter's rank rows,  y[m][n] = base[m][n] + scale[a] sum_r t[m][s(n)][r] B[a, n, r]
//
// for the adapter a of token m and the slice s(n) of column n.  Tokens come in blocks of BM rows of one adapter
// (qg_moe_align's map).  The first product makes t in float32, partial sums over `ksplit` parts of K, each
// in a place of its own, so that no order is left to chance.  Few tokens (blocks of 16): the second one adds the parts
// itself, two launches in all, which bound them (1 token, 7168 to 7168, rank 16: 4.2 + 4.3 us).  Many: a launch between
// adds them once, and both products pass their operands through LDS.  Bound by bytes, of which the second product's
// outputs, read and written, are most (8192 tokens, 4096 to 2 x 2816, rank 128, 252 MB: 43 + 10 + 65 us).
//
// Both products run on 16x16x32 MFMAs with the adapter's rows as first operand, so that a lane's sums belong to
// one token: four ranks side by side of t, and, with the columns of two tiles interleaved, eight columns
// side by side of y.
//
// t is split into two 16-bit numbers, high and low part, which together carry at least 16 (bf16) or 22 (f16) bits
// of it: one number alone would cost the last bit of y.  f16 parts are taken from t over a power of two of the
// token, so that no t leaves the type's range.
#include <type_traits>

#include "qg_device.h"
#include "qg_kernels.h"
#include "qg_rows.h"

namespace qg {

namespace {

constexpr int kWaves = 4;

template <int T, int BM, int RT>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2))) void lora_shrink_kernel(LoraArgs a) {
  constexpr int AF = T == O_F16 ? A_F16 : A_BF16;
  constexpr int TT = BM / 16;
  constexpr int STEP = 64;                                    // K of a wave's step: one 128-byte line of every row
  __shared__ __attribute__((aligned(16))) float sum[kWaves][BM][RT * 16 + 4];
  const int64_t row0 = (int64_t)blockIdx.x * BM;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  int f[TT];                                                  // (the map is written to its end: read before it is asked for)
#pragma unroll
  for (int t = 0; t < TT; ++t) f[t] = a.sorted_ids[row0 + 16 * t + r];
  const int f0 = a.sorted_ids[row0];
  const int adapter = a.expert_ids[blockIdx.x];               // (blocks are of 16 rows here)
  if (row0 >= (int64_t)*a.num_post_pad) return;
  const int rank = a.ranks ? max(0, min(a.ranks[adapter], a.max_rank)) : a.max_rank;

  const uint16_t* xp[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t)                                // a block's first row is a token; its sums are not used twice
    xp[t] = (const uint16_t*)a.x + (int64_t)(f[t] < 0 || f[t] >= a.tokens ? f0 : f[t]) * a.x_stride + 8 * g;
  const uint16_t* ap[RT];
  bool has[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int row = (blockIdx.z * RT + t) * 16 + r;           // of all slices' rows
    has[t] = row < a.rank_rows && row % a.max_rank < rank;
    ap[t] = (const uint16_t*)a.a + ((int64_t)adapter * a.rank_rows + (has[t] ? row : 0)) * a.k + 8 * g;
  }
  f32x4 acc[RT][TT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int u = 0; u < TT; ++u) acc[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int steps = (a.k + STEP - 1) / STEP;
  const int per = (steps + a.ksplit - 1) / a.ksplit;
  const int first = (int)blockIdx.y * per, end = min(steps, first + per);
  struct Ops { u32x4 x[2][TT], w[2][RT]; };
  auto load = [&](int s, Ops& o) __attribute__((always_inline)) {
    const int k0 = s * STEP;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = s < end && k0 + 32 * h + 8 * g < a.k;   // (k % 8 == 0)
#pragma unroll
      for (int t = 0; t < RT; ++t) o.w[h][t] = in && has[t] ? ldg16(ap[t] + k0 + 32 * h) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int t = 0; t < TT; ++t) o.x[h][t] = in ? ldg16(xp[t] + k0 + 32 * h) : u32x4{0, 0, 0, 0};
    }
  };
  auto multiply = [&](const Ops& o) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int u = 0; u < TT; ++u) acc[t][u] = mfma16x16x32<AF>(o.w[h][t], o.x[h][u], acc[t][u]);
  };
  Ops now, next;
  load(first + wave, now);
  for (int s = first + wave; s < end; s += 2 * kWaves) {
    load(s + kWaves, next);
    multiply(now);
    load(s + 2 * kWaves, now);
    multiply(next);
  }
  // the waves' sums, in their order
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int u = 0; u < TT; ++u) *(f32x4*)&sum[wave][16 * u + r][16 * t + 4 * g] = acc[t][u];
  __syncthreads();
  for (int i = tid; i < BM * RT * 4; i += 64 * kWaves) {
    const int row = i / (RT * 4), c = i - row * (RT * 4);
    f32x4 v = *(const f32x4*)&sum[0][row][4 * c];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += *(const f32x4*)&sum[w][row][4 * c];
    const int at = blockIdx.z * RT * 16 + 4 * c;
    if (at < a.rank_pitch)
      *(f32x4*)(a.part + ((int64_t)blockIdx.y * a.cap_rows + row0 + row) * a.rank_pitch + at) = v;
  }
}

// Place of 16-byte chunk c of row `row` in an LDS image of rows of CH chunks, such that the lanes that an LDS read of 16
// bytes per lane serves together (0-3, 12-15, 20-23, 24-27, then 4-11, 16-19, 28-31, and so on) use every bank once when
// lane l reads chunk l / 16 + a constant of row l % 16.
template <int CH>
__device__ __forceinline__ int swizzled(int row, int c) {
  if constexpr (CH == 2) return c;
  else if constexpr (CH == 4) return c ^ (-(row >> 2) & 3);
  else if constexpr (CH == 8) return c ^ ((row >> 1) & 7);
  else return c ^ (row & 15);
}

// The first product for blocks of many tokens.  What its lanes multiply are 16 rows' 16 bytes, and loads in that order
// (neighbouring lanes in different rows) take the cache an access per lane: with both operands loaded so, 16 bytes per
// clock and CU bound it (8192 tokens, K = 4096, 256 rank rows 95 us, 16 rank rows 26 us).  So both go into LDS, whole
// lines of rows side by side, through a ring of NS stages of STEP values of K.  WT waves share the tokens, 4 / WT the
// rank rows: tokens while there are few rank rows (each wave then reads all of them), rank rows above.
template <int T, int BM, int RTALL, int WT>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2))) void lora_shrink_staged_kernel(LoraArgs a) {
  constexpr int AF = T == O_F16 ? A_F16 : A_BF16;
  constexpr int TT = BM / 16 / WT, RT = RTALL / (kWaves / WT);
  constexpr int STEP = BM == 16 ? 128 : BM == 64 ? 64 : 32, CH = STEP / 8;
  constexpr int ROWS = BM + 16 * RTALL, STAGE = ROWS * STEP * 2, NS = STAGE <= 16384 ? 4 : 3;
  constexpr int NI = STAGE / 1024 / kWaves;                    // 1 KiB loads of a wave per stage
  static_assert(NI * 1024 * kWaves == STAGE, "whole loads");
  __shared__ __attribute__((aligned(16))) uint8_t ring[NS * STAGE];
  const int64_t row0 = (int64_t)blockIdx.x * BM;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int f0 = a.sorted_ids[row0], adapter = a.expert_ids[row0 >> a.block_shift];
  // (a tile may be a part of a block; tokens come first in an adapter's rows: without one there is nothing behind)
  if (row0 >= (int64_t)*a.num_post_pad || f0 < 0 || f0 >= a.tokens) return;
  const int rank = a.ranks ? max(0, min(a.ranks[adapter], a.max_rank)) : a.max_rank;
  const int rank0 = blockIdx.z * RTALL * 16;

  // what this lane loads of a stage: chunk `at` (first of K) of a token's row or of an adapter's; rows that do not count
  // are the first's once more (of tokens: sums that are not used; of ranks: taken out of the operand below)
  const uint16_t* src[NI];
  int at[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int piece = (i * kWaves + wave) * 64 + lane, row = piece / CH, c = swizzled<CH>(row, piece % CH);
    at[i] = 8 * c;
    if ((i * kWaves + wave) * 64 < BM * CH) {
      const int f = a.sorted_ids[row0 + row];
      src[i] = (const uint16_t*)a.x + (int64_t)(f < 0 || f >= a.tokens ? f0 : f) * a.x_stride;
    } else {
      const int q = rank0 + row - BM;
      src[i] = (const uint16_t*)a.a + ((int64_t)adapter * a.rank_rows + (q < a.rank_rows && q % a.max_rank < rank ? q : 0)) * a.k;
    }
  }
  const int tok0 = (WT == 1 ? 0 : wave) * TT * 16, rt0 = (WT == 1 ? wave : 0) * RT;   // this wave's share
  bool has[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int q = rank0 + (rt0 + t) * 16 + r;
    has[t] = q < a.rank_rows && q % a.max_rank < rank;
  }
  f32x4 acc[RT][TT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int u = 0; u < TT; ++u) acc[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int steps = (a.k + STEP - 1) / STEP;
  const int per = (steps + a.ksplit - 1) / a.ksplit;
  const int first = (int)blockIdx.y * per, end = min(steps, first + per);
  auto load = [&](int s, int slot) __attribute__((always_inline)) {   // (past the end: the last once more, never read)
    const int k0 = min(s, end - 1) * STEP;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      gload16_lds(src[i] + min(k0 + at[i], a.k - 8), ring + slot * STAGE + (i * kWaves + wave) * 1024);
    __builtin_amdgcn_sched_barrier(0);
  };
  if (first < end) {
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) load(first + i, i);
    int slot = 0;
    for (int s = first; s < end; ++s) {
      wait_loads<(NS - 2) * NI>();                             // this wave's part of stage s
      group_barrier();                                         // the whole of it, and stage s - 1 has been read by all
      load(s + NS - 1, slot == 0 ? NS - 1 : slot - 1);
      const uint8_t* const sb = ring + slot * STAGE;
#pragma unroll
      for (int h = 0; h < STEP / 32; ++h) {
        const bool in = s * STEP + 32 * h + 8 * g < a.k;       // (k % 8 == 0)
        u32x4 xv[TT];
#pragma unroll
        for (int u = 0; u < TT; ++u) {
          const int row = tok0 + 16 * u + r;
          xv[u] = *(const u32x4*)(sb + (row * CH + swizzled<CH>(row, 4 * h + g)) * 16);
          xv[u] = in ? xv[u] : u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const int row = BM + (rt0 + t) * 16 + r;
          u32x4 wv = *(const u32x4*)(sb + (row * CH + swizzled<CH>(row, 4 * h + g)) * 16);
          wv = in && has[t] ? wv : u32x4{0, 0, 0, 0};
#pragma unroll
          for (int u = 0; u < TT; ++u) acc[t][u] = mfma16x16x32<AF>(wv, xv[u], acc[t][u]);
        }
      }
      slot = slot == NS - 1 ? 0 : slot + 1;
    }
  }
  wait_loads<0>();                                             // the last stages land before the LDS is another workgroup's
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int q = rank0 + (rt0 + t) * 16 + 4 * g;
    if (q >= a.rank_pitch) continue;
#pragma unroll
    for (int u = 0; u < TT; ++u)
      *(f32x4*)(a.part + ((int64_t)blockIdx.y * a.cap_rows + row0 + tok0 + 16 * u + r) * a.rank_pitch + q) = acc[t][u];
  }
}

// Four ranks' sums of a token, as two 16-bit numbers each, into its row of LDS (`low` elements between the parts); LPR
// neighbouring lanes hold a token's ranks.  f16: over the power of two of the token's largest, which joins its scale.
template <int T, int LPR>
__device__ __forceinline__ void split_row(f32x4 v, int first, int rank, float scale, uint16_t* high, int low, float* row_scale) {
  constexpr int AF = T == O_F16 ? A_F16 : A_BF16;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = first + j < rank ? v[j] : 0.f;   // (0 * x, and x may be infinite)
  if constexpr (T == O_F16) {
    float amax = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
    for (int off = 1; off < LPR; off <<= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
    const int e = amax > 0.f && amax < __builtin_inff() ? __builtin_amdgcn_frexp_expf(amax) : 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __builtin_ldexpf(v[j], -e);
    scale = __builtin_ldexpf(scale, e);
  }
  float lo[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float hi = to_f32<T>(f32_to_out<T>(v[j]));
    lo[j] = fabsf(hi) < __builtin_inff() ? v[j] - hi : 0.f;
  }
  *(u32x2*)high = u32x2{pack2<AF>(v[0], v[1]), pack2<AF>(v[2], v[3])};
  *(u32x2*)(high + low) = u32x2{pack2<AF>(lo[0], lo[1]), pack2<AF>(lo[2], lo[3])};
  if (row_scale) *row_scale = scale;
}

// RS: MFMAs (of 32 ranks) per tile, 0: up to 16 ranks, whose high and low parts share one MFMA.  A wave takes every
// kWaves-th pair of column tiles, the operands of the next pair on their way meanwhile.
template <int T, int BM, int RS>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2))) void lora_expand_kernel(LoraArgs a) {
  constexpr int AF = T == O_F16 ? A_F16 : A_BF16;
  constexpr int TT = BM / 16;
  constexpr int RP = RS == 0 ? 16 : 32 * RS;                  // ranks with padding
  constexpr int KS = RS == 0 ? 1 : RS;
  constexpr int KC = KS < 2 ? KS : 2, CH = KS / KC;           // operands are taken in CH chunks of KC MFMAs' ranks
  constexpr int PITCH = 2 * RP + 8;                           // 16-bit elements: [high RP | low RP], rows 16 bytes apart in banks
  __shared__ __attribute__((aligned(16))) uint16_t st[BM * PITCH];
  __shared__ float row_scale[BM];
  const int block = (int)blockIdx.x / a.col_tiles;
  const int64_t row0 = (int64_t)block * BM;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  int tok[TT];
#pragma unroll
  for (int u = 0; u < TT; ++u) tok[u] = a.sorted_ids[row0 + 16 * u + r];
  const int adapter = a.expert_ids[block];
  if (row0 >= (int64_t)*a.num_post_pad) return;
  const int rank = a.ranks ? max(0, min(a.ranks[adapter], a.max_rank)) : a.max_rank;
  // the workgroup's slice and columns
  const int cols = 32 * kWaves * a.col_pairs;
  int slice = 0, col0 = 0, tile = (int)blockIdx.x - block * a.col_tiles, col_end = 0;
  for (int begin = 0;; ++slice) {
    col_end = a.slice_end[slice];
    const int tiles = (col_end - begin + cols - 1) / cols;
    if (tile < tiles) { col0 = begin + tile * cols; break; }
    tile -= tiles;
    begin = col_end;
  }
#pragma unroll
  for (int u = 0; u < TT; ++u) tok[u] = tok[u] < a.tokens ? tok[u] : -1;

  // a pair of column tiles: row rho of tile j is column 8 (rho / 4) + 4 j + rho % 4, so that a lane's sums are 8 columns
  // side by side
  typedef u32x4 Weights[KC][2];
  typedef u32x4 Rows[TT];
  const uint16_t* const bw = (const uint16_t*)a.b + (int64_t)adapter * a.n * a.max_rank;
  auto load_b = [&](int p, int ch, Weights& w) __attribute__((always_inline)) {
    const int n0 = col0 + (p * kWaves + wave) * 32;
#pragma unroll
    for (int k = 0; k < KC; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int n = n0 + 8 * (r >> 2) + 4 * j + (r & 3);
        const int c = RS == 0 ? g & 1 : 4 * (ch * KC + k) + g;   // chunk of 8 ranks
        w[k][j] = p < a.col_pairs && n < col_end && 8 * c < rank ? ldg16(bw + (int64_t)n * a.max_rank + 8 * c) : u32x4{0, 0, 0, 0};
      }
  };
  auto load_y = [&](int p, Rows& y) __attribute__((always_inline)) {
    const int n = col0 + (p * kWaves + wave) * 32 + 8 * g;
#pragma unroll
    for (int u = 0; u < TT; ++u)
      y[u] = p < a.col_pairs && n < col_end && tok[u] >= 0 ? ldg16((const uint16_t*)a.base + tok[u] * a.base_stride + n)
                                                           : u32x4{0, 0, 0, 0};
  };
  Weights w0, w1;
  Rows y0, y1;
  load_b(0, 0, w0);
  load_y(0, y0);

  // t of the block's tokens: LPR lanes per row, four ranks each
  constexpr int LPR = RP / 4;
  for (int i = tid; i < BM * LPR; i += 64 * kWaves) {
    const int row = i / LPR, c = i - row * LPR;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (4 * c < a.max_rank) {
      const float* p = a.part + (row0 + row) * a.rank_pitch + (int64_t)slice * a.max_rank + 4 * c;
#pragma unroll 4
      for (int s = 0; s < a.ksplit; ++s) v += *(const f32x4*)(p + (int64_t)s * a.cap_rows * a.rank_pitch);
    }
    split_row<T, LPR>(v, 4 * c, rank, a.scales ? a.scales[adapter] : 1.0f, st + row * PITCH + 4 * c, RP, c == 0 ? row_scale + row : nullptr);
  }
  __syncthreads();

  const bool cut = rank % 8 != 0;
  f32x4 acc[TT][2];
  auto multiply = [&](int ch, Weights& w) __attribute__((always_inline)) {
    if (cut) {   // ranks of a chunk of 8 behind the adapter's own: out of the operand (they may hold anything)
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        const int left = rank - 8 * (RS == 0 ? g & 1 : 4 * (ch * KC + k) + g);
        if (left < 8)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) w[k][j][e] &= left > 2 * e + 1 ? 0xFFFFFFFFu : left > 2 * e ? 0xFFFFu : 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < TT; ++u) {
      const uint16_t* const t = st + (16 * u + r) * PITCH + 32 * ch * KC + 8 * g;
      if (RS >= 4) __builtin_amdgcn_sched_barrier(0);           // (else all reads move up, and registers run out)
      if (ch == 0) acc[u][0] = acc[u][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KC; ++k) {
        const u32x4 hi = *(const u32x4*)(t + 32 * k);         // (RS 0: high and low part)
        acc[u][0] = mfma16x16x32<AF>(w[k][0], hi, acc[u][0]);
        acc[u][1] = mfma16x16x32<AF>(w[k][1], hi, acc[u][1]);
        if constexpr (RS != 0) {
          const u32x4 lo = *(const u32x4*)(t + RP + 32 * k);
          acc[u][0] = mfma16x16x32<AF>(w[k][0], lo, acc[u][0]);
          acc[u][1] = mfma16x16x32<AF>(w[k][1], lo, acc[u][1]);
        }
      }
    }
  };
  auto store = [&](int p, const Rows& rows) __attribute__((always_inline)) {
    const int n = col0 + (p * kWaves + wave) * 32 + 8 * g;
#pragma unroll
    for (int u = 0; u < TT; ++u) {
      const float sc = row_scale[16 * u + r];
      float y[8];
      unpack8<T>(rows[u], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(acc[u][e >> 2][e & 3], sc, y[e]);
      if (tok[u] >= 0 && n < col_end) *(u32x4*)((uint16_t*)a.y + tok[u] * a.y_stride + n) = pack8<T>(y);
    }
  };
  if constexpr (CH == 1) {
    for (int p = 0; p < a.col_pairs; p += 2) {
      load_b(p + 1, 0, w1);
      load_y(p + 1, y1);
      multiply(0, w0);
      store(p, y0);
      if (p + 1 >= a.col_pairs) break;
      load_b(p + 2, 0, w0);
      load_y(p + 2, y0);
      multiply(0, w1);
      store(p + 1, y1);
    }
  } else {
    for (int p = 0; p < a.col_pairs; ++p) {
#pragma unroll
      for (int ch = 0; ch < CH; ++ch) {
        const bool last = ch == CH - 1;
        load_b(last ? p + 1 : p, last ? 0 : ch + 1, ch & 1 ? w0 : w1);
        if (last) load_y(p + 1, y1);
        multiply(ch, ch & 1 ? w1 : w0);
      }
      store(p, y0);
#pragma unroll
      for (int u = 0; u < TT; ++u) y0[u] = y1[u];
    }
  }
}

// Between the two products of many tokens: the parts of K added up in their order, and split into two 16-bit numbers, once
// (every workgroup of the second product would do it for its columns).  A row of a slice: [high RP | low RP] and its scale.
template <int T, int RP>
__global__ __launch_bounds__(256) void lora_join_kernel(LoraArgs a) {
  constexpr int LPR = RP / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / LPR;
  const int c = (int)(i - row * LPR), slice = blockIdx.y;
  if (row >= (int64_t)*a.num_post_pad) return;                // (whole blocks of rows: lanes of a row leave together)
  const int adapter = a.expert_ids[row >> a.block_shift];
  const int rank = a.ranks ? max(0, min(a.ranks[adapter], a.max_rank)) : a.max_rank;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (4 * c < a.max_rank) {
    const float* p = a.part + row * a.rank_pitch + (int64_t)slice * a.max_rank + 4 * c;
#pragma unroll 4
    for (int s = 0; s < a.ksplit; ++s) v += *(const f32x4*)(p + (int64_t)s * a.cap_rows * a.rank_pitch);
  }
  const int64_t at = (int64_t)slice * a.cap_rows + row;
  split_row<T, LPR>(v, 4 * c, rank, a.scales ? a.scales[adapter] : 1.0f, a.t16 + at * 2 * RP + 4 * c, RP, c == 0 ? a.t_scale + at : nullptr);
}

// The second product for blocks of many tokens.  Like the first's, its operands' and outputs' natural order (neighbouring
// lanes in different rows) would take the cache an access per lane, so a wave passes B's rows of its 32 columns through
// LDS on their way in (a ring of NB pairs of column tiles of its own, no barrier) and the sums on their way out, 16
// tokens at a time: rows of y are then read and written 64 bytes at a time by neighbouring lanes.
template <int T, int BM, int RS>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2))) void lora_expand_staged_kernel(LoraArgs a) {
  constexpr int AF = T == O_F16 ? A_F16 : A_BF16;
  constexpr int TT = BM / 16, W = kWaves;
  constexpr int RP = RS == 0 ? 16 : 32 * RS, KS = RS == 0 ? 1 : RS, CH = RP / 8;
  constexpr int CT = 2 * CH;                                  // chunks of a row of t: [high | low]
  constexpr int BSTAGE = 32 * RP * 2, NBL = BSTAGE / 1024, NB = RS >= 4 ? 1 : 2;
  constexpr int DP = 36;                                      // floats of a row of sums
  __shared__ __attribute__((aligned(16))) uint16_t st[BM * 2 * RP];
  __shared__ __attribute__((aligned(16))) uint8_t sb[W * NB * BSTAGE];
  __shared__ __attribute__((aligned(16))) float sd[W * 16 * DP];
  const int block = (int)blockIdx.x / a.col_tiles;
  const int64_t row0 = (int64_t)block * BM;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  int tok[TT];                                                // of the rows that this lane reads and writes
  const int f0 = a.sorted_ids[row0];
#pragma unroll
  for (int u = 0; u < TT; ++u) tok[u] = a.sorted_ids[row0 + 16 * u + (lane >> 2)];
  const int adapter = a.expert_ids[row0 >> a.block_shift];
  if (row0 >= (int64_t)*a.num_post_pad || f0 < 0 || f0 >= a.tokens) return;
  const int rank = a.ranks ? max(0, min(a.ranks[adapter], a.max_rank)) : a.max_rank;
  const int cols = 32 * W * a.col_pairs;
  int slice = 0, col0 = 0, tile = (int)blockIdx.x - block * a.col_tiles, col_end = 0;
  for (int begin = 0;; ++slice) {
    col_end = a.slice_end[slice];
    const int tiles = (col_end - begin + cols - 1) / cols;
    if (tile < tiles) { col0 = begin + tile * cols; break; }
    tile -= tiles;
    begin = col_end;
  }
  const uint16_t* const bw = (const uint16_t*)a.b + (int64_t)adapter * a.n * a.max_rank;
  uint8_t* const my_b = sb + wave * NB * BSTAGE;
  float* const my_d = sd + wave * 16 * DP;
  // (loads stay inside the tensors: columns and chunks behind the end are the last ones once more)
  auto load_b = [&](int p) __attribute__((always_inline)) {
    const int n0 = col0 + (p * W + wave) * 32;
#pragma unroll
    for (int i = 0; i < NBL; ++i) {
      const int piece = i * 64 + lane, row = piece / CH, c = swizzled<CH>(row, piece % CH);
      gload16_lds(bw + (int64_t)min(n0 + row, col_end - 1) * a.max_rank + min(8 * c, a.max_rank - 8),
                  my_b + (NB == 1 ? 0 : p & 1) * BSTAGE + i * 1024);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  typedef u32x4 Rows[TT];
  const uint16_t* in[TT];
  uint16_t* out[TT];                                          // (null: no token)
#pragma unroll
  for (int u = 0; u < TT; ++u) {
    const bool some = tok[u] >= 0 && tok[u] < a.tokens;
    in[u] = (const uint16_t*)a.base + (int64_t)(some ? tok[u] : f0) * a.base_stride;
    out[u] = some ? (uint16_t*)a.y + (int64_t)tok[u] * a.y_stride : nullptr;
  }
  auto load_y = [&](int p, Rows& y) __attribute__((always_inline)) {
    const int n = min(col0 + (p * W + wave) * 32 + 8 * (lane & 3), col_end - 8);
#pragma unroll
    for (int u = 0; u < TT; ++u) y[u] = ldg16(in[u] + n);
    __builtin_amdgcn_sched_barrier(0);
  };
  Rows y0, y1;
  load_b(0);
  load_y(0, y0);

  // t of the tile's tokens, as it lies in memory but for the order of its 16-byte chunks
  const int64_t t_row = (int64_t)slice * a.cap_rows + row0;
#pragma unroll
  for (int i = 0; i < BM * CT / 64 / W; ++i) {
    const int piece = (i * W + wave) * 64 + lane, row = piece / CT;
    gload16_lds(a.t16 + (t_row + row) * (2 * RP) + 8 * swizzled<CT>(row, piece % CT), st + (i * W + wave) * 512);
  }
  float scale[TT];
#pragma unroll
  for (int u = 0; u < TT; ++u) scale[u] = a.t_scale[t_row + 16 * u + r];
  wait_loads<0>();
  group_barrier();

  auto pair = [&](int p, const Rows& y) __attribute__((always_inline)) {
    const int n0 = col0 + (p * W + wave) * 32;
    const uint8_t* const b = my_b + (NB == 1 ? 0 : p & 1) * BSTAGE;
    u32x4 w[KS][2];
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = 16 * j + r, c = RS == 0 ? g & 1 : 4 * k + g, left = rank - 8 * c;
        w[k][j] = *(const u32x4*)(b + (row * CH + swizzled<CH>(row, c)) * 16);
        if (rank < RP && left < 8)                            // ranks behind the adapter's own: out (they may hold anything)
#pragma unroll
          for (int e = 0; e < 4; ++e) w[k][j][e] &= left > 2 * e + 1 ? 0xFFFFFFFFu : left > 2 * e ? 0xFFFFu : 0u;
      }
#pragma unroll
    for (int u = 0; u < TT; ++u) {
      const int row = 16 * u + r;
      auto t = [&](int c) __attribute__((always_inline)) { return *(const u32x4*)(st + (row * CT + swizzled<CT>(row, c)) * 8); };
      f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const u32x4 hi = t(4 * k + g);                          // (RS 0: high and low part)
        acc[0] = mfma16x16x32<AF>(w[k][0], hi, acc[0]);
        acc[1] = mfma16x16x32<AF>(w[k][1], hi, acc[1]);
        if constexpr (RS != 0) {
          const u32x4 lo = t(CH + 4 * k + g);
          acc[0] = mfma16x16x32<AF>(w[k][0], lo, acc[0]);
          acc[1] = mfma16x16x32<AF>(w[k][1], lo, acc[1]);
        }
      }
      *(f32x4*)(my_d + r * DP + 4 * g) = acc[0] * scale[u];
      *(f32x4*)(my_d + r * DP + 16 + 4 * g) = acc[1] * scale[u];
      asm volatile("" ::: "memory");                          // (a wave's LDS accesses keep their order)
      __builtin_amdgcn_wave_barrier();
      float v[8];
      unpack8<T>(y[u], v);
      const float* const d = my_d + (lane >> 2) * DP + 8 * (lane & 3);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += d[e];
      asm volatile("" ::: "memory");
      __builtin_amdgcn_wave_barrier();
      const int n = n0 + 8 * (lane & 3);
      if (out[u] && n < col_end) *(u32x4*)(out[u] + n) = pack8<T>(v);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  if constexpr (NB == 2) {
    for (int p = 0; p < a.col_pairs; p += 2) {
      load_b(p + 1);
      load_y(p + 1, y1);
      wait_loads<2 * TT + NBL>();                             // pair p's B: behind it are its rows of y and the next pair's loads
      pair(p, y0);
      if (p + 1 >= a.col_pairs) break;
      load_b(p + 2);
      load_y(p + 2, y0);
      wait_loads<2 * TT + NBL>();
      pair(p + 1, y1);
    }
  } else {
    for (int p = 0; p < a.col_pairs; ++p) {
      if (p > 0) load_b(p);
      load_y(p + 1, y1);
      wait_loads<TT>();
      pair(p, y0);
#pragma unroll
      for (int u = 0; u < TT; ++u) y0[u] = y1[u];
    }
  }
  wait_loads<0>();                                            // the last loads land before the LDS is another workgroup's
}

template <int T, int BM, int RT>
void launch_shrink(const LoraArgs& a, unsigned blocks, hipStream_t st) {
  const unsigned groups = (unsigned)((a.rank_rows + 16 * RT - 1) / (16 * RT));
  hipLaunchKernelGGL((lora_shrink_kernel<T, BM, RT>), dim3(blocks, a.ksplit, groups), dim3(64 * kWaves), 0, st, a);
}

template <int T, int BM, int RTALL, int WT>
void launch_staged(const LoraArgs& a, unsigned blocks, hipStream_t st) {
  const unsigned groups = (unsigned)((a.rank_rows + 16 * RTALL - 1) / (16 * RTALL)), tiles = blocks * ((1u << a.block_shift) / BM);
  hipLaunchKernelGGL((lora_shrink_staged_kernel<T, BM, RTALL, WT>), dim3(tiles, a.ksplit, groups), dim3(64 * kWaves), 0, st, a);
}

template <int T, int BM, int RS>
void launch_expand(LoraArgs a, unsigned blocks, hipStream_t st) {
  const unsigned tiles = blocks * ((1u << a.block_shift) / BM);
  // pairs of column tiles per wave: two where that leaves four workgroups per CU (8192 tokens, 5632 columns, rank 128: one 77 us,
  // two 65, four 68; 256 tokens, 6144 columns, rank 64: 12.3, 10.1, 10.0)
  a.col_pairs = (int64_t)tiles * (a.n / (64 * kWaves)) >= 1024 ? 2 : 1;
  const int cols = 32 * kWaves * a.col_pairs;
  a.col_tiles = 0;
  for (int s = 0, begin = 0; s < a.slices; begin = a.slice_end[s], ++s) a.col_tiles += (a.slice_end[s] - begin + cols - 1) / cols;
  const dim3 grid(tiles * (unsigned)a.col_tiles);
  if constexpr (BM == 16) {
    hipLaunchKernelGGL((lora_expand_kernel<T, BM, RS>), grid, dim3(64 * kWaves), 0, st, a);
  } else {
    constexpr int RP = RS == 0 ? 16 : 32 * RS;
    const int64_t threads = (int64_t)blocks * (1 << a.block_shift) * (RP / 4);
    hipLaunchKernelGGL((lora_join_kernel<T, RP>), dim3((unsigned)((threads + 255) / 256), a.slices), dim3(256), 0, st, a);
    hipLaunchKernelGGL((lora_expand_staged_kernel<T, BM, RS>), grid, dim3(64 * kWaves), 0, st, a);
  }
}

// Blocks of 16 tokens: a few per adapter.
template <int T>
void launch_few(const LoraArgs& a, unsigned blocks, hipStream_t st) {
  if (a.rank_rows <= 16) launch_shrink<T, 16, 1>(a, blocks, st);
  else if (a.rank_rows <= 32) launch_shrink<T, 16, 2>(a, blocks, st);
  else launch_staged<T, 16, 4, 1>(a, blocks, st);
  if (a.max_rank <= 16) launch_expand<T, 16, 0>(a, blocks, st);
  else if (a.max_rank <= 32) launch_expand<T, 16, 1>(a, blocks, st);
  else if (a.max_rank <= 64) launch_expand<T, 16, 2>(a, blocks, st);
  else if (a.max_rank <= 128) launch_expand<T, 16, 4>(a, blocks, st);
  else launch_expand<T, 16, 8>(a, blocks, st);
}

// Blocks of 64 or 128: tiles of 128 tokens where there are ranks enough for the adapter's rows to be the larger operand.
template <int T>
void launch_many(const LoraArgs& a, unsigned blocks, hipStream_t st) {
  const int tile = lora_tile(1 << a.block_shift, a.rank_rows);
  if (a.rank_rows <= 32) launch_staged<T, 64, 2, 4>(a, blocks, st);
  else if (a.rank_rows <= 64) launch_staged<T, 64, 4, 4>(a, blocks, st);
  else if (a.rank_rows <= 128) tile == 128 ? launch_staged<T, 128, 8, 1>(a, blocks, st) : launch_staged<T, 64, 8, 1>(a, blocks, st);
  else tile == 128 ? launch_staged<T, 128, 16, 1>(a, blocks, st) : launch_staged<T, 64, 16, 1>(a, blocks, st);
  if (a.max_rank <= 16) launch_expand<T, 64, 0>(a, blocks, st);
  else if (a.max_rank <= 32) launch_expand<T, 64, 1>(a, blocks, st);
  else if (a.max_rank <= 64) launch_expand<T, 64, 2>(a, blocks, st);
  else if (a.max_rank <= 128) launch_expand<T, 64, 4>(a, blocks, st);
  else launch_expand<T, 64, 8>(a, blocks, st);
}

}  // namespace

int lora_tile(int block_m, int rank_rows) { return block_m == 128 && rank_rows > 64 ? 128 : block_m < 64 ? block_m : 64; }
int lora_padded_rank(int max_rank) { return max_rank <= 16 ? 16 : max_rank <= 32 ? 32 : max_rank <= 64 ? 64 : max_rank <= 128 ? 128 : 256; }
int lora_group(int block_m, int rank_rows) { return block_m == 16 || rank_rows <= 64 ? 64 : rank_rows <= 128 ? 128 : 256; }

void launch_lora(const LoraArgs& a, int type, unsigned blocks, hipStream_t st) {
  if (a.block_shift == 4) type == O_BF16 ? launch_few<O_BF16>(a, blocks, st) : launch_few<O_F16>(a, blocks, st);
  else type == O_BF16 ? launch_many<O_BF16>(a, blocks, st) : launch_many<O_F16>(a, blocks, st);
}

}  // namespace qg
