// Low-rank adapters of many requests beside a projection that they share:
//
//   t[m][s] = x[m] A[a, s]^T over the adapter's rank rows,  y[m][n] = base[m][n] + scale[a] sum_r t[m][s(n)][r] B[a, n, r]
//
// for the adapter a of token m and the slice s(n) of column n.  Tokens come in blocks of BM rows of one adapter
// (qg_moe_align's map).  Two launches: the first makes t in float32 (partial sums over `ksplit` parts of K, each
// in a place of its own, so that no order is left to chance), the second adds the parts and multiplies by B.
//
// Both products run on 16x16x32 MFMAs with the adapter's rows as first operand, so that a lane's sums belong to
// one token: four ranks side by side of t, and, with the columns of two tiles interleaved, eight columns
// side by side of y.  Operands go from memory to registers: an adapter's rows are read by one workgroup (few
// tokens) or stay in the caches (many).
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
__global__ __launch_bounds__(64 * kWaves) void lora_shrink_kernel(LoraArgs a) {
  constexpr int AF = T == O_F16 ? A_F16 : A_BF16;
  constexpr int TT = BM / 16;
  constexpr int STEP = 64;                                    // K of a wave's step: one 128-byte line of every row
  __shared__ __attribute__((aligned(16))) float sum[kWaves][BM][RT * 16 + 4];
  const int64_t row0 = (int64_t)blockIdx.x * BM;
  if (row0 >= (int64_t)*a.num_post_pad) return;
  const int adapter = a.expert_ids[blockIdx.x];
  const int rank = a.ranks ? max(0, min(a.ranks[adapter], a.max_rank)) : a.max_rank;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;

  const uint16_t* xp[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    int f = a.sorted_ids[row0 + 16 * t + r];
    if (f < 0 || f >= a.tokens) f = a.sorted_ids[row0];       // a block's first row is a token; its sums are not used
    xp[t] = (const uint16_t*)a.x + f * a.x_stride + 16 * g;
  }
  const uint16_t* ap[RT];
  bool has[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int row = (blockIdx.z * RT + t) * 16 + r;           // of all slices' rows
    has[t] = row < a.rank_rows && row % a.max_rank < rank;
    ap[t] = (const uint16_t*)a.a + ((int64_t)adapter * a.rank_rows + (has[t] ? row : 0)) * a.k + 16 * g;
  }
  f32x4 acc[RT][TT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int u = 0; u < TT; ++u) acc[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int steps = (a.k + STEP - 1) / STEP;
  const int per = (steps + a.ksplit - 1) / a.ksplit;
  const int first = (int)blockIdx.y * per, end = min(steps, first + per);
  for (int s = first + wave; s < end; s += kWaves) {
    const int k0 = s * STEP;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = k0 + 16 * g + 8 * h < a.k;              // (k % 8 == 0)
      u32x4 xv[TT], av[RT];
#pragma unroll
      for (int t = 0; t < TT; ++t) xv[t] = in ? ldg16(xp[t] + k0 + 8 * h) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int t = 0; t < RT; ++t) av[t] = in && has[t] ? ldg16(ap[t] + k0 + 8 * h) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int u = 0; u < TT; ++u) acc[t][u] = mfma16x16x32<AF>(av[t], xv[u], acc[t][u]);
    }
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

// RS: MFMAs (of 32 ranks) per tile, 0: up to 16 ranks, whose high and low parts share one MFMA.
template <int T, int BM, int NP, int RS>
__global__ __launch_bounds__(64 * kWaves) void lora_expand_kernel(LoraArgs a) {
  constexpr int AF = T == O_F16 ? A_F16 : A_BF16;
  constexpr int TT = BM / 16;
  constexpr int RP = RS == 0 ? 16 : 32 * RS;                  // ranks with padding
  constexpr int KS = RS == 0 ? 1 : RS;
  constexpr int PITCH = 2 * RP + 8;                           // 16-bit elements: [high RP | low RP], rows 16 bytes apart in banks
  __shared__ __attribute__((aligned(16))) uint16_t st[BM * PITCH];
  __shared__ float row_scale[BM];
  __shared__ int row_tok[BM];
  const int block = (int)blockIdx.x / a.col_tiles;
  const int64_t row0 = (int64_t)block * BM;
  if (row0 >= (int64_t)*a.num_post_pad) return;
  const int adapter = a.expert_ids[block];
  const int rank = a.ranks ? max(0, min(a.ranks[adapter], a.max_rank)) : a.max_rank;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  // the workgroup's slice and columns
  constexpr int COLS = 32 * NP * kWaves;
  int slice = 0, col0 = 0, tile = (int)blockIdx.x - block * a.col_tiles, col_end = 0;
  for (int begin = 0;; ++slice) {
    col_end = a.slice_end[slice];
    const int tiles = (col_end - begin + COLS - 1) / COLS;
    if (tile < tiles) { col0 = begin + tile * COLS; break; }
    tile -= tiles;
    begin = col_end;
  }

  // t of the block's tokens: LPR lanes per row, four ranks each
  constexpr int LPR = RP / 4;
  for (int i = tid; i < BM * LPR; i += 64 * kWaves) {
    const int row = i / LPR, c = i - row * LPR;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (4 * c < a.max_rank) {
      const float* p = a.part + (row0 + row) * a.rank_pitch + (int64_t)slice * a.max_rank + 4 * c;
      for (int s = 0; s < a.ksplit; ++s) v += *(const f32x4*)(p + (int64_t)s * a.cap_rows * a.rank_pitch);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = 4 * c + j < rank ? v[j] : 0.f;   // (0 * x, and x may be infinite)
    }
    float scale = a.scales ? a.scales[adapter] : 1.0f;
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
    *(u32x2*)(st + row * PITCH + 4 * c) = u32x2{pack2<AF>(v[0], v[1]), pack2<AF>(v[2], v[3])};
    *(u32x2*)(st + row * PITCH + RP + 4 * c) = u32x2{pack2<AF>(lo[0], lo[1]), pack2<AF>(lo[2], lo[3])};
    if (c == 0) {
      const int f = a.sorted_ids[row0 + row];
      row_scale[row] = scale;
      row_tok[row] = f >= 0 && f < a.tokens ? f : -1;
    }
  }
  __syncthreads();

#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int n0 = col0 + (wave * NP + p) * 32;
    if (n0 >= col_end) break;
    // row rho of tile j is column 8 (rho / 4) + 4 j + rho % 4: a lane's sums are 8 columns side by side
    u32x4 bv[KS][2];
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int n = n0 + 8 * (r >> 2) + 4 * j + (r & 3);
        const int c = RS == 0 ? g & 1 : 4 * k + g;            // chunk of 8 ranks
        const int left = rank - 8 * c;                        // ranks of the chunk that count
        u32x4 v = {0, 0, 0, 0};
        if (n < col_end && left > 0) v = ldg16((const uint16_t*)a.b + ((int64_t)adapter * a.n + n) * a.max_rank + 8 * c);
        if (left < 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] &= left > 2 * e + 1 ? 0xFFFFFFFFu : left > 2 * e ? 0xFFFFu : 0u;
        }
        bv[k][j] = v;
      }
#pragma unroll
    for (int u = 0; u < TT; ++u) {
      const int row = 16 * u + r;
      f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        if constexpr (RS == 0) {
          const u32x4 tv = *(const u32x4*)(st + row * PITCH + 8 * g);
          acc[0] = mfma16x16x32<AF>(bv[k][0], tv, acc[0]);
          acc[1] = mfma16x16x32<AF>(bv[k][1], tv, acc[1]);
        } else {
          const u32x4 hi = *(const u32x4*)(st + row * PITCH + 32 * k + 8 * g);
          const u32x4 lo = *(const u32x4*)(st + row * PITCH + RP + 32 * k + 8 * g);
          acc[0] = mfma16x16x32<AF>(bv[k][0], hi, acc[0]);
          acc[1] = mfma16x16x32<AF>(bv[k][1], hi, acc[1]);
          acc[0] = mfma16x16x32<AF>(bv[k][0], lo, acc[0]);
          acc[1] = mfma16x16x32<AF>(bv[k][1], lo, acc[1]);
        }
      }
      const int tok = row_tok[row], n = n0 + 8 * g;
      if (tok < 0 || n >= col_end) continue;
      const float sc = row_scale[row];
      float y[8];
      unpack8<T>(ldg16((const uint16_t*)a.base + tok * a.base_stride + n), y);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(acc[e >> 2][e & 3], sc, y[e]);
      *(u32x4*)((uint16_t*)a.y + tok * a.y_stride + n) = pack8<T>(y);
    }
  }
}

template <int T, int BM, int RT>
void launch_shrink(const LoraArgs& a, unsigned blocks, hipStream_t st) {
  const unsigned groups = (unsigned)((a.rank_rows + 16 * RT - 1) / (16 * RT));
  hipLaunchKernelGGL((lora_shrink_kernel<T, BM, RT>), dim3(blocks, a.ksplit, groups), dim3(64 * kWaves), 0, st, a);
}

template <int T, int BM, int NP, int RS>
void launch_expand(LoraArgs a, unsigned blocks, hipStream_t st) {
  constexpr int COLS = 32 * NP * kWaves;
  a.col_tiles = 0;
  for (int s = 0, begin = 0; s < a.slices; begin = a.slice_end[s], ++s) a.col_tiles += (a.slice_end[s] - begin + COLS - 1) / COLS;
  hipLaunchKernelGGL((lora_expand_kernel<T, BM, NP, RS>), dim3(blocks * (unsigned)a.col_tiles), dim3(64 * kWaves), 0, st, a);
}

template <int T, int BM, int NP>
void launch_block(const LoraArgs& a, unsigned blocks, hipStream_t st) {
  if (a.rank_rows <= 16) launch_shrink<T, BM, 1>(a, blocks, st);
  else if (a.rank_rows <= 32) launch_shrink<T, BM, 2>(a, blocks, st);
  else launch_shrink<T, BM, 4>(a, blocks, st);
  if (a.max_rank <= 16) launch_expand<T, BM, NP, 0>(a, blocks, st);
  else if (a.max_rank <= 32) launch_expand<T, BM, NP, 1>(a, blocks, st);
  else if (a.max_rank <= 64) launch_expand<T, BM, NP, 2>(a, blocks, st);
  else if (a.max_rank <= 128) launch_expand<T, BM, NP, 4>(a, blocks, st);
  else launch_expand<T, BM, NP, 8>(a, blocks, st);
}

}  // namespace

bool launch_lora(const LoraArgs& a, int type, int block_m, unsigned blocks, hipStream_t st) {
  if (block_m == 16) type == O_BF16 ? launch_block<O_BF16, 16, 1>(a, blocks, st) : launch_block<O_F16, 16, 1>(a, blocks, st);
  else if (block_m == 64) type == O_BF16 ? launch_block<O_BF16, 64, 2>(a, blocks, st) : launch_block<O_F16, 64, 2>(a, blocks, st);
  else return false;
  return true;
}

}  // namespace qg
