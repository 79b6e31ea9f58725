// int8 x int8 product of few rows, dense or an MoE block's: the weights are read once, or once per 64 rows,
// past the activations.
//
//   sum[m][n] = sum_k x[m][k] w[n][k] in 32-bit integers, y = out(float(sum) * sw[n] * sx[m]).
//
// Bound by reading the weights, and by what a CU loads (about 65 bytes per ns), of which every workgroup's
// copy of the activations is a part.  A workgroup takes up to 64 rows x CW columns, and its waves take the
// 128-wide K steps in turn: a wave shares nothing with the others until the end, so the loop has no
// barrier, only waits for its own loads.  Activations go HBM -> LDS (buffer_load ... lds) into the
// wave's own ring of four stages, 16-byte chunks XOR-swizzled by row bits 1..3; weights go HBM -> VGPR,
// four steps ahead like the activations.  At the end the waves' sums meet in LDS, as integers, so that
// their order does not matter.
//
// Measured in a graph, with 3 sets of weights in turn, which stay in the 256 MB last-level cache, / with 1 GiB of
// them: N = K = 7168, 1 row 9.5 / 9.7 us (5.4 / 5.3 TB/s of weights), 16 rows 11.0 / 11.3, 32 rows 10.8 / 13.5,
// 64 rows 12.8 / 16.6-18.1, 128 rows 15.7 / 21.5; N = K = 4096, 1 row 4.5 / 5.2, 64 rows 8.1 / 9.1, 128 rows 9.1 / 10.6.
// MoE, E = 64 top-6, N = 2816, K = 4096: 1 token 15.1 us (6 experts, 4.6 TB/s), 64 tokens 106.3 (6.9 TB/s); the kernel
// that streams weights through workgroups sharing staged activations took 17.8 and 112.2.
#include <type_traits>

#include "qg_device.h"
#include "qg_int8_steps.h"
#include "qg_kernels.h"

namespace qg {

namespace {

// RB: rows staged (8, 16, 32 or 64; those that fill no MFMA tile repeat others and are left out at the
// end), CW: columns (16, 32 or 64, by MFMA tiles of 16 or 32), NTW: non-temporal weight loads
template <int OF, int RB, int CW, bool MOE, bool NTW>
__global__ __launch_bounds__(64 * kParts) void int8_rows_kernel(MfmaArgs a) {
  constexpr int KP = kParts;
  constexpr int TW = CW < 32 ? CW : 32, NT = CW / TW;              // MFMA tile, column tiles
  constexpr int MT = RB > TW ? RB / TW : 1;                        // row tiles
  constexpr int TR = RB < TW ? RB : TW;                            // rows of a tile that are staged
  constexpr int G = 64 / TW, KJ = 8 / G;                           // 16-byte chunks of K per MFMA, MFMAs per step
  constexpr int AP = RB / 8;                                       // 16-byte activation pieces per lane and step
  constexpr int ROWB = 128;                                        // bytes of a row per step
  constexpr int STAGE = RB * ROWB;                                 // per wave
  constexpr int LOADS = AP + KJ * NT;                              // per step
  constexpr int BLOCK = RB == 8 ? 4 : RB;                          // MoE: rows of a block
  __shared__ __attribute__((aligned(16))) uint8_t sA0[KP * STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t sA1[KP * STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t sA2[KP * STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t sA3[KP * STAGE];
  __shared__ __attribute__((aligned(16))) float sRowScale[64];
  __shared__ __attribute__((aligned(16))) float sColScale[64];
  __shared__ int sRowOut[MOE ? 64 : 1];                            // output row of each row (-1: none)
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & (TW - 1), g = lane / TW;
  // (rows past RB: further row tiles, those of the same columns on the same XCD)
  int mtile = 0, ntile = (int)blockIdx.x, expert = 0;
  if constexpr (MOE) {
    if ((int64_t)blockIdx.y * BLOCK >= *a.num_post_pad) return;
    expert = a.expert_ids[blockIdx.y];
  } else if (RB == 64 && a.m > RB) {
    const int mtiles = (int)((a.m + RB - 1) / RB);
    xcd_tile(blockIdx.x, mtiles, (int)gridDim.x / mtiles, (int64_t)RB * a.k, (int64_t)CW * a.k, mtile, ntile);
  }
  const int row0 = mtile * RB, col0 = ntile * CW;
  const int nsteps = a.k / ROWB;
  const int cnt = wave_steps(nsteps, wave);                        // this wave's steps
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w + (int64_t)expert * a.w_expert_bytes, (uint32_t)a.w_expert_bytes);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, (uint32_t)(a.x_rows * a.k));
  // output row (MoE: of the token's slot) of a row, -1: none
  auto out_of = [&](int row) __attribute__((always_inline)) -> int {
    if constexpr (MOE) {
      const int f = row < BLOCK ? a.sorted_ids[(int64_t)blockIdx.y * BLOCK + row] : a.sentinel;
      return f < a.sentinel ? f : -1;
    } else {
      return row < RB && row0 + row < a.m ? row0 + row : -1;
    }
  };
  auto in_of = [&](int out) __attribute__((always_inline)) { return MOE && out >= 0 ? out / a.topk : out; };

  int a_off[AP];
#pragma unroll
  for (int i = 0; i < AP; ++i) {
    const int p = lane + 64 * i, row = p >> 3;
    const int in = in_of(out_of(row));
    a_off[i] = in >= 0 ? in * a.k + 16 * ((p & 7) ^ ((row >> 1) & 7)) : -1;
  }
  int b_off[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
    b_off[t] = (int)(((int64_t)((col0 + TW * t + r) >> 4) * (a.k >> 4) + g) * 256 + (r & 15) * 16);
  // the scales, for the end
  if (wave == 0) {
    const int out = out_of(lane), in = in_of(out);
    bload4_lds(make_rsrc(a.x_scale, (uint32_t)(a.x_rows * 4)), sRowScale, in >= 0 ? 4 * in : kOOB);
    if constexpr (MOE) sRowOut[lane] = out;
  }
  if (wave == 1)
    bload4_lds(make_rsrc((const float*)a.s + (int64_t)expert * a.n + col0, 4 * CW), sColScale, lane < CW ? 4 * lane : kOOB);
  __builtin_amdgcn_sched_barrier(0);

  auto stg = [&](int i) __attribute__((always_inline)) -> uint8_t* {
    return (i == 0 ? sA0 : i == 1 ? sA1 : i == 2 ? sA2 : sA3) + wave * STAGE;
  };
  i32x4 B[4][KJ][NT];
  // (past the end: zeros)
  auto load = [&](int i, auto S_) __attribute__((always_inline)) {
    constexpr int S = decltype(S_)::value;
    const int step = wave_step(wave, i);
#pragma unroll
    for (int c = 0; c < AP; ++c)
      bload16_lds(xr, stg(S) + 1024 * c, a_off[c] < 0 || i >= cnt ? kOOB : a_off[c] + step * ROWB);
#pragma unroll
    for (int j = 0; j < KJ; ++j)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        B[S][j][t] = __builtin_bit_cast(i32x4, bload16_s<NTW>(wr, i >= cnt ? kOOB : b_off[t],
                                                            weight_step_offset(wave, i, cnt, G * j)));
    __builtin_amdgcn_sched_barrier(0);
  };
  using Acc = std::conditional_t<TW == 32, i32x16, i32x4>;
  Acc acc[MT][NT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < TW * TW / 64; ++i) acc[mt][t][i] = 0;
  load(0, std::integral_constant<int, 0>{});
  load(1, std::integral_constant<int, 1>{});
  load(2, std::integral_constant<int, 2>{});
  load(3, std::integral_constant<int, 3>{});
  auto step = [&](int i, auto S_) __attribute__((always_inline)) {
    constexpr int S = decltype(S_)::value;
    wait_loads<3 * LOADS>();                                       // all but the three steps after this one
    const uint8_t* st = stg(S);
#pragma unroll
    for (int j = 0; j < KJ; ++j)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int row = TW * mt + (r & (TR - 1));
        const i32x4 A = *(const i32x4*)(st + row * ROWB + 16 * ((G * j + g) ^ ((row >> 1) & 7)));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if constexpr (TW == 32) acc[mt][t] = mfma32x32x32_i8(B[S][j][t], A, acc[mt][t]);
          else acc[mt][t] = mfma16x16x64_i8(__builtin_bit_cast(u32x4, B[S][j][t]), __builtin_bit_cast(u32x4, A), acc[mt][t]);
        }
      }
    __builtin_amdgcn_sched_barrier(0);
    load(i + kAhead, S_);
  };
  int i = 0;
  for (; i + 4 <= cnt; i += 4) {
    step(i, std::integral_constant<int, 0>{});
    step(i + 1, std::integral_constant<int, 1>{});
    step(i + 2, std::integral_constant<int, 2>{});
    step(i + 3, std::integral_constant<int, 3>{});
  }
  if (i < cnt) step(i, std::integral_constant<int, 0>{});
  if (i + 1 < cnt) step(i + 1, std::integral_constant<int, 1>{});
  if (i + 2 < cnt) step(i + 2, std::integral_constant<int, 2>{});
  wait_loads<0>();

  // Each wave's sums into its first stages, one per column tile, 16-byte pieces XOR-swizzled by the row: with
  // the weights as the MFMAs' first operand lane (r, g) holds columns 4 (G q + g) .. of row r.
  constexpr int PPR = TW / 4;                                      // pieces per row of a tile
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int q = 0; q < PPR / G; ++q)
        if (r < TR)
          *(i32x4*)(stg(t) + 16 * (PPR * (TW * mt + r) + ((G * q + g) ^ (r & (PPR - 1))))) =
              i32x4{acc[mt][t][4 * q], acc[mt][t][4 * q + 1], acc[mt][t][4 * q + 2], acc[mt][t][4 * q + 3]};
  __syncthreads();
  for (int p = tid; p < RB * PPR * NT; p += 64 * KP) {
    const int row = p / (PPR * NT), c = p % (PPR * NT);            // piece c of the row: columns 4 c ..
    int64_t out = row0 + row;
    if constexpr (MOE) {
      out = row < BLOCK ? sRowOut[row] : -1;
      if (out < 0) continue;
    } else if (out >= a.m) {
      break;
    }
    const uint8_t* src = (NT == 1 || c < PPR ? sA0 : sA1) + 16 * (PPR * row + ((c & (PPR - 1)) ^ (row & (PPR - 1))));
    i32x4 v = *(const i32x4*)src;
#pragma unroll
    for (int w = 1; w < KP; ++w) v += *(const i32x4*)(src + w * STAGE);
    const f32x4 sw = *(const f32x4*)&sColScale[4 * c];
    const float sx = sRowScale[row];
    u32x2 o;
    o[0] = scaled_out2<OF>(v[0], v[1], sw[0], sw[1], sx);
    o[1] = scaled_out2<OF>(v[2], v[3], sw[2], sw[3], sx);
    *(u32x2*)((uint16_t*)a.y + out * a.n + col0 + 4 * c) = o;
  }
}

template <int OF, int RB, int CW>
void launch_one(const MfmaArgs& a, bool ntw, hipStream_t st) {
  const dim3 grid((unsigned)(a.n / CW * ((a.m + RB - 1) / RB))), block(64 * kParts);
  if (ntw) hipLaunchKernelGGL((int8_rows_kernel<OF, RB, CW, false, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((int8_rows_kernel<OF, RB, CW, false, false>), grid, block, 0, st, a);
}

// 16 columns while they are at most one workgroup per CU, else 32, which load the activations half as
// often (16 rows, 16 / 32 columns: N = K = 4096 4.6 / 4.9 us, N = 2048, K = 14336 7.2 / 9.6; N = K = 5120 7.1 /
// 6.2, N = K = 7168 11.5 / 10.0), and 64 for several row tiles when 32 are more than one round.
template <int OF, int RB>
void launch_width(const MfmaArgs& a, bool ntw, hipStream_t st) {
  const int64_t tiles = (a.m + RB - 1) / RB * a.n;
  if (tiles <= 4096) return launch_one<OF, RB, 16>(a, ntw, st);
  if constexpr (RB == 64) {
    if (tiles > 8192) return launch_one<OF, RB, 64>(a, ntw, st);
  }
  launch_one<OF, RB, 32>(a, ntw, st);
}

// Weights past the caches where they are too many to stay there from one call to the next and activations
// are few (N = K = 7168, 3 / 16 sets of weights in turn, past / through: 5 rows 8.9 / 9.5 against 9.1 / 10.5 us,
// 16 rows 9.9 / 10.3 against 9.6 / 11.0; 64 rows 15.2 / 15.7 against 12.2 / 17.1; N = 8192, K = 14336, 32 rows
// 22.2 / 22.5 against 23.3 / 23.7; N = K = 4096, 5 rows 5.4 / 5.6 against 4.4 / 5.4); through them where several
// row tiles read them (N = K = 8192, 128 rows 23.7 / 23.7 against 18.3 / 24.9).
template <int OF>
void launch_rows(const MfmaArgs& a, hipStream_t st) {
  const int64_t bytes = a.w_expert_bytes;
  const bool ntw = a.m <= 64 && bytes >= (a.m <= 16 ? (int64_t)1 << 25 : (int64_t)1 << 26);
  if (a.m <= 8) launch_width<OF, 8>(a, ntw, st);
  else if (a.m <= 16) launch_width<OF, 16>(a, ntw, st);
  else if (a.m <= 32) launch_width<OF, 32>(a, ntw, st);
  else launch_width<OF, 64>(a, ntw, st);
}

// 32 columns for blocks of 4 and 16 rows (64 tokens of the above with 16 / 32 / 64 columns: 123 / 107 / 113 us), 64 for
// blocks of 64 (400 tokens 328 / 208 / 160).
template <int OF, int RB, int CW>
void launch_moe(const MfmaArgs& a, unsigned blocks, bool ntw, hipStream_t st) {
  const dim3 grid(a.n / CW, blocks), block(64 * kParts);
  if (ntw) hipLaunchKernelGGL((int8_rows_kernel<OF, RB, CW, true, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((int8_rows_kernel<OF, RB, CW, true, false>), grid, block, 0, st, a);
}

template <int OF>
bool launch_moe_rows(const MfmaArgs& a, const MoeRows& m, hipStream_t st) {
  if (m.block == 4) launch_moe<OF, 8, 32>(a, m.blocks, m.once, st);
  else if (m.block == 16) launch_moe<OF, 16, 32>(a, m.blocks, m.once, st);
  else if (m.block == 32 && !m.wide) launch_moe<OF, 32, 32>(a, m.blocks, m.once, st);
  else if (m.block == 32) launch_moe<OF, 32, 64>(a, m.blocks, m.once, st);
  else if (m.block == 64) launch_moe<OF, 64, 64>(a, m.blocks, m.once, st);
  else return false;
  return true;
}

}  // namespace

bool launch_rows_gemm_int8(const MfmaArgs& a, int of, hipStream_t st) {
  if (of == O_BF16) launch_rows<O_BF16>(a, st);
  else if (of == O_F16) launch_rows<O_F16>(a, st);
  else return false;
  return true;
}

bool launch_moe_rows_int8(const MfmaArgs& a, const MoeRows& m, int of, hipStream_t st) {
  if (of == O_BF16) return launch_moe_rows<O_BF16>(a, m, st);
  if (of == O_F16) return launch_moe_rows<O_F16>(a, m, st);
  return false;
}

}  // namespace qg
