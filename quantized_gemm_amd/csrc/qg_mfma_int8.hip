// MFMA-bound int8 x int8 product for more rows than the few-rows kernel serves: dense
// tiles (with K split over workgroups where the tiles are few) and MoE blocks.
//
//   sum[m][n] = sum_k x[m][k] w[n][k] in 32-bit integers (exact, so every tile and split gives the
//   same), y = out(float(sum) * sw[n] * sx[m]).
//
// Nothing is converted on the way, so the tile is chosen for the operands' feed: BM rows x 256
// columns, 4 waves of all BM rows x 64 columns.  Per 128-wide K step a CU reads BM x 128 bytes of
// activations and 256 x 128 bytes of weights, each once, and its waves read the activations from
// LDS four times; eight waves of 32 columns, as the paths that convert weights take, read them
// eight times.  256-row tiles run one wave per SIMD with the accumulators in the 256 AGPRs;
// 128- and 64-row tiles run two.
//
// Activations go HBM -> LDS (buffer_load ... lds) into a ring of four 128-byte-wide stages, 16-byte
// chunks XOR-swizzled by row bits 1..3 (conflict-free 16-byte fragment reads); weights go HBM ->
// VGPR, one 16-byte unit of the prepared image being one lane's operand of one 32x32x32 MFMA.
//
// The weights are the MFMAs' first operand, so a lane's products share one activation row (lane (r, g)
// of a tile: row r, columns 8 (i / 4) + 4 g + i % 4): one row scale per lane and row tile, and four
// outputs of a row side by side, written into the epilogue's LDS rows 8 bytes at a time.
//
// A step is four sub-steps of 32 K.  Sub-step j multiplies, per row tile, NT MFMAs, and right after
// them reads that tile's fragment of sub-step j + 1 into the same registers: a fragment is read a
// whole sub-step before it is needed.  So that sub-step 3 can read the next stage, stages are handed
// over in the middle of a step: after sub-step 1 each wave waits for its own loads of stage
// step + 1 and passes the barrier; past it that stage is visible to all, and the stage that
// step - 1 read is free for step + 3, whose loads go out in sub-steps 2 and 3.  The weights of
// sub-step j are reloaded two steps ahead during the sub-step after it.
//
// 4096 rows, N = K = 7168: 174-176 us (2.4 POP/s), 316 k cycles at a clock that the power limit holds at 1.81 GHz
// (1.38 kW); on zeros, which switch little, the same launches take 129 us, 308 k cycles at 2.39 GHz (1.01 kW).
// The MFMAs are busy 201 k of those cycles, and the 448 tiles are two rounds of 256 workgroups, the second
// three quarters full.
//
// MoE: workgroups go to the 8 XCDs round-robin, each with its own L2, so each XCD takes an eighth of
// the tiles in order, groups of 8 row blocks with the block walked fastest: the tiles that run
// together share activation rows and, where an expert has several blocks, its weights (E = 64
// top-6, N = 2816, K = 4096: 4000 tokens 468 -> 325 us, 400 tokens 158 -> 140 us; E = 32 top-4,
// N = 7168, K = 2048, 8192 tokens in groups of 1 / 2 / 8: 620 / 545 / 540 us).  Where most experts have one
// block, whose weights are then read once, they are loaded past the caches (NTW: 400 tokens 140 ->
// 134 us; with two blocks per expert 108 -> 119 us).
#include <type_traits>

#include "qg_device.h"
#include "qg_kernels.h"

namespace qg {

namespace {

constexpr int kI8Stages = 4;

// waves per SIMD: what the accumulators and LDS stages of a tile leave room for
constexpr int waves_of(int bm, int nt) { return bm == 256 ? 1 : bm == 64 && nt == 1 ? 4 : 2; }

// NT: 32-column MFMA tiles per wave; NTW: non-temporal weight loads
template <int OF, int BM, int NT, bool MOE, bool SPLIT, bool NTW>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(waves_of(BM, NT), waves_of(BM, NT))))
void int8_gemm_kernel(MfmaArgs a) {
  constexpr int MT = BM / 32;                 // 32-row MFMA tiles per wave
  constexpr int WCOL = 32 * NT;
  constexpr int COLS = 4 * WCOL;              // columns per workgroup
  constexpr int ROWB = 128;                   // bytes of a row per step
  constexpr int STAGE = BM * ROWB;
  constexpr int APT = STAGE / 16 / 256;       // 16-byte activation pieces per thread and step
  // one array per stage, so that the compiler sees which stage a read and a load touch
  __shared__ __attribute__((aligned(16))) uint8_t sA0[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t sA1[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t sA2[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t sA3[STAGE];
  __shared__ int sRowOut[MOE ? BM : 1];       // output row of each tile row (-1: none)
  __shared__ __attribute__((aligned(16))) float sRowScale[SPLIT ? 4 : BM];
  __shared__ __attribute__((aligned(16))) float sColScale[SPLIT ? 4 : COLS];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, g = lane >> 5;

  int expert = 0, ntile;
  int64_t rowbase;
  if constexpr (MOE) {
    const int ntiles = (a.n + COLS - 1) / COLS;
    const int total = *a.num_post_pad / BM * ntiles;
    const int chunk = (total + 7) >> 3, l = (int)blockIdx.x >> 3;
    const int tile = ((int)blockIdx.x & 7) * chunk + l;
    if (l >= chunk || tile >= total) return;
    const int group = tile / (8 * ntiles), gl = tile - group * (8 * ntiles);
    const int gb = min(8, total / ntiles - 8 * group);             // row blocks of the group
    ntile = gl / gb;
    const int block = 8 * group + gl - ntile * gb;
    rowbase = (int64_t)block * BM;
    expert = a.expert_ids[block];
  } else {
    int mtile;
    const int mtiles = (int)((a.m + BM - 1) / BM);
    xcd_tile(blockIdx.x, mtiles, (int)gridDim.x / mtiles, (int64_t)BM * a.k, (int64_t)COLS * a.k, mtile, ntile);
    rowbase = (int64_t)mtile * BM;
  }
  // input row of a tile row, -1: none
  auto token_of = [&](int row) __attribute__((always_inline)) -> int {
    if constexpr (MOE) {
      const int f = a.sorted_ids[rowbase + row];
      return f < a.sentinel ? f / a.topk : -1;
    } else {
      return rowbase + row < a.m ? (int)rowbase + row : -1;
    }
  };

  const int col0 = ntile * COLS + WCOL * wave;                  // first column of this wave
  const int nsteps = SPLIT ? a.k / ROWB / a.ksplit : a.k / ROWB;
  const int kstep0 = SPLIT ? (int)blockIdx.z * nsteps : 0;
  const __amdgpu_buffer_rsrc_t wr =
      make_rsrc(a.w + (int64_t)expert * a.w_expert_bytes, (uint32_t)a.w_expert_bytes);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, (uint32_t)(a.x_rows * a.k));

  // activation piece p of a step: row p / 8, physical 16-byte chunk p % 8; the load of thread tid's
  // i-th piece lands in slot p = tid + 256 i.  Rows without a token read out of range: zeros.
  int a_off[APT];
#pragma unroll
  for (int i = 0; i < APT; ++i) {
    const int p = tid + 256 * i, row = p >> 3;
    const int lc = (p & 7) ^ ((row >> 1) & 7);                     // logical chunk
    const int tok = token_of(row);
    a_off[i] = tok < 0 ? -1 : (int)((int64_t)tok * a.k) + kstep0 * ROWB + 16 * lc;
  }
  // the scales of the tile's rows and columns, for the epilogue; they land before the first stage
  if constexpr (!SPLIT) {
    if (tid < BM) {
      const int tok = token_of(tid);
      bload4_lds(make_rsrc(a.x_scale, (uint32_t)(a.x_rows * 4)), sRowScale + (tid & ~63), tok < 0 ? kOOB : 4 * tok);
    }
    const int col = ntile * COLS + tid;
    if (tid < COLS)
      bload4_lds(make_rsrc((const float*)a.s + (int64_t)expert * a.n, (uint32_t)a.n * 4), sColScale + (tid & ~63),
                 col < a.n ? 4 * col : kOOB);
  }
  if constexpr (MOE) {
    for (int i = tid; i < BM; i += 256) {
      const int f = a.sorted_ids[rowbase + i];
      sRowOut[i] = f < a.sentinel ? f : -1;
    }
  }
  __builtin_amdgcn_sched_barrier(0);
  const int wave_slot = wave * 1024;
  // (loads of steps past the end store zeros that nothing reads)
  auto issue_a = [&](int step, uint8_t* stage, int i) __attribute__((always_inline)) {
    bload16_lds(xr, stage + 4096 * i + wave_slot, a_off[i] < 0 || step >= nsteps ? kOOB : a_off[i] + step * ROWB);
  };
  // weight unit j of a step: k = 32 j + 16 g .. of the step, this lane's column of tile t
  int b_off[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int col = col0 + 32 * t + r;
    b_off[t] = col < a.n ? (int)(((int64_t)(col >> 4) * (a.k >> 4) + kstep0 * 8 + g) * 256 + (col & 15) * 16) : kOOB;
  }
  i32x4 B[2][4][NT];                                               // slot = step % 2
  auto load_b = [&](int step, int slot, int j) __attribute__((always_inline)) {
    // (past the end: the last step's again, which nothing reads)
    const int so = min(step, nsteps - 1) * 2048;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      B[slot][j][t] = __builtin_bit_cast(i32x4, bload16_s<NTW>(wr, b_off[t], so + 512 * j));
  };

  i32x16 acc[MT][NT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[mt][t][i] = 0;

  auto stg = [&](int i) __attribute__((always_inline)) -> uint8_t* {
    return i == 0 ? sA0 : i == 1 ? sA1 : i == 2 ? sA2 : sA3;
  };
  i32x4 A[MT];
  auto read_a = [&](const uint8_t* st, int j, int mt) __attribute__((always_inline)) {
    const int row = 32 * mt + r;
    A[mt] = *(const i32x4*)(st + row * ROWB + 16 * ((2 * j + g) ^ ((row >> 1) & 7)));
  };

  // Loads in issue order: A(0) B(0) A(1) B(1).0-2 A(2), then per step s: B(s+1).3 in sub-step 0,
  // B(s+2).0 in 1, B(s+2).1 and half of A(s+3) in 2, B(s+2).2 and the rest in 3.
  auto all_a = [&](int step, uint8_t* st) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < APT; ++i) issue_a(step, st, i);
    __builtin_amdgcn_sched_barrier(0);
  };
  all_a(0, sA0);
#pragma unroll
  for (int j = 0; j < 4; ++j) load_b(0, 0, j);
  __builtin_amdgcn_sched_barrier(0);
  all_a(1, sA1);
#pragma unroll
  for (int j = 0; j < 3; ++j) load_b(1, 1, j);
  __builtin_amdgcn_sched_barrier(0);
  all_a(2, sA2);
  // loads issued after the last piece of a stage up to the wait for it: for stage 0 B(0), A(1),
  // B(1).0-2 and A(2); for stage s + 1 in the middle of step s at least one step's loads and B's of
  // two more sub-steps (stage 1: B(1).0-2, A(2) and B's of two sub-steps)
  constexpr int VM0 = 7 * NT + 2 * APT;
  constexpr int VM1 = 5 * NT + APT;
  wait_loads<VM0>();
  group_barrier();
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) read_a(sA0, 0, mt);
  __builtin_amdgcn_sched_barrier(0);

  auto step_body = [&](const int step, auto S_) __attribute__((always_inline)) {
    constexpr int S = decltype(S_)::value;                         // step % 4
    uint8_t* const st0 = stg(S);
    uint8_t* const st1 = stg((S + 1) & 3);
    uint8_t* const st3 = stg((S + 3) & 3);
    constexpr int SB = S & 1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j == 2) {
        __builtin_amdgcn_sched_barrier(0);
        wait_loads<VM1>();
        group_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[mt][t] = mfma32x32x32_i8(B[SB][j][t], A[mt], acc[mt][t]);
        // (after the sub-step's first tile: the registers of the unit before are free)
        if (mt == 0) {
          if (j == 0) load_b(step + 1, SB ^ 1, 3);
          else load_b(step + 2, SB, j - 1);
        }
        if (j >= 2) {
          constexpr int HALF = APT / 2;
#pragma unroll
          for (int i = 0; i < HALF; ++i)
            if (i * MT / HALF == mt) issue_a(step + 3, st3, (j - 2) * HALF + i);
        }
        if (j < 3) read_a(st0, j + 1, mt);
        else read_a(st1, 0, mt);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  int step = 0;
  for (; step + kI8Stages <= nsteps; step += kI8Stages) {
    step_body(step, std::integral_constant<int, 0>{});
    step_body(step + 1, std::integral_constant<int, 1>{});
    step_body(step + 2, std::integral_constant<int, 2>{});
    step_body(step + 3, std::integral_constant<int, 3>{});
  }
  if (step < nsteps) step_body(step, std::integral_constant<int, 0>{});
  if (step + 1 < nsteps) step_body(step + 1, std::integral_constant<int, 1>{});
  if (step + 2 < nsteps) step_body(step + 2, std::integral_constant<int, 2>{});
  // the out-of-range loads of the last steps still write zeros into LDS
  wait_loads<0>();
  __syncthreads();

  // ---- epilogue: 32 rows of the wave's columns at a time through a stage of its own, then 16-byte
  // pieces of rows, GR row tiles together so that their LDS round trips overlap
  if (col0 >= a.n) return;                                         // n % 64 == 0: all or none of a wave's columns
  uint8_t* const ep = stg(wave);
  auto out_row = [&](int row) __attribute__((always_inline)) -> int64_t {
    if constexpr (MOE) return sRowOut[row];
    else return rowbase + row < a.m ? rowbase + row : -1;
  };
  if constexpr (SPLIT) {
    // 16-byte pieces XOR-swizzled by the row
    constexpr int PPR = WCOL / 4;                                  // pieces per row
    static_assert(32 * PPR * 16 <= STAGE, "a row tile fits a stage");
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *(i32x4*)(ep + 16 * PPR * r + 16 * ((8 * t + 2 * q + g) ^ (r & (PPR - 1)))) =
              i32x4{acc[mt][t][4 * q], acc[mt][t][4 * q + 1], acc[mt][t][4 * q + 2], acc[mt][t][4 * q + 3]};
#pragma unroll
      for (int q = 0; q < PPR / 2; ++q) {
        const int rl = (64 / PPR) * q + lane / PPR, c16 = lane % PPR;
        const int64_t orow = out_row(32 * mt + rl);
        const u32x4 val = *(const u32x4*)(ep + 16 * PPR * rl + 16 * (c16 ^ (rl & (PPR - 1))));
        if (orow >= 0) *(u32x4*)(a.part + ((int64_t)blockIdx.z * a.m + orow) * a.n + col0 + 4 * c16) = val;
      }
    }
  } else {
    constexpr int PITCH = WCOL * 2 + 16;
    constexpr int PPR = WCOL / 8;                                  // 16-byte pieces per row
    constexpr int GR = BM == 64 ? 1 : 2;
    static_assert(GR * 32 * PITCH <= STAGE, "the row tiles fit a stage");
    f32x4 sw[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) sw[t][q] = *(const f32x4*)&sColScale[WCOL * wave + 32 * t + 8 * q + 4 * g];
#pragma unroll
    for (int m0 = 0; m0 < MT; m0 += GR) {
#pragma unroll
      for (int mm = 0; mm < GR; ++mm) {
        const int mt = m0 + mm;
        const float sx = sRowScale[32 * mt + r];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            u32x2 o;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              o[h] = scaled_out2<OF>(acc[mt][t][4 * q + 2 * h], acc[mt][t][4 * q + 2 * h + 1], sw[t][q][2 * h],
                                     sw[t][q][2 * h + 1], sx);
            *(u32x2*)(ep + (32 * mm + r) * PITCH + (32 * t + 8 * q + 4 * g) * 2) = o;
          }
      }
#pragma unroll
      for (int q = 0; q < GR * PPR / 2; ++q) {
        const int rl = (64 / PPR) * q + lane / PPR, c16 = lane % PPR;
        const int64_t orow = out_row(32 * m0 + rl);
        const u32x4 val = *(const u32x4*)(ep + rl * PITCH + 16 * c16);
        if (orow >= 0) *(u32x4*)((uint16_t*)a.y + orow * a.n + col0 + 8 * c16) = val;
      }
    }
  }
}

template <int OF, int BM, int NT, bool MOE, bool SPLIT, bool NTW>
void launch_one(const MfmaArgs& a, const MfmaTile& t, hipStream_t st) {
  const dim3 grid = MOE ? dim3((t.grid_x * t.grid_y + 7) / 8 * 8) : dim3(t.grid_x, 1, SPLIT ? t.ksplit : 1);
  hipLaunchKernelGGL((int8_gemm_kernel<OF, BM, NT, MOE, SPLIT, NTW>), grid, dim3(256), 0, st, a);
}

template <int OF, int BM, int NT>
bool launch_dense(const MfmaArgs& a, const MfmaTile& t, hipStream_t st) {
  if (t.ksplit <= 1) launch_one<OF, BM, NT, false, false, false>(a, t, st);
  else if constexpr (BM == 64) launch_one<OF, BM, NT, false, true, false>(a, t, st);
  else return false;
  return true;
}

template <int OF>
bool launch_int8(const MfmaArgs& a, const MfmaTile& t, bool moe, hipStream_t st) {
  if (moe) {
    if (t.cols != 256 || (t.bm != 128 && t.bm != 256)) return false;
    if (t.bm == 128 && t.once) launch_one<OF, 128, 2, true, false, true>(a, t, st);
    else if (t.bm == 128) launch_one<OF, 128, 2, true, false, false>(a, t, st);
    else if (t.once) launch_one<OF, 256, 2, true, false, true>(a, t, st);
    else launch_one<OF, 256, 2, true, false, false>(a, t, st);
    return true;
  }
  if (t.cols == 256 && t.bm == 256) return launch_dense<OF, 256, 2>(a, t, st);
  if (t.cols == 256 && t.bm == 128) return launch_dense<OF, 128, 2>(a, t, st);
  if (t.cols == 256 && t.bm == 64) return launch_dense<OF, 64, 2>(a, t, st);
  if (t.cols == 128 && t.bm == 128) return launch_dense<OF, 128, 1>(a, t, st);
  if (t.cols == 128 && t.bm == 64) return launch_dense<OF, 64, 1>(a, t, st);
  return false;
}

}  // namespace

bool mfma_int8(const MfmaArgs& a, const MfmaTile& t, int wp, int af, int of, int stype, bool zero, bool moe,
               hipStream_t st) {
  if (wp != WP_INT8 || af != A_INT8 || stype != S_F32 || zero) return false;
  if (of == O_BF16) return launch_int8<O_BF16>(a, t, moe, st);
  if (of == O_F16) return launch_int8<O_F16>(a, t, moe, st);
  return false;
}

}  // namespace qg
