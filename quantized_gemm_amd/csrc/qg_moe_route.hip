// Routing of tokens to experts: scores, choice and weights of one row of logits per token.
//
//   score s[e]  = exp(l[e] - max) / sum (softmax over the row) or 1 / (1 + exp(-l[e]));
//   choice c[e] = s[e] + bias[e], or the order of the logits where there is no bias (both scores
//                 rise with the logit, and comparing logits is exact);
//   groups      = equal runs of experts, valued by their best choice or the sum of their two best
//                 (of scores where there is no bias); experts outside the topk_groups best are out;
//   the topk best choices in descending order, ties to the lowest index, and their scores,
//   renormalized and scaled.
//
// What is chosen is what 64-bit scores choose.  Logits decide exactly in 32 bits.  Choice values by scores
// are compared as 30- or 28-bit fixed-point numbers, and every comparison that the choice rests on (a
// chosen value with the next one, the last kept group with the best one left out) has to be clear of
// their rounding; a token with one too close to call, equal values most often, is done again with 64-bit
// keys.  (32-bit float scores left 1-3% of the tokens of 256 experts too close, and as all waves run at
// once, their second pass was half of the kernel's time: 8192 tokens 25 us.)  Weights are 64-bit scores
// of the chosen, rounded once.
//
// One wave per token, the experts of a group on lanes of their own: with G groups, rounded up to a
// power of two, 64 / G lanes each, lane l of a group holding its experts l, l + 64 / G, ...  Group values
// are then reductions over lanes, and no LDS is used.  Bound by latency and instruction issue, not by
// bytes (8192 tokens of 256 float32 logits are 8.4 MB), so larger batches take four tokens per wave, one
// per row of 16 lanes, whose reductions are four lane moves: see moe_route_rows_kernel.
// Measured, launches in a graph: 1 token of 128 experts 3.3-3.7 us (a launch by itself), 4096 of 128 float32
// 5.0 us, 8192 of 256 float32 with bias and groups 10.2 us (0.87 TB/s), 8192 of 512 float32 15.0 us.
#include "qg_device.h"
#include "qg_kernels.h"

namespace qg {

namespace {

constexpr int kRouteMaxExperts = 512;

template <int T>
__device__ __forceinline__ float logit_of(const void* p, int64_t i) {
  if constexpr (T == S_F32) return ((const float*)p)[i];
  else if constexpr (T == S_BF16) return bf16_bits_to_f32(((const uint16_t*)p)[i]);
  else return f16_bits_to_f32(((const uint16_t*)p)[i]);
}

// Keys: 32-bit integers in the order of floats or fixed-point numbers (one instruction per comparison
// across lanes, without the canonicalizing of float maxima), or doubles.
template <typename K> struct KeyOf;
template <> struct KeyOf<int> {
  static constexpr int kNone = -0x7FFFFFFF - 1;    // not eligible: below every other key
  static __device__ __forceinline__ int of(float x) {
    const int b = __float_as_int(x);
    return b ^ ((b >> 31) & 0x7FFFFFFF);
  }
  static __device__ __forceinline__ float value(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF)); }
};
template <> struct KeyOf<double> {
  static constexpr double kNone = -__builtin_inf();
};
__device__ __forceinline__ int kmax(int x, int y) { return max(x, y); }
__device__ __forceinline__ int kmin(int x, int y) { return min(x, y); }
__device__ __forceinline__ double kmax(double x, double y) { return fmax(x, y); }
__device__ __forceinline__ double kmin(double x, double y) { return fmin(x, y); }

// The value of another lane of the row of 16 (quad permutations and mirrors), or of the last lane of the
// row or half before, kNone where ROWS leaves a row out.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ int lane_move(int x) {
  return __builtin_amdgcn_update_dpp(KeyOf<int>::kNone, x, CTRL, ROWS, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ uint32_t lane_move(uint32_t x, uint32_t none) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)x, CTRL, 0xF, 0xF, false);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140, kLast16 = 0x142, kLast32 = 0x143;

// Maximum over the wave, in every lane.
__device__ __forceinline__ int wave_max(int x) {
  x = max(x, lane_move<kXor1>(x));
  x = max(x, lane_move<kXor2>(x));
  x = max(x, lane_move<kHalfMirror>(x));
  x = max(x, lane_move<kMirror>(x));
  x = max(x, lane_move<kLast16, 0xA>(x));   // rows 1 and 3
  x = max(x, lane_move<kLast32, 0xC>(x));   // rows 2 and 3
  return __builtin_amdgcn_readlane(x, 63);
}
__device__ __forceinline__ double wave_max(double x) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x = fmax(x, __shfl_xor(x, off, 64));
  return x;
}
template <typename F>
__device__ __forceinline__ F wave_sum(F x) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
  return x;
}
__device__ __forceinline__ int read_lane(int x, int lane) { return __builtin_amdgcn_readlane(x, lane); }
__device__ __forceinline__ double read_lane(double x, int lane) { return __shfl(x, lane, 64); }

// The two largest of two pairs.
template <typename K>
__device__ __forceinline__ void merge2(K& b1, K& b2, K o1, K o2) {
  b2 = kmax(kmin(b1, o1), kmax(b2, o2));
  b1 = kmax(b1, o1);
}

struct RouteLane {          // where a lane's experts lie
  int log2, lanes;          // lanes per group
  int group, l;             // this lane's group and place in it
  int size;                 // experts per group
};

// The two largest keys of each group, in all of its lanes.
__device__ __forceinline__ void group_best(const RouteLane& p, int& b1, int& b2) {
  // (a mirror joins the other half as an exchange would: halves are uniform by then)
  if (p.lanes > 1) merge2(b1, b2, lane_move<kXor1>(b1), lane_move<kXor1>(b2));
  if (p.lanes > 2) merge2(b1, b2, lane_move<kXor2>(b1), lane_move<kXor2>(b2));
  if (p.lanes > 4) merge2(b1, b2, lane_move<kHalfMirror>(b1), lane_move<kHalfMirror>(b2));
  if (p.lanes > 8) merge2(b1, b2, lane_move<kMirror>(b1), lane_move<kMirror>(b2));
  if (p.lanes > 16) merge2(b1, b2, __shfl_xor(b1, 16, 64), __shfl_xor(b2, 16, 64));   // (at most 32: two groups)
}
__device__ __forceinline__ void group_best(const RouteLane& p, double& b1, double& b2) {
  for (int off = 1; off < p.lanes; off <<= 1) merge2(b1, b2, __shfl_xor(b1, off, 64), __shfl_xor(b2, off, 64));
}

// Scores of V logits to 2^-34, for fixed-point choice values: exp(l - mx) (softmax, still to be divided by
// the row's sum) or 1 / (1 + exp(-l)), 0 for experts that are out.  The exponential is 2^n e^r with
// |r| <= ln 2 / 2 and e^r by its Taylor series to r^9 / 9!, which leaves 2^-37.  Without branches, so that
// the V chains of dependent operations run through one another.
__device__ __forceinline__ double quick_exp(double x) {            // |x| <= 700
  const double n = rint(x * 1.4426950408889634);
  const double r = fma(n, -0.69314718055994531, x);
  double e = 1.0 / 362880;
  constexpr double kFact[] = {40320, 5040, 720, 120, 24, 6, 2, 1, 1};
#pragma unroll
  for (int i = 0; i < 9; ++i) e = fma(e, r, 1.0 / kFact[i]);
  return __builtin_ldexp(e, (int)n);
}
template <int V>
__device__ __forceinline__ void quick_scores(bool softmax, const float (&l)[V], float mx, double (&s)[V]) {
  if (softmax) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const double e = quick_exp(fmax((double)l[i] - (double)mx, -700.0));   // (-inf - -inf: -700)
      s[i] = l[i] > -__builtin_inff() ? e : 0.0;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const double d = 1.0 + quick_exp((double)fminf(fmaxf(-l[i], -700.f), 700.f));
      double y = __builtin_amdgcn_rcp(d);
      y = fma(fma(-d, y, 1.0), y, y);
      y = fma(fma(-d, y, 1.0), y, y);
      s[i] = l[i] > -__builtin_inff() ? y : 0.0;
    }
  }
}

// Fixed-point choice values of a row: key = 1 + (c - lo) * inv, of kBits bits.
struct FixedPoint {
  double lo, inv;
  bool ok;                  // the biases have a finite range
  // blo, bhi: the least and largest bias of the row's eligible experts (scores lie in [0, 1])
  __device__ __forceinline__ FixedPoint(float blo, float bhi, int bits) {
    lo = fmin((double)blo, 0.0);
    const double range = fmax((double)bhi, 0.0) - lo + 1.0;
    ok = range < 1e300;
    inv = ok ? (double)((1u << bits) - 2) / range : 0.0;
  }
  __device__ __forceinline__ uint32_t key(double c) const { return 1u + (uint32_t)((c - lo) * inv); }
};

// Chooses by the keys k[] (groups by gk[], zero: the key of a choice value 0): the id and key of the j-th
// chosen on lane j, -1 where there is none.  gap > 0: fixed-point keys; false where two that the choice
// rests on are not more than gap apart (gap 0: keys decide, always true).
template <typename K, int V>
__device__ __forceinline__ bool choose(const RouteArgs& a, const RouteLane& p, K (&k)[V], const K (&gk)[V], K zero, int gap,
                                       int& my_id, K& my_key) {
  const K none = KeyOf<K>::kNone;
  const int lane = threadIdx.x & 63;
  bool sure = true;
  if (a.groups > 1) {
    K b1 = none, b2 = none;
#pragma unroll
    for (int i = 0; i < V; ++i) merge2(b1, b2, gk[i], none);
    group_best(p, b1, b2);
    const K gv = a.group_top == 1 || b1 == none ? b1 : b1 + (b2 == none ? zero : b2);
    int rank = 0;                                                  // groups before this lane's
    for (int g = 0; g < a.groups; ++g) {
      const K o = read_lane(gv, g << p.log2);
      rank += (o > gv) || (o == gv && g < p.group) ? 1 : 0;
    }
    const bool kept = rank < a.topk_groups && p.group < a.groups;
    if (gap > 0) {
      // (the least kept value: the one of rank topk_groups - 1)
      const K low = wave_max(rank == a.topk_groups - 1 && p.group < a.groups ? gv : none);
      const K next = wave_max(kept || p.group >= a.groups ? none : gv);
      sure = next == none || low - next > 3 * gap;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) k[i] = kept ? k[i] : none;
  }
  my_id = -1;
  my_key = none;
  K before = none;
  for (int j = 0; j <= a.topk; ++j) {
    if (j == a.topk && gap == 0) break;
    K top = k[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = kmax(top, k[i]);
    const K best = wave_max(top);
    if (gap > 0 && j > 0) sure = sure && (best == none || before - best > gap);
    if (j == a.topk || best == none) break;
    before = best;
    // the lowest index among equals: within a lane by i, among lanes (rarely several) by index
    int mine = V - 1;
#pragma unroll
    for (int i = V - 2; i >= 0; --i) mine = k[i] == best ? i : mine;
    const int e = p.group * p.size + (mine << p.log2) + p.l;
    uint64_t m = __ballot(top == best);
    int at = __ffsll((unsigned long long)m) - 1;
    int id = __builtin_amdgcn_readlane(e, at);
    for (m &= m - 1; m; m &= m - 1) {
      const int w = __ffsll((unsigned long long)m) - 1, o = __builtin_amdgcn_readlane(e, w);
      at = o < id ? w : at;
      id = min(id, o);
    }
    const bool won = lane == at;
#pragma unroll
    for (int i = 0; i < V; ++i) k[i] = won && mine == i ? none : k[i];
    my_id = lane == j ? id : my_id;
    my_key = lane == j ? best : my_key;
  }
  return sure;
}

// The float32 logit a row holds for an expert: +inf as the largest finite value, NaN as -inf (not eligible),
// -0 as 0 (keys order bits, and the two are equal).
__device__ __forceinline__ float eligible(float x) {
  return x > -__builtin_inff() ? fminf(x, 3.402823466e38f) + 0.f : -__builtin_inff();
}
template <int T>
__device__ __forceinline__ float eligible_logit(const RouteArgs& a, int64_t t, int e) {
  return eligible(logit_of<T>(a.logits, t * a.stride + e));
}

// One token by a whole wave, up to V experts per lane.
template <int T, int V>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t t, int lanes_log2) {
  const int lane = threadIdx.x & 63;
  const float finf = __builtin_inff();
  RouteLane p;
  p.log2 = lanes_log2;
  p.lanes = 1 << lanes_log2;
  p.group = lane >> lanes_log2;
  p.l = lane & (p.lanes - 1);
  p.size = a.experts / a.groups;
  float l[V], b[V];
  float mx = -finf;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = (i << p.log2) + p.l, e = p.group * p.size + j;
    const bool in = p.group < a.groups && j < p.size;
    l[i] = in ? eligible_logit<T>(a, t, e) : -finf;
    b[i] = in && a.bias ? a.bias[e] : 0.f;
    mx = fmaxf(mx, l[i]);
  }
  if (a.softmax) mx = KeyOf<int>::value(wave_max(KeyOf<int>::of(mx)));
  constexpr int kNone = KeyOf<int>::kNone;
  int id, key, k[V], gk[V];
  float lg;                                                        // the logit of lane j's expert
  if (!a.bias && (a.groups == 1 || a.group_top == 1)) {
#pragma unroll
    for (int i = 0; i < V; ++i) k[i] = gk[i] = l[i] > -finf ? KeyOf<int>::of(l[i]) : kNone;
    choose<int, V>(a, p, k, gk, 0, 0, id, key);
    lg = KeyOf<int>::value(key);
  } else {
    double s[V], sum = 0;
    float blo = finf, bhi = -finf;
    quick_scores<V>(a.softmax, l, mx, s);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      sum += s[i];
      const bool ok = l[i] > -finf && b[i] > -finf;
      blo = ok ? fminf(blo, b[i]) : blo;
      bhi = ok ? fmaxf(bhi, b[i]) : bhi;
    }
    const double scale = a.softmax ? 1.0 / wave_sum(sum) : 1.0;
    const FixedPoint f(-KeyOf<int>::value(wave_max(KeyOf<int>::of(-blo))),
                       KeyOf<int>::value(wave_max(KeyOf<int>::of(bhi))), 30);
    bool sure = f.ok;
    if (sure) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int fixed = (int)f.key(s[i] * scale + (double)b[i]);
        k[i] = gk[i] = l[i] > -finf && b[i] > -finf ? fixed : kNone;
      }
      sure = choose<int, V>(a, p, k, gk, (int)f.key(0.0), 1, id, key);
    }
    if (!sure) {
      double kd[V], gd[V], key64, total = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool in = l[i] > -finf;
        kd[i] = !in ? 0.0 : a.softmax ? exp((double)l[i] - (double)mx) : 1.0 / (1.0 + exp(-(double)l[i]));
        total += kd[i];
      }
      if (a.softmax) total = wave_sum(total);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool ok = l[i] > -finf && b[i] > -finf;
        gd[i] = ok ? (a.softmax ? kd[i] / total : kd[i]) + (double)b[i] : KeyOf<double>::kNone;
        kd[i] = a.bias || !ok ? gd[i] : (double)l[i];
      }
      choose<double, V>(a, p, kd, gd, 0.0, 0, id, key64);
    }
    lg = eligible_logit<T>(a, t, max(id, 0));
  }
  // weights: lane j's expert
  double s = 0;
  if (id >= 0) s = a.softmax ? exp((double)lg - (double)mx) : 1.0 / (1.0 + exp(-(double)lg));
  double total = 1;
  if (a.renorm) {
    total = s;                                                     // (0 on the lanes past topk)
    for (int off = 1; off < a.topk; off <<= 1) total += __shfl_xor(total, off, 64);
  } else if (a.softmax) {
    total = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) total += l[i] > -finf ? exp((double)l[i] - (double)mx) : 0.0;
    total = wave_sum(total);
  }
  if (lane < a.topk) {
    a.ids[t * a.topk + lane] = id;
    a.weights[t * a.topk + lane] = total > 0 ? (float)(s / total * (double)a.scale) : 0.f;
  }
}

template <int T, int V>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs a, int lanes_log2) {
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t < a.tokens) route_token<T, V>(a, t, lanes_log2);
}

// Maximum and minimum over a row of 16 lanes, in all of them (mirrors join the halves, uniform by then).
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  x = max(x, lane_move<kXor1>(x, 0u));
  x = max(x, lane_move<kXor2>(x, 0u));
  x = max(x, lane_move<kHalfMirror>(x, 0u));
  return max(x, lane_move<kMirror>(x, 0u));
}
__device__ __forceinline__ uint32_t row_min(uint32_t x) { return ~row_max(~x); }
template <typename F>
__device__ __forceinline__ F row_sum(F x, int lanes) {
  for (int off = 1; off < lanes; off <<= 1) x += __shfl_xor(x, off, 64);
  return x;
}

// V values of a row from element e on, at an address that is a multiple of 16 bytes (16-bit ones: 8).
template <int T, int V>
__device__ __forceinline__ void load_run(const void* p, int64_t e, float (&v)[V]) {
  if constexpr (T == S_F32) {
    const f32x4* q = (const f32x4*)((const float*)p + e);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const f32x4 x = q[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = x[j];
    }
  } else {
    const u32x2* q = (const u32x2*)((const uint16_t*)p + e);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const u32x2 x = q[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint16_t bits = (uint16_t)(x[j >> 1] >> (16 * (j & 1)));
        v[4 * i + j] = logit_of<T>(&bits, 0);
      }
    }
  }
}

// Counts the groups before this lane's, gv being each group's value in all of its lanes: those of greater value, or of an equal one and lower index.
template <int R>
__device__ __forceinline__ void count_before(uint32_t gv, int group, int lanes, int& before) {
  if constexpr (R < 16) {
    if ((R & (lanes - 1)) == 0) {                                  // (turns by whole groups: one lane of each)
      const uint32_t o = lane_move<0x120 + R>(gv, 0u);
      const int og = (int)lane_move<0x120 + R>((uint32_t)group, 0u);
      before += (o > gv) || (o == gv && og < group) ? 1 : 0;
    }
    count_before<R + 1>(gv, group, lanes, before);
  }
}

// Four tokens per wave, token r on lanes 16 r .. 16 r + 15, up to V experts per lane: for choices by
// scores (fixed-point ones, checked; a token too close to call goes to route_token) and for choices by
// 16-bit logits, whose float32 images leave bits for the expert's index.
//
// Keys are unsigned integers in the order of values, 0 for experts that are out, and no two of a lane
// alike: by scores 28 bits of the value and 15 - i for the lane's i-th expert, by 16-bit logits the
// float's upper bits and 511 - e.  The j-th best is then the largest key below the one before it, found
// without taking that one out: of all u - before, modulo 2^32, those of smaller keys are the larger
// ones, in order.
template <int T, int V>
__global__ __launch_bounds__(256) void moe_route_rows_kernel(RouteArgs a, int lanes_log2, bool runs,
                                                             int wave_lanes_log2) {
  const int lane = threadIdx.x & 63, l16 = lane & 15;
  const int64_t t0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * 4;
  if (t0 >= a.tokens) return;
  const bool valid = t0 + (lane >> 4) < a.tokens;
  const int64_t t = valid ? t0 + (lane >> 4) : a.tokens - 1;
  const float finf = __builtin_inff();
  const int lanes = 1 << lanes_log2, group = l16 >> lanes_log2, gl = l16 & (lanes - 1);
  const int size = a.experts / a.groups;
  const bool by_score = T == S_F32 || a.bias || (a.groups > 1 && a.group_top == 2);
  auto key_of = [](float x) __attribute__((always_inline)) { return (uint32_t)KeyOf<int>::of(x) ^ 0x80000000u; };
  auto value_of = [](uint32_t u) __attribute__((always_inline)) { return KeyOf<int>::value((int)(u ^ 0x80000000u)); };
  // The lane's i-th expert is its group's at(i): runs of V, read 16 bytes at a time, where they fill the
  // group and are aligned, else every lanes-th (places past a group's experts read its last one and are out).
  // With 8 groups a scalar load touches 32 lines: 8192 tokens of 256 logits 14.3 us so, 10.0 us by runs.
  const int at_step = runs ? 1 : lanes, l_step = runs ? V : 1;
  auto at = [&](int i) __attribute__((always_inline)) { return i * at_step + gl * l_step; };
  float l[V], b[V], mx = -finf;
  const int first = (group < a.groups ? group : 0) * size;
  if (runs) {
    const int64_t e = first + gl * V;                               // (groups past the last one read the first)
    load_run<T, V>(a.logits, t * a.stride + e, l);
    if (a.bias) load_run<S_F32, V>(a.bias, e, b);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = first + min(at(i), size - 1);
      l[i] = logit_of<T>(a.logits, t * a.stride + e);
      if (a.bias) b[i] = a.bias[e];
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float x = eligible(l[i]);
    l[i] = (group < a.groups) & (at(i) < size) ? x : -finf;
    b[i] = a.bias ? b[i] : 0.f;
    mx = fmaxf(mx, l[i]);
  }
  if (a.softmax) mx = value_of(row_max(key_of(mx)));
  uint32_t u[V], b1 = 0, b2 = 0, zero = 0;                         // keys; a group's two best; the key of 0
  bool sure = true;
  if (by_score) {
    double s[V], sum = 0;
    float blo = finf, bhi = -finf;
    quick_scores<V>(a.softmax, l, mx, s);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      sum += s[i];
      const bool ok = l[i] > -finf && b[i] > -finf;
      blo = ok ? fminf(blo, b[i]) : blo;
      bhi = ok ? fmaxf(bhi, b[i]) : bhi;
    }
    const double scale = a.softmax ? 1.0 / row_sum(sum, 16) : 1.0;
    const FixedPoint f(-value_of(row_max(key_of(-blo))), value_of(row_max(key_of(bhi))), 28);
    sure = f.ok;
    zero = f.key(0.0);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t fixed = f.key(s[i] * scale + (double)b[i]) << 4 | (15u - i);
      u[i] = (int)f.ok & (l[i] > -finf) & (b[i] > -finf) ? fixed : 0u;
      b2 = max(b2, min(b1, u[i]));
      b1 = max(b1, u[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = group * size + at(i);
      u[i] = l[i] > -finf ? (key_of(l[i]) & ~511u) | (511u - e) : 0u;
      b1 = max(b1, u[i]);
    }
  }
  if (a.groups > 1) {
    auto join = [&](uint32_t o1, uint32_t o2) __attribute__((always_inline)) {
      b2 = max(min(b1, o1), max(b2, o2));
      b1 = max(b1, o1);
    };
    if (lanes > 1) join(lane_move<kXor1>(b1, 0u), lane_move<kXor1>(b2, 0u));
    if (lanes > 2) join(lane_move<kXor2>(b1, 0u), lane_move<kXor2>(b2, 0u));
    if (lanes > 4) join(lane_move<kHalfMirror>(b1, 0u), lane_move<kHalfMirror>(b2, 0u));
    const uint32_t gv = group >= a.groups || b1 == 0 ? 0u
                        : a.group_top == 1 || !by_score ? b1 : (b1 >> 4) + (b2 == 0 ? zero : b2 >> 4);
    int rank = 0;
    count_before<1>(gv, group, lanes, rank);
    const bool kept = rank < a.topk_groups && group < a.groups;
    if (by_score) {
      const uint32_t low = row_max(rank == a.topk_groups - 1 && group < a.groups ? gv : 0u);
      const uint32_t next = row_max(kept ? 0u : gv);
      const int bits = a.group_top == 1 ? 4 : 0;
      sure = sure && (next == 0 || (low >> bits) - (next >> bits) > 3);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = kept ? u[i] : 0u;
  }
  int id = -1;
  uint32_t prev = 0;
  for (int j = 0; j <= a.topk; ++j) {
    uint32_t d = u[0] - prev;
#pragma unroll
    for (int i = 1; i < V; ++i) d = max(d, u[i] - prev);
    const uint32_t dm = row_max(d), best = prev + dm;
    const bool found = best != 0 && (j == 0 || best < prev);
    if (by_score && j > 0) sure = sure && (!found || (prev >> 4) - (best >> 4) > 1);
    if (j == a.topk) break;
    int e;
    if (by_score) {
      const bool here = found && d == dm;
      const uint64_t holders = __ballot(here), rows = __ballot(found);
      sure = sure && 16 * __popcll(holders) == __popcll(rows);     // the same key on two lanes of a row: too close
      const int i = 15 - (int)(best & 15u);
      e = (int)row_min(here ? (uint32_t)(group * size + at(i)) : ~0u);
    } else {
      e = 511 - (int)(best & 511u);
    }
    id = l16 == j && found ? e : id;
    prev = found ? best : 1u;                                      // (below 1 there are only experts that are out)
  }
  // weights, as in route_token
  double s = 0;
  if (id >= 0) {
    const double lg = eligible_logit<T>(a, t, id);
    s = a.softmax ? exp(lg - (double)mx) : 1.0 / (1.0 + exp(-lg));
  }
  double total = 1;
  if (a.renorm) {
    total = row_sum(s, a.topk);
  } else if (a.softmax) {
    total = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) total += l[i] > -finf ? exp((double)l[i] - (double)mx) : 0.0;
    total = row_sum(total, 16);
  }
  if (valid && sure && l16 < a.topk) {
    a.ids[t * a.topk + l16] = id;
    a.weights[t * a.topk + l16] = total > 0 ? (float)(s / total * (double)a.scale) : 0.f;
  }
  const uint64_t again = __ballot(valid && !sure);
  for (int r = 0; r < 4; ++r)
    if ((again >> (16 * r)) & 1) route_token<T, (V + 3) / 4>(a, t0 + r, wave_lanes_log2);
}

int lanes_per_group(int lanes, int groups) {   // log2
  int log2 = 0;
  while ((lanes >> (log2 + 1)) >= groups) ++log2;
  return log2;
}

// Rows of 16 lanes from kRowTokens tokens, four per SIMD: below, a token per wave takes less time by
// itself.  Wave per token against rows: 2048 tokens of 256 sigmoid scores with bias and groups 6.8 / 7.3 us,
// 4096 9.1 / 7.5, 8192 14.4 / 10.0; 64 softmax scores with bias 4.8 / 5.1, 6.1 / 5.1, 8.8 / 6.1; 128 bf16
// logits 4.1 / 4.4, 4.9 / 4.5, 7.0 / 4.7.
constexpr int64_t kRowTokens = 4096;

template <int T, int V>
void launch_rows(const RouteArgs& a, int lanes_log2, int wave_lanes_log2, hipStream_t st) {
  constexpr int kAlign = T == S_F32 ? 16 : 8, kBytes = T == S_F32 ? 4 : 2;
  const bool runs = (V << lanes_log2) * a.groups == a.experts && (uintptr_t)a.logits % kAlign == 0 &&
                    a.stride * kBytes % kAlign == 0 && (uintptr_t)a.bias % 16 == 0;
  hipLaunchKernelGGL((moe_route_rows_kernel<T, V>), dim3((unsigned)((a.tokens + 15) / 16)), dim3(256), 0, st, a, lanes_log2,
                     runs, wave_lanes_log2);
}

template <int T>
bool launch_route(const RouteArgs& a, hipStream_t st) {
  const int size = a.experts / a.groups;
  const int log2 = lanes_per_group(64, a.groups);
  if (a.tokens >= kRowTokens && a.topk <= 16 && a.groups <= 16 &&
      (T != S_F32 || a.bias || (a.groups > 1 && a.group_top == 2))) {
    const int row_log2 = lanes_per_group(16, a.groups);
    const int v = (size + (1 << row_log2) - 1) >> row_log2;
    if (v <= 4) launch_rows<T, 4>(a, row_log2, log2, st);
    else if (v <= 8) launch_rows<T, 8>(a, row_log2, log2, st);
    else if (v <= 16) launch_rows<T, 16>(a, row_log2, log2, st);
    if (v <= 16) return true;
  }
  const dim3 grid((unsigned)((a.tokens + 3) / 4));
  const int v = (size + (1 << log2) - 1) >> log2;                  // experts per lane
  if (v <= 1) hipLaunchKernelGGL((moe_route_kernel<T, 1>), grid, dim3(256), 0, st, a, log2);
  else if (v <= 2) hipLaunchKernelGGL((moe_route_kernel<T, 2>), grid, dim3(256), 0, st, a, log2);
  else if (v <= 4) hipLaunchKernelGGL((moe_route_kernel<T, 4>), grid, dim3(256), 0, st, a, log2);
  else if (v <= 8) hipLaunchKernelGGL((moe_route_kernel<T, 8>), grid, dim3(256), 0, st, a, log2);
  else if (v <= 16) hipLaunchKernelGGL((moe_route_kernel<T, 16>), grid, dim3(256), 0, st, a, log2);
  else return false;
  return true;
}

}  // namespace

// A launch takes fewer than 2^32 threads, 64 per token.
constexpr int64_t kTokensPerLaunch = 1 << 24;

bool launch_moe_route(const RouteArgs& a, int in_t, hipStream_t st) {
  if (a.experts > kRouteMaxExperts) return false;
  for (int64_t t = 0; t < a.tokens; t += kTokensPerLaunch) {
    RouteArgs b = a;
    b.logits = (const char*)a.logits + t * a.stride * (in_t == S_F32 ? 4 : 2);
    b.ids += t * a.topk;
    b.weights += t * a.topk;
    b.tokens = a.tokens - t < kTokensPerLaunch ? a.tokens - t : kTokensPerLaunch;
    if (in_t == S_F32 ? !launch_route<S_F32>(b, st)
        : in_t == S_BF16 ? !launch_route<S_BF16>(b, st)
        : in_t == S_F16 ? !launch_route<S_F16>(b, st) : true)
      return false;
  }
  return true;
}

}  // namespace qg
