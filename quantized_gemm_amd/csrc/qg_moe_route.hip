// Routing of tokens to experts: scores, choice and weights of one row of logits per token.
//
//   score s[e]  = exp(l[e] - max) / sum (softmax over the row) or 1 / (1 + exp(-l[e]));
//   choice c[e] = s[e] + bias[e], or the order of the logits where there is no bias (both scores
//                 rise with the logit, and comparing logits is exact);
//   groups      = equal runs of experts, valued by their best choice or the sum of their two best
//                 scores; experts outside the topk_groups best groups are out;
//   the topk best choices in descending order, ties to the lowest index, and their scores,
//   renormalized and scaled.
//
// Two experts whose scores differ by less than float32 resolves are common enough in a batch of
// rows to decide which one is chosen, so scores and choices are held in 64 bits.
//
// One wave per token: lane l holds experts l, l + 64, ...
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

template <int T, int V>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  __shared__ double s_choice[4][64 * V];
  const double ninf = -__builtin_inf();
  if (t >= a.tokens) return;
  double l[V];
  double mx = ninf;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    float x = e < a.experts ? logit_of<T>(a.logits, t * a.stride + e) : -__builtin_inff();
    x = x > 3.402823466e38f ? 3.402823466e38f : x;          // +inf: the largest finite value
    l[i] = x > -__builtin_inff() ? (double)x : ninf;        // NaN: not eligible
    mx = fmax(mx, l[i]);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) mx = fmax(mx, __shfl_xor(mx, off, 64));
  double s[V], c[V];
  if (a.softmax) {
    double sum = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = l[i] > ninf ? exp(l[i] - mx) : 0.0;
      sum += s[i];
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = sum > 0 ? s[i] / sum : 0.0;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = l[i] > ninf ? 1.0 / (1.0 + exp(-l[i])) : 0.0;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    c[i] = l[i];
    if (a.bias && l[i] > ninf) {
      const float b = a.bias[e];
      c[i] = b > -__builtin_inff() ? s[i] + (double)b : ninf;
    }
  }
  if (a.groups > 1) {
    // a group's value from the choice values, or from the scores where two are added without a bias
    const bool scores = a.group_top == 2 && !a.bias;
#pragma unroll
    for (int i = 0; i < V; ++i) s_choice[wave][lane + 64 * i] = scores ? (c[i] > ninf ? s[i] : ninf) : c[i];
    __builtin_amdgcn_wave_barrier();
    const int size = a.experts / a.groups;
    double gv = ninf;
    if (lane < a.groups) {
      double b1 = ninf, b2 = ninf;
      for (int j = 0; j < size; ++j) {
        const double v = s_choice[wave][lane * size + j];
        b2 = fmax(b2, fmin(b1, v));
        b1 = fmax(b1, v);
      }
      gv = a.group_top == 2 && b2 > ninf ? b1 + b2 : b1;
    }
    uint64_t kept = 0;
    for (int j = 0; j < a.topk_groups; ++j) {
      double best = gv;
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) best = fmax(best, __shfl_xor(best, off, 64));
      if (!(best > ninf)) break;
      const int g = __ffsll((unsigned long long)__ballot(gv == best)) - 1;
      kept |= 1ull << g;
      if (lane == g) gv = ninf;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      if (e < a.experts && !((kept >> (e / size)) & 1)) c[i] = ninf;
    }
  }
  // the topk best, one at a time; lane j keeps the j-th
  int my_id = -1;
  double my_s = 0;
  for (int j = 0; j < a.topk; ++j) {
    double best = ninf;
#pragma unroll
    for (int i = 0; i < V; ++i) best = fmax(best, c[i]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) best = fmax(best, __shfl_xor(best, off, 64));
    if (!(best > ninf)) break;
    int id = -1;
    double sc = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint64_t m = __ballot(c[i] == best);
      if (id < 0 && m) {
        const int w = __ffsll((unsigned long long)m) - 1;
        id = w + 64 * i;
        sc = __shfl(s[i], w, 64);
        if (lane == w) c[i] = ninf;
      }
    }
    if (lane == j) {
      my_id = id;
      my_s = sc;
    }
  }
  double sum = my_s;
  if (a.renorm) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
    my_s = sum > 0 ? my_s / sum : 0.0;
  }
  if (lane < a.topk) {
    a.ids[t * a.topk + lane] = my_id;
    a.weights[t * a.topk + lane] = (float)(my_s * (double)a.scale);
  }
}

template <int T>
bool launch_route(const RouteArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)((a.tokens + 3) / 4));
  if (a.experts <= 64) hipLaunchKernelGGL((moe_route_kernel<T, 1>), grid, dim3(256), 0, st, a);
  else if (a.experts <= 128) hipLaunchKernelGGL((moe_route_kernel<T, 2>), grid, dim3(256), 0, st, a);
  else if (a.experts <= 256) hipLaunchKernelGGL((moe_route_kernel<T, 4>), grid, dim3(256), 0, st, a);
  else if (a.experts <= kRouteMaxExperts) hipLaunchKernelGGL((moe_route_kernel<T, 8>), grid, dim3(256), 0, st, a);
  else return false;
  return true;
}

}  // namespace

bool launch_moe_route(const RouteArgs& a, int in_t, hipStream_t st) {
  if (in_t == S_F32) return launch_route<S_F32>(a, st);
  if (in_t == S_BF16) return launch_route<S_BF16>(a, st);
  if (in_t == S_F16) return launch_route<S_F16>(a, st);
  return false;
}

}  // namespace qg
