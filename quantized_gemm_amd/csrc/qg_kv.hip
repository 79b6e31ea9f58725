// Rows of keys and values into a paged cache in MXFP4, and back.
//
// A row's head of D values is D / 32 blocks, each one power of two (UE8M0) and 32 e2m1 codes, by the rule of
// mxfp4_encode32: nothing is rounded but the values to their codes.  A block that is not finite keeps
// the exponent byte of NaN.  A thread takes 8 values (one word of codes), four threads a block.
//
// Bound by bytes (4 of rows and 1.06 of codes per key and value); a decoding batch by the launch.  8 heads of 128: 64 tokens
// 2.6 us each way, 8192 tokens 13.8 us to append and 12.1 to read (42 MB: 3.1 and 3.5 TB/s; tokens found by a 32-bit
// division, by one of 64 bits 5% more).
#include "qg_device.h"
#include "qg_kernels.h"
#include "qg_rows.h"

namespace qg {

namespace {

// Where 8 values (word w) of a token's head are: codes and exponent byte.
struct KvPlace { uint8_t *codes, *scale; };
__device__ __forceinline__ KvPlace place_of(const KvArgs& a, bool value, int64_t slot, int head, int w) {
  const int page = 1 << a.page_shift, dim = a.dim;
  const int64_t half = (int64_t)page * (dim / 2), tail = (int64_t)page * (dim / 32);
  uint8_t* const base = a.cache + ((slot >> a.page_shift) * a.heads + head) * (2 * (half + tail));
  const int t = (int)(slot & (page - 1));
  KvPlace p;
  if (value) {
    p.codes = base + half + (((int64_t)(t >> 2) * (dim / 8) + w) * 4 + (t & 3)) * 4;
    p.scale = base + 2 * half + tail + ((t >> 2) * (dim / 32) + (w >> 2)) * 4 + (t & 3);
  } else {
    p.codes = base + (int64_t)t * (dim / 2) + 4 * w;
    p.scale = base + 2 * half + t * (dim / 32) + (w >> 2);
  }
  return p;
}

// Thread i's token, and in it keys or values, head and word.  (a launch has fewer than 2^32 threads)
struct Item {
  int64_t token;
  bool value;
  int hw, head, w;                                  // hw: word of the row
  __device__ __forceinline__ Item(const KvArgs& a) {
    const int shift = a.dim_shift - 3;
    const uint32_t half = (uint32_t)a.heads << shift, i = blockIdx.x * 256u + threadIdx.x, n = i / (2 * half), c = i - n * (2 * half);
    token = n;
    value = c >= half;
    hw = (int)(value ? c - half : c);
    head = hw >> shift;
    w = hw & ((1 << shift) - 1);
  }
};

template <int T>
__global__ __launch_bounds__(256) void kv_append_kernel(KvArgs a) {
  const Item t(a);
  if (t.token >= a.tokens) return;
  const int64_t slot = a.slots[t.token];
  float v[8];
  unpack8<T>(ldg16(t.value ? (const uint16_t*)a.v + t.token * a.v_stride + 8 * t.hw : (const uint16_t*)a.k + t.token * a.k_stride + 8 * t.hw), v);
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = __builtin_elementwise_maximum(amax, fabsf(v[e]));
  amax = __builtin_elementwise_maximum(amax, neighbour<0xB1>(amax));
  amax = __builtin_elementwise_maximum(amax, neighbour<0x4E>(amax));
  uint32_t codes;
  const uint32_t e8 = mxfp4_encode8(v, amax, codes);
  if (slot < 0 || slot >= a.num_slots) return;
  const KvPlace p = place_of(a, t.value, slot, t.head, t.w);
  *(uint32_t*)p.codes = codes;
  if ((t.w & 3) == 0) *p.scale = (uint8_t)e8;
}

template <int T>
__global__ __launch_bounds__(256) void kv_read_kernel(KvArgs a) {
  constexpr int AF = T == O_F16 ? A_F16 : A_BF16;
  const Item t(a);
  if (t.token >= a.tokens) return;
  const int64_t slot = a.slots[t.token];
  u32x4 o = {0, 0, 0, 0};
  if (slot >= 0 && slot < a.num_slots) {
    const KvPlace p = place_of(a, t.value, slot, t.head, t.w);
    o = fp4_to_16<AF>(*(const uint32_t*)p.codes, scale_bits_to_f32<S_UE8M0>(*p.scale));
  }
  uint16_t* const row = (uint16_t*)(t.value ? a.v_out : a.k_out) + t.token * (int64_t)(a.heads * a.dim);
  *(u32x4*)(row + 8 * t.hw) = o;
}

}  // namespace

// a launch takes fewer than 2^32 threads
template <typename F>
static void in_parts(const KvArgs& all, F one) {
  const int64_t per = (int64_t)2 * all.heads * (all.dim / 8), most = ((int64_t)1 << 31) / per;
  for (int64_t t = 0; t < all.tokens; t += most) {
    KvArgs a = all;
    a.tokens = all.tokens - t < most ? all.tokens - t : most;
    a.slots += t;
    const int64_t width = (int64_t)all.heads * all.dim;
    if (a.k) a.k = (const uint16_t*)a.k + t * a.k_stride;
    if (a.v) a.v = (const uint16_t*)a.v + t * a.v_stride;
    if (a.k_out) a.k_out = (uint16_t*)a.k_out + t * width;
    if (a.v_out) a.v_out = (uint16_t*)a.v_out + t * width;
    one(a, dim3((unsigned)((a.tokens * per + 255) / 256)));
  }
}

void launch_kv_append(const KvArgs& a, int type, hipStream_t st) {
  in_parts(a, [&](const KvArgs& p, dim3 grid) {
    if (type == O_BF16) hipLaunchKernelGGL(kv_append_kernel<O_BF16>, grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL(kv_append_kernel<O_F16>, grid, dim3(256), 0, st, p);
  });
}

void launch_kv_read(const KvArgs& a, int type, hipStream_t st) {
  in_parts(a, [&](const KvArgs& p, dim3 grid) {
    if (type == O_BF16) hipLaunchKernelGGL(kv_read_kernel<O_BF16>, grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL(kv_read_kernel<O_F16>, grid, dim3(256), 0, st, p);
  });
}

}  // namespace qg
