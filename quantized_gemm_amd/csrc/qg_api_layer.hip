// Host side of the operators around the products of a decoder layer (include/qg.h): norms around a block, low-rank
// adapters, the 4-bit cache and the attention that reads it.  Validation happens here, before anything is launched.
#include <math.h>

#include <algorithm>

#include "qg.h"
#include "qg_device.h"
#include "qg_host.h"
#include "qg_kernels.h"

using namespace qg;

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 32;
constexpr int64_t kLoraMaxTokens = (int64_t)1 << 24;
constexpr int kCUs = 256;
constexpr float kLog2e = 1.44269504088896f;

int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

bool type16(int32_t t) { return t == QG_O_F16 || t == QG_O_BF16; }

// A row stride in elements: 0 means `width`; else at least that, in steps of 8 (16 bytes and more).
bool stride_of(int64_t given, int64_t width, int64_t* out) {
  *out = given == 0 ? width : given;
  return given == 0 || (given >= width && given % 8 == 0 && given <= kMaxStride);
}

bool finite(float v) { return v - v == 0.0f; }

// Tokens' blocks of the map: as many as qg_moe_capacity allows.
int64_t block_capacity(int64_t tokens, int64_t adapters, int64_t block_m, int64_t* rows) {
  int64_t blocks = 0;
  *rows = 0;
  qg_moe_capacity(tokens, 1, (int32_t)adapters, (int32_t)block_m, rows, &blocks);
  return blocks;
}

qg_status check_lora(const qg_lora_desc* d) {
  if (!d) return QG_ERR_INVALID_ARG;
  if (!type16(d->type) || d->num_adapters <= 0 || d->max_rank <= 0 || d->num_slices <= 0 || d->n <= 0 || d->k <= 0)
    return QG_ERR_INVALID_ARG;
  if (d->num_adapters > 512 || d->max_rank > kLoraMaxRank || d->num_slices > kLoraMaxSlices) return QG_ERR_UNSUPPORTED;
  if (d->max_rank % 8 != 0 || d->n % 8 != 0 || d->k % 8 != 0) return QG_ERR_UNSUPPORTED;
  if (d->n > (1 << 24) || d->k > (1 << 24)) return QG_ERR_UNSUPPORTED;
  int64_t s;
  if (!stride_of(d->x_stride, d->k, &s) || !stride_of(d->base_stride, d->n, &s) || !stride_of(d->y_stride, d->n, &s))
    return QG_ERR_INVALID_ARG;
  for (int32_t i = 0, begin = 0; i < d->num_slices; begin = (int32_t)d->slice_end[i], ++i) {
    if (d->slice_end[i] <= begin || d->slice_end[i] > d->n) return QG_ERR_INVALID_ARG;
    if (i + 1 < d->num_slices && d->slice_end[i] % 32 != 0) return QG_ERR_UNSUPPORTED;
  }
  return d->slice_end[d->num_slices - 1] == d->n ? QG_OK : QG_ERR_INVALID_ARG;
}

bool lora_block(int32_t m) { return m == 16 || m == 64 || m == 128; }

// Parts of K, each of 512 (blocks of 16 with more than 32 rank rows: 1024) or more: as many workgroups as are on the GPU at once, and
// no few more, which would take as long again.  With more than 64 rank rows that is one per CU (8192 tokens, K = 4096, 256
// rank rows: 3 parts 45 us, 4 parts 59, 5 parts 55, 7 parts 50, and each part's sums are written and read again), else
// two (16 rank rows: 2 parts 28.6 us, 3 parts 22.7, 5 parts 22.9; 64 rank rows 32.8, 25.8, 26.4).
int lora_split(const qg_lora_desc* d, int64_t tokens, int32_t block_m) {
  const int rows = d->num_slices * d->max_rank, group = lora_group(block_m, rows);
  const int64_t tiles = (tokens / lora_tile(block_m, rows) + 1) * ((rows + group - 1) / group);
  const int64_t want = (block_m > 16 && rows > 64 ? 1 : 2) * kCUs / tiles, most = std::min<int64_t>(8, d->k / (block_m == 16 && rows > 32 ? 1024 : 512));
  return (int)std::max<int64_t>(1, std::min(want, most));
}

qg_status check_kv(const qg_kv_desc* d) {
  if (!d) return QG_ERR_INVALID_ARG;
  if (!type16(d->type) || d->kv_heads <= 0 || d->num_pages <= 0 || d->page_tokens <= 0) return QG_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return QG_ERR_UNSUPPORTED;
  if (d->page_tokens < 16 || d->page_tokens > 256 || (d->page_tokens & (d->page_tokens - 1)) != 0) return QG_ERR_UNSUPPORTED;
  if (d->kv_heads > 1024 || d->num_pages > (((int64_t)1 << 31) - 1) / d->page_tokens) return QG_ERR_UNSUPPORTED;
  return QG_OK;
}

KvArgs kv_args(const qg_kv_desc* d, const int32_t* slots, int64_t tokens, const void* cache) {
  KvArgs a{};
  a.cache = (uint8_t*)cache;
  a.slots = slots;
  a.tokens = tokens;
  a.num_slots = d->num_pages * d->page_tokens;
  a.heads = d->kv_heads;
  a.dim = d->head_dim;
  a.dim_shift = log2_of(d->head_dim);
  a.page_shift = log2_of(d->page_tokens);
  return a;
}

}  // namespace

extern "C" {

qg_status qg_norm_rows(const qg_norm_desc* d, int64_t rows, const void* y, const void* res, void* res_out, const void* gate,
                       const void* post_weight, const void* weight, const void* bias, void* out, void* codes, void* scale,
                       void* stream) {
  if (!d || rows < 0) return QG_ERR_INVALID_ARG;
  if (d->norm < 0 || d->norm > QG_N_LAYER || d->post_norm < 0 || d->post_norm > QG_N_LAYER || !type16(d->type))
    return QG_ERR_INVALID_ARG;
  if (d->res_type != QG_L_F16 && d->res_type != QG_L_BF16 && d->res_type != QG_L_F32) return QG_ERR_INVALID_ARG;
  if (d->code_type != 0 && d->code_type != QG_A_FP8_E4M3 && d->code_type != QG_A_INT8 && d->code_type != QG_A_FP4_E2M1)
    return QG_ERR_INVALID_ARG;
  if (!(d->eps >= 1e-30f) || !finite(d->eps) || !finite(d->weight_offset) || !finite(d->res_scale) || d->k <= 0)
    return QG_ERR_INVALID_ARG;
  NormArgs a{};
  if (!stride_of(d->y_stride, d->k, &a.y_stride) || !stride_of(d->res_stride, d->k, &a.res_stride) ||
      !stride_of(d->out_stride, d->k, &a.out_stride))
    return QG_ERR_INVALID_ARG;
  if (d->gate_stride != 0 && !stride_of(d->gate_stride, d->k, &a.gate_stride)) return QG_ERR_INVALID_ARG;
  // 16-bit residuals are of the rows' type
  const bool res32 = d->res_type == QG_L_F32;
  if (!res32 && (d->res_type == QG_L_F16) != (d->type == QG_O_F16)) return QG_ERR_UNSUPPORTED;
  if (d->k % 8 != 0 || d->k > kNormRowMax || (d->code_type == QG_A_FP4_E2M1 && d->k % 32 != 0)) return QG_ERR_UNSUPPORTED;
  if (rows > ((int64_t)1 << 31) - 1) return QG_ERR_UNSUPPORTED;
  if (rows == 0) return QG_OK;
  if ((!y && !res) || (!res_out && !out && !codes)) return QG_ERR_INVALID_ARG;
  if (!y && (gate || post_weight || d->post_norm != 0)) return QG_ERR_INVALID_ARG;
  if (post_weight && d->post_norm == 0) return QG_ERR_INVALID_ARG;
  if (d->norm == 0 && (weight || bias || out || codes)) return QG_ERR_INVALID_ARG;
  if ((codes != nullptr) != (d->code_type != 0) || (codes != nullptr) != (scale != nullptr)) return QG_ERR_INVALID_ARG;
  for (const void* p : {y, res, (const void*)res_out, gate, post_weight, weight, bias, (const void*)out, (const void*)codes})
    if (!aligned16(p)) return QG_ERR_INVALID_ARG;
  if (d->code_type != QG_A_FP4_E2M1 && ((uintptr_t)scale & 3u) != 0) return QG_ERR_INVALID_ARG;
  // an output in an input's place: row by row, or rows are overwritten before they are read
  auto apart = [&](int64_t s, int64_t t) { return rows > 1 && s != t; };
  if (out && (out == res_out || (out == y && apart(a.out_stride, a.y_stride)) ||
              (out == res && (res32 || apart(a.out_stride, a.res_stride)))))
    return QG_ERR_INVALID_ARG;
  if (res_out && res_out == y && (res32 || apart(a.res_stride, a.y_stride))) return QG_ERR_INVALID_ARG;
  qg_status s = check_arch();
  if (s != QG_OK) return s;
  a.y = y; a.res = res; a.gate = gate; a.post_weight = post_weight; a.weight = weight; a.bias = bias;
  a.res_out = res_out; a.out = out; a.codes = codes; a.scale = scale;
  a.rows = rows; a.k = d->k;
  a.norm = d->norm == QG_N_LAYER ? kNormLayer : d->norm == QG_N_RMS ? kNormRms : 0;
  a.post = d->post_norm == QG_N_LAYER ? kNormLayer : d->post_norm == QG_N_RMS ? kNormRms : 0;
  a.code = d->code_type == 0 ? 0 : d->code_type == QG_A_FP8_E4M3 ? A_FP8 : d->code_type == QG_A_INT8 ? A_INT8 : A_FP4;
  a.eps = d->eps; a.weight_offset = d->weight_offset; a.res_scale = d->res_scale;
  launch_norm_rows(a, d->type == QG_O_F16 ? O_F16 : O_BF16, res32, (hipStream_t)stream);
  return launched();
}

int32_t qg_lora_block_m(int64_t tokens, int32_t num_adapters) {
  if (tokens < 0 || num_adapters <= 0) return 0;
  return tokens >= (int64_t)256 * num_adapters ? 128 : tokens >= (int64_t)32 * num_adapters ? 64 : 16;
}

// Workspace: the parts of K's sums and, for blocks of 64 and 128 tokens, their 16-bit parts and scales.
static size_t lora_workspace(const qg_lora_desc* d, int64_t tokens, int32_t block_m, LoraArgs* a) {
  int64_t rows;
  block_capacity(tokens, d->num_adapters, block_m, &rows);
  const int64_t pitch = ((int64_t)d->num_slices * d->max_rank + 15) / 16 * 16;
  const size_t part = (size_t)lora_split(d, tokens, block_m) * (size_t)rows * (size_t)pitch * sizeof(float);
  const size_t both = block_m == 16 ? 0 : (size_t)d->num_slices * (size_t)rows * (size_t)lora_padded_rank(d->max_rank) * 4;
  if (a && a->part) {
    a->t16 = (uint16_t*)((uint8_t*)a->part + part);            // (rows are multiples of 16: every part starts at 16 bytes)
    a->t_scale = (float*)((uint8_t*)a->part + part + both);
  }
  return part + both + (block_m == 16 ? 0 : (size_t)d->num_slices * (size_t)rows * sizeof(float));
}

size_t qg_lora_workspace_bytes(const qg_lora_desc* d, int64_t tokens, int32_t block_m) {
  if (check_lora(d) != QG_OK || tokens <= 0 || tokens > kLoraMaxTokens || !lora_block(block_m)) return 0;
  return lora_workspace(d, tokens, block_m, nullptr);
}

qg_status qg_lora(const qg_lora_desc* d, const void* x, const void* a_weight, const void* b_weight, const int32_t* ranks,
                  const float* scales, const int32_t* sorted_ids, const int32_t* expert_ids, const int32_t* num_post_pad,
                  int64_t tokens, int32_t block_m, const void* base, void* y, void* ws, size_t ws_bytes, void* stream) {
  qg_status s = check_lora(d);
  if (s != QG_OK) return s;
  if (tokens < 0) return QG_ERR_INVALID_ARG;
  if (!lora_block(block_m)) return QG_ERR_UNSUPPORTED;
  if (tokens > kLoraMaxTokens) return QG_ERR_UNSUPPORTED;
  if (tokens == 0) return QG_OK;
  if (!x || !a_weight || !b_weight || !sorted_ids || !expert_ids || !num_post_pad || !base || !y) return QG_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(a_weight) || !aligned16(b_weight) || !aligned16(base) || !aligned16(y) ||
      (((uintptr_t)ranks | (uintptr_t)scales | (uintptr_t)sorted_ids | (uintptr_t)expert_ids | (uintptr_t)num_post_pad) & 3u) != 0)
    return QG_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws) || ws_bytes < qg_lora_workspace_bytes(d, tokens, block_m)) return QG_ERR_WORKSPACE;
  LoraArgs a{};
  stride_of(d->x_stride, d->k, &a.x_stride);
  stride_of(d->base_stride, d->n, &a.base_stride);
  stride_of(d->y_stride, d->n, &a.y_stride);
  if (y == base && tokens > 1 && a.y_stride != a.base_stride) return QG_ERR_INVALID_ARG;   // (rows overwritten before they are read)
  const int64_t blocks = block_capacity(tokens, d->num_adapters, block_m, &a.cap_rows);
  if (blocks * std::max(1, block_m / 64) * (d->n / 128 + d->num_slices) >= (int64_t)1 << 23) return QG_ERR_UNSUPPORTED;   // a launch takes fewer than 2^32 threads
  s = check_arch();
  if (s != QG_OK) return s;
  a.x = x; a.a = a_weight; a.b = b_weight; a.base = base; a.y = y;
  a.ranks = ranks; a.scales = scales; a.sorted_ids = sorted_ids; a.expert_ids = expert_ids; a.num_post_pad = num_post_pad;
  a.part = (float*)ws;
  a.n = d->n; a.k = (int)d->k; a.tokens = (int)tokens; a.max_rank = d->max_rank; a.slices = d->num_slices;
  a.rank_rows = d->num_slices * d->max_rank;
  a.rank_pitch = (a.rank_rows + 15) / 16 * 16;
  a.ksplit = lora_split(d, tokens, block_m);
  lora_workspace(d, tokens, block_m, &a);
  a.block_shift = log2_of(block_m);
  for (int i = 0; i < d->num_slices; ++i) a.slice_end[i] = (int)d->slice_end[i];
  QG_LOG("lora tokens=%lld n=%lld k=%lld rank=%d x %d -> block=%d ksplit=%d", (long long)tokens, (long long)d->n,
         (long long)d->k, d->num_slices, d->max_rank, block_m, a.ksplit);
  launch_lora(a, d->type == QG_O_F16 ? O_F16 : O_BF16, (unsigned)blocks, (hipStream_t)stream);
  return launched();
}

size_t qg_kv_cache_bytes(const qg_kv_desc* d) {
  if (check_kv(d) != QG_OK) return 0;
  return (size_t)d->num_pages * (size_t)d->kv_heads * (size_t)kv_head_bytes(d->page_tokens, d->head_dim);
}

qg_status qg_kv_append(const qg_kv_desc* d, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                       const int32_t* slots, int64_t tokens, void* cache, void* stream) {
  qg_status s = check_kv(d);
  if (s != QG_OK) return s;
  const int64_t width = (int64_t)d->kv_heads * d->head_dim;
  KvArgs a = kv_args(d, slots, tokens, cache);
  if (tokens < 0 || !stride_of(k_stride, width, &a.k_stride) || !stride_of(v_stride, width, &a.v_stride))
    return QG_ERR_INVALID_ARG;
  if (tokens > ((int64_t)1 << 31) - 1) return QG_ERR_UNSUPPORTED;
  if (tokens == 0) return QG_OK;
  if (!k || !v || !slots || !cache || !aligned16(k) || !aligned16(v) || !aligned16(cache) || ((uintptr_t)slots & 3u) != 0)
    return QG_ERR_INVALID_ARG;
  s = check_arch();
  if (s != QG_OK) return s;
  a.k = k; a.v = v;
  launch_kv_append(a, d->type == QG_O_F16 ? O_F16 : O_BF16, (hipStream_t)stream);
  return launched();
}

qg_status qg_kv_read(const qg_kv_desc* d, const void* cache, const int32_t* slots, int64_t tokens, void* k, void* v,
                     void* stream) {
  qg_status s = check_kv(d);
  if (s != QG_OK) return s;
  if (tokens < 0) return QG_ERR_INVALID_ARG;
  if (tokens > ((int64_t)1 << 31) - 1) return QG_ERR_UNSUPPORTED;
  if (tokens == 0) return QG_OK;
  if (!k || !v || !slots || !cache || !aligned16(k) || !aligned16(v) || !aligned16(cache) || ((uintptr_t)slots & 3u) != 0)
    return QG_ERR_INVALID_ARG;
  s = check_arch();
  if (s != QG_OK) return s;
  KvArgs a = kv_args(d, slots, tokens, cache);
  a.k_out = k; a.v_out = v;
  launch_kv_read(a, d->type == QG_O_F16 ? O_F16 : O_BF16, (hipStream_t)stream);
  return launched();
}

static qg_status check_attention(const qg_kv_desc* d, int32_t q_heads, int64_t batch, int64_t max_q, int64_t tokens,
                                 int64_t max_len) {
  const qg_status s = check_kv(d);
  if (s != QG_OK) return s;
  if (q_heads <= 0 || q_heads % d->kv_heads != 0 || batch < 0 || max_q <= 0 || tokens < 0 || max_len < 0) return QG_ERR_INVALID_ARG;
  if (q_heads / d->kv_heads > 256 || batch > 65535 || max_q > (1 << 24) || tokens > (1 << 24) || max_len > (1 << 30)) return QG_ERR_UNSUPPORTED;
  return QG_OK;
}

size_t qg_attention_workspace_bytes(const qg_kv_desc* d, int32_t q_heads, int64_t batch, int64_t max_q, int64_t tokens,
                                    int64_t max_len) {
  if (check_attention(d, q_heads, batch, max_q, tokens, max_len) != QG_OK || batch == 0) return 0;
  const int splits =
      attn_split(batch, q_heads, d->kv_heads, max_q, max_len, d->head_dim, d->type == QG_O_F16 ? O_F16 : O_BF16).parts;
  return splits > 1 ? (size_t)splits * (size_t)tokens * (size_t)q_heads * (size_t)(d->head_dim + 2) * sizeof(float) : 0;
}

qg_status qg_attention(const qg_kv_desc* d, const void* q, int64_t q_stride, int32_t q_heads, const void* cache,
                       const int32_t* block_table, int64_t table_stride, const int32_t* seq_lens, const int32_t* q_offsets,
                       int64_t batch, int64_t max_q, int64_t tokens, int64_t max_len, float scale, void* out,
                       int64_t out_stride, void* ws, size_t ws_bytes, void* stream) {
  qg_status s = check_attention(d, q_heads, batch, max_q, tokens, max_len);
  if (s != QG_OK) return s;
  AttnArgs a{};
  const int64_t width = (int64_t)q_heads * d->head_dim;
  if (!finite(scale * kLog2e) || !stride_of(q_stride, width, &a.q_stride) || !stride_of(out_stride, width, &a.out_stride))
    return QG_ERR_INVALID_ARG;
  if (table_stride < 0 || table_stride > kMaxStride || table_stride * d->page_tokens < max_len) return QG_ERR_INVALID_ARG;
  if (!q_offsets && (max_q != 1 || tokens != batch)) return QG_ERR_INVALID_ARG;
  if (batch == 0 || tokens == 0) return QG_OK;
  if (!q || !out || !cache || !seq_lens || (!block_table && max_len > 0)) return QG_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(cache) ||
      (((uintptr_t)block_table | (uintptr_t)seq_lens | (uintptr_t)q_offsets) & 3u) != 0)
    return QG_ERR_INVALID_ARG;
  const int type = d->type == QG_O_F16 ? O_F16 : O_BF16;
  const AttnSplit split = attn_split(batch, q_heads, d->kv_heads, max_q, max_len, d->head_dim, type);
  a.nsplit = split.parts;
  a.chunk = split.chunk;
  if (a.nsplit > 1 &&
      (!ws || !aligned16(ws) || ws_bytes < qg_attention_workspace_bytes(d, q_heads, batch, max_q, tokens, max_len)))
    return QG_ERR_WORKSPACE;
  a.group = q_heads / d->kv_heads;
  a.group_inv = (uint32_t)((((uint64_t)1 << 32) + a.group - 1) / a.group);
  // grid axes of 65535 workgroups, launches of fewer than 2^32 threads
  const int64_t tiles = split.row_tiles * split.parts;
  if (tiles > 65535 || tiles * batch * d->kv_heads >= ((int64_t)1 << 24) || max_q > 65535) return QG_ERR_UNSUPPORTED;
  s = check_arch();
  if (s != QG_OK) return s;
  a.cache = (const uint8_t*)cache; a.table = block_table; a.lens = seq_lens; a.q_offsets = q_offsets;
  a.q = q; a.out = out; a.part = (float*)ws;
  a.table_stride = table_stride; a.num_pages = d->num_pages; a.tokens = tokens; a.rows = tokens * q_heads;
  a.batch = (int)batch; a.q_heads = q_heads; a.kv_heads = d->kv_heads; a.dim = d->head_dim;
  a.page_shift = log2_of(d->page_tokens); a.max_q = (int)max_q; a.max_len = (int)max_len;
  // (scores of tokens that are not seen are -infinity, before the scale: times 0 they would be NaN)
  a.scale_log2 = std::max(fabsf(scale) * kLog2e, 0x1p-149f);
  a.q_sign = scale < 0 ? 0x80008000u : 0;
  QG_LOG("attention batch=%lld heads=%d/%d dim=%d max_q=%lld max_len=%lld -> splits=%d", (long long)batch, q_heads,
         d->kv_heads, d->head_dim, (long long)max_q, (long long)max_len, a.nsplit);
  if (!launch_attention(a, type, (hipStream_t)stream)) return QG_ERR_UNSUPPORTED;
  return launched();
}

}  // extern "C"
