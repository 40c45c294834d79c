// api_decode.cu -- the C ABI of the decoding-step operators: the 4-bit paged key/value cache (append, read back,
// attention) and the processing of logits.  Host side only: argument checks and launches.
#include <cmath>

#include "../../include/softmax_rows.h"
#include "kv4.h"
#include "launch.h"
#include "logits.h"

namespace rwo {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int64_t kMaxPositions = (int64_t(1) << 31) - 256;  // positions and rows are 32-bit in the kernels
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

// Sizes of a cache and its sequences; *noop where there is no token.
int check_cache(const kv4_cache* c, bool* noop) {
  *noop = false;
  if (!c) return SOFTMAX_ERR_INVALID_ARG;
  if (c->num_pages < 0 || c->heads < 1 || c->page_size < 1 || c->head_dim < 1 || c->batch < 0 || c->table_width < 0 || c->tokens < 0)
    return SOFTMAX_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return SOFTMAX_ERR_UNSUPPORTED;
  if (c->page_size % kKv4Block || c->heads > 65535 || c->num_pages > kMaxRows || c->batch > (1 << 24)) return SOFTMAX_ERR_UNSUPPORTED;
  if (c->page_size > kMaxPositions || (c->table_width > 0 && c->page_size > kMaxPositions / c->table_width)) return SOFTMAX_ERR_UNSUPPORTED;
  if (c->tokens > kMaxRows / c->heads) return SOFTMAX_ERR_UNSUPPORTED;
  if (c->num_pages > 0 && c->page_size / kKv4Block > INT64_MAX / 20 / c->head_dim / c->heads / c->num_pages) return SOFTMAX_ERR_INVALID_ARG;
  if (!c->cu_tokens && c->tokens != c->batch) return SOFTMAX_ERR_INVALID_ARG;
  if (c->tokens == 0 || c->batch == 0) {
    *noop = true;
    return SOFTMAX_OK;
  }
  if (c->num_pages < 1 || c->table_width < 1 || !c->data || !c->page_table || !c->seq_lens) return SOFTMAX_ERR_INVALID_ARG;
  if (!aligned(c->data, 16) || !aligned(c->page_table, 4) || !aligned(c->seq_lens, 4) || !aligned(c->cu_tokens, 4))
    return SOFTMAX_ERR_MISALIGNED;
  return SOFTMAX_OK;
}

Kv4View view_of(const kv4_cache* c, const DeviceInfo& dev) {
  Kv4View v;
  v.data = static_cast<unsigned char*>(c->data);
  v.table = c->page_table;
  v.lens = c->seq_lens;
  v.cu = c->cu_tokens;
  v.num_pages = c->num_pages;
  v.width = c->table_width;
  v.tokens = c->tokens;
  v.batch = int(c->batch);
  v.heads = int(c->heads);
  v.d = int(c->head_dim);
  v.page_blocks = int(c->page_size / kKv4Block);
  v.status = dev.status;
  return v;
}

// Rows [tokens][heads][d]: 16-byte aligned at every token and head.
int check_rows(const kv4_rows* r, int64_t tokens, int64_t heads) {
  if (!r || !r->data) return SOFTMAX_ERR_INVALID_ARG;
  if (!aligned(r->data, 16) || r->token_stride % 8 || r->head_stride % 8) return SOFTMAX_ERR_MISALIGNED;
  const int64_t a = r->token_stride < 0 ? -r->token_stride : r->token_stride, b = r->head_stride < 0 ? -r->head_stride : r->head_stride;
  if (a < 0 || b < 0 || a > INT64_MAX / 8 / tokens || b > INT64_MAX / 8 / heads) return SOFTMAX_ERR_INVALID_ARG;
  return SOFTMAX_OK;
}
Kv4Rows rows_of(const kv4_rows* r) { return r ? Kv4Rows{r->data, r->token_stride, r->head_stride} : Kv4Rows{}; }

int check_16bit(int dtype) {
  if (dtype != SOFTMAX_F32 && dtype != SOFTMAX_BF16 && dtype != SOFTMAX_F16) return SOFTMAX_ERR_INVALID_ARG;
  return dtype == SOFTMAX_F32 ? SOFTMAX_ERR_UNSUPPORTED : SOFTMAX_OK;
}

}  // namespace
}  // namespace rwo

using namespace rwo;

extern "C" {

int kv4_append(const kv4_cache* cache, const kv4_rows* k, const kv4_rows* v, const kv4_rows* q, const kv4_rows* q_out, int64_t q_heads,
               const float* cos_sin, int64_t positions, int64_t rotated, int flags, int dtype, void* stream) {
  bool noop = false;
  int st = check_16bit(dtype);
  if (st == SOFTMAX_OK) st = check_cache(cache, &noop);
  if (st != SOFTMAX_OK) return st;
  if ((flags & ~KV4_FLAG_NEIGHBOURS) || q_heads < 0 || (!q) != (!q_out) || (q && q_heads < 1)) return SOFTMAX_ERR_INVALID_ARG;
  if (!q) q_heads = 0;
  if (q_heads > 65535 || cache->tokens > kMaxRows / (q_heads + 2 * cache->heads)) return SOFTMAX_ERR_UNSUPPORTED;
  if (cos_sin) {
    if (rotated < 1 || rotated > cache->head_dim || positions < 1) return SOFTMAX_ERR_INVALID_ARG;
    if (rotated % 8) return SOFTMAX_ERR_UNSUPPORTED;
    if (!aligned(cos_sin, 16)) return SOFTMAX_ERR_MISALIGNED;
    if (positions > INT64_MAX / 4 / rotated) return SOFTMAX_ERR_INVALID_ARG;
  }
  if (noop) return SOFTMAX_OK;
  if ((st = check_rows(k, cache->tokens, cache->heads)) != SOFTMAX_OK || (st = check_rows(v, cache->tokens, cache->heads)) != SOFTMAX_OK) return st;
  if (q && ((st = check_rows(q, cache->tokens, q_heads)) != SOFTMAX_OK || (st = check_rows(q_out, cache->tokens, q_heads)) != SOFTMAX_OK)) return st;
  const DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != SOFTMAX_OK) return st;
  const cudaError_t err = launch_kv4_append(view_of(cache, *dev), rows_of(k), rows_of(v), rows_of(q), rows_of(q_out), int(q_heads), cos_sin,
                                            positions, int(rotated), (flags & KV4_FLAG_NEIGHBOURS) != 0, dtype,
                                            static_cast<cudaStream_t>(stream), *dev);
  return err == cudaSuccess ? SOFTMAX_OK : cuda_failure(err);
}

int kv4_gather(const kv4_cache* cache, const kv4_rows* k, const kv4_rows* v, int dtype, void* stream) {
  bool noop = false;
  int st = check_16bit(dtype);
  if (st == SOFTMAX_OK) st = check_cache(cache, &noop);
  if (st != SOFTMAX_OK || noop) return st;
  if ((st = check_rows(k, cache->tokens, cache->heads)) != SOFTMAX_OK || (st = check_rows(v, cache->tokens, cache->heads)) != SOFTMAX_OK) return st;
  const DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != SOFTMAX_OK) return st;
  const cudaError_t err = launch_kv4_gather(view_of(cache, *dev), rows_of(k), rows_of(v), dtype, static_cast<cudaStream_t>(stream), *dev);
  return err == cudaSuccess ? SOFTMAX_OK : cuda_failure(err);
}

static int check_attention(int64_t batch, int64_t tokens, int64_t q_heads, int64_t heads, int64_t head_dim) {
  if (batch < 0 || tokens < 0 || q_heads < 1 || heads < 1 || q_heads % heads) return SOFTMAX_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return SOFTMAX_ERR_UNSUPPORTED;
  if (q_heads > 65535 || batch > (1 << 24) || tokens > kMaxRows / q_heads) return SOFTMAX_ERR_UNSUPPORTED;
  return SOFTMAX_OK;
}

int64_t attention_kv4_workspace(int64_t batch, int64_t tokens, int64_t q_heads, int64_t heads, int64_t head_dim) {
  if (check_attention(batch, tokens, q_heads, heads, head_dim) != SOFTMAX_OK) return -1;
  if (batch == 0 || tokens == 0) return 0;
  const DeviceInfo* dev = nullptr;
  if (current_device(&dev) != SOFTMAX_OK) return -1;
  return int64_t(attention_kv4_scratch(batch, tokens, int(q_heads), int(heads), int(head_dim), *dev));
}

int attention_kv4(const kv4_cache* cache, const kv4_rows* q, void* o, float* lse_out, int64_t q_heads, float scale, int dtype,
                  void* workspace, int64_t workspace_bytes, void* stream) {
  bool noop = false;
  int st = check_16bit(dtype);
  if (st == SOFTMAX_OK) st = check_cache(cache, &noop);
  if (st == SOFTMAX_OK) st = check_attention(cache->batch, cache->tokens, q_heads, cache->heads, cache->head_dim);
  if (st != SOFTMAX_OK) return st;
  if (scale == 0.f) scale = float(1.0 / sqrt(double(cache->head_dim)));  // the attention default, 1 / sqrt(d)
  if (!(scale > 0.f) || !(scale <= 3.4028234663852886e38f)) return SOFTMAX_ERR_INVALID_ARG;
  if (noop) return SOFTMAX_OK;
  if ((st = check_rows(q, cache->tokens, q_heads)) != SOFTMAX_OK) return st;
  if (!o || !workspace) return SOFTMAX_ERR_INVALID_ARG;
  if (!aligned(o, 16) || !aligned(workspace, 256) || !aligned(lse_out, 4)) return SOFTMAX_ERR_MISALIGNED;
  const DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != SOFTMAX_OK) return st;
  if (workspace_bytes < int64_t(attention_kv4_scratch(cache->batch, cache->tokens, int(q_heads), int(cache->heads), int(cache->head_dim), *dev)))
    return SOFTMAX_ERR_INVALID_ARG;
  const cudaError_t err = launch_attention_kv4(view_of(cache, *dev), rows_of(q), o, lse_out, int(q_heads), scale, dtype, workspace,
                                               static_cast<cudaStream_t>(stream), *dev);
  return err == cudaSuccess ? SOFTMAX_OK : cuda_failure(err);
}

int logits_process_rows(const logits_rows* a, int64_t M, int64_t N, int dtype, int out, void* stream) {
  if (!a || M < 0 || N < 1) return SOFTMAX_ERR_INVALID_ARG;
  if (dtype != SOFTMAX_F32 && dtype != SOFTMAX_BF16 && dtype != SOFTMAX_F16) return SOFTMAX_ERR_INVALID_ARG;
  if (out < LOGITS_OUT_LOGITS || out > LOGITS_OUT_LOG_SOFTMAX) return SOFTMAX_ERR_INVALID_ARG;
  const int64_t s = elem_bytes(dtype), ldx = a->ldx ? a->ldx : N, ldy = a->ldy ? a->ldy : N, words = (N + 31) / 32;
  const int64_t ldm = a->ld_mask ? a->ld_mask : words;
  if (ldx < N || ldy < N || ldm < words || a->token_width < 0 || a->bias_count < 0) return SOFTMAX_ERR_INVALID_ARG;
  if (M > 0 && (ldx > INT64_MAX / s / M || ldy > INT64_MAX / s / M || ldm > INT64_MAX / 4 / M)) return SOFTMAX_ERR_INVALID_ARG;
  // 32-bit tokens; counts and bias indices share a 32-bit word
  if (N > kMaxPositions || M > (1 << 26) || a->token_width >= kMaxHistory || a->bias_count > kMaxBias) return SOFTMAX_ERR_UNSUPPORTED;
  if (M == 0) return SOFTMAX_OK;
  if (!a->x || !a->y) return SOFTMAX_ERR_INVALID_ARG;
  if (a->token_width > 0 && a->tokens && !a->token_lens) return SOFTMAX_ERR_INVALID_ARG;
  if (a->bias_count > 0 && (!a->bias_ids || !a->bias_values)) return SOFTMAX_ERR_INVALID_ARG;
  if (!aligned(a->x, uintptr_t(s)) || !aligned(a->y, uintptr_t(s))) return SOFTMAX_ERR_MISALIGNED;
  for (const void* p : {static_cast<const void*>(a->lse_out), static_cast<const void*>(a->tokens), static_cast<const void*>(a->prompt_lens),
                        static_cast<const void*>(a->token_lens), static_cast<const void*>(a->repetition), static_cast<const void*>(a->frequency),
                        static_cast<const void*>(a->presence), static_cast<const void*>(a->bias_ids), static_cast<const void*>(a->bias_values),
                        static_cast<const void*>(a->mask), static_cast<const void*>(a->scale)})
    if (!aligned(p, 4)) return SOFTMAX_ERR_MISALIGNED;
  const DeviceInfo* dev = nullptr;
  int st = current_device(&dev);
  if (st != SOFTMAX_OK) return st;
  LogitsProblem p;
  p.x = a->x;
  p.y = a->y;
  p.lse = a->lse_out;
  p.M = M;
  p.N = N;
  p.x_pitch = ldx;
  p.y_pitch = ldy;
  p.dtype = dtype;
  p.out = out;
  if (a->tokens && a->token_width > 0) {
    p.tokens = a->tokens;
    p.token_pitch = a->token_width;
    p.prompt_lens = a->prompt_lens;
    p.token_lens = a->token_lens;
    p.repetition = a->repetition;
    p.frequency = a->frequency;
    p.presence = a->presence;
  }
  if (a->bias_count > 0) {
    p.bias_ids = a->bias_ids;
    p.bias_values = a->bias_values;
    p.bias_count = int(a->bias_count);
  }
  p.mask = a->mask;
  p.mask_pitch = ldm;
  p.scale = a->scale;
  p.stream = static_cast<cudaStream_t>(stream);
  const cudaError_t err = launch_logits(p, *dev);
  return err == cudaSuccess ? SOFTMAX_OK : cuda_failure(err);
}

}  // extern "C"
