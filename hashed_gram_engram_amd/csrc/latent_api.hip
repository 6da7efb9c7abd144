// C ABI of the latent cache and its attention: synchronous argument checks, then one or two launches on the
// caller's stream.  No device memory is allocated here.
#include <hip/hip_runtime.h>
#include <math.h>
#include <string.h>

#include "../../include/engram.h"
#include "latent.h"
#include "launch.h"
#include "serving.h"

using namespace engram;

namespace {

constexpr float kLog2e = 1.44269504f;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

engram_status launched(hipError_t e) { return e == hipSuccess ? ENGRAM_OK : ENGRAM_E_HIP; }

hipStream_t hip_stream(engram_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

// Elements between rows of `row` elements: at least so many, whole 16 bytes, offsets far from 64 bits.
bool stride_ok(int64_t stride, int64_t row) { return stride >= row && stride % 8 == 0 && stride <= (int64_t(1) << 28); }

// The checks that both attentions and the read share; fills `q`.
engram_status requests(const engram_latent_layout* l, const int32_t* token_start, const int32_t* start_pos, int64_t R,
                       int64_t n_tokens, LatentRequests* q) {
  memset(q, 0, sizeof(*q));
  if (R < 0 || R > kMaxRequests || n_tokens < 0 || n_tokens > (int64_t(1) << 30) / l->heads) return ENGRAM_E_SHAPE;
  if (R > 0 && (!token_start || !start_pos)) return ENGRAM_E_NULL;
  if (!aligned(token_start, 4) || !aligned(start_pos, 4)) return ENGRAM_E_ALIGN;
  q->token_start = token_start;
  q->start_pos = start_pos;
  q->R = int(R);
  q->n_tokens = int(n_tokens);
  q->min_tokens = 1;
  q->set_pages(1 << 30, 1, 0);  // (without pages: positions below 2^30)
  q->window = l->window < (1 << 30) ? l->window : 1 << 30;  // (no position lies further back)
  return ENGRAM_OK;
}

engram_status latent_pages_check(const engram_page_layout* p) {
  const engram_status st = engram_page_layout_check(p);
  if (st != ENGRAM_OK) return st;
  return p->n_blocks > 0x7FFFFFFF / p->block_size ? ENGRAM_E_LAYOUT : ENGRAM_OK;  // slots are counted in 32 bits
}

engram_status pages_of(const engram_page_layout* p, const int32_t* block_table, LatentRequests* q) {
  if (q->R > 0 && !block_table) return ENGRAM_E_NULL;
  if (!aligned(block_table, 4)) return ENGRAM_E_ALIGN;
  q->block_table = block_table;
  q->set_pages(p->block_size, p->max_blocks, p->n_blocks);
  return ENGRAM_OK;
}

}  // namespace

extern "C" {

engram_status engram_latent_layout_check(const engram_latent_layout* l) {
  if (l == nullptr) return ENGRAM_E_NULL;
  if (l->heads < 1 || l->heads > 1024) return ENGRAM_E_LAYOUT;
  if (l->latent_dim != 128 && l->latent_dim != 256 && l->latent_dim != 512) return ENGRAM_E_LAYOUT;
  if (l->rope_dim != 32 && l->rope_dim != 64) return ENGRAM_E_LAYOUT;
  if (l->head_dim != 64 && l->head_dim != 128) return ENGRAM_E_LAYOUT;
  if (l->cache_format != ENGRAM_CACHE_BF16 && l->cache_format != ENGRAM_CACHE_MXFP8) return ENGRAM_E_LAYOUT;
  if (l->window < 0 || !(fabsf(l->scale) < 0x1p127f)) return ENGRAM_E_LAYOUT;  // (times log2 e it stays finite)
  return ENGRAM_OK;
}

size_t engram_latent_row_bytes(const engram_latent_layout* l) {
  if (engram_latent_layout_check(l) != ENGRAM_OK) return 0;
  return size_t(latent_row_bytes(l->latent_dim, l->rope_dim, l->cache_format == ENGRAM_CACHE_MXFP8));
}

engram_status engram_latent_write(const engram_latent_layout* l, const engram_page_layout* p, const uint16_t* latent,
                                  int64_t latent_stride, const uint16_t* rope, int64_t rope_stride,
                                  const int64_t* slots, int64_t n_tokens, void* cache, int32_t* err_count,
                                  engram_stream_t stream) {
  engram_status st = engram_latent_layout_check(l);
  if (st != ENGRAM_OK) return st;
  if ((st = latent_pages_check(p)) != ENGRAM_OK) return st;
  if (n_tokens < 0 || n_tokens > (int64_t(1) << 30)) return ENGRAM_E_SHAPE;
  if (n_tokens == 0) return ENGRAM_OK;
  if (!latent || !rope || !slots || !cache) return ENGRAM_E_NULL;
  if (!aligned(latent, 16) || !aligned(rope, 16) || !aligned(cache, 16) || !aligned(slots, 8) || !aligned(err_count, 4))
    return ENGRAM_E_ALIGN;
  if (!stride_ok(latent_stride, l->latent_dim) || !stride_ok(rope_stride, l->rope_dim)) return ENGRAM_E_SHAPE;
  DeviceInfo di;
  if ((st = device_info(&di)) != ENGRAM_OK) return st;
  LatentWriteArgs a;
  memset(&a, 0, sizeof(a));
  a.latent = latent;
  a.rope = rope;
  a.slots = slots;
  a.cache = static_cast<uint8_t*>(cache);
  a.err_count = err_count;
  a.latent_stride = latent_stride;
  a.rope_stride = rope_stride;
  a.n_slots = p->n_blocks * p->block_size;
  a.n_tokens = int(n_tokens);
  a.latent_dim = l->latent_dim;
  a.rope_dim = l->rope_dim;
  a.fp8 = l->cache_format == ENGRAM_CACHE_MXFP8;
  return launched(launch_latent_write(a, hip_stream(stream)));
}

engram_status engram_latent_read(const engram_latent_layout* l, const engram_page_layout* p, const void* cache,
                                 const int32_t* token_start, const int32_t* start_pos, int64_t R,
                                 const int32_t* block_table, int64_t n_tokens, int32_t min_tokens, int64_t max_rows,
                                 int32_t* row_start, uint16_t* latent, uint16_t* rope, int32_t* err_count,
                                 engram_stream_t stream) {
  engram_status st = engram_latent_layout_check(l);
  if (st != ENGRAM_OK) return st;
  if ((st = latent_pages_check(p)) != ENGRAM_OK) return st;
  LatentReadArgs a;
  memset(&a, 0, sizeof(a));
  if ((st = requests(l, token_start, start_pos, R, n_tokens, &a.rq)) != ENGRAM_OK) return st;
  if ((st = pages_of(p, block_table, &a.rq)) != ENGRAM_OK) return st;
  if (min_tokens < 1 || max_rows < 0 || max_rows > (int64_t(1) << 30)) return ENGRAM_E_SHAPE;
  if (!cache || !row_start || (max_rows > 0 && (!latent || !rope))) return ENGRAM_E_NULL;
  if (!aligned(cache, 16) || !aligned(latent, 16) || !aligned(rope, 16) || !aligned(row_start, 4) || !aligned(err_count, 4))
    return ENGRAM_E_ALIGN;
  DeviceInfo di;
  if ((st = device_info(&di)) != ENGRAM_OK) return st;
  a.rq.min_tokens = min_tokens;
  a.cache = static_cast<const uint8_t*>(cache);
  a.row_start = row_start;
  a.latent = latent;
  a.rope = rope;
  a.err_count = err_count;
  a.max_rows = max_rows;
  a.latent_dim = l->latent_dim;
  a.rope_dim = l->rope_dim;
  a.fp8 = l->cache_format == ENGRAM_CACHE_MXFP8;
  return launched(launch_latent_read(a, di.cus, hip_stream(stream)));
}

size_t engram_latent_attention_workspace_bytes(const engram_latent_layout* l) {
  if (engram_latent_layout_check(l) != ENGRAM_OK) return 0;
  DeviceInfo di;
  const int cus = device_info(&di) == ENGRAM_OK ? di.cus : 256;
  return size_t(absorbed_workspace_bytes(l->latent_dim, cus));
}

engram_status engram_latent_attention(const engram_latent_layout* l, const engram_page_layout* p, const uint16_t* q,
                                      int64_t q_stride, const void* cache, const int32_t* token_start,
                                      const int32_t* start_pos, int64_t R, const int32_t* block_table,
                                      int64_t n_tokens, int32_t max_tokens, uint16_t* out, int64_t out_stride,
                                      float* lse, void* workspace, size_t workspace_bytes, int32_t* err_count,
                                      engram_stream_t stream) {
  engram_status st = engram_latent_layout_check(l);
  if (st != ENGRAM_OK) return st;
  if ((st = latent_pages_check(p)) != ENGRAM_OK) return st;
  AbsorbedArgs a;
  memset(&a, 0, sizeof(a));
  if ((st = requests(l, token_start, start_pos, R, n_tokens, &a.rq)) != ENGRAM_OK) return st;
  if ((st = pages_of(p, block_table, &a.rq)) != ENGRAM_OK) return st;
  if (max_tokens < 0) return ENGRAM_E_SHAPE;
  if (R == 0 || n_tokens == 0) return ENGRAM_OK;
  if (!q || !cache || !out) return ENGRAM_E_NULL;
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(err_count, 4))
    return ENGRAM_E_ALIGN;
  if (!stride_ok(q_stride, int64_t(l->heads) * (l->latent_dim + l->rope_dim)) ||
      !stride_ok(out_stride, int64_t(l->heads) * l->latent_dim))
    return ENGRAM_E_SHAPE;
  DeviceInfo di;
  if ((st = device_info(&di)) != ENGRAM_OK) return st;
  if (workspace == nullptr || !aligned(workspace, 16) ||
      workspace_bytes < size_t(absorbed_workspace_bytes(l->latent_dim, di.cus)))
    return ENGRAM_E_WORKSPACE;
  a.rq.max_tokens = max_tokens;
  a.q = q;
  a.cache = static_cast<const uint8_t*>(cache);
  a.out = out;
  a.lse = lse;
  a.err_count = err_count;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.scale_log2 = fmaxf(fabsf(l->scale) * kLog2e, 1e-44f);
  a.q_sign = l->scale < 0.0f ? 0x80008000u : 0u;
  a.heads = l->heads;
  a.latent_dim = l->latent_dim;
  a.rope_dim = l->rope_dim;
  a.fp8 = l->cache_format == ENGRAM_CACHE_MXFP8;
  a.workspace = static_cast<char*>(workspace);
  return launched(launch_latent_absorbed(a, di.cus, hip_stream(stream)));
}

size_t engram_latent_attention_expanded_workspace_bytes(const engram_latent_layout* l, int64_t R, int64_t n_tokens,
                                                        int64_t n_rows) {
  if (engram_latent_layout_check(l) != ENGRAM_OK || R < 1 || R > kMaxRequests || n_tokens < 1 ||
      n_tokens > (int64_t(1) << 30) / l->heads || n_rows < 0 || n_rows > (int64_t(1) << 30))
    return 0;
  DeviceInfo di;
  const int cus = device_info(&di) == ENGRAM_OK ? di.cus : 256;
  return size_t(expanded_workspace_bytes(R, n_tokens, n_rows, l->heads, l->head_dim, cus));
}

size_t engram_latent_attention_expanded_workspace_bytes_up_to(const engram_latent_layout* l, int64_t n_tokens, int64_t n_rows) {
  if (engram_latent_layout_check(l) != ENGRAM_OK || n_tokens < 1 || n_tokens > (int64_t(1) << 30) / l->heads || n_rows < 0 ||
      n_rows > (int64_t(1) << 30))
    return 0;
  DeviceInfo di;
  const int cus = device_info(&di) == ENGRAM_OK ? di.cus : 256;
  return size_t(expanded_workspace_bytes_up_to(n_tokens, n_rows, l->heads, l->head_dim, cus));
}

engram_status engram_latent_attention_expanded(const engram_latent_layout* l, const uint16_t* q, int64_t q_stride,
                                               const uint16_t* kv, int64_t kv_stride, const uint16_t* rope,
                                               int64_t rope_stride, const int32_t* row_start, int64_t n_rows,
                                               const int32_t* token_start, const int32_t* start_pos, int64_t R,
                                               int64_t n_tokens, int32_t min_tokens, uint16_t* out,
                                               int64_t out_stride, float* lse, void* workspace,
                                               size_t workspace_bytes, engram_stream_t stream) {
  engram_status st = engram_latent_layout_check(l);
  if (st != ENGRAM_OK) return st;
  ExpandedArgs a;
  memset(&a, 0, sizeof(a));
  if ((st = requests(l, token_start, start_pos, R, n_tokens, &a.rq)) != ENGRAM_OK) return st;
  if (min_tokens < 1 || n_rows < 0 || n_rows > (int64_t(1) << 30)) return ENGRAM_E_SHAPE;
  // a launch of 2^32 threads and more loses some without an error: at most 256 for each tile of 64 tokens and head
  if ((n_tokens / 64 + (R < n_tokens ? R : n_tokens)) * l->heads >= int64_t(1) << 24) return ENGRAM_E_SHAPE;
  if (R == 0 || n_tokens == 0) return ENGRAM_OK;
  if (!q || !row_start || !out || (n_rows > 0 && (!kv || !rope))) return ENGRAM_E_NULL;
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(rope, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(row_start, 4))
    return ENGRAM_E_ALIGN;
  if (!stride_ok(q_stride, int64_t(l->heads) * (l->head_dim + l->rope_dim)) ||
      !stride_ok(out_stride, int64_t(l->heads) * l->head_dim))
    return ENGRAM_E_SHAPE;
  if (n_rows > 0 && (!stride_ok(kv_stride, int64_t(l->heads) * 2 * l->head_dim) || !stride_ok(rope_stride, l->rope_dim)))
    return ENGRAM_E_SHAPE;
  DeviceInfo di;
  if ((st = device_info(&di)) != ENGRAM_OK) return st;
  const int64_t need = expanded_workspace_bytes(R, n_tokens, n_rows, l->heads, l->head_dim, di.cus);
  if (need > 0 && (workspace == nullptr || workspace_bytes < size_t(need) || !aligned(workspace, 16))) return ENGRAM_E_WORKSPACE;
  a.rq.min_tokens = min_tokens;
  a.q = q;
  a.kv = kv;
  a.rope = rope;
  a.row_start = row_start;
  a.out = out;
  a.lse = lse;
  a.q_stride = q_stride;
  a.kv_stride = kv_stride;
  a.rope_stride = rope_stride;
  a.out_stride = out_stride;
  a.n_rows = int(n_rows);
  a.scale_log2 = fmaxf(fabsf(l->scale) * kLog2e, 1e-44f);
  a.q_sign = l->scale < 0.0f ? 0x80008000u : 0u;
  a.heads = l->heads;
  a.head_dim = l->head_dim;
  a.rope_dim = l->rope_dim;
  a.workspace = static_cast<float*>(workspace);
  return launched(launch_latent_expanded(a, di.cus, hip_stream(stream)));
}

}  // extern "C"
