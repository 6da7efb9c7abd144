// C ABI of the serving operators: synchronous argument checks, then one launch on the caller's
// stream (two for a product that splits K).  No device memory is allocated here.
#include <hip/hip_runtime.h>
#include <math.h>
#include <string.h>

#include "../../include/engram.h"
#include "launch.h"
#include "serving.h"

using namespace engram;

namespace {

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

engram_status launched(hipError_t e) { return e == hipSuccess ? ENGRAM_OK : ENGRAM_E_HIP; }

hipStream_t hip_stream(engram_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

engram_status engram_page_layout_check(const engram_page_layout* l) {
  if (l == nullptr) return ENGRAM_E_NULL;
  if (l->block_size < 1 || l->max_blocks < 1 || l->n_blocks < 1 || l->n_blocks > (int64_t(1) << 30)) return ENGRAM_E_LAYOUT;
  if (int64_t(l->block_size) * l->max_blocks > (int64_t(1) << 30)) return ENGRAM_E_LAYOUT;
  return ENGRAM_OK;
}

engram_status engram_norm_layout_check(const engram_norm_layout* l) {
  if (l == nullptr) return ENGRAM_E_NULL;
  if (l->hc < 1 || l->hc > 64 || l->dim < 8 || l->dim % 8 != 0 || l->dim > 40960) return ENGRAM_E_LAYOUT;
  if (l->y_streams != 1 && l->y_streams != l->hc) return ENGRAM_E_LAYOUT;
  if (l->stream_format != ENGRAM_STREAM_BF16 && l->stream_format != ENGRAM_STREAM_FP32) return ENGRAM_E_LAYOUT;
  if (l->gate < ENGRAM_GATE_NONE || l->gate > ENGRAM_GATE_FEATURE) return ENGRAM_E_LAYOUT;
  if ((l->post_norm & ~1) != 0 || (l->pre_norm & ~1) != 0) return ENGRAM_E_LAYOUT;
  if (!isfinite(l->alpha) || !isfinite(l->beta)) return ENGRAM_E_LAYOUT;
  if (!(l->post_eps >= 0.0f) || !isfinite(l->post_eps) || !(l->pre_eps >= 0.0f) || !isfinite(l->pre_eps))
    return ENGRAM_E_LAYOUT;
  return ENGRAM_OK;
}

engram_status engram_linear_layout_check(const engram_linear_layout* l) {
  if (l == nullptr) return ENGRAM_E_NULL;
  if (l->in_features < 8 || l->in_features % 8 != 0 || l->in_features > (1 << 20)) return ENGRAM_E_LAYOUT;
  if (l->out_features < 1 || l->out_features > (1 << 24)) return ENGRAM_E_LAYOUT;
  if (l->activation < ENGRAM_ACT_NONE || l->activation > ENGRAM_ACT_SIGMOID) return ENGRAM_E_LAYOUT;
  if ((l->glu & ~1) != 0) return ENGRAM_E_LAYOUT;
  if (l->stream_format != ENGRAM_STREAM_BF16 && l->stream_format != ENGRAM_STREAM_FP32) return ENGRAM_E_LAYOUT;
  return ENGRAM_OK;
}

engram_status engram_batch_plan(const engram_page_layout* l, const int32_t* new_lens, const int32_t* cached_lens,
                                int64_t R, int32_t* block_table, int32_t* free_list, const int32_t* free_count,
                                int64_t max_tokens, const engram_batch_plan_out* plan, int32_t* err_count,
                                engram_stream_t stream) {
  engram_status st = engram_page_layout_check(l);
  if (st != ENGRAM_OK) return st;
  if (R < 0 || R > kMaxRequests || max_tokens < 0 || max_tokens > 0x7FFFFFFF - 1024) return ENGRAM_E_SHAPE;
  if (plan == nullptr || !free_list || !free_count || !plan->token_start || !plan->free_left) return ENGRAM_E_NULL;
  if (R > 0 && (!new_lens || !cached_lens || !block_table || !plan->start_pos || !plan->seq_lens || !plan->status))
    return ENGRAM_E_NULL;
  if (max_tokens > 0 && (!plan->slots || !plan->positions || !plan->requests || !plan->live)) return ENGRAM_E_NULL;
  const void* words[] = {new_lens,        cached_lens,    block_table,  free_list,       free_count,     plan->token_start,
                         plan->start_pos, plan->seq_lens, plan->status, plan->free_left, plan->positions, plan->requests,
                         err_count};
  for (const void* p : words)
    if (!aligned(p, 4)) return ENGRAM_E_ALIGN;
  if (!aligned(plan->slots, 8)) return ENGRAM_E_ALIGN;
  // every workgroup reads the lengths and the count: none of them may be written in place
  const void* in[] = {new_lens, cached_lens, free_count};
  const void* out[] = {plan->start_pos, plan->seq_lens, plan->status, plan->token_start, plan->free_left};
  for (const void* p : in)
    for (const void* q : out)
      if (p != nullptr && p == q) return ENGRAM_E_SHAPE;
  DeviceInfo di;
  if ((st = device_info(&di)) != ENGRAM_OK) return st;
  PlanArgs a;
  memset(&a, 0, sizeof(a));
  a.new_lens = new_lens;
  a.cached_lens = cached_lens;
  a.block_table = block_table;
  a.free_list = free_list;
  a.free_count = free_count;
  a.R = int(R);
  a.block_size = l->block_size;
  a.max_blocks = l->max_blocks;
  a.n_blocks = int(l->n_blocks);
  a.max_tokens = int(max_tokens);
  a.token_start = plan->token_start;
  a.start_pos = plan->start_pos;
  a.seq_lens = plan->seq_lens;
  a.status = plan->status;
  a.free_left = plan->free_left;
  a.slots = plan->slots;
  a.positions = plan->positions;
  a.requests = plan->requests;
  a.live = plan->live;
  a.err_count = err_count;
  return launched(launch_batch_plan(a, hip_stream(stream)));
}

engram_status engram_hash_ids_paged(const engram_hash_layout* hl, const engram_page_layout* pl,
                                    const uint32_t* token_map, const int64_t* multipliers, const int64_t* primes,
                                    const int64_t* offsets, const int64_t* input_ids, const uint8_t* token_mask,
                                    int64_t n_tokens, const int64_t* slots, const int32_t* positions,
                                    const int32_t* requests, const int32_t* start_pos, int64_t R,
                                    const int32_t* block_table, int64_t* history, int64_t* hash_ids,
                                    int32_t* err_count, engram_stream_t stream) {
  if (hl == nullptr) return ENGRAM_E_NULL;
  engram_status st = engram_page_layout_check(pl);
  if (st != ENGRAM_OK) return st;
  if (hl->n_layers < 1 || hl->max_ngram < 2 || hl->max_ngram > 8 || hl->n_heads < 1 || hl->vocab < 1 ||
      int64_t(hl->n_layers) * (hl->max_ngram - 1) * hl->n_heads > (1 << 20))
    return ENGRAM_E_LAYOUT;
  if (n_tokens < 0 || n_tokens > 0x7FFFFFFF || R < 0 || R > 0x7FFFFFFF) return ENGRAM_E_SHAPE;
  if (n_tokens == 0) return ENGRAM_OK;
  if (!token_map || !multipliers || !primes || !offsets || !input_ids || !slots || !positions || !requests ||
      !history || !hash_ids || (R > 0 && (!start_pos || !block_table)))
    return ENGRAM_E_NULL;
  const void* words[] = {token_map, positions, requests, start_pos, block_table, err_count};
  for (const void* p : words)
    if (!aligned(p, 4)) return ENGRAM_E_ALIGN;
  const void* longs[] = {multipliers, primes, offsets, input_ids, slots, history, hash_ids};
  for (const void* p : longs)
    if (!aligned(p, 8)) return ENGRAM_E_ALIGN;
  DeviceInfo di;
  if ((st = device_info(&di)) != ENGRAM_OK) return st;
  HashPagedArgs a;
  memset(&a, 0, sizeof(a));
  a.token_map = token_map;
  a.multipliers = multipliers;
  a.primes = primes;
  a.offsets = offsets;
  a.input_ids = input_ids;
  a.token_mask = token_mask;
  a.slots = slots;
  a.positions = positions;
  a.requests = requests;
  a.start_pos = start_pos;
  a.block_table = block_table;
  a.history = history;
  a.hash_ids = hash_ids;
  a.err_count = err_count;
  a.n_tokens = n_tokens;
  a.vocab = hl->vocab;
  a.n_blocks = pl->n_blocks;
  a.R = int(R);
  a.block_size = pl->block_size;
  a.max_blocks = pl->max_blocks;
  a.n_layers = hl->n_layers;
  a.max_ngram = hl->max_ngram;
  a.n_heads = hl->n_heads;
  a.pad_id = hl->pad_id;
  return launched(launch_hash_ids_paged(a, hip_stream(stream)));
}

engram_status engram_residual_norm(const engram_norm_layout* l, const void* x, const uint16_t* y, int64_t y_stride,
                                   const void* gate, int64_t gate_stride, const float* post_weight,
                                   const float* pre_weight, const uint8_t* token_mask, int64_t B, int64_t T,
                                   void* out, uint16_t* h, engram_stream_t stream) {
  engram_status st = engram_norm_layout_check(l);
  if (st != ENGRAM_OK) return st;
  if (B < 0 || T < 0 || (B != 0 && T > (int64_t(1) << 40) / B)) return ENGRAM_E_SHAPE;
  const int64_t M = B * T;
  if (M == 0) return ENGRAM_OK;
  if (M > 0x7FFFFFFF / l->hc) return ENGRAM_E_SHAPE;
  if (!x || (y != nullptr) != (out != nullptr) || (l->pre_norm != 0) != (h != nullptr)) return ENGRAM_E_NULL;
  if (y == nullptr && h == nullptr) return ENGRAM_E_NULL;  // nothing to compute
  if (y != nullptr && (l->gate != ENGRAM_GATE_NONE) != (gate != nullptr)) return ENGRAM_E_NULL;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(out, 16) || !aligned(h, 16) || !aligned(post_weight, 16) ||
      !aligned(pre_weight, 16) || !aligned(gate, l->gate == ENGRAM_GATE_FEATURE ? 16 : 4))
    return ENGRAM_E_ALIGN;
  const int64_t yrow = int64_t(l->y_streams) * l->dim;
  if (y != nullptr && (y_stride < yrow || y_stride % 8 != 0)) return ENGRAM_E_SHAPE;
  if (y != nullptr && l->gate == ENGRAM_GATE_FEATURE && (gate_stride < yrow || gate_stride % 8 != 0))
    return ENGRAM_E_SHAPE;
  DeviceInfo di;
  if ((st = device_info(&di)) != ENGRAM_OK) return st;
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x;
  a.y = y;
  a.gate = gate;
  a.post_weight = post_weight;
  a.pre_weight = pre_weight;
  a.token_mask = token_mask;
  a.out = out;
  a.h = h;
  a.M = M;
  a.y_stride = y_stride;
  a.gate_stride = gate_stride;
  a.hc = l->hc;
  a.dim = l->dim;
  a.y_streams = l->y_streams;
  a.gate_kind = y != nullptr ? l->gate : ENGRAM_GATE_NONE;
  a.post_norm = l->post_norm;
  a.fp32 = l->stream_format == ENGRAM_STREAM_FP32;
  a.alpha = l->alpha;
  a.beta = l->beta;
  a.post_eps = l->post_eps;
  a.pre_eps = l->pre_eps;
  return launched(launch_residual_norm(a, di.cus, hip_stream(stream)));
}

size_t engram_linear_workspace_bytes(const engram_linear_layout* l, int64_t M) {
  if (engram_linear_layout_check(l) != ENGRAM_OK || M <= 0 || M > 0x7FFFFFFF) return 0;
  DeviceInfo di;
  const int cus = device_info(&di) == ENGRAM_OK ? di.cus : 256;
  return size_t(linear_workspace_bytes(M, l->in_features, l->out_features, l->glu != 0, cus));
}

size_t engram_linear_workspace_bytes_up_to(const engram_linear_layout* l, int64_t M) {
  if (engram_linear_layout_check(l) != ENGRAM_OK || M <= 0 || M > 0x7FFFFFFF) return 0;
  DeviceInfo di;
  const int cus = device_info(&di) == ENGRAM_OK ? di.cus : 256;
  return size_t(linear_workspace_bytes_up_to(M, l->in_features, l->out_features, l->glu != 0, cus));
}

engram_status engram_linear(const engram_linear_layout* l, const uint16_t* x, int64_t x_stride, const uint16_t* w,
                            const float* bias, const void* residual, int64_t residual_stride, int64_t M, void* out,
                            int64_t out_stride, void* workspace, size_t workspace_bytes, engram_stream_t stream) {
  engram_status st = engram_linear_layout_check(l);
  if (st != ENGRAM_OK) return st;
  if (M < 0 || M > 0x7FFFFFFF) return ENGRAM_E_SHAPE;
  if (M == 0) return ENGRAM_OK;
  if (!x || !w || !out) return ENGRAM_E_NULL;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 16) || !aligned(residual, 16) || !aligned(out, 16))
    return ENGRAM_E_ALIGN;
  if (x_stride < l->in_features || x_stride % 8 != 0 || x_stride > (int64_t(1) << 28) || out_stride < l->out_features) return ENGRAM_E_SHAPE;
  if (residual != nullptr && residual_stride < l->out_features) return ENGRAM_E_SHAPE;
  // offsets into a tensor stay far from 64 bits
  const int64_t far = (int64_t(1) << 56) / M;
  if (out_stride > far || (residual != nullptr && residual_stride > far)) return ENGRAM_E_SHAPE;
  if (residual == out && residual_stride != out_stride) return ENGRAM_E_SHAPE;
  DeviceInfo di;
  if ((st = device_info(&di)) != ENGRAM_OK) return st;
  LinearArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.residual = residual;
  a.out = out;
  a.M = M;
  a.x_stride = x_stride;
  a.residual_stride = residual_stride;
  a.out_stride = out_stride;
  a.K = l->in_features;
  a.N = l->out_features;
  a.act = l->activation;
  a.glu = l->glu;
  a.fp32 = l->stream_format == ENGRAM_STREAM_FP32;
  const int64_t need = linear_workspace_bytes(M, a.K, a.N, a.glu != 0, di.cus);
  if (need > 0 && (workspace == nullptr || workspace_bytes < size_t(need) || !aligned(workspace, 16)))
    return ENGRAM_E_WORKSPACE;
  a.partials = static_cast<float*>(workspace);
  return launched(launch_linear(a, di.cus, hip_stream(stream)));
}

}  // extern "C"
