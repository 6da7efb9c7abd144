// Kernel argument blocks and launchers of the serving operators (host side).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace engram {

constexpr int kMaxRequests = 4096;  // requests of one plan: their sums live in a workgroup's LDS

struct PlanArgs {
  const int32_t* new_lens;
  const int32_t* cached_lens;
  int32_t* block_table;  // [R, max_blocks]
  int32_t* free_list;    // [n_blocks]
  const int32_t* free_count;
  int R, block_size, max_blocks, n_blocks;
  int max_tokens;
  int32_t* token_start;
  int32_t* start_pos;
  int32_t* seq_lens;
  int32_t* status;
  int32_t* free_left;
  int64_t* slots;
  int32_t* positions;
  int32_t* requests;
  uint8_t* live;
  int32_t* err_count;
};
hipError_t launch_batch_plan(const PlanArgs& a, hipStream_t stream);

struct HashPagedArgs {
  const uint32_t* token_map;
  const int64_t* multipliers;
  const int64_t* primes;
  const int64_t* offsets;
  const int64_t* input_ids;
  const uint8_t* token_mask;
  const int64_t* slots;
  const int32_t* positions;
  const int32_t* requests;
  const int32_t* start_pos;
  const int32_t* block_table;
  int64_t* history;
  int64_t* hash_ids;
  int32_t* err_count;
  int64_t n_tokens, vocab, n_blocks;
  int R, block_size, max_blocks;
  int n_layers, max_ngram, n_heads, pad_id;
};
hipError_t launch_hash_ids_paged(const HashPagedArgs& a, hipStream_t stream);

struct NormArgs {
  const void* x;
  const uint16_t* y;  // null: no block before
  const void* gate;
  const float* post_weight;  // null: ones
  const float* pre_weight;
  const uint8_t* token_mask;
  void* out;    // null without y
  uint16_t* h;  // null without pre_norm
  int64_t M, y_stride, gate_stride;
  int hc, dim, y_streams, gate_kind, post_norm, fp32;
  float alpha, beta, post_eps, pre_eps;
};
hipError_t launch_residual_norm(const NormArgs& a, int cus, hipStream_t stream);

struct LinearArgs {
  const uint16_t* x;
  const uint16_t* w;
  const float* bias;
  const void* residual;
  void* out;
  int64_t M, x_stride, residual_stride, out_stride;
  int K, N;  // N: output features (the weight has 2 N rows with glu)
  int act, glu, fp32;
  // split over K: parts > 1 leave their fp32 blocks in `partials`, a second kernel joins them
  int parts;
  float* partials;
};
// Bytes of `partials` (16-byte aligned) that launch_linear needs on a device of `cus` compute units; 0
// where it does not split K.
int64_t linear_workspace_bytes(int64_t M, int K, int N, bool glu, int cus);
int64_t linear_workspace_bytes_up_to(int64_t M, int K, int N, bool glu, int cus);  // the most for 1 .. M rows
hipError_t launch_linear(const LinearArgs& a, int cus, hipStream_t stream);  // (sets a.parts itself)

}  // namespace engram
