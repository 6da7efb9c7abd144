// Kernel argument blocks and launchers of the latent cache and its attention (host side).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace engram {

// A step's requests in a plan's pages.
struct LatentRequests {
  const int32_t* token_start;  // [R + 1]
  const int32_t* start_pos;    // [R]
  const int32_t* block_table;  // [R, max_blocks]
  int R, n_tokens;
  int block_size, max_blocks, n_blocks;
  int min_tokens, max_tokens;  // requests with so many new tokens take part
  int window;                  // 0: none
  uint32_t page_mul, page_shift;  // of page_of
  int stage_pages, stage_rest;    // 32 positions: whole pages, and positions more
  // pos / block_size of a position below 2^30: page_mul = ceil(2^(30 + s) / block_size) with s the bits of block_size - 1, so
  // that page_mul block_size - 2^(30 + s) < 2^s and the quotient is off by less than 1 / block_size
  __host__ __device__ int page_of(int pos) const { return int((uint64_t(uint32_t(pos)) * page_mul) >> page_shift); }
  void set_pages(int block, int blocks, int64_t pool) {
    block_size = block;
    max_blocks = blocks;
    n_blocks = int(pool);
    int s = 0;
    while ((int64_t(1) << s) < block) ++s;
    page_mul = uint32_t(((uint64_t(1) << (30 + s)) + block - 1) / block);
    page_shift = 30 + s;
    stage_pages = 32 / block;
    stage_rest = 32 % block;
  }
};

// Bytes of a cache row.
constexpr int latent_row_bytes(int latent_dim, int rope_dim, bool fp8) {
  return fp8 ? latent_dim + 16 + 2 * rope_dim : 2 * (latent_dim + rope_dim);
}

struct LatentWriteArgs {
  const uint16_t* latent;
  const uint16_t* rope;
  const int64_t* slots;
  uint8_t* cache;
  int32_t* err_count;
  int64_t latent_stride, rope_stride, n_slots;
  int n_tokens, latent_dim, rope_dim, fp8;
};
hipError_t launch_latent_write(const LatentWriteArgs& a, hipStream_t stream);

struct LatentReadArgs {
  LatentRequests rq;
  const uint8_t* cache;
  int32_t* row_start;
  uint16_t* latent;
  uint16_t* rope;
  int32_t* err_count;
  int64_t max_rows;
  int latent_dim, rope_dim, fp8;
};
hipError_t launch_latent_read(const LatentReadArgs& a, int cus, hipStream_t stream);

struct AbsorbedArgs {
  LatentRequests rq;
  const uint16_t* q;
  const uint8_t* cache;
  uint16_t* out;
  float* lse;
  int32_t* err_count;
  int64_t q_stride, out_stride;
  float scale_log2;  // magnitude of the scores' scale, times log2 e, above zero (a masked score is -infinity times it)
  uint32_t q_sign;   // 0x80008000: queries are negated (a negative scale)
  int heads, latent_dim, rope_dim, fp8;
  char* workspace;
};
int64_t absorbed_workspace_bytes(int latent_dim, int cus);
hipError_t launch_absorbed_rows(const AbsorbedArgs& a, int G, bool wide, hipStream_t stream);  // 33 rows and more a request
hipError_t launch_latent_absorbed(const AbsorbedArgs& a, int cus, hipStream_t stream);

struct ExpandedArgs {
  LatentRequests rq;  // (no pages)
  const uint16_t* q;
  const uint16_t* kv;
  const uint16_t* rope;
  const int32_t* row_start;  // [R + 1]
  uint16_t* out;
  float* lse;
  int64_t q_stride, kv_stride, rope_stride, out_stride;
  int n_rows;
  float scale_log2;
  uint32_t q_sign;
  int heads, head_dim, rope_dim;
  float* workspace;
  // set by the launcher: tiles of the grid, and the parts that a tile's keys are shared out in
  int tiles, parts;
};
int64_t expanded_workspace_bytes(int64_t R, int64_t n_tokens, int64_t n_rows, int heads, int head_dim, int cus);
int64_t expanded_workspace_bytes_up_to(int64_t n_tokens, int64_t n_rows, int heads, int head_dim, int cus);  // for fewer, too
hipError_t launch_latent_expanded(ExpandedArgs a, int cus, hipStream_t stream);

}  // namespace engram
