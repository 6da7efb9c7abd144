// The hash step for the ragged tokens of a plan: engram_hash_ids' rule, with the look-back history
// in pages.
//
// A workgroup takes up to 32 consecutive tokens.  First one thread per (token, look-back) fetches
// the compressed id (all of them at once: each is a chain of up to four dependent reads) into LDS;
// then a thread per token applies the blocking rule; then each thread takes one column (layer,
// n-gram, head) and some of the tokens, so that a wave's stores of a token are contiguous.
//
// The remainder by the column's prime p: with v = floor((2^64 - 1) / p), computed once per thread,
// q = mulhi(h, v) is at most 1 below floor(h / p) for any h < 2^64 (v >= (2^64 - p) / p, so h v / 2^64
// >= h / p - h / 2^64 > h / p - 1), so one conditional subtraction gives h mod p.  A negative h (the hash is a signed 64-bit value, the
// remainder a floor modulo) uses h mod p = p - 1 - (-h - 1) mod p, where -h - 1 = ~h >= 0.
//
// What bounds it: latency for a decode step; at 8192 tokens the 3.1 MB of row ids and about 280
// cycles of 64-bit multiplies per wave and id.
#include "common.h"
#include "launch.h"
#include "serving.h"

namespace engram {

namespace {

constexpr int kHashThreads = 256;
constexpr int kHashTokens = 32;  // most tokens of a workgroup
constexpr int kMaxLookBack = 8;

__device__ __forceinline__ uint64_t mod_by(uint64_t h, uint64_t p, uint64_t v) {
  const uint64_t r = h - __umul64hi(h, v) * p;
  return r >= p ? r - p : r;
}

__global__ __launch_bounds__(kHashThreads) void k_hash_ids_paged(HashPagedArgs a, int per_group) {
  __shared__ int64_t src[kHashTokens][kMaxLookBack];
  const int tid = threadIdx.x;
  const int64_t i0 = int64_t(blockIdx.x) * per_group;
  const int n = int(a.n_tokens - i0 < per_group ? a.n_tokens - i0 : per_group);
  auto compressed = [&](int64_t i, bool count) -> int64_t {
    const int64_t id = a.input_ids[i];
    if (id < 0 || id >= a.vocab) {
      if (count && a.err_count != nullptr) atomicAdd(a.err_count, 1);
      return kDead;
    }
    if (a.token_mask != nullptr && a.token_mask[i] == 0) return kDead;
    return int64_t(a.token_map[id]);
  };
  const int ng = a.max_ngram;
  for (int w = tid; w < n * ng; w += kHashThreads) {
    const int t = w / ng, sh = w - t * ng;
    const int64_t i = i0 + t;
    const int r = a.requests[i];
    int64_t c = kDead;
    if (r >= 0 && r < a.R) {
      const int pos = a.positions[i], q = pos - sh;
      if (q < 0) {
      } else if (q >= a.start_pos[r]) {
        if (i >= sh) c = compressed(i - sh, sh == 0);
      } else {
        const int b = q / a.block_size;
        const int64_t page = b < a.max_blocks ? a.block_table[int64_t(r) * a.max_blocks + b] : -1;
        if (page >= 0 && page < a.n_blocks) c = a.history[page * a.block_size + (q - b * a.block_size)];
        else if (a.err_count != nullptr) atomicAdd(a.err_count, 1);
      }
      // positions of this call only: no look-back of this call reads them
      if (sh == 0) {
        const int64_t slot = a.slots[i];
        if (slot >= 0 && slot < a.n_blocks * a.block_size) a.history[slot] = c;
      }
    }
    src[t][sh] = c;
  }
  __syncthreads();
  if (tid < n) {
    // the first dead look-back, or the one before the sequence start, hides every longer one
    bool blocked = false;
    for (int sh = 0; sh < ng; ++sh) {
      blocked = blocked || src[tid][sh] == kDead;
      if (blocked) src[tid][sh] = int64_t(a.pad_id);
    }
  }
  __syncthreads();
  const int cols = (ng - 1) * a.n_heads, all = a.n_layers * cols;
  const int width = all < kHashThreads ? all : kHashThreads;
  const int lanes = kHashThreads / width, mine = tid / width;
  if (mine >= lanes) return;
  for (int c = tid - mine * width; c < all; c += width) {
    const int layer = c / cols, col = c - layer * cols, order = col / a.n_heads + 1;
    const int64_t p = a.primes[c], off = a.offsets[c];
    uint64_t m[kMaxLookBack];
#pragma unroll
    for (int s = 0; s < kMaxLookBack; ++s)  // look-backs past the column's order add nothing
      m[s] = s <= order ? uint64_t(a.multipliers[int64_t(layer) * ng + s]) : 0u;
    const uint64_t v = p > 0 ? ~uint64_t(0) / uint64_t(p) : 0;
    int64_t* out = a.hash_ids + (int64_t(layer) * a.n_tokens + i0) * cols + col;
    for (int t = mine; t < n; t += lanes) {
      uint64_t h = 0;
#pragma unroll
      for (int s = 0; s < kMaxLookBack; ++s)
        if (s < ng) h ^= uint64_t(src[t][s]) * m[s];
      int64_t row = -1;
      if (p > 0) {
        const bool neg = int64_t(h) < 0;
        const int64_t r = int64_t(mod_by(neg ? ~h : h, uint64_t(p), v));
        row = (neg ? p - 1 - r : r) + off;
      } else if (a.err_count != nullptr) {
        atomicAdd(a.err_count, 1);
      }
      out[int64_t(t) * cols] = row;
    }
  }
}

}  // namespace

hipError_t launch_hash_ids_paged(const HashPagedArgs& a, hipStream_t stream) {
  if (a.n_tokens <= 0) return hipSuccess;
  if (a.max_ngram < 2 || a.max_ngram > kMaxLookBack) return hipErrorInvalidValue;
  int per_group = a.n_tokens >= 2048 ? kHashTokens : 8;
  const int64_t grid = (a.n_tokens + per_group - 1) / per_group;
  if (!launch_fits(grid, kHashThreads)) return hipErrorInvalidValue;
  HashPagedArgs args = a;
  void* params[] = {&args, &per_group};
  return hipLaunchKernel(reinterpret_cast<const void*>(&k_hash_ids_paged), dim3(unsigned(grid)), dim3(kHashThreads),
                         params, 0, stream);
}

}  // namespace engram
