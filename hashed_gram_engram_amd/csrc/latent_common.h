// Device helpers shared by the latent cache's kernels.
#pragma once

#include "common.h"
#include "latent.h"

namespace engram {

// What a request does in a step: its new tokens and the positions that they see, [lo, hi).
struct Span {
  int first, tokens;  // flat tokens
  int pos;            // position of the first
  int lo, hi;
};
__device__ __forceinline__ Span span_of(const LatentRequests& q, int r) {
  const int cap = q.max_blocks * q.block_size;
  int a = q.token_start[r], b = q.token_start[r + 1];
  a = a < 0 ? 0 : (a > q.n_tokens ? q.n_tokens : a);
  b = b < a ? a : (b > q.n_tokens ? q.n_tokens : b);
  int p = q.start_pos[r];
  p = p < 0 ? 0 : (p > cap ? cap : p);
  Span s;
  s.first = a;
  s.tokens = b - a < cap - p ? b - a : cap - p;
  if (b - a < q.min_tokens || (q.max_tokens > 0 && b - a > q.max_tokens)) s.tokens = 0;
  s.pos = p;
  s.lo = q.window > 0 && p + 1 > q.window ? p + 1 - q.window : 0;
  s.hi = p + s.tokens;
  return s;
}

// The slot of a request's position; -1 where its page is outside the pool.
__device__ __forceinline__ int64_t slot_of(const LatentRequests& q, int r, int pos) {
  const int b = q.page_of(pos);
  const int page = q.block_table[int64_t(r) * q.max_blocks + b];
  return page >= 0 && page < q.n_blocks ? int64_t(page) * q.block_size + (pos - b * q.block_size) : -1;
}

// Sixteen e4m3 codes times 2^(scale - 127) -> sixteen bf16, exact wherever bf16 holds the product.  The
// conversion takes the scale's exponent field, so 2^-127 (a subnormal) and NaN take the multiplication.
__device__ __forceinline__ uint32_t scaled_pair(uint32_t c, float s, bool high) {
  return high ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, s, false));
}
__device__ __forceinline__ void latent16(u32x4 c, uint32_t scale, u32x4& o0, u32x4& o1) {
  const float s = __uint_as_float(scale << 23);
  o0 = u32x4{scaled_pair(c.x, s, false), scaled_pair(c.x, s, true), scaled_pair(c.y, s, false), scaled_pair(c.y, s, true)};
  o1 = u32x4{scaled_pair(c.z, s, false), scaled_pair(c.z, s, true), scaled_pair(c.w, s, false), scaled_pair(c.w, s, true)};
  if (__builtin_expect(scale == 0u || scale == 255u, 0)) dequant16(c, e8m0_to_f32(scale), o0, o1);
}

// Eight codes, of a scale that engram_latent_write makes (1 .. 247).
__device__ __forceinline__ u32x4 latent8(u32x2 c, uint32_t scale) {
  const float s = __uint_as_float(scale << 23);
  return u32x4{scaled_pair(c.x, s, false), scaled_pair(c.x, s, true), scaled_pair(c.y, s, false), scaled_pair(c.y, s, true)};
}

// Running sums over the lanes of a wave, and over the threads of a workgroup of THREADS (tmp: one word per
// wave; free again behind the caller's next barrier).
__device__ __forceinline__ int64_t wave_scan64(int64_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int64_t u = __shfl_up(v, o, kWave);
    if (lane >= o) v += u;
  }
  return v;
}
template <int THREADS>
__device__ __forceinline__ int64_t block_scan64(int64_t v, int64_t* tmp, int64_t* total) {
  const int wv = threadIdx.x >> 6;
  const int64_t in = wave_scan64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) tmp[wv] = in;
  __syncthreads();
  int64_t before = in - v, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / kWave; ++w) {
    if (w < wv) before += tmp[w];
    all += tmp[w];
  }
  *total = all;
  return before;  // of the threads before this one
}

}  // namespace engram
