// The latent cache: a step's rows into the pages, and a step's requests' rows back.
//
// Write.  A lane takes 8 features (16 bytes).  MXFP8: the 4 lanes of a block of 32 features share its largest
// magnitude; the scale's byte follows from that value's exponent field E and significand: 448 = 1.75 2^8, so
// 2^(E - 127 - 8) suffices up to a significand of 1.75 and its double beyond.  The scaling is exact (a power of
// two), so each code is rounded once.
//
// Read.  Rows lie one request after the other; every workgroup sums the requests' lengths in LDS for itself
// (at most 4096 of them), finds its rows' requests by bisection and copies 16 bytes of a cache row a lane.
//
// What bounds them: memory (24 requests of up to 8192 positions, MXFP8 rows of 512 + 64: written in 9 us and read in 59,
// 258 MB together, 3.8 TB/s where a copy of 2 GiB reaches 4.9); small calls, the launch and (read) a chain of
// dependent loads: lengths, table, row (six requests of up to 700 positions: 4 and 8 us).
#include "latent_common.h"
#include "serving.h"

namespace engram {

namespace {

constexpr int kThreads = 256;
constexpr int kWriteTokens = 4;  // per workgroup and turn
// A launch of 2^32 threads and more loses some without an error: from 2^24 tokens on workgroups take several turns.
constexpr int kWriteGroups = 1 << 22;

__device__ __forceinline__ uint32_t abs_bits_finite(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
  return b < 0x7F800000u ? b : 0u;
}

__global__ __launch_bounds__(kThreads) void k_latent_write(LatentWriteArgs a) {
  const int lat = a.latent_dim / 8, chunks = lat + a.rope_dim / 8;  // multiples of 4: a block of 32 stays in 4 lanes
  const int row = latent_row_bytes(a.latent_dim, a.rope_dim, a.fp8 != 0);
  for (int t0 = blockIdx.x * kWriteTokens; t0 < a.n_tokens; t0 += gridDim.x * kWriteTokens) {
    for (int i = threadIdx.x; i < kWriteTokens * chunks; i += kThreads) {
      const int t = t0 + i / chunks, c = i % chunks;
      const bool on = t < a.n_tokens;
      int64_t slot = on ? a.slots[t] : -1;
      if (slot >= a.n_slots) {
        if (c == 0 && a.err_count != nullptr) atomicAdd(a.err_count, 1);
        slot = -1;
      }
      u32x4 v = {0u, 0u, 0u, 0u};
      if (slot >= 0)
        v = *reinterpret_cast<const u32x4*>(c < lat ? a.latent + t * a.latent_stride + c * 8 : a.rope + t * a.rope_stride + (c - lat) * 8);
      uint8_t* to = a.cache + (slot < 0 ? 0 : slot) * row;
      if (!a.fp8 || c >= lat) {
        if (slot >= 0) *reinterpret_cast<u32x4*>(to + (a.fp8 ? a.latent_dim + 16 + (c - lat) * 16 : c * 16)) = v;
        continue;  // (whole groups of 4 lanes)
      }
      float x[8];
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = bf16_lo(v[e]);
        x[2 * e + 1] = bf16_hi(v[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = abs_bits_finite(x[e]);
        top = b > top ? b : top;
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        const uint32_t b = uint32_t(__shfl_xor(int(top), o, kWave));
        top = b > top ? b : top;
      }
      int scale = int(top >> 23) - 8 + ((top & 0x007FFFFFu) > 0x00600000u ? 1 : 0);
      scale = scale < 1 ? 1 : scale;  // (what 2^-126 leaves of smaller values is still exact: bf16 has none below 2^-133)
      const float up = __uint_as_float(uint32_t(254 - scale) << 23);  // 2^(127 - scale)
      // 248 and more would become 256, which the largest scale takes past bf16: 240 there
      const float most = scale == 247 ? 240.0f : 448.0f;
      u32x2 code;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __builtin_amdgcn_fmed3f(x[4 * h + e] * up, -most, most);
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!(__builtin_fabsf(x[4 * h + e]) <= kFltMax)) w |= 0x7F << (8 * e);  // (not finite)
        code[h] = uint32_t(w);
      }
      if (slot >= 0) {
        *reinterpret_cast<u32x2*>(to + c * 8) = code;
        if ((c & 3) == 0) to[a.latent_dim + (c >> 2)] = uint8_t(scale);
      }
    }
  }
}

constexpr int kReadRows = 32;  // per workgroup and turn

// First r with end[r] > i.
__device__ __forceinline__ int first_above(const int32_t* end, int n, int i) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > i) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

template <bool FP8>
__global__ __launch_bounds__(kThreads) void k_latent_read(LatentReadArgs a) {
  __shared__ int32_t end[kMaxRequests];  // rows up to and with each request
  __shared__ int64_t tmp[kThreads / kWave];
  __shared__ int64_t from[kReadRows];    // slot of each row of the turn
  const int tid = threadIdx.x;
  const bool lead = blockIdx.x == 0;
  const int items = (a.rq.R + kThreads - 1) / kThreads, r0 = tid * items;
  int64_t mine = 0, total;
  for (int r = r0; r < r0 + items && r < a.rq.R; ++r) {
    const Span s = span_of(a.rq, r);
    mine += s.tokens > 0 ? s.hi - s.lo : 0;
  }
  int64_t at = block_scan64<kThreads>(mine, tmp, &total);
  // (the sums only grow, so that the first request past max_rows cuts off every later one)
  int64_t kept = 0;
  for (int r = r0; r < r0 + items && r < a.rq.R; ++r) {
    const Span s = span_of(a.rq, r);
    const int64_t n = s.tokens > 0 ? s.hi - s.lo : 0;
    if (at + n <= a.max_rows) {
      at += n;
      kept = at;
      end[r] = int32_t(at);
    } else {
      at = int64_t(1) << 62;
      end[r] = -1;
      if (lead && n > 0 && a.err_count != nullptr) atomicAdd(a.err_count, 1);
    }
  }
  // the rows that are left: the largest sum that fits
  __syncthreads();
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const int64_t u = __shfl_xor(kept, o, kWave);
    kept = u > kept ? u : kept;
  }
  if ((tid & 63) == 0) tmp[tid >> 6] = kept;
  __syncthreads();
  int64_t left = 0;
#pragma unroll
  for (int w = 0; w < kThreads / kWave; ++w) left = tmp[w] > left ? tmp[w] : left;
  const int rows = int(left);
  for (int r = tid; r < a.rq.R; r += kThreads)
    if (end[r] < 0) end[r] = rows;
  __syncthreads();
  if (lead) {
    for (int r = tid; r < a.rq.R; r += kThreads) a.row_start[r + 1] = end[r];
    if (tid == 0) a.row_start[0] = 0;
  }

  const int row = latent_row_bytes(a.latent_dim, a.rope_dim, FP8);
  const int lat = FP8 ? a.latent_dim / 16 : a.latent_dim / 8, pieces = lat + a.rope_dim / 8;  // of 16 bytes
  for (int i0 = blockIdx.x * kReadRows; i0 < rows; i0 += gridDim.x * kReadRows) {
    if (tid < kReadRows && i0 + tid < rows) {
      const int r = first_above(end, a.rq.R, i0 + tid);
      const Span s = span_of(a.rq, r);
      const int64_t slot = slot_of(a.rq, r, s.lo + i0 + tid - (r > 0 ? end[r - 1] : 0));
      from[tid] = slot;
      if (slot < 0 && a.err_count != nullptr) atomicAdd(a.err_count, 1);
    }
    __syncthreads();
    const int n = (rows - i0 < kReadRows ? rows - i0 : kReadRows) * pieces;
#pragma unroll 4
    for (int k = tid; k < n; k += kThreads) {
      const int t = k / pieces, c = k - t * pieces;
      const int64_t slot = from[t], to = i0 + t;
      const uint8_t* src = a.cache + (slot < 0 ? 0 : slot) * row;
      const bool is_rope = c >= lat;
      u32x4 v = *reinterpret_cast<const u32x4*>(src + (is_rope && FP8 ? a.latent_dim + 16 + (c - lat) * 16 : c * 16));
      if (slot < 0) v = u32x4{0u, 0u, 0u, 0u};
      if (is_rope) {
        *reinterpret_cast<u32x4*>(a.rope + to * a.rope_dim + (c - lat) * 8) = v;
      } else if constexpr (FP8) {
        u32x4 o0, o1;
        latent16(v, slot < 0 ? 1u : src[a.latent_dim + (c >> 1)], o0, o1);
        u32x4* out = reinterpret_cast<u32x4*>(a.latent + to * a.latent_dim + c * 16);
        out[0] = o0;
        out[1] = o1;
      } else {
        *reinterpret_cast<u32x4*>(a.latent + to * a.latent_dim + c * 8) = v;
      }
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_latent_write(const LatentWriteArgs& a, hipStream_t stream) {
  const int turns = (a.n_tokens + kWriteTokens - 1) / kWriteTokens, grid = turns < kWriteGroups ? turns : kWriteGroups;
  k_latent_write<<<dim3(grid), dim3(kThreads), 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_latent_read(const LatentReadArgs& a, int cus, hipStream_t stream) {
  const int64_t turns = (a.max_rows + kReadRows - 1) / kReadRows;
  const int grid = int(turns < 1 ? 1 : (turns < 8 * cus ? turns : 8 * cus));
  if (a.fp8) k_latent_read<true><<<dim3(grid), dim3(kThreads), 0, stream>>>(a);
  else k_latent_read<false><<<dim3(grid), dim3(kThreads), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace engram
