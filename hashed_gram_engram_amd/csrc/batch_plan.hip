// Block tables and slot maps of a ragged step, from its requests' lengths.
//
// Everything a token needs follows from four running sums over the requests: pages given back,
// tokens asked for, pages needed, and (of the admitted requests) tokens and pages.  The inputs are
// not changed by the call (the new lengths and count go out to other arrays, released pages go
// above the stack's top, new table entries past the held ones), so every workgroup computes the
// sums for itself and then writes its own share of tokens and table entries: one launch, no wait
// between workgroups.
//
// What bounds it: latency.  A step of 16,384 tokens writes 0.3 MB; the time is the launch and a
// chain of dependent reads (lengths, sums, a search in LDS, a table entry, the write).
#include "common.h"
#include "serving.h"

namespace engram {

namespace {

constexpr int kPlanThreads = 256;

// Sums saturate at 2^31 - 1 (lengths near 2^30 times 4096 requests pass 32 bits): sums of non-negative
// values capped like this do not depend on their order, and nothing that fits (tokens, pages) reaches the cap.
constexpr uint32_t kCapped = 0x7FFFFFFF;
__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) {
  const uint32_t s = a + b;
  return s < kCapped ? s : kCapped;
}

// Inclusive sum over the wave's lanes: within rows of 16 lanes, then row 0 into 1 and 2 into 3, then
// lane 31 into the upper half.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v = add(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x111, 0xF, 0xF, false)));  // row_shr 1
  v = add(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x112, 0xF, 0xF, false)));
  v = add(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x114, 0xF, 0xF, false)));
  v = add(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x118, 0xF, 0xF, false)));
  v = add(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x142, 0xA, 0xF, false)));  // row_bcast 15
  v = add(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x143, 0xC, 0xF, false)));  // row_bcast 31
  return v;
}

// Sums of a and b over the threads before this one, and over all threads (total).  tmp: free again after
// the call's last barrier.
struct Sums {
  uint32_t a, b, all_a, all_b;
};
__device__ __forceinline__ Sums scan2(uint32_t a, uint32_t b, uint32_t (*tmp)[2]) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const uint32_t ia = wave_scan(a), ib = wave_scan(b);
  __syncthreads();
  if (lane == 63) {
    tmp[wv][0] = ia;
    tmp[wv][1] = ib;
  }
  __syncthreads();
  // the sums before this lane: shifted by one, not subtracted (a capped sum has no difference)
  const uint32_t ua = uint32_t(__shfl_up(int(ia), 1, kWave)), ub = uint32_t(__shfl_up(int(ib), 1, kWave));
  Sums s;
  s.a = lane > 0 ? ua : 0u;  // (every lane takes part in the shuffle)
  s.b = lane > 0 ? ub : 0u;
  s.all_a = s.all_b = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / kWave; ++w) {
    if (w < wv) {
      s.a = add(s.a, tmp[w][0]);
      s.b = add(s.b, tmp[w][1]);
    }
    s.all_a = add(s.all_a, tmp[w][0]);
    s.all_b = add(s.all_b, tmp[w][1]);
  }
  return s;
}

// First r with end[r] > i (end ascending, n entries; n if none).
__device__ __forceinline__ int first_above(const int32_t* end, int n, int i) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > i) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// ITEMS consecutive requests per thread.
template <int ITEMS>
__global__ __launch_bounds__(kPlanThreads) void k_batch_plan(PlanArgs a) {
  constexpr int kCap = kPlanThreads * ITEMS;
  // the held lengths are looked up again below; for the most requests they no longer fit 64 KB of LDS
  constexpr bool kKeep = ITEMS < 16;
  __shared__ int32_t back_end[kCap], tok_end[kCap], blk_end[kCap];  // inclusive sums
  __shared__ int32_t length[kKeep ? kCap : 1];
  __shared__ uint32_t tmp[kPlanThreads / kWave][2];
  const int tid = threadIdx.x;
  const int bs = a.block_size, cap = a.max_blocks * bs;
  const int r0 = tid * ITEMS;
  const bool lead = blockIdx.x == 0;
  int free0 = a.free_count[0];
  free0 = free0 < 0 ? 0 : (free0 > a.n_blocks ? a.n_blocks : free0);

  int held[ITEMS], have[ITEMS], want[ITEMS], stat[ITEMS];
  uint32_t back[ITEMS], tok[ITEMS];  // this thread's sums up to each request
  bool gone[ITEMS];
  uint32_t sb = 0, st = 0;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int r = r0 + k;
    const int n = r < a.R ? a.new_lens[r] : 0;
    held[k] = r < a.R ? a.cached_lens[r] : 0;
    const bool bad = held[k] < 0 || held[k] > cap || (n > 0 && n > cap - held[k]);
    have[k] = bad ? 0 : (held[k] + bs - 1) / bs;
    gone[k] = n < 0 && !bad;
    want[k] = bad || n < 0 ? 0 : n;
    stat[k] = bad ? 3 : 0;
    sb = add(sb, gone[k] ? have[k] : 0);
    back[k] = sb;
    st = add(st, want[k]);
    tok[k] = st;
    if constexpr (kKeep) length[r] = held[k];
  }
  const Sums first = scan2(sb, st, tmp);
  const uint32_t all_back = first.all_a, room = uint32_t(a.n_blocks - free0);
  const int avail = free0 + int(all_back < room ? all_back : room);

  // by tokens, then by pages
  int need[ITEMS];
  uint32_t blk[ITEMS], sn = 0;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    back_end[r0 + k] = int32_t(add(first.a, back[k]));
    if (want[k] > 0 && add(first.b, tok[k]) > uint32_t(a.max_tokens)) {
      stat[k] = 1;
      want[k] = 0;
    }
    need[k] = want[k] > 0 ? (held[k] + want[k] + bs - 1) / bs - have[k] : 0;
    sn = add(sn, need[k]);
    blk[k] = sn;
  }
  const Sums asked = scan2(sn, 0u, tmp);
  st = sn = 0;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    if (need[k] > 0 && add(asked.a, blk[k]) > uint32_t(avail)) {
      stat[k] = 2;
      want[k] = 0;
      need[k] = 0;
    }
    st += want[k];
    tok[k] = st;
    sn += need[k];
    blk[k] = sn;
  }
  const Sums given = scan2(st, sn, tmp);
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int r = r0 + k;
    tok_end[r] = int32_t(given.a + tok[k]);
    blk_end[r] = int32_t(given.b + blk[k]);
    if (lead && r < a.R) {
      a.token_start[r + 1] = int32_t(given.a + tok[k]);
      a.start_pos[r] = held[k];
      a.seq_lens[r] = gone[k] ? 0 : held[k] + want[k];
      a.status[r] = stat[k];
      if (stat[k] != 0 && a.err_count != nullptr) atomicAdd(a.err_count, 1);
    }
  }
  __syncthreads();
  const int n_tok = int(given.all_a), n_new = int(given.all_b);
  if (lead && tid == 0) {
    a.token_start[0] = 0;
    a.free_left[0] = avail - n_new;
    if (a.err_count != nullptr && all_back > room) atomicAdd(a.err_count, int(all_back - room));
  }

  // entry j of the stack after the released pages came back: below free0 the caller's list, above
  // it the released requests' entries
  auto released = [&](int j) {
    const int r = first_above(back_end, a.R, j);
    const int before = r > 0 ? back_end[r - 1] : 0;
    return a.block_table[int64_t(r) * a.max_blocks + (j - before)];
  };
  auto stack = [&](int idx) { return idx < free0 ? a.free_list[idx] : released(idx - free0); };
  auto length_of = [&](int r) { return kKeep ? length[kKeep ? r : 0] : a.cached_lens[r]; };
  auto pages_of = [&](int r) {  // pages the request holds already
    return (length_of(r) + bs - 1) / bs;
  };

  const int step = int(gridDim.x) * kPlanThreads;
  const int g = int(blockIdx.x) * kPlanThreads + tid;
  for (int64_t j = g; j < avail - free0; j += step) a.free_list[free0 + j] = released(int(j));
  for (int64_t e = g; e < n_new; e += step) {
    const int r = first_above(blk_end, a.R, int(e));
    const int before = r > 0 ? blk_end[r - 1] : 0;
    a.block_table[int64_t(r) * a.max_blocks + pages_of(r) + (e - before)] = stack(avail - 1 - int(e));
  }
  for (int64_t i = g; i < a.max_tokens; i += step) {
    int64_t slot = -1;
    int pos = -1, req = -1;
    if (i < n_tok) {
      req = first_above(tok_end, a.R, int(i));
      pos = length_of(req) + int(i) - (req > 0 ? tok_end[req - 1] : 0);
      const int b = pos / bs, old = pages_of(req);
      const int page = b < old ? a.block_table[int64_t(req) * a.max_blocks + b]
                               : stack(avail - 1 - ((req > 0 ? blk_end[req - 1] : 0) + b - old));
      if (page >= 0 && page < a.n_blocks) slot = int64_t(page) * bs + (pos - b * bs);
      else if (a.err_count != nullptr) atomicAdd(a.err_count, 1);
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
    a.requests[i] = req;
    a.live[i] = i < n_tok ? 1 : 0;
  }
}

}  // namespace

hipError_t launch_batch_plan(const PlanArgs& a, hipStream_t stream) {
  if (a.R < 0 || a.R > kMaxRequests || a.max_tokens < 0) return hipErrorInvalidValue;
  // one token per thread: a token is a chain of reads (16,384 tokens of 512 requests: 14.6 us with four
  // tokens per thread, 9.3 us with one; every workgroup's own sums cost less than the wait)
  int64_t grid = (int64_t(a.max_tokens) + kPlanThreads - 1) / kPlanThreads;
  grid = grid < 1 ? 1 : (grid > 4096 ? 4096 : grid);
  PlanArgs args = a;
  void* params[] = {&args};
  const void* fn = a.R <= kPlanThreads       ? reinterpret_cast<const void*>(&k_batch_plan<1>)
                   : a.R <= 4 * kPlanThreads ? reinterpret_cast<const void*>(&k_batch_plan<4>)
                                             : reinterpret_cast<const void*>(&k_batch_plan<16>);
  return hipLaunchKernel(fn, dim3(unsigned(grid)), dim3(kPlanThreads), params, 0, stream);
}

}  // namespace engram
