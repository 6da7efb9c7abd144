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
constexpr int kTokensPerGroup = 1024;  // tokens of one workgroup: 4 per thread, coalesced

// Inclusive sums of a and b over the workgroup's threads (64 bits: lengths near 2^30 times 4096
// requests pass 32).  tmp: 2 x (kPlanThreads / 64) words, free again after the call.
__device__ __forceinline__ void scan2(int64_t& a, int64_t& b, int64_t (*tmp)[kPlanThreads / kWave]) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int64_t pa = __shfl_up(a, o, kWave), pb = __shfl_up(b, o, kWave);
    if (lane >= o) {
      a += pa;
      b += pb;
    }
  }
  __syncthreads();
  if (lane == 63) {
    tmp[0][wv] = a;
    tmp[1][wv] = b;
  }
  __syncthreads();
  for (int w = 0; w < wv; ++w) {
    a += tmp[0][w];
    b += tmp[1][w];
  }
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
  __shared__ int32_t back_end[kCap], tok_end[kCap], blk_end[kCap];  // inclusive sums
  __shared__ int64_t tmp[2][kPlanThreads / kWave];
  __shared__ int64_t total[2];
  const int tid = threadIdx.x;
  const int bs = a.block_size, cap = a.max_blocks * bs;
  const int r0 = tid * ITEMS;
  const bool lead = blockIdx.x == 0;

  int held[ITEMS], have[ITEMS], want[ITEMS], stat[ITEMS];
  int64_t back[ITEMS], tok[ITEMS];
  bool gone[ITEMS];
  int64_t sb = 0, st = 0;
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
    sb += gone[k] ? have[k] : 0;
    back[k] = sb;
    st += want[k];
    tok[k] = st;
  }
  {
    int64_t eb = sb, et = st;
    scan2(eb, et, tmp);
    if (tid == kPlanThreads - 1) total[0] = eb;
    eb -= sb;
    et -= st;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      back[k] += eb;
      tok[k] += et;
      // past 2^31 nothing is looked up: a stack has fewer entries
      back_end[r0 + k] = int32_t(back[k] < 0x7FFFFFFF ? back[k] : 0x7FFFFFFF);
    }
  }
  __syncthreads();
  int free0 = a.free_count[0];
  free0 = free0 < 0 ? 0 : (free0 > a.n_blocks ? a.n_blocks : free0);
  const int64_t all_back = total[0];
  const int avail = int(all_back < a.n_blocks - free0 ? all_back + free0 : a.n_blocks);

  // by tokens, then by pages
  int need[ITEMS];
  int64_t blk[ITEMS], sn = 0;
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    if (want[k] > 0 && tok[k] > a.max_tokens) {
      stat[k] = 1;
      want[k] = 0;
    }
    need[k] = want[k] > 0 ? (held[k] + want[k] + bs - 1) / bs - have[k] : 0;
    sn += need[k];
    blk[k] = sn;
  }
  {
    int64_t en = sn, unused = 0;
    scan2(en, unused, tmp);
    en -= sn;
    st = sn = 0;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      if (need[k] > 0 && blk[k] + en > avail) {
        stat[k] = 2;
        want[k] = 0;
        need[k] = 0;
      }
      st += want[k];
      tok[k] = st;
      sn += need[k];
      blk[k] = sn;
    }
  }
  {
    int64_t et = st, en = sn;
    scan2(et, en, tmp);
    if (tid == kPlanThreads - 1) {
      total[0] = et;
      total[1] = en;
    }
    et -= st;
    en -= sn;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int r = r0 + k;
      tok_end[r] = int32_t(tok[k] + et);
      blk_end[r] = int32_t(blk[k] + en);
      if (lead && r < a.R) {
        a.token_start[r + 1] = int32_t(tok[k] + et);
        a.start_pos[r] = held[k];
        a.seq_lens[r] = gone[k] ? 0 : held[k] + want[k];
        a.status[r] = stat[k];
        if (stat[k] != 0 && a.err_count != nullptr) atomicAdd(a.err_count, 1);
      }
    }
  }
  __syncthreads();
  const int n_tok = int(total[0]), n_new = int(total[1]);
  if (lead && tid == 0) {
    a.token_start[0] = 0;
    a.free_left[0] = avail - n_new;
    if (a.err_count != nullptr && all_back > a.n_blocks - free0) {
      const int64_t dropped = all_back - (a.n_blocks - free0);
      atomicAdd(a.err_count, int(dropped < 0x7FFFFFFF ? dropped : 0x7FFFFFFF));
    }
  }

  // entry j of the stack after the released pages came back: below free0 the caller's list, above
  // it the released requests' entries
  auto released = [&](int j) {
    const int r = first_above(back_end, a.R, j);
    const int before = r > 0 ? back_end[r - 1] : 0;
    return a.block_table[int64_t(r) * a.max_blocks + (j - before)];
  };
  auto stack = [&](int idx) { return idx < free0 ? a.free_list[idx] : released(idx - free0); };
  auto pages_of = [&](int r) {  // pages the request holds already
    return (a.cached_lens[r] + bs - 1) / bs;
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
      pos = a.cached_lens[req] + int(i) - (req > 0 ? tok_end[req - 1] : 0);
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
  int64_t grid = (int64_t(a.max_tokens) + kTokensPerGroup - 1) / kTokensPerGroup;
  grid = grid < 1 ? 1 : (grid > 1024 ? 1024 : grid);
  PlanArgs args = a;
  void* params[] = {&args};
  const void* fn = a.R <= kPlanThreads       ? reinterpret_cast<const void*>(&k_batch_plan<1>)
                   : a.R <= 4 * kPlanThreads ? reinterpret_cast<const void*>(&k_batch_plan<4>)
                                             : reinterpret_cast<const void*>(&k_batch_plan<16>);
  return hipLaunchKernel(fn, dim3(unsigned(grid)), dim3(kPlanThreads), params, 0, stream);
}

}  // namespace engram
