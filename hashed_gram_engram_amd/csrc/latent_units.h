// The absorbed attention's work sharing: units of one stage (STAGE positions) of one tile (M rows) each, in order of
// requests, tiles and positions; workgroup w of n takes units [w U / n, (w + 1) U / n) of the step's U.  So each has the same
// share, whatever the requests' lengths.  A workgroup finishes the tiles whose stages it has alone; of others it
// leaves a part (at most two: of a tile that began before its first unit, and of one that goes on behind its last).
#pragma once

#include "latent_common.h"

namespace engram {

typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4_t;

constexpr float kInf = __builtin_inff();
// The reference of a softmax is set 2^16 above the highest score and moves when a score passes it, so accumulators are rarely
// scaled.  Weights are 1 at most (whatever values fp32 can add up stay in range), and 2^-16 costs nothing in fp32 sums and
// bf16 weights.
constexpr float kGrow = 16.0f;
__device__ __forceinline__ float moved_reference(float m_run, float m_new) { return m_new > m_run ? m_new + kGrow : m_run; }

// A product that is rounded by itself, not fused into what it is added to.
__device__ __forceinline__ float rounded_product(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}

// Scores times the scale are taken to a reference of more than 2^24 rounded: the reference is the rounded product of the highest
// score, and a fused product less it would be that rounding's error, which from 2^31 on passes the exponents of fp32 (weights
// of infinity, or all zero).  Below 2^24 the error is at most 1 and the same for all weights.
constexpr float kBigScore = 16777216.0f;

// 16-byte chunk c of row r lies at position c ^ swizzle(r): 16 rows' reads of one chunk cover all 64 banks once
// (rows start at even multiples of 128 bytes or odd ones by turns), and so do 8 rows' transposed reads of
// a pair of chunks.
__device__ __forceinline__ int latent_swizzle(int r) { return (r & 6) | ((r >> 3) & 1); }

// The maximum (sum) over the four lanes i, 16 + i, 32 + i, 48 + i.
__device__ __forceinline__ float quad_max(float v) {
  const uint32_t b = __float_as_uint(v);
  const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const uint32_t m = __float_as_uint(fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1])));
  const auto q = __builtin_amdgcn_permlane16_swap(m, m, false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float quad_sum(float v) {
  const uint32_t b = __float_as_uint(v);
  const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const uint32_t m = __float_as_uint(__uint_as_float(h[0]) + __uint_as_float(h[1]));
  const auto q = __builtin_amdgcn_permlane16_swap(m, m, false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// The address in LDS of `at`.
__device__ __forceinline__ uint32_t lds_address(const void* at) { return uint32_t(uintptr_t((lds_ptr_t)at)); }

// Copies 16 or 4 bytes a lane from memory to LDS, lane l's to `to` + l times that; `to` is the same in every lane.  Whoever
// reads them waits first: the compiler does not know of them (its own waits, for loads into registers, then only wait
// for more than they need).  m0 is set for each copy; kernels with these use nothing else that keeps it.  (The compiler
// has a builtin, but then lets every transposed read of LDS wait for all copies in flight.)
template <int BYTES>
__device__ __forceinline__ void copy_to_lds(const void* from, uint32_t to) {
  to = __builtin_amdgcn_readfirstlane(to);
  if constexpr (BYTES == 16) asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from));
  else asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(from));
}
// 16 bytes a lane from `off` bytes after `from`, which is the same in every lane.
__device__ __forceinline__ void copy_to_lds(const void* from, uint32_t off, uint32_t to) {
  to = __builtin_amdgcn_readfirstlane(to);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(off), "s"(from));
}
__device__ __forceinline__ void wait_lds_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void wait_all_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ bool any_not_finite(u32x4 v) {  // of eight bf16
  bool odd = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) odd |= (v[e] & 0x7F80u) == 0x7F80u || (v[e] & 0x7F800000u) == 0x7F800000u;
  return odd;
}
// The union of all threads' rows (uniform).  A barrier lies between two calls.
__device__ __forceinline__ uint64_t any_rows(uint64_t rows, int64_t* misc) {
  unsigned long long* word = reinterpret_cast<unsigned long long*>(misc);
  if (threadIdx.x == 0) *word = 0;
  wait_lds_barrier();
  if (rows != 0) atomicOr(word, static_cast<unsigned long long>(rows));
  wait_lds_barrier();
  const uint64_t all = *word;
  return uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(all >> 32)))) << 32 | uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(all)));
}

// A part of a tile in the workspace, for the join.
struct Part {
  int32_t first, row0, rows;  // first flat token of the request, first row of the tile, rows of the request (0: no part)
  int32_t end;                // of a tile's first part: the workgroup that has its last
};

// The workspace of G workgroups: parts, then maxima and sums (2 M fp32 a part), then accumulators (M DC fp32).
struct PartSpace {
  Part* parts;
  float* ml;
  f32x4* acc;
};
__device__ __forceinline__ PartSpace part_space(char* workspace, int G, int M) {
  PartSpace s;
  s.parts = reinterpret_cast<Part*>(workspace);
  s.ml = reinterpret_cast<float*>(workspace + int64_t(G) * 2 * sizeof(Part));
  s.acc = reinterpret_cast<f32x4*>(workspace + int64_t(G) * 2 * (sizeof(Part) + M * 8));
  return s;
}
constexpr int64_t part_space_bytes(int64_t G, int M, int latent_dim) {
  return G * 2 * (int64_t(sizeof(Part)) + M * 8 + int64_t(M) * latent_dim * 4);
}

template <int M, int STAGE>
__device__ __forceinline__ void tiles_of(const Span& s, int heads, int* tiles, int* stages) {
  *tiles = (s.tokens * heads + M - 1) / M;
  *stages = (s.hi - s.lo + STAGE - 1) / STAGE;
}

// This workgroup's units [u, u1): they begin with unit `rem` of request r.  misc: 8 words of LDS.
struct Units {
  int64_t u, u1, rem, total;
  int r, w, n;
  __device__ __forceinline__ int64_t begin(int k) const { return total / n * k + total % n * k / n; }
  __device__ __forceinline__ int owner(int64_t unit) const {  // (units below 2^54)
    int k = int(uint64_t(unit) * n / total);
    while (begin(k + 1) <= unit) ++k;
    while (begin(k) > unit) --k;
    return k;
  }
};
template <int THREADS, int M, int STAGE>
__device__ __forceinline__ bool my_units(const LatentRequests& q, int heads, Part* parts, int64_t* misc, Units* out) {
  const int tid = threadIdx.x, items = (q.R + THREADS - 1) / THREADS, r0 = tid * items, G = gridDim.x;
  auto units_of = [&](int k) -> int64_t {
    int tiles, stages;
    tiles_of<M, STAGE>(span_of(q, k), heads, &tiles, &stages);
    return int64_t(tiles) * stages;
  };
  const int64_t first = r0 < q.R ? units_of(r0) : 0;  // (up to THREADS requests: each has one)
  int64_t mine = first, total;
  for (int k = r0 + 1; k < r0 + items && k < q.R; ++k) mine += units_of(k);
  const int64_t before = block_scan64<THREADS>(mine, misc + 2, &total);
  // where every workgroup has work, an XCD takes neighbours (they share tiles' rows); else all XCDs take some
  const int n = total < G ? int(total) : G;
  int w = blockIdx.x;
  if (n == G && (G & 7) == 0) w = (w & 7) * (G >> 3) + (w >> 3);
  if (tid == 0) {
    parts[2 * w].rows = 0;
    parts[2 * w + 1].rows = 0;
  }
  if (w >= n) return false;
  out->w = w;
  out->n = n;
  out->total = total;
  out->u = out->begin(w);  // (each of the n has a unit at least: a tile's parts are neighbours)
  out->u1 = out->begin(w + 1);
  if (out->u >= before && out->u < before + mine) {
    int64_t at = before, units = first;
    int k = r0;
    while (out->u >= at + units) {
      at += units;
      units = units_of(++k);
    }
    misc[0] = k;
    misc[1] = out->u - at;
  }
  __syncthreads();
  out->r = __builtin_amdgcn_readfirstlane(int(misc[0]));
  const int64_t rem = misc[1];
  out->rem = (int64_t(__builtin_amdgcn_readfirstlane(int(rem >> 32))) << 32) | uint32_t(__builtin_amdgcn_readfirstlane(int(rem)));
  return true;
}

// The first request behind r with work (R if none); all threads.
template <int THREADS>
__device__ __forceinline__ int next_request(const LatentRequests& q, int r, int64_t* misc) {
  for (int from = r + 1; from < q.R; from += THREADS) {
    wait_lds_barrier();
    if (threadIdx.x == 0) misc[0] = q.R;
    wait_lds_barrier();
    const int k = from + int(threadIdx.x);
    if (k < q.R && span_of(q, k).tokens > 0)
      atomicMin(reinterpret_cast<unsigned long long*>(misc), static_cast<unsigned long long>(k));
    wait_lds_barrier();
    const int found = __builtin_amdgcn_readfirstlane(int(misc[0]));
    if (found < q.R) return found;
  }
  return q.R;
}

// Stages [c0, c0 + n) of one tile.
struct Segment {
  Span s;
  int tile, c0, n, stages;
  int64_t units;        // of the request
  int row0, rows;       // first row of the tile, rows of the request
  int lo, hi;           // positions that any of the tile's rows sees
  int p_min, p_max;     // positions of its first and last row's tokens
  int base;             // position of stage 0
  int fresh;            // the first position that no earlier tile of the request sees
};
template <int M, int STAGE>
__device__ __forceinline__ Segment segment_of(const LatentRequests& q, int heads, const Units& un) {
  Segment t;
  int tiles;
  t.s = span_of(q, un.r);
  tiles_of<M, STAGE>(t.s, heads, &tiles, &t.stages);
  t.units = int64_t(tiles) * t.stages;
  t.tile = int(un.rem / t.stages);
  t.c0 = int(un.rem - int64_t(t.tile) * t.stages);
  t.n = int(un.u1 - un.u < t.stages - t.c0 ? un.u1 - un.u : t.stages - t.c0);
  t.row0 = t.tile * M;
  t.rows = t.s.tokens * heads;
  const int last_row = t.row0 + M < t.rows ? t.row0 + M - 1 : t.rows - 1;
  t.p_min = t.s.pos + t.row0 / heads;
  t.p_max = t.s.pos + last_row / heads;
  t.base = t.s.lo;
  t.lo = q.window > 0 && t.p_min + 1 > q.window ? t.p_min + 1 - q.window : 0;
  t.hi = t.p_max + 1;
  t.fresh = t.tile == 0 ? t.lo : t.s.pos + (t.row0 - 1) / heads + 1;
  return t;
}

// Adds a tile's parts in order: part 2 w + 1 of the workgroup w in which it begins, and parts 2 k of w + 1 .. end.  `block`
// is the place of an accumulator (rows 16 blk .., features 16 fb ..) in a part, in blocks of 16 x 16.
// An item is a block of 16 rows of a tile; of tiles with many parts, 16 features of one, and its four waves share the
// parts.  The workgroups (a few per CU) find the items from the parts' descriptions and go over them.  Weights come
// first, in LDS; the sums then have several loads in flight.
constexpr int kMaxGroups = 1024, kManyParts = 24;
template <int DC, int M, class Block>
__device__ __forceinline__ void join_parts(const AbsorbedArgs& a, int G, Block block) {
  constexpr int kFB = DC / 16, kPer = kFB / 4, kThreads = 256;
  __shared__ int begin[kMaxGroups + 1];
  __shared__ float weight[kMaxGroups][16];
  __shared__ float red[4][2][16];
  __shared__ f32x4 sums[4][kWave];
  __shared__ int64_t tmp[4];
  const PartSpace space = part_space(a.workspace, G, M);
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, i16 = lane & 15, g = lane >> 4;
  const int groups = (G + kThreads - 1) / kThreads;
  int64_t mine = 0, total;
  for (int w = tid * groups; w < tid * groups + groups && w < G; ++w) {
    const Part p = space.parts[2 * w + 1];
    const int left = p.rows - p.row0, blocks = p.rows == 0 ? 0 : (left < M ? (left + 15) / 16 : M / 16);
    mine += p.end - w + 1 > kManyParts ? blocks * kFB : blocks;
  }
  int at = int(block_scan64<kThreads>(mine, tmp, &total));
  for (int w = tid * groups; w < tid * groups + groups && w < G; ++w) {
    const Part p = space.parts[2 * w + 1];
    const int left = p.rows - p.row0, blocks = p.rows == 0 ? 0 : (left < M ? (left + 15) / 16 : M / 16);
    begin[w] = at;
    at += p.end - w + 1 > kManyParts ? blocks * kFB : blocks;
  }
  if (tid == 0) begin[G] = int(total);
  __syncthreads();
  for (int item = blockIdx.x; item < int(total); item += gridDim.x) {
    int lo = 0, hi = G - 1;  // the last w with begin[w] <= item (those without items have the same begin as the next)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (begin[mid] <= item) lo = mid;
      else hi = mid - 1;
    }
    const int w = lo;
    const Part p = space.parts[2 * w + 1];
    const int count = p.end - w + 1;
    const bool many = count > kManyParts;
    const int in = item - begin[w], blk = many ? in / kFB : in, fb = many ? in % kFB : 0;
    auto part = [&](int k) -> int64_t { return k == 0 ? 2 * w + 1 : 2 * (w + k); };
    const float* ml = space.ml + blk * 16 + i16;
    float m = -kInf;
    for (int k = tid >> 4; k < count; k += 16) {
      const float v = ml[part(k) * 2 * M];
      weight[k][i16] = v;
      m = fmaxf(m, v);
    }
    m = quad_max(m);
    if (g == 0) red[wv][0][i16] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0][0][i16], red[1][0][i16]), fmaxf(red[2][0][i16], red[3][0][i16]));
    const float ref = m == -kInf ? 0.0f : m;
    float l = 0.0f;
    for (int k = tid >> 4; k < count; k += 16) {
      const float f = __builtin_amdgcn_exp2f(weight[k][i16] - ref);
      weight[k][i16] = f;
      l += f * ml[part(k) * 2 * M + M];
    }
    l = quad_sum(l);
    if (g == 0) red[wv][1][i16] = l;
    __syncthreads();
    l = red[0][1][i16] + red[1][1][i16] + red[2][1][i16] + red[3][1][i16];
    const int row = p.row0 + blk * 16 + i16;
    const int tok = row / a.heads, head = row - tok * a.heads;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t* out = a.out + (p.first + tok) * a.out_stride + int64_t(head) * DC + 4 * g;
    auto store = [&](int f, f32x4 v) {
      v *= inv;
      if (row < p.rows) *reinterpret_cast<u32x2*>(out + f * 16) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    };
    if (many) {
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
      const f32x4* from = space.acc + block(blk, fb) * kWave + lane;
#pragma unroll 8
      for (int k = wv; k < count; k += 4) acc += weight[k][i16] * from[part(k) * (M * DC / 4)];
      sums[wv][lane] = acc;
      __syncthreads();
      if (wv == 0) store(fb, (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]));
    } else {
      f32x4 acc[kPer] = {};
      for (int k = 0; k < count; ++k) {
        const float f = weight[k][i16];
        const f32x4* from = space.acc + part(k) * (M * DC / 4) + lane;
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] += f * from[block(blk, wv * kPer + e) * kWave];
      }
#pragma unroll
      for (int e = 0; e < kPer; ++e) store(wv * kPer + e, acc[e]);
    }
    if (a.lse != nullptr && fb == 0 && wv == 0 && g == 0 && row < p.rows)
      a.lse[int64_t(p.first + tok) * a.heads + head] = l == 0.0f ? -kInf : (m + __builtin_amdgcn_logf(l)) * 0.69314718f;
    __syncthreads();
  }
}

}  // namespace engram
