// Absorbed latent attention over the pages: out = softmax(scale q (c, k)^T) c, one latent row c a position.
//
// A row of a tile is a (token, head) pair of one request, M = 16 MB rows to a tile; a tile goes over its
// positions in stages of 64 rows of the cache, which lie in LDS as bf16 (FP8 rows are converted on the way in,
// exactly), read twice: along the features for the scores, and transposed (ds_read_tr16) for the values.
//  scores   S^T = C Q^T: a wave takes 16 (MB 4: 32) of the positions and keeps its queries in registers; a lane
//           then holds 4 consecutive positions of one query.
//  softmax  running maximum and sum in the base 2; the waves share each stage's maxima through LDS; a maximum
//           that grows by less than 2^8 leaves the reference where it is (weights up to 2^8 cost nothing in
//           fp32 sums and bf16 weights), so that accumulators are rarely rescaled.
//  values   out^T += C^T P^T: a wave takes a quarter of the latent's features for every query; the weights
//           pass through LDS as bf16, the order of positions in the product being that of the score fragments.
//
// Work is shared out in units of one stage of one tile: workgroup w of G takes units [w U / G, (w + 1) U / G) of
// the step's U, whatever the requests' lengths, so every CU has the same share.  What a workgroup holds of a
// tile that it does not finish alone goes to the workspace (fp32 sums, maxima), and k_absorbed_join
// adds a tile's parts in order.
//
// Rows that take no part (outside the tile's positions, on a bad page) are zeros in LDS and their scores
// -infinity.  Where the tokens of a tile see different positions, a value that is not finite must not reach those that do
// not see it (0 times infinity): such stages are looked through and, if they hold one, added by plain_values.
#include "latent_common.h"
#include "serving.h"

namespace engram {

namespace {

typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4_t;

constexpr int kThreads = 256;
constexpr int kTB = 64;           // positions per stage
constexpr float kGrow = 8.0f;     // the reference maximum moves when it is passed by more (log2)
constexpr float kInf = __builtin_inff();

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

// 16-byte chunk c of row r lies at position c ^ swizzle(r): 16 rows' reads of one chunk cover all 64 banks once
// (rows start at even multiples of 128 bytes or odd ones by turns), and so do 8 rows' transposed
// reads of a pair of chunks.
__device__ __forceinline__ int swizzle(int r) { return (r & 6) | ((r >> 3) & 1); }

// What a workgroup leaves in the workspace, for the join.
struct Part {
  int32_t first, row0, rows;  // flat token, first row and number of rows of the request; rows 0: no part
  int32_t last;               // the part that ends its tile
};

template <int DC, int MB>
struct Shape {
  static constexpr int M = 16 * MB;
  static constexpr int kChunks = (DC + 64) / 8, kRowB = kChunks * 16;  // of a row in LDS
  static constexpr int kKB = DC / 32;                                  // K blocks of the latent
  static constexpr int kFB = DC / 64;                                  // 16-feature blocks of a wave's quarter
  static constexpr int kQSplit = MB == 4 ? 2 : 1;                      // the waves share the queries in so many parts
  static constexpr int kMBQ = MB / kQSplit, kTBQ = kQSplit, kTG = 4 / kQSplit;
  static constexpr int kStageB = kTB * kRowB;
  static constexpr int kP = 2 * kStageB;                               // offsets into LDS
  static constexpr int kMax = kP + M * kTB * 2;
  static constexpr int kSlots = kMax + 4 * M * 4;
  static constexpr int kAlive = kSlots + 4 * kTB * 8;
  static constexpr int kMisc = kAlive + 4 * 8;
  static constexpr int kBytes = kMisc + 64;
  // per workgroup in the workspace: two parts of accumulators, maxima and sums, and their descriptions
  static constexpr int64_t kAccB = int64_t(M) * DC * 4, kMLB = M * 8;
};

struct Tile {
  Span s;
  int r, row0, rows;    // first row of the tile, rows of the request
  int lo, hi;           // positions that any of its rows sees
  int p_min, p_max;     // positions of its first and last row's tokens
  int base;             // position of unit 0 (the request's first)
};

template <int DC, int MB, bool FP8>
__global__ __launch_bounds__(kThreads, DC == 128 ? 2 : 1) void k_absorbed(AbsorbedArgs a) {
  using S = Shape<DC, MB>;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int rh = wv % S::kQSplit, tg = wv / S::kQSplit;
  const int rkb = a.rope_dim / 32;
  const int row_b = latent_row_bytes(DC, a.rope_dim, FP8);
  int64_t* slots = reinterpret_cast<int64_t*>(lds + S::kSlots);
  uint64_t* alive = reinterpret_cast<uint64_t*>(lds + S::kAlive);
  float* smax = reinterpret_cast<float*>(lds + S::kMax);
  int64_t* misc = reinterpret_cast<int64_t*>(lds + S::kMisc);

  // ---- this workgroup's units
  auto shape_of = [&](const Span& s, int* tiles, int* stages) {
    *tiles = (s.tokens * a.heads + S::M - 1) / S::M;
    *stages = (s.hi - s.lo + kTB - 1) / kTB;
  };
  const int G = gridDim.x;
  int w = blockIdx.x;
  Part* parts = reinterpret_cast<Part*>(a.workspace);
  float* ml = reinterpret_cast<float*>(a.workspace + int64_t(G) * 2 * sizeof(Part));
  f32x4* accs = reinterpret_cast<f32x4*>(a.workspace + int64_t(G) * 2 * (sizeof(Part) + S::kMLB));
  int64_t u, u1;
  int r;
  int64_t rem;
  {
    const int items = (a.rq.R + kThreads - 1) / kThreads, r0 = tid * items;
    int64_t mine = 0, total;
    for (int k = r0; k < r0 + items && k < a.rq.R; ++k) {
      int tiles, stages;
      shape_of(span_of(a.rq, k), &tiles, &stages);
      mine += int64_t(tiles) * stages;
    }
    const int64_t before = block_scan64<kThreads>(mine, misc + 2, &total);
    // where every workgroup has work, an XCD takes neighbours (they share tiles' rows); else all XCDs take some
    const int n = total < G ? int(total) : G;
    if (n == G && (G & 7) == 0) w = (w & 7) * (G >> 3) + (w >> 3);
    if (tid == 0) {
      parts[2 * w].rows = 0;
      parts[2 * w + 1].rows = 0;
    }
    if (w >= n) return;
    u = total / n * w + total % n * w / n;  // (so each of the n has a unit at least, and a tile's parts are neighbours)
    u1 = total / n * (w + 1) + total % n * (w + 1) / n;
    if (u >= before && u < before + mine) {
      int64_t at = before;
      for (int k = r0; k < r0 + items && k < a.rq.R; ++k) {
        int tiles, stages;
        shape_of(span_of(a.rq, k), &tiles, &stages);
        const int64_t n = int64_t(tiles) * stages;
        if (u < at + n) {
          misc[0] = k;
          misc[1] = u - at;
          break;
        }
        at += n;
      }
    }
    __syncthreads();
    r = __builtin_amdgcn_readfirstlane(int(misc[0]));
    rem = misc[1];
    rem = (int64_t(__builtin_amdgcn_readfirstlane(int(rem >> 32))) << 32) | uint32_t(__builtin_amdgcn_readfirstlane(int(rem)));
  }

  while (u < u1) {
    // ---- the next segment: stages [c0, c0 + n) of one tile
    Tile t;
    t.r = r;
    t.s = span_of(a.rq, r);
    int tiles, stages;
    shape_of(t.s, &tiles, &stages);
    const int64_t units = int64_t(tiles) * stages;
    const int tile = int(rem / stages), c0 = int(rem - int64_t(tile) * stages);
    const int n = int(u1 - u < stages - c0 ? u1 - u : stages - c0);
    t.row0 = tile * S::M;
    t.rows = t.s.tokens * a.heads;
    const int last_row = t.row0 + S::M < t.rows ? t.row0 + S::M - 1 : t.rows - 1;
    t.p_min = t.s.pos + t.row0 / a.heads;
    t.p_max = t.s.pos + last_row / a.heads;
    t.base = t.s.lo;
    t.lo = a.rq.window > 0 && t.p_min + 1 > a.rq.window ? t.p_min + 1 - a.rq.window : 0;
    t.hi = t.p_max + 1;

    // ---- queries: fragments in registers, and the position of each row's token (-1: no row)
    u32x4 qf[S::kMBQ][S::kKB + 2];
    int qpos[S::kMBQ];
#pragma unroll
    for (int mb = 0; mb < S::kMBQ; ++mb) {
      const int row = t.row0 + (rh * S::kMBQ + mb) * 16 + i16;
      const bool on = row < t.rows;
      const int tok = on ? row / a.heads : 0, head = on ? row - tok * a.heads : 0;
      qpos[mb] = on ? t.s.pos + tok : -1;
      const uint16_t* src = a.q + (t.s.first + tok) * a.q_stride + int64_t(head) * (DC + a.rope_dim) + 8 * g;
#pragma unroll
      for (int kb = 0; kb < S::kKB + 2; ++kb)
        qf[mb][kb] = on && kb < S::kKB + rkb ? *reinterpret_cast<const u32x4*>(src + 32 * kb) : u32x4{0u, 0u, 0u, 0u};
    }
    f32x4 acc[S::kFB][MB];
    float m_run[MB], l_own[S::kMBQ];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      m_run[mb] = -kInf;
#pragma unroll
      for (int fb = 0; fb < S::kFB; ++fb) acc[fb][mb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int mb = 0; mb < S::kMBQ; ++mb) l_own[mb] = 0.0f;

    // ---- staging
    auto find_slot = [&](int c) -> int64_t {  // (wave 0) slot of the lane's row of stage c
      const int pos = t.base + c * kTB + lane;
      if (c >= c0 + n || pos < t.lo || pos >= t.hi) return -1;
      const int64_t slot = slot_of(a.rq, r, pos);
      if (slot < 0 && tile == 0 && a.err_count != nullptr) atomicAdd(a.err_count, 1);
      return slot;
    };
    auto put_slot = [&](int c, int64_t slot) {
      slots[(c & 3) * kTB + lane] = slot;
      const uint64_t on = __ballot(slot >= 0);
      if (lane == 0) alive[c & 3] = on;
    };
    // FP8: 16 codes a lane, in registers until the stage's buffer is free
    constexpr int kNP = DC / 16, kPer = kNP / 4;
    u32x4 code[FP8 ? kPer : 1], rope[2];
    uint32_t scale[FP8 ? kPer : 1];
    auto load_stage = [&](int c) {
      const int64_t* sl = slots + (c & 3) * kTB;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int64_t slot = sl[tid / kNP + k * (kThreads / kNP)];
        const uint8_t* src = a.cache + (slot < 0 ? 0 : slot) * row_b;
        code[k] = *reinterpret_cast<const u32x4*>(src + (tid % kNP) * 16);
        scale[k] = src[DC + (tid % kNP) / 2];
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int rp = 4 * rkb, id = tid + k * kThreads;
        if (k < rkb) {
          const int64_t slot = sl[id / rp];
          rope[k] = *reinterpret_cast<const u32x4*>(a.cache + (slot < 0 ? 0 : slot) * row_b + DC + 16 + (id % rp) * 16);
        }
      }
    };
    auto store_stage = [&](int c, char* buf) {
      const uint64_t on = alive[c & 3];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int row = tid / kNP + k * (kThreads / kNP), sw = swizzle(row);
        u32x4 o0, o1;
        latent16(code[k], scale[k], o0, o1);
        if (!((on >> row) & 1)) o0 = o1 = u32x4{0u, 0u, 0u, 0u};
        char* to = buf + row * S::kRowB;
        *reinterpret_cast<u32x4*>(to + ((2 * (tid % kNP)) ^ sw) * 16) = o0;
        *reinterpret_cast<u32x4*>(to + ((2 * (tid % kNP) + 1) ^ sw) * 16) = o1;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int rp = 4 * rkb, id = tid + k * kThreads, row = id / rp;
        if (k < rkb)
          *reinterpret_cast<u32x4*>(buf + row * S::kRowB + ((DC / 8 + id % rp) ^ swizzle(row)) * 16) =
              (on >> row) & 1 ? rope[k] : u32x4{0u, 0u, 0u, 0u};
      }
    };
    // BF16: straight into LDS, 16 bytes a lane in the order of the buffer
    auto copy_stage = [&](int c, char* buf) {
      const int64_t* sl = slots + (c & 3) * kTB;
#pragma unroll
      for (int k = 0; k < S::kChunks / 4; ++k) {
        const int id = (k * 4 + wv) * 64 + lane, row = id / S::kChunks;
        int ch = (id - row * S::kChunks) ^ swizzle(row);
        ch = ch < DC / 8 + 4 * rkb ? ch : 0;  // (a place that is not read)
        const int64_t slot = sl[row];
        __builtin_amdgcn_global_load_lds((const void*)(a.cache + (slot < 0 ? 0 : slot) * row_b + ch * 16),
                                         (lds_ptr_t)(buf + (k * 4 + wv) * 1024), 16, 0, 0);
      }
    };
    auto clear_dead = [&](int c, char* buf) {  // of what this lane copied
      const uint64_t on = alive[c & 3];
      if (on == ~uint64_t(0)) return;
#pragma unroll 1
      for (int k = 0; k < S::kChunks / 4; ++k) {
        const int id = (k * 4 + wv) * 64 + lane;
        if (!((on >> (id / S::kChunks)) & 1)) *reinterpret_cast<u32x4*>(buf + id * 16) = u32x4{0u, 0u, 0u, 0u};
      }
    };

    wait_lds_barrier();  // the last segment's reads of LDS are over
    if (wv == 0) {
      put_slot(c0, find_slot(c0));
      put_slot(c0 + 1, find_slot(c0 + 1));
    }
    wait_lds_barrier();
    if constexpr (FP8) {
      load_stage(c0);
      store_stage(c0, lds);
      if (n > 1) load_stage(c0 + 1);
    } else {
      copy_stage(c0, lds);
    }

    for (int j = 0; j < n; ++j) {
      const int c = c0 + j;
      char* buf = lds + (j & 1) * S::kStageB;
      char* next = lds + ((j & 1) ^ 1) * S::kStageB;
      if constexpr (!FP8) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        clear_dead(c, buf);
      }
      if constexpr (FP8) wait_lds_barrier();
      else wait_all_barrier();
      if constexpr (!FP8)
        if (j + 1 < n) copy_stage(c + 1, next);
      int64_t slot2 = -1;
      if (wv == 0) slot2 = find_slot(c + 2);

      // ---- scores
      f32x4 s[S::kTBQ][S::kMBQ];
#pragma unroll
      for (int tb = 0; tb < S::kTBQ; ++tb)
#pragma unroll
        for (int mb = 0; mb < S::kMBQ; ++mb) s[tb][mb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      const int sw = swizzle(i16);
#pragma unroll
      for (int kb = 0; kb < S::kKB + 2; ++kb) {
        if (kb == S::kKB + 1 && rkb == 1) continue;
#pragma unroll
        for (int tb = 0; tb < S::kTBQ; ++tb) {
          const u32x4 k = *reinterpret_cast<const u32x4*>(buf + ((tg * S::kTBQ + tb) * 16 + i16) * S::kRowB + ((kb * 4 + g) ^ sw) * 16);
#pragma unroll
          for (int mb = 0; mb < S::kMBQ; ++mb) s[tb][mb] = mfma16x16x32(k, qf[mb][kb], s[tb][mb]);
        }
      }
      const uint64_t on = alive[c & 3];
      const int j0 = t.base + c * kTB;
      const bool differ = t.p_min != t.p_max && (j0 + kTB - 1 > t.p_min || (a.rq.window > 0 && j0 <= t.p_max - a.rq.window));
      const bool edge = on != ~uint64_t(0) || differ;
#pragma unroll
      for (int tb = 0; tb < S::kTBQ; ++tb)
#pragma unroll
        for (int mb = 0; mb < S::kMBQ; ++mb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[tb][mb][e] *= a.scale_log2;
            if (edge) {
              const int row = (tg * S::kTBQ + tb) * 16 + 4 * g + e, pos = j0 + row;
              const bool seen = ((on >> row) & 1) && pos <= qpos[mb] && (a.rq.window <= 0 || pos > qpos[mb] - a.rq.window);
              s[tb][mb][e] = seen ? s[tb][mb][e] : -kInf;
            }
          }
#pragma unroll
      for (int mb = 0; mb < S::kMBQ; ++mb) {
        float m = -kInf;
#pragma unroll
        for (int tb = 0; tb < S::kTBQ; ++tb)
#pragma unroll
          for (int e = 0; e < 4; ++e) m = fmaxf(m, s[tb][mb][e]);
        m = fmaxf(m, __shfl_xor(m, 16, kWave));
        m = fmaxf(m, __shfl_xor(m, 32, kWave));
        if (g == 0) smax[tg * S::M + (rh * S::kMBQ + mb) * 16 + i16] = m;
      }
      if (wv == 0) put_slot(c + 2, slot2);
      wait_lds_barrier();

      // ---- the reference maxima, then the weights
      float m_new[MB];
      bool grow = false;
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        float m = smax[mb * 16 + i16];
#pragma unroll
        for (int k = 1; k < S::kTG; ++k) m = fmaxf(m, smax[k * S::M + mb * 16 + i16]);
        m_new[mb] = m;
        grow |= m > m_run[mb] + kGrow;
      }
      if (__any(grow)) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          const float m = fmaxf(m_run[mb], m_new[mb]);
          const float alpha = m == -kInf ? 1.0f : __builtin_amdgcn_exp2f(m_run[mb] - m);
          m_run[mb] = m;
#pragma unroll
          for (int fb = 0; fb < S::kFB; ++fb) acc[fb][mb] *= alpha;
          if (mb / S::kMBQ == rh) {
#pragma unroll
            for (int k = 0; k < S::kMBQ; ++k)
              if (mb % S::kMBQ == k) l_own[k] *= alpha;
          }
        }
      }
#pragma unroll
      for (int mb = 0; mb < S::kMBQ; ++mb) {
        float ref = 0.0f;
#pragma unroll
        for (int k = 0; k < S::kQSplit; ++k)
          if (rh == k) ref = m_run[k * S::kMBQ + mb];
        ref = ref == -kInf ? 0.0f : ref;
        const int row = (rh * S::kMBQ + mb) * 16 + i16;
#pragma unroll
        for (int tb = 0; tb < S::kTBQ; ++tb) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = __builtin_amdgcn_exp2f(s[tb][mb][e] - ref);
            l_own[mb] += p[e];
          }
          const int blk = tg * S::kTBQ + tb;  // positions 16 blk + 4 g .. : half blk & 1 of K block blk / 2
          *reinterpret_cast<u32x2*>(lds + S::kP + row * kTB * 2 + (((blk >> 1) * 4 + g) ^ ((row >> 1) & 7)) * 16 + (blk & 1) * 8) =
              u32x2{pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3])};
        }
      }
      if constexpr (FP8) {
        if (j + 1 < n) store_stage(c + 1, next);
        if (j + 2 < n) load_stage(c + 2);
      }
      bool odd = false;  // a value that is not finite, where rows see different positions
      if (differ) {
        for (int k = tid; k < kTB * DC / 8; k += kThreads) {
          const int row = k / (DC / 8), ch = k % (DC / 8);
          const u32x4 v = *reinterpret_cast<const u32x4*>(buf + row * S::kRowB + (ch ^ swizzle(row)) * 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) odd |= (v[e] & 0x7F80u) == 0x7F80u || (v[e] & 0x7F800000u) == 0x7F800000u;
        }
        if (tid == 0) misc[0] = 0;
        wait_lds_barrier();
        if (odd) misc[0] = 1;
      }
      wait_lds_barrier();
      if (differ) odd = misc[0] != 0;

      // ---- values
      if (__builtin_expect(!odd, 1)) {
#pragma unroll
        for (int ks = 0; ks < kTB / 32; ++ks) {
          u32x4 p[MB];
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            const int row = mb * 16 + i16;
            p[mb] = *reinterpret_cast<const u32x4*>(lds + S::kP + row * kTB * 2 + ((ks * 4 + g) ^ ((row >> 1) & 7)) * 16);
          }
          const int vrow = 4 * g + (i16 >> 2), vsw = swizzle(vrow);
#pragma unroll
          for (int fb = 0; fb < S::kFB; ++fb) {
            const int ch = (wv * (DC / 4) + fb * 16) / 8 + ((i16 & 3) >> 1);
            char* at = buf + (ks * 32 + vrow) * S::kRowB + (ch ^ vsw) * 16 + (i16 & 1) * 8;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)at);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)(at + 16 * S::kRowB));
            const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
            const u32x4 v = {l2.x, l2.y, h2.x, h2.y};
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) acc[fb][mb] = mfma16x16x32(v, p[mb], acc[fb][mb]);
          }
        }
      } else {
        // plain_values: each weight times its row, only where the query sees it
#pragma unroll 1
        for (int row = 0; row < kTB; ++row) {
          const int pos = j0 + row;
          const int off = ((row >> 5) * 4 + ((row >> 2) & 3)) * 16, in = ((row >> 4) & 1) * 8 + (row & 3) * 2;
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            const int q = t.row0 + mb * 16 + i16, qp = q < t.rows ? t.s.pos + q / a.heads : -1;
            if (!((on >> row) & 1) || pos > qp || (a.rq.window > 0 && pos <= qp - a.rq.window)) continue;
            const float p = bf16_lo(*reinterpret_cast<const uint16_t*>(lds + S::kP + (mb * 16 + i16) * kTB * 2 +
                                                                        (off ^ ((((mb * 16 + i16) >> 1) & 7) * 16)) + in));
#pragma unroll
            for (int fb = 0; fb < S::kFB; ++fb) {
              const int f = wv * (DC / 4) + fb * 16 + 4 * g;
              const u32x2 v = *reinterpret_cast<const u32x2*>(buf + row * S::kRowB + ((f >> 3) ^ swizzle(row)) * 16 + (f & 7) * 2);
              acc[fb][mb] += f32x4{p * bf16_lo(v.x), p * bf16_hi(v.x), p * bf16_lo(v.y), p * bf16_hi(v.y)};
            }
          }
        }
      }
    }

    // ---- the sums of all positions, then the outputs or a part
#pragma unroll
    for (int mb = 0; mb < S::kMBQ; ++mb) {
      float l = l_own[mb];
      l += __shfl_xor(l, 16, kWave);
      l += __shfl_xor(l, 32, kWave);
      if (g == 0) smax[tg * S::M + (rh * S::kMBQ + mb) * 16 + i16] = l;
    }
    wait_lds_barrier();
    float l_all[MB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      l_all[mb] = smax[mb * 16 + i16];
#pragma unroll
      for (int k = 1; k < S::kTG; ++k) l_all[mb] += smax[k * S::M + mb * 16 + i16];
    }
    if (c0 == 0 && n == stages) {
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const int row = t.row0 + mb * 16 + i16;
        if (row >= t.rows) continue;
        const int tok = row / a.heads, head = row - tok * a.heads;
        const float inv = l_all[mb] == 0.0f ? 0.0f : 1.0f / l_all[mb];
        uint16_t* out = a.out + (t.s.first + tok) * a.out_stride + int64_t(head) * DC + wv * (DC / 4) + 4 * g;
#pragma unroll
        for (int fb = 0; fb < S::kFB; ++fb)
          *reinterpret_cast<u32x2*>(out + fb * 16) = u32x2{pack_bf16x2(acc[fb][mb][0] * inv, acc[fb][mb][1] * inv),
                                                           pack_bf16x2(acc[fb][mb][2] * inv, acc[fb][mb][3] * inv)};
        if (a.lse != nullptr && wv == 0 && g == 0)
          a.lse[int64_t(t.s.first + tok) * a.heads + head] =
              l_all[mb] == 0.0f ? -kInf : (m_run[mb] + __builtin_amdgcn_logf(l_all[mb])) * 0.69314718f;
      }
    } else {
      const int64_t at = 2 * w + (c0 == 0 ? 1 : 0);
      f32x4* to = accs + at * (S::M * DC / 4) + wv * (S::kFB * MB * kWave) + lane;
#pragma unroll
      for (int fb = 0; fb < S::kFB; ++fb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) to[(fb * MB + mb) * kWave] = acc[fb][mb];
      if (wv == 0 && g == 0) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          ml[at * 2 * S::M + mb * 16 + i16] = m_run[mb];
          ml[at * 2 * S::M + S::M + mb * 16 + i16] = l_all[mb];
        }
      }
      if (tid == 0) parts[at] = Part{t.s.first, t.row0, t.rows, c0 + n == stages ? 1 : 0};
    }

    // ---- on to the next request with work, if this one is done
    u += n;
    rem += n;
    if (u < u1 && rem == units) {
      rem = 0;
      for (int from = r + 1;; from += kThreads) {
        wait_lds_barrier();
        if (tid == 0) misc[0] = a.rq.R;
        wait_lds_barrier();
        if (from + tid < a.rq.R && span_of(a.rq, from + tid).tokens > 0) atomicMin(reinterpret_cast<unsigned long long*>(misc), (unsigned long long)(from + tid));
        wait_lds_barrier();
        r = __builtin_amdgcn_readfirstlane(int(misc[0]));
        if (r < a.rq.R || from + kThreads >= a.rq.R) break;
      }
      if (r >= a.rq.R) break;  // (cannot be: the units say that there is one)
    }
  }
}

// Adds the parts of the tile that begins in workgroup blockIdx.x's last segment, if others finish it.  A wave takes 16 features of 16 rows.
template <int DC, int MB>
__global__ __launch_bounds__(kWave) void k_absorbed_join(AbsorbedArgs a, int G) {
  using S = Shape<DC, MB>;
  const Part* parts = reinterpret_cast<const Part*>(a.workspace);
  const float* ml = reinterpret_cast<const float*>(a.workspace + int64_t(G) * 2 * sizeof(Part));
  const f32x4* accs = reinterpret_cast<const f32x4*>(a.workspace + int64_t(G) * 2 * (sizeof(Part) + S::kMLB));
  const int w = blockIdx.x, lane = threadIdx.x, i16 = lane & 15, g = lane >> 4;
  const Part p = parts[2 * w + 1];
  if (p.rows == 0) return;
  const int mb = blockIdx.y % MB, fbw = blockIdx.y / MB, wv = fbw / S::kFB, fb = fbw % S::kFB;
  const int row = p.row0 + mb * 16 + i16;
  int end = w + 1;  // the part that ends the tile
  while (end < G - 1 && !(parts[2 * end].rows != 0 && parts[2 * end].last)) ++end;
  float m = ml[(2 * w + 1) * 2 * S::M + mb * 16 + i16];
  for (int k = w + 1; k <= end; ++k) m = fmaxf(m, ml[int64_t(2 * k) * 2 * S::M + mb * 16 + i16]);
  const float ref = m == -kInf ? 0.0f : m;
  float l = 0.0f;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int k = w; k <= end; ++k) {
    const int64_t at = k == w ? 2 * w + 1 : 2 * k;
    const float f = __builtin_amdgcn_exp2f(ml[at * 2 * S::M + mb * 16 + i16] - ref);
    l += f * ml[at * 2 * S::M + S::M + mb * 16 + i16];
    acc += f * accs[at * (S::M * DC / 4) + (wv * S::kFB * MB + fb * MB + mb) * kWave + lane];
  }
  if (row >= p.rows) return;
  const int tok = row / a.heads, head = row - tok * a.heads;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  acc *= inv;
  *reinterpret_cast<u32x2*>(a.out + (p.first + tok) * a.out_stride + int64_t(head) * DC + wv * (DC / 4) + fb * 16 + 4 * g) =
      u32x2{pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3])};
  if (a.lse != nullptr && fbw == 0 && g == 0)
    a.lse[int64_t(p.first + tok) * a.heads + head] = l == 0.0f ? -kInf : (m + __builtin_amdgcn_logf(l)) * 0.69314718f;
}

template <int DC, int MB, bool FP8>
hipError_t run(const AbsorbedArgs& a, int G, hipStream_t stream) {
  using S = Shape<DC, MB>;
  static_assert(S::kBytes <= 160 * 1024, "LDS of a CU");
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_absorbed<DC, MB, FP8>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e != hipSuccess) return e;
  k_absorbed<DC, MB, FP8><<<dim3(G), dim3(kThreads), S::kBytes, stream>>>(a);
  k_absorbed_join<DC, MB><<<dim3(G, 4 * S::kFB * MB), dim3(kWave), 0, stream>>>(a, G);
  return hipGetLastError();
}

template <int DC, int MB>
hipError_t run(const AbsorbedArgs& a, int G, hipStream_t stream) {
  return a.fp8 ? run<DC, MB, true>(a, G, stream) : run<DC, MB, false>(a, G, stream);
}

template <int DC>
hipError_t run(const AbsorbedArgs& a, int cus, hipStream_t stream) {
  const int G = DC == 128 ? 2 * cus : cus;
  // rows of a request: its tokens (the step's share of one) times the heads
  int64_t tokens = (a.rq.n_tokens + a.rq.R - 1) / a.rq.R;
  if (a.rq.max_tokens > 0 && tokens > a.rq.max_tokens) tokens = a.rq.max_tokens;
  const int64_t rows = tokens * a.heads;
  if (rows <= 16) return run<DC, 1>(a, G, stream);
  if (rows <= 32) return run<DC, 2>(a, G, stream);
  return run<DC, 4>(a, G, stream);
}

}  // namespace

int64_t absorbed_workspace_bytes(int latent_dim, int cus) {
  const int G = latent_dim == 128 ? 2 * cus : cus;
  return int64_t(G) * 2 * (int64_t(sizeof(Part)) + 64 * 8 + int64_t(64) * latent_dim * 4);
}

hipError_t launch_latent_absorbed(const AbsorbedArgs& a, int cus, hipStream_t stream) {
  if (a.latent_dim == 128) return run<128>(a, cus, stream);
  if (a.latent_dim == 256) return run<256>(a, cus, stream);
  return run<512>(a, cus, stream);
}

}  // namespace engram
