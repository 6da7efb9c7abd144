// Expanded latent attention: per head, keys (kv part, shared rope part) and values (kv part) of each row.
//
// A workgroup takes M = 16 RB NW tokens of one request and one head; each of its NW waves holds the queries of
// 16 RB tokens in registers.  Keys and values come through LDS in stages of 64 rows, copied straight from
// memory, two buffers.  S^T = K Q^T leaves a lane with 4 consecutive keys of one query, which is an operand
// of out^T += V^T P^T as it stands if the keys of that product are counted in the same order: the weights never
// leave the registers, and a query's maximum and sum are shared by 4 lanes of one wave.  Values are read
// transposed (ds_read_tr16).  The softmax is in the base 2; a maximum that grows by less than 2^16 leaves the
// reference where it is.
//
// Where few tiles meet many rows, each tile's stages are shared out in parts; their fp32 sums go to the workspace
// and k_expanded_join adds them in order.
//
// Rows past the last stay zeros in LDS; where a stage holds a value that is not finite and tokens see different
// rows of it, the product is taken row by row, only where it is seen (0 times infinity would not be 0).
#include "latent_units.h"

namespace engram {

namespace {

constexpr int kTB = 64;

template <int HD, int NW, int RB>
struct Shape {
  static constexpr int kThreads = NW * kWave, M = 16 * RB * NW;
  static constexpr int kKC = (HD + 64) / 8, kVC = HD / 8;  // 16-byte chunks of a key and of a value in LDS
  static constexpr int kKB = (HD + 64) / 32;
  static constexpr int kKeyTurn = kKC % 16 == 0 ? 4 : 2;   // K blocks that a swizzle moves a chunk among
  static constexpr int kValueTurn = kVC / 2;                  // 16-feature blocks, the same (8 or 4 pairs of chunks)
  static constexpr int kV = kTB * kKC * 16;                // offset of the values
  static constexpr int kStageB = kTB * (kKC + kVC) * 16;
  static constexpr int kBytes = 2 * kStageB;
};

// Chunk c of row r lies at c ^ swizzle: 16 rows' reads of a chunk of a key, and 8 rows' transposed reads of a
// pair of chunks of a value, then cover all 64 banks once.
template <int CHUNKS>
__device__ __forceinline__ int key_swizzle(int r) { return CHUNKS % 16 == 0 ? r & 15 : (r >> 1) & 7; }
template <int CHUNKS>
__device__ __forceinline__ int value_swizzle(int r) { return CHUNKS % 16 == 0 ? (r & 7) << 1 : r & 6; }

struct Tile {
  Span s;
  int first_row, rows;  // of the request
  int base;             // position of its first row
  int t0, tokens;       // of the tile
  int lo, hi;           // rows that any of them sees
};

// The tile of this workgroup (uniform); false where there is none.
template <int THREADS, int M>
__device__ __forceinline__ bool find_tile(const ExpandedArgs& a, int index, int64_t* tmp, Tile* t) {
  const int tid = threadIdx.x, items = (a.rq.R + THREADS - 1) / THREADS, r0 = tid * items;
  int64_t mine = 0, total;
  for (int r = r0; r < r0 + items && r < a.rq.R; ++r) mine += (span_of(a.rq, r).tokens + M - 1) / M;
  int64_t at = block_scan64<THREADS>(mine, tmp, &total);
  if (index >= total) return false;
  if (index >= at && index < at + mine) {
    for (int r = r0; r < r0 + items && r < a.rq.R; ++r) {
      const int n = (span_of(a.rq, r).tokens + M - 1) / M;
      if (index < at + n) {
        tmp[THREADS / kWave] = r;
        tmp[THREADS / kWave + 1] = index - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  const int r = __builtin_amdgcn_readfirstlane(int(tmp[THREADS / kWave]));
  const int tile = __builtin_amdgcn_readfirstlane(int(tmp[THREADS / kWave + 1]));
  t->s = span_of(a.rq, r);
  int b = a.row_start[r], e = a.row_start[r + 1];
  b = b < 0 ? 0 : (b > a.n_rows ? a.n_rows : b);
  e = e < b ? b : (e > a.n_rows ? a.n_rows : e);
  t->first_row = b;
  t->rows = e - b;
  t->base = t->s.pos + t->s.tokens - t->rows;
  t->t0 = tile * M;
  t->tokens = t->s.tokens - t->t0 < M ? t->s.tokens - t->t0 : M;
  const int p0 = t->s.pos + t->t0;
  int lo = a.rq.window > 0 ? p0 - a.rq.window + 1 - t->base : 0, hi = p0 + t->tokens - t->base;
  t->lo = lo < 0 ? 0 : lo;
  t->hi = hi > t->rows ? t->rows : hi;
  if (t->hi < t->lo) t->hi = t->lo;
  return true;
}

__device__ __forceinline__ uint32_t in_order(uint32_t b, uint32_t n) {  // an XCD takes a run of neighbours
  const uint32_t q = n >> 3, rem = n & 7, x = b & 7;
  return x * q + (x < rem ? x : rem) + (b >> 3);
}

template <int HD, int NW, int RB>
__global__ __launch_bounds__(NW* kWave, NW / 4) void k_expanded(ExpandedArgs a) {
  using S = Shape<HD, NW, RB>;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ int64_t tmp[NW + 2];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int rkb = a.rope_dim / 32;
  // heads, then tiles (the last, which sees the most, first), then parts
  uint32_t id = in_order(blockIdx.x, gridDim.x);
  const int part = int(id % a.parts);
  id /= a.parts;
  const int head = int(id / a.tiles);
  Tile t;
  if (!find_tile<S::kThreads, S::M>(a, a.tiles - 1 - int(id - head * a.tiles), tmp, &t)) return;
  const int stages_all = (t.hi - t.lo + kTB - 1) / kTB;
  const int c0 = int(int64_t(stages_all) * part / a.parts), c1 = int(int64_t(stages_all) * (part + 1) / a.parts);

  // queries: token wv * 16 RB + 16 mb + i16 of the tile
  u32x4 qf[RB][S::kKB];
  int qrow[RB];  // the last row that the token sees, -1: no token
#pragma unroll
  for (int mb = 0; mb < RB; ++mb) {
    const int tok = (wv * RB + mb) * 16 + i16;
    const bool on = tok < t.tokens;  // (tokens past the last repeat it)
    qrow[mb] = on ? t.s.pos + t.t0 + tok - t.base : -1;
    const uint16_t* src = a.q + int64_t(t.s.first + t.t0 + (on ? tok : t.tokens - 1)) * a.q_stride + head * (HD + a.rope_dim) + 8 * g;
#pragma unroll
    for (int kb = 0; kb < S::kKB; ++kb) qf[mb][kb] = *reinterpret_cast<const u32x4*>(src + 32 * (kb < HD / 32 + rkb ? kb : 0)) ^ a.q_sign;
  }
  // the rows that this wave's tokens see
  const int w0 = wv * RB * 16, wn = t.tokens - w0 < RB * 16 ? t.tokens - w0 : RB * 16;
  const int t_min = t.s.pos + t.t0 - t.base;  // the last row that the tile's first token sees
  const int w_min = t.s.pos + t.t0 + w0 - t.base, w_max = w_min + wn - 1;  // (wn <= 0: no token)

  // (a chunk's place differs from row to row in the low bits of its number only: addresses are one xor away from these)
  const int key_at = i16 * S::kKC * 16 + (g ^ key_swizzle<S::kKC>(i16)) * 16;
  const int vrow = 4 * g + (i16 >> 2);
  const int value_at = vrow * S::kVC * 16 + (((i16 & 3) >> 1) ^ value_swizzle<S::kVC>(vrow)) * 16 + (i16 & 1) * 8;

  f32x4 acc[HD / 16][RB];
  float m_run[RB], l_own[RB];
#pragma unroll
  for (int mb = 0; mb < RB; ++mb) {
    m_run[mb] = -kInf;
    l_own[mb] = 0.0f;
#pragma unroll
    for (int fb = 0; fb < HD / 16; ++fb) acc[fb][mb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // Copies: 16 bytes a lane, in the order of the buffer; keys, then values.  A lane's place in the rows moves on by a stage
  // at a time; only the last stage may have fewer rows, those past the end then repeat the last.
  constexpr int kKeyCopies = kTB * S::kKC / S::kThreads, kCopies = kKeyCopies + kTB * S::kVC / S::kThreads;
  static_assert(kTB * S::kKC % S::kThreads == 0 && kTB * S::kVC % S::kThreads == 0, "whole copies");
  const uint16_t* from[kCopies];
  uint32_t step[kCopies];  // bytes from row to row
  auto row_of = [&](int k) { return k < kKeyCopies ? (k * S::kThreads + tid) / S::kKC : ((k - kKeyCopies) * S::kThreads + tid) / S::kVC; };
#pragma unroll
  for (int k = 0; k < kCopies; ++k) {
    const int row = row_of(k);
    const uint16_t* base;
    if (k < kKeyCopies) {
      const int ch = (k * S::kThreads + tid - row * S::kKC) ^ key_swizzle<S::kKC>(row);
      const bool own = ch < HD / 8;
      base = own ? a.kv + head * 2 * HD + ch * 8 : a.rope + (ch - HD / 8 < 4 * rkb ? ch - HD / 8 : 0) * 8;
      step[k] = uint32_t(own ? a.kv_stride : a.rope_stride) * 2;
    } else {
      const int ch = ((k - kKeyCopies) * S::kThreads + tid - row * S::kVC) ^ value_swizzle<S::kVC>(row);
      base = a.kv + head * 2 * HD + HD + ch * 8;
      step[k] = uint32_t(a.kv_stride) * 2;
    }
    from[k] = base + int64_t(t.first_row + t.lo + c0 * kTB + row) * (step[k] / 2);
  }
  auto copy_stage = [&](int c, char* buf) {
    const int left = t.hi - (t.lo + c * kTB);
#pragma unroll
    for (int k = 0; k < kCopies; ++k) {
      const uint16_t* at = from[k];
      if (left < kTB) {
        const int row = row_of(k);
        if (row >= left) at -= int64_t(row - left + 1) * (step[k] / 2);
      }
      __builtin_amdgcn_global_load_lds((const void*)at, (lds_ptr_t)(buf + (k * NW + wv) * 1024), 16, 0, 0);
      from[k] += uint64_t(step[k]) * (kTB / 2);
    }
  };

  __syncthreads();
  if (c0 < c1) copy_stage(c0, lds);
  for (int c = c0; c < c1; ++c) {
    char* buf = lds + ((c - c0) & 1) * S::kStageB;
    const int j0 = t.lo + c * kTB, live = t.hi - j0;  // rows of the stage
    if (live < kTB) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll 1
      for (int k = 0; k < kCopies - kKeyCopies; ++k) {
        const int at = k * S::kThreads + tid;
        if (at / S::kVC >= live) *reinterpret_cast<u32x4*>(buf + S::kV + at * 16) = u32x4{0u, 0u, 0u, 0u};
      }
    }
    wait_all_barrier();
    if (c + 1 < c1) copy_stage(c + 1, lds + ((c - c0 + 1) & 1) * S::kStageB);
    // nothing of it is seen by this wave's tokens; whether the tile's tokens see different rows of it
    const bool skip = wn <= 0 || j0 > w_max || (a.rq.window > 0 && j0 + kTB <= w_min - a.rq.window + 1);
    const bool t_differ = t.tokens > 1 && (j0 + kTB - 1 > t_min || (a.rq.window > 0 && j0 <= t_min + t.tokens - 1 - a.rq.window));

    f32x4 s[kTB / 16][RB];
    u32x4 p[kTB / 32][RB];
    if (!skip) {
    // ---- scores
#pragma unroll
    for (int tb = 0; tb < kTB / 16; ++tb)
#pragma unroll
      for (int mb = 0; mb < RB; ++mb) s[tb][mb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // (a step's keys are read one step before its products: 128 cycles of this wave, and as many of its neighbour's)
    auto key = [&](int kb, int tb) {
      return *reinterpret_cast<const u32x4*>(buf + (key_at ^ (kb % S::kKeyTurn * 64)) + kb / S::kKeyTurn * S::kKeyTurn * 64 + tb * 16 * S::kKC * 16);
    };
    u32x4 kf[2][kTB / 16];
#pragma unroll
    for (int tb = 0; tb < kTB / 16; ++tb) kf[0][tb] = key(0, tb);
#pragma unroll
    for (int kb = 0; kb < S::kKB; ++kb) {
      if (kb + 1 < S::kKB)
#pragma unroll
        for (int tb = 0; tb < kTB / 16; ++tb) kf[(kb + 1) & 1][tb] = key(kb + 1, tb);
      if (kb < HD / 32 + 1 || rkb == 2)
#pragma unroll
        for (int tb = 0; tb < kTB / 16; ++tb)
#pragma unroll
          for (int mb = 0; mb < RB; ++mb) s[tb][mb] = mfma16x16x32(kf[kb & 1][tb], qf[mb][kb], s[tb][mb]);
      __builtin_amdgcn_sched_barrier(0);
    }
    const bool differ = j0 + kTB - 1 > w_min || (a.rq.window > 0 && j0 <= w_max - a.rq.window);
    if (live < kTB || differ || wn < RB * 16) {
#pragma unroll
      for (int tb = 0; tb < kTB / 16; ++tb)
#pragma unroll
        for (int mb = 0; mb < RB; ++mb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = j0 + tb * 16 + 4 * g + e;
            const bool seen = row < t.hi && row <= qrow[mb] && (a.rq.window <= 0 || row > qrow[mb] - a.rq.window);
            s[tb][mb][e] = seen ? s[tb][mb][e] : -kInf;
          }
    }
    // ---- softmax
    float m_new[RB];
    bool grow = false;
#pragma unroll
    for (int mb = 0; mb < RB; ++mb) {
      float m = -kInf;
#pragma unroll
      for (int tb = 0; tb < kTB / 16; ++tb)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = fmaxf(m, s[tb][mb][e]);
      m = quad_max(m) * a.scale_log2;  // (the scale is positive: its sign is in the queries)
      m_new[mb] = m;
      grow |= m > m_run[mb] + kGrow;
    }
    if (__any(grow)) {
#pragma unroll
      for (int mb = 0; mb < RB; ++mb) {
        const float m = fmaxf(m_run[mb], m_new[mb]);
        const float alpha = m == -kInf ? 1.0f : __builtin_amdgcn_exp2f(m_run[mb] - m);
        m_run[mb] = m;
        l_own[mb] *= alpha;
#pragma unroll
        for (int fb = 0; fb < HD / 16; ++fb) acc[fb][mb] *= alpha;
      }
    }
#pragma unroll
    for (int mb = 0; mb < RB; ++mb) {
      const float ref = m_run[mb] == -kInf ? 0.0f : m_run[mb];
#pragma unroll
      for (int tb = 0; tb < kTB / 16; ++tb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[tb][mb][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[tb][mb][e], a.scale_log2, -ref));
          l_own[mb] += s[tb][mb][e];
        }
        p[tb >> 1][mb][(tb & 1) * 2] = pack_bf16x2(s[tb][mb][0], s[tb][mb][1]);
        p[tb >> 1][mb][(tb & 1) * 2 + 1] = pack_bf16x2(s[tb][mb][2], s[tb][mb][3]);
      }
    }
    }
    // ---- values that are not finite, where the tile's tokens see different rows: added row by row where they are
    // seen, and zeros for the product
    char* vb = buf + S::kV;
    if (t_differ) {
      for (int half = 0; half < 2; ++half) {
        uint32_t odd = 0;
        for (int k = tid; k < 32 * S::kVC; k += S::kThreads)
          if (any_not_finite(*reinterpret_cast<const u32x4*>(vb + (half * 32 * S::kVC + k) * 16))) odd |= 1u << (k / S::kVC);
        odd = any_rows(odd, tmp);
        if (__builtin_expect(odd == 0, 1)) continue;
#pragma unroll 1
        for (uint32_t left = skip ? 0 : odd; left != 0; left &= left - 1) {
          const int row = half * 32 + __builtin_ctz(left), at = j0 + row;
#pragma unroll
          for (int mb = 0; mb < RB; ++mb) {
            float w = 0.0f;
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if ((row >> 4) * 4 + (row & 3) == k) w = s[k >> 2][mb][k & 3];
            w = __shfl(w, ((row >> 2) & 3) * 16 + i16, kWave);
            const bool seen = at < t.hi && at <= qrow[mb] && (a.rq.window <= 0 || at > qrow[mb] - a.rq.window);
#pragma unroll
            for (int fb = 0; fb < HD / 16; ++fb) {
              const u32x2 v = *reinterpret_cast<const u32x2*>(vb + row * S::kVC * 16 + ((fb * 2 + (g >> 1)) ^ value_swizzle<S::kVC>(row)) * 16 + (g & 1) * 8);
              acc[fb][mb][0] += seen ? w * bf16_lo(v.x) : 0.0f;
              acc[fb][mb][1] += seen ? w * bf16_hi(v.x) : 0.0f;
              acc[fb][mb][2] += seen ? w * bf16_lo(v.y) : 0.0f;
              acc[fb][mb][3] += seen ? w * bf16_hi(v.y) : 0.0f;
            }
          }
        }
        wait_lds_barrier();
        for (int k = tid; k < 32 * S::kVC; k += S::kThreads)
          if ((odd >> (k / S::kVC)) & 1) *reinterpret_cast<u32x4*>(vb + (half * 32 * S::kVC + k) * 16) = u32x4{0u, 0u, 0u, 0u};
        wait_lds_barrier();
      }
    }
    if (skip) continue;
    // ---- values
    auto value = [&](int k) {  // rows 32 (k / (HD / 16)) .., features 16 (k % (HD / 16)) ..
      const int fb = k % (HD / 16);
      const char* at = vb + (value_at ^ (fb % S::kValueTurn * 32)) + fb / S::kValueTurn * S::kValueTurn * 32 + k / (HD / 16) * 32 * S::kVC * 16;
      const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)at));
      const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)(at + 16 * S::kVC * 16)));
      return u32x4{lo.x, lo.y, hi.x, hi.y};
    };
    constexpr int kDeep = 5, kSteps = kTB / 32 * (HD / 16);
    u32x4 vf[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep - 1; ++k) vf[k] = value(k);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      if (k + kDeep - 1 < kSteps) vf[(k + kDeep - 1) % kDeep] = value(k + kDeep - 1);
#pragma unroll
      for (int mb = 0; mb < RB; ++mb)
        acc[k % (HD / 16)][mb] = mfma16x16x32(vf[k % kDeep], p[k / (HD / 16)][mb], acc[k % (HD / 16)][mb]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // ---- outputs, or a part: [part, token, head, HD + 2] fp32 with the maximum and the sum at the end
#pragma unroll
  for (int mb = 0; mb < RB; ++mb) {
    const float l = quad_sum(l_own[mb]);
    const int tok = (wv * RB + mb) * 16 + i16;
    if (tok >= t.tokens) continue;
    const int64_t token = t.s.first + t.t0 + tok;
    if (a.parts == 1) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      uint16_t* out = a.out + token * a.out_stride + head * HD + 4 * g;
#pragma unroll
      for (int fb = 0; fb < HD / 16; ++fb)
        *reinterpret_cast<u32x2*>(out + fb * 16) = u32x2{pack_bf16x2(acc[fb][mb][0] * inv, acc[fb][mb][1] * inv),
                                                         pack_bf16x2(acc[fb][mb][2] * inv, acc[fb][mb][3] * inv)};
      if (a.lse != nullptr && g == 0)
        a.lse[token * a.heads + head] = l == 0.0f ? -kInf : (m_run[mb] + __builtin_amdgcn_logf(l)) * 0.69314718f;
    } else {
      const int64_t rows = int64_t(a.rq.n_tokens) * a.heads, row = token * a.heads + head;
      float* to = a.workspace + (part * rows + row) * HD + 4 * g;
#pragma unroll
      for (int fb = 0; fb < HD / 16; ++fb) *reinterpret_cast<f32x4*>(to + fb * 16) = acc[fb][mb];
      if (g == 0) *reinterpret_cast<f32x2*>(a.workspace + a.parts * rows * HD + (part * rows + row) * 2) = f32x2{m_run[mb], l};
    }
  }
}

// Adds a tile's parts in order: a workgroup takes 16 tokens of a tile, a wave one at a time.  Lane p has part p's maximum
// and sum (at most 32 parts).
template <int HD, int M>
__global__ __launch_bounds__(256) void k_expanded_join(ExpandedArgs a) {
  __shared__ int64_t tmp[4 + 2];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int tile = int(blockIdx.x % a.tiles), head = int(blockIdx.x / a.tiles);
  Tile t;
  if (!find_tile<256, M>(a, tile, tmp, &t)) return;
  constexpr int kPer = HD / 64;
  typedef float vec __attribute__((ext_vector_type(kPer)));
  const int64_t rows = int64_t(a.rq.n_tokens) * a.heads;
  const int last = blockIdx.y * 16 + 16 < t.tokens ? blockIdx.y * 16 + 16 : t.tokens;
  for (int tok = blockIdx.y * 16 + wv; tok < last; tok += 4) {
    const int64_t token = t.s.first + t.t0 + tok, row = token * a.heads + head;
    float m = -kInf, l = 0.0f;
    if (lane < a.parts) {
      const f32x2 ml = *reinterpret_cast<const f32x2*>(a.workspace + a.parts * rows * HD + (lane * rows + row) * 2);
      m = ml.x;
      l = ml.y;
    }
    float top = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, kWave));
    top = __shfl(top, 0, kWave);
    const float f = __builtin_amdgcn_exp2f(m - (top == -kInf ? 0.0f : top));
    l *= f;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) l += __shfl_xor(l, o, kWave);
    l = __shfl(l, 0, kWave);
    vec v = {};
    const float* from = a.workspace + row * HD + lane * kPer;
    for (int p0 = 0; p0 < a.parts; p0 += 8) {  // (indexes past the last part repeat it, unused)
      vec part[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) part[k] = *reinterpret_cast<const vec*>(from + (p0 + k < a.parts ? p0 + k : a.parts - 1) * rows * HD);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), p0 + k));
        if (p0 + k < a.parts) v += w * part[k];
      }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t* out = a.out + token * a.out_stride + head * HD + lane * kPer;
    if constexpr (kPer == 2) *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(v[0] * inv, v[1] * inv);
    else *out = uint16_t(pack_bf16x2(v[0] * inv, 0.0f));
    if (a.lse != nullptr && lane == 0) a.lse[row] = l == 0.0f ? -kInf : (top + __builtin_amdgcn_logf(l)) * 0.69314718f;
  }
}

struct Choice {
  bool large;  // 256 tokens per tile, else 64
  int tiles, parts;
};
Choice choose(int64_t R, int64_t n_tokens, int64_t n_rows, int heads, int cus) {
  Choice c;
  // tiles of 256 where they fill the device or nearly all are whole
  c.large = n_tokens / 256 * heads >= cus || n_tokens / R >= 512;
  const int64_t M = c.large ? 256 : 64, some = R < n_tokens ? R : n_tokens;
  c.tiles = int(n_tokens / M + some);
  const int64_t tiles = (n_tokens + M * some - 1) / (M * some) * some * heads, stages = n_rows / R / kTB;
  int64_t parts = tiles >= cus ? 1 : (2 * cus + tiles - 1) / tiles;
  parts = parts < stages / 4 ? parts : stages / 4;
  c.parts = int(parts < 1 ? 1 : (parts > 32 ? 32 : parts));
  return c;
}

template <int HD, int NW, int RB>
hipError_t run(const ExpandedArgs& a, hipStream_t stream) {
  using S = Shape<HD, NW, RB>;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_expanded<HD, NW, RB>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e != hipSuccess) return e;
  const dim3 block(S::kThreads);
  k_expanded<HD, NW, RB><<<dim3(uint32_t(a.tiles) * a.heads * a.parts), block, S::kBytes, stream>>>(a);
  if (a.parts > 1) k_expanded_join<HD, S::M><<<dim3(uint32_t(a.tiles) * a.heads, S::M / 16), dim3(256), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

int64_t expanded_workspace_bytes(int64_t R, int64_t n_tokens, int64_t n_rows, int heads, int head_dim, int cus) {
  const Choice c = choose(R, n_tokens, n_rows, heads, cus);
  return c.parts > 1 ? int64_t(c.parts) * n_tokens * heads * (head_dim + 2) * 4 : 0;
}

hipError_t launch_latent_expanded(ExpandedArgs a, int cus, hipStream_t stream) {
  const Choice c = choose(a.rq.R, a.rq.n_tokens, a.n_rows, a.heads, cus);
  a.tiles = c.tiles;
  a.parts = c.parts;
  if (a.head_dim == 128) return c.large ? run<128, 8, 2>(a, stream) : run<128, 4, 1>(a, stream);
  return c.large ? run<64, 8, 2>(a, stream) : run<64, 4, 1>(a, stream);
}

}  // namespace engram
