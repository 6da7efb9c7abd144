// Expanded latent attention: per head, keys (kv part, shared rope part) and values (kv part) of each row.
//
// A workgroup takes M = 16 RB NW tokens of one request and one head; each of its NW waves holds the queries of
// 16 RB tokens in registers.  Keys and values come through LDS in stages of 64 rows, copied straight from
// memory.  S^T = K Q^T leaves a lane with 4 consecutive keys of one query, which is an operand
// of out^T += V^T P^T as it stands if the keys of that product are counted in the same order: the weights never
// leave the registers, and a query's maximum and sum are shared by 4 lanes of one wave.  Values are read
// transposed (ds_read_tr16).  The softmax is in the base 2; its reference is set 2^16 above the maximum and
// moves when it is passed.  The weights are rounded to bf16 for the second product, their sum is of the unrounded ones.
//
// Large tiles: eight waves, two on each SIMD, the second four half a stage behind (a barrier after each half), so that one of
// a SIMD's two is at its products while the other is at its softmax: 8192 tokens by 64 heads of 128 features take 1.43 ms
// in a trace (1.64 with all eight in step), 1.27 ms or 1.09 PFLOP/s in long rows of calls.  With neither softmax, copies nor
// reads of LDS the products alone take 1.04 (in a trace): they run at the power limit.
//
// Where few tiles meet many rows, each tile's stages are shared out in parts; their fp32 sums go to the workspace
// and k_expanded_join adds them in order.
//
// Rows past the last stay zeros in LDS; where a stage holds a value that is not finite and tokens see different
// rows of it, the product is taken row by row, only where it is seen (0 times infinity would not be 0).
#include <type_traits>

#include "latent_units.h"

namespace engram {

namespace {

constexpr int kTB = 64;

template <int HD, int NW, int RB>
struct Shape {
  static constexpr int kThreads = NW * kWave, M = 16 * RB * NW;
  // a stage in LDS: the rows' own parts of the keys, their rope parts (64 places), and their values
  static constexpr int kChunks = HD / 8;  // 16-byte chunks of a row's own part of a key, and of its value
  static constexpr int kRowB = HD * 2;
  static constexpr int kKB = (HD + 64) / 32;
  static constexpr int kRope = kTB * kRowB, kV = kRope + kTB * 128;  // offsets
  static constexpr int kStageB = kV + kTB * kRowB;
  static constexpr int kTurn = kChunks / 2;  // 16-feature blocks of a value among which a swizzle moves a pair of chunks
  // Eight waves: two on each SIMD, and the second four are half a stage behind, so that one of a SIMD's two is at its
  // products while the other is at its softmax.
  static constexpr bool kTurns = NW == 8;
  static constexpr int kBuffers = kTurns ? 3 : 2;
  static constexpr int kBytes = kBuffers * kStageB;
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
__global__ __launch_bounds__(NW* kWave, 2) void k_expanded(ExpandedArgs a) {
  using S = Shape<HD, NW, RB>;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ int64_t tmp[NW + 2];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int rkb = a.rope_dim / 32;
  // pairs of heads, then tiles (the last, which sees the most, first), then the pair's heads, then parts: neighbours share
  // rows in their L2
  uint32_t id = in_order(blockIdx.x, gridDim.x);
  const int part = int(id % a.parts);
  id /= a.parts;
  const int pair = int(id / (2 * a.tiles)), in = int(id - pair * 2 * a.tiles), of = pair * 2 + 1 < a.heads ? 2 : 1;
  const int head = pair * 2 + in % of;
  Tile t;
  if (!find_tile<S::kThreads, S::M>(a, a.tiles - 1 - in / of, tmp, &t)) return;
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

  // (a swizzle changes bits of a chunk's number, so a row's chunks are one xor away from the first)
  const int key_at = i16 * S::kRowB + (g ^ key_swizzle<S::kChunks>(i16)) * 16;
  const int rope_at = S::kRope + i16 * 128 + (g ^ key_swizzle<8>(i16)) * 16;
  const int vrow = 4 * g + (i16 >> 2);
  const int value_at = S::kV + vrow * S::kRowB + (((i16 & 3) >> 1) ^ value_swizzle<S::kChunks>(vrow)) * 16 + (i16 & 1) * 8;

  f32x4 acc[HD / 16][RB];
  float m_run[RB], l_own[RB];
#pragma unroll
  for (int mb = 0; mb < RB; ++mb) {
    m_run[mb] = -kInf;
    l_own[mb] = 0.0f;
#pragma unroll
    for (int fb = 0; fb < HD / 16; ++fb) acc[fb][mb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  // Copies, by four of the waves: 16 bytes a lane in the order of the buffer, a few whole rows by each.  A lane's place from a
  // copy's first row on is the same in all copies of a kind, which go through the rows in order, stage after stage.
  // Only the last stage may have fewer rows: its last one is repeated.
  constexpr int kPer = 64 / S::kChunks;  // rows of a copy
  constexpr int kOwn = kTB / (kPer * 4), kRopes = kTB / (8 * 4), kCopies = 2 * kOwn + kRopes;
  static_assert(kPer * 4 % 16 == 0, "the same swizzles in all copies of a wave");
  const bool late = S::kTurns && wv >= 4;
  const int cw = S::kTurns ? wv - 4 : wv, row_l = lane / S::kChunks, rope_l = lane >> 3;
  const int rope_ch = (lane & 7) ^ key_swizzle<8>(cw * 8 + rope_l);
  const uint32_t kv_step = uint32_t(a.kv_stride) * 2, rope_step = uint32_t(a.rope_stride) * 2;  // bytes from row to row
  const uint32_t key_off = row_l * kv_step + (lane % S::kChunks ^ key_swizzle<S::kChunks>(cw * kPer + row_l)) * 16;
  const uint32_t value_off = row_l * kv_step + (HD / 8 + (lane % S::kChunks ^ value_swizzle<S::kChunks>(cw * kPer + row_l))) * 16;
  const uint32_t rope_off = rope_l * rope_step + (rope_ch < 4 * rkb ? rope_ch : 0) * 16;
  const int64_t first_copied = t.first_row + t.lo + c0 * kTB;
  const char* kv_from = reinterpret_cast<const char*>(a.kv + head * 2 * HD + (first_copied + cw * kPer) * a.kv_stride);
  const char* rope_from = reinterpret_cast<const char*>(a.rope + (first_copied + cw * 8) * a.rope_stride);
  const uint32_t to = lds_address(lds) + cw * 1024;
  auto copy_stage = [&](int c, uint32_t buf) {
    const int left = t.hi - (t.lo + c * kTB);
    auto copy = [&](int n, bool rope, uint32_t off, uint32_t at) {
      const char* from = rope ? rope_from : kv_from;
      if (left < kTB) {
        const int row = (n * 4 + cw) * (rope ? 8 : kPer), back = row < left ? 0 : row - (left - 1);
        const int over = (rope ? rope_l : row_l) - (left - 1 - (row - back));
        const uint32_t step = rope ? rope_step : kv_step;
        if (over > 0) off -= over * step;
        from -= int64_t(back) * step;
      }
      copy_to_lds(from, off, to + buf + at + n * 4096);
    };
#pragma unroll
    for (int n = 0; n < kOwn; ++n) {
      copy(n, false, key_off, 0);
      copy(n, false, value_off, S::kV);
      kv_from += uint64_t(kv_step) * (4 * kPer);
    }
#pragma unroll
    for (int n = 0; n < kRopes; ++n) {
      copy(n, true, rope_off, S::kRope);
      rope_from += uint64_t(rope_step) * 32;
    }
  };
  // This lane's copies of stage c are there; its values past the last row are made zeros.
  auto arrive = [&](int c, char* buf) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const int live = t.hi - (t.lo + c * kTB);
    if (live < kTB) {
#pragma unroll 1
      for (int k = 0; k < kOwn; ++k) {
        const int at = (k * 4 + cw) * kWave + lane;
        if (at / S::kChunks >= live) *reinterpret_cast<u32x4*>(buf + S::kV + at * 16) = u32x4{0u, 0u, 0u, 0u};
      }
    }
  };
  // Rows of stage c with values that are not finite, looked for where the tile's tokens see different rows.
  auto scan = [&](int c, const char* buf) {
    const int j0 = t.lo + c * kTB;
    if (!(t.tokens > 1 && (j0 + kTB - 1 > t_min || (a.rq.window > 0 && j0 <= t_min + t.tokens - 1 - a.rq.window)))) return uint64_t{0};
    uint64_t mine = 0;
#pragma unroll 1
    for (int k = tid; k < kTB * S::kChunks; k += S::kThreads)
      if (any_not_finite(*reinterpret_cast<const u32x4*>(buf + S::kV + k * 16))) mine |= uint64_t{1} << (k / S::kChunks);
    return any_rows(mine, tmp);
  };
  auto clear = [&](char* buf, uint64_t odd) {  // those rows, once every wave has added what it sees of them
    wait_lds_barrier();
#pragma unroll 1
    for (int k = tid; k < kTB * S::kChunks; k += S::kThreads)
      if ((odd >> (k / S::kChunks)) & 1) *reinterpret_cast<u32x4*>(buf + S::kV + k * 16) = u32x4{0u, 0u, 0u, 0u};
    wait_lds_barrier();
  };
  auto unseen = [&](int c) {  // by all of this wave's tokens
    const int j0 = t.lo + c * kTB;
    return wn <= 0 || j0 > w_max || (a.rq.window > 0 && j0 + kTB <= w_min - a.rq.window + 1);
  };

  f32x4 s[kTB / 16][RB];
  u32x4 p[kTB / 32][RB];
  // out += values (of vbuf) by the weights, and scores = keys (of kbuf) by the queries, as one run of operands of RB
  // products each, read kDeep - 1 operands ahead.
  constexpr int kValueSteps = kTB / 32 * (HD / 16), kKeySteps = S::kKB * (kTB / 16);
  auto products = [&](auto with_values, auto with_keys, const char* vbuf, const char* kbuf) {
    constexpr int kFirst = with_values ? kValueSteps : 0, kSteps = kFirst + (with_keys ? kKeySteps : 0);
    auto read = [&](int k) {
      if (k < kFirst) {  // rows 32 (k / (HD / 16)) .., features 16 (k % (HD / 16)) ..
        const int fb = k % (HD / 16);
        const char* at = vbuf + (value_at ^ (fb % S::kTurn * 32)) + fb / S::kTurn * S::kTurn * 32 + k / (HD / 16) * 32 * S::kRowB;
        const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)at));
        const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)(at + 16 * S::kRowB)));
        return u32x4{lo.x, lo.y, hi.x, hi.y};
      }
      const int kb = (k - kFirst) / (kTB / 16), tb = (k - kFirst) % (kTB / 16);
      if (kb < HD / 32) return *reinterpret_cast<const u32x4*>(kbuf + (key_at ^ (kb * 64)) + tb * 16 * S::kRowB);
      return *reinterpret_cast<const u32x4*>(kbuf + (rope_at ^ ((kb - HD / 32) * 64)) + tb * 16 * 128);
    };
    constexpr int kDeep = S::kTurns ? 9 : 5;
    u32x4 f[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep - 1; ++k) f[k] = read(k);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      if (k + kDeep - 1 < kSteps) f[(k + kDeep - 1) % kDeep] = read(k + kDeep - 1);
      if (k < kFirst) {
#pragma unroll
        for (int mb = 0; mb < RB; ++mb)
          acc[k % (HD / 16)][mb] = mfma16x16x32(f[k % kDeep], p[k / (HD / 16)][mb], acc[k % (HD / 16)][mb]);
      } else {
        const int kb = (k - kFirst) / (kTB / 16), tb = (k - kFirst) % (kTB / 16);
        if (kb < HD / 32 + 1 || rkb == 2)
#pragma unroll
          for (int mb = 0; mb < RB; ++mb) s[tb][mb] = mfma16x16x32(f[k % kDeep], qf[mb][kb], kb == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : s[tb][mb]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto mask = [&](int c) {
    const int j0 = t.lo + c * kTB;
    const bool differ = j0 + kTB - 1 > w_min || (a.rq.window > 0 && j0 <= w_max - a.rq.window);
    if (t.hi - j0 < kTB || differ || wn < RB * 16) {
#pragma unroll
      for (int mb = 0; mb < RB; ++mb) {
        // rows first .. first + n - 1 are seen, of rows from 0 on
        const int first = a.rq.window > 0 && qrow[mb] >= a.rq.window ? qrow[mb] - a.rq.window + 1 : 0;
        const int end = qrow[mb] + 1 < t.hi ? qrow[mb] + 1 : t.hi, n = end > first ? end - first : 0;
        const int at = j0 + 4 * g - first;
#pragma unroll
        for (int tb = 0; tb < kTB / 16; ++tb)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[tb][mb][e] = uint32_t(at + tb * 16 + e) < uint32_t(n) ? s[tb][mb][e] : -kInf;
      }
    }
  };
  bool big = false;  // any of the references
  auto softmax = [&]() {
    float m_new[RB];
    bool grow = false;
#pragma unroll
    for (int mb = 0; mb < RB; ++mb) {
      float m = -kInf;
#pragma unroll
      for (int tb = 0; tb < kTB / 16; ++tb)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = fmaxf(m, s[tb][mb][e]);
      m = rounded_product(quad_max(m), a.scale_log2);  // (the scale is positive: its sign is in the queries)
      m_new[mb] = m;
      grow |= m > m_run[mb];
    }
    if (__any(grow)) {
      bool high = false;
#pragma unroll
      for (int mb = 0; mb < RB; ++mb) {
        const float m = moved_reference(m_run[mb], m_new[mb]);
        const float alpha = m == -kInf ? 1.0f : __builtin_amdgcn_exp2f(m_run[mb] - m);
        m_run[mb] = m;
        l_own[mb] *= alpha;
#pragma unroll
        for (int fb = 0; fb < HD / 16; ++fb) acc[fb][mb] *= alpha;
        high |= m != -kInf && !(__builtin_fabsf(m) < kBigScore);
      }
      big = __any(high);
    }
    float scale = a.scale_log2;
    if (__builtin_expect(big, 0)) {
#pragma unroll
      for (int mb = 0; mb < RB; ++mb)
#pragma unroll
        for (int tb = 0; tb < kTB / 16; ++tb)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[tb][mb][e] = rounded_product(s[tb][mb][e], scale);
      scale = 1.0f;
    }
#pragma unroll
    for (int mb = 0; mb < RB; ++mb) {
      const float ref = m_run[mb] == -kInf ? 0.0f : m_run[mb];
#pragma unroll
      for (int tb = 0; tb < kTB / 16; ++tb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[tb][mb][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[tb][mb][e], scale, -ref));
          l_own[mb] += s[tb][mb][e];
        }
        p[tb >> 1][mb][(tb & 1) * 2] = pack_bf16x2(s[tb][mb][0], s[tb][mb][1]);
        p[tb >> 1][mb][(tb & 1) * 2 + 1] = pack_bf16x2(s[tb][mb][2], s[tb][mb][3]);
      }
    }
  };
  // Rows that are not finite, one by one where they are seen.
  auto add_odd = [&](int c, const char* buf, uint64_t odd) {
#pragma unroll 1
    for (uint64_t left = odd; left != 0; left &= left - 1) {
      const int row = __builtin_ctzll(left), at = t.lo + c * kTB + row;
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
          const u32x2 v = *reinterpret_cast<const u32x2*>(buf + S::kV + row * S::kRowB + ((fb * 2 + (g >> 1)) ^ value_swizzle<S::kChunks>(row)) * 16 + (g & 1) * 8);
          acc[fb][mb][0] += seen ? w * bf16_lo(v.x) : 0.0f;
          acc[fb][mb][1] += seen ? w * bf16_hi(v.x) : 0.0f;
          acc[fb][mb][2] += seen ? w * bf16_lo(v.y) : 0.0f;
          acc[fb][mb][3] += seen ? w * bf16_hi(v.y) : 0.0f;
        }
      }
    }
  };
  constexpr auto yes = std::true_type{};
  constexpr auto no = std::false_type{};

  __syncthreads();
  if constexpr (S::kTurns) {
    // Phases, a barrier after each: in phase 2c the first four waves are at the products (values of stage c - 1, scores of
    // stage c) and the others at the softmax of c - 1; in phase 2c + 1 the other way round.  A stage is read in the phases
    // 2c .. 2c + 3, and stage c + 3 is copied to its place in phase 2c + 4 by the waves at the softmax.  The stages
    // [plain0, plain1) are whole and seen by all tokens of the tile.
    const int plain0 = a.rq.window > 0 ? (t_min + t.tokens - 1 - a.rq.window - t.lo + kTB) / kTB : 0;
    const int plain1 = t.tokens < S::M ? 0 : ((t_min + 1 < t.hi ? t_min + 1 : t.hi) - t.lo) / kTB;
    auto plain = [&](int c) { return c >= plain0 && c < plain1; };
    uint64_t odd = 0, odd_next = 0;
    bool saw = false;  // this wave's tokens, something of the stage before
    int buf = 0, next = S::kStageB, last = 2 * S::kStageB;
    if (c0 < c1) {
      // (before the first stage: weights of zero and values of zero)
      for (int k = tid; k < kTB * S::kChunks; k += S::kThreads) *reinterpret_cast<u32x4*>(lds + last + S::kV + k * 16) = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int kb = 0; kb < kTB / 32; ++kb)
#pragma unroll
        for (int mb = 0; mb < RB; ++mb) p[kb][mb] = u32x4{0u, 0u, 0u, 0u};
      if (late) {
        copy_stage(c0, buf);
        arrive(c0, lds + buf);
      }
      wait_lds_barrier();
      if (late) {
        if (c0 + 1 < c1) copy_stage(c0 + 1, next);
        odd = scan(c0, lds + buf);
        wait_lds_barrier();
      }
      for (int c = c0; c < c1; ++c) {
        const int after = next + S::kStageB < S::kBytes ? next + S::kStageB : 0;
        const bool more = c + 1 < c1;
        if (!late) {
          if (!plain(c)) odd_next = scan(c, lds + buf);
          if (odd != 0) clear(lds + last, odd);
          odd = odd_next;
          odd_next = 0;
        }
        const bool sees = plain(c) || !unseen(c);
        if (sees || saw) {
          __builtin_amdgcn_s_setprio(1);
          products(yes, yes, lds + last, lds + buf);
          __builtin_amdgcn_s_setprio(0);
        }
        saw = sees;
        if (!plain(c)) mask(c);
        if (late && more) arrive(c + 1, lds + next);
        wait_lds_barrier();
        if (late) {
          odd_next = more && !plain(c + 1) ? scan(c + 1, lds + next) : 0;
          if (c + 2 < c1) copy_stage(c + 2, after);
        }
        if (sees) {
          softmax();
        } else {
#pragma unroll
          for (int kb = 0; kb < kTB / 32; ++kb)
#pragma unroll
            for (int mb = 0; mb < RB; ++mb) p[kb][mb] = u32x4{0u, 0u, 0u, 0u};
        }
        if (odd != 0) add_odd(c, lds + buf, odd);
        if (late) {
          if (odd != 0) clear(lds + buf, odd);
          odd = odd_next;
        }
        wait_lds_barrier();
        last = buf;
        buf = next;
        next = after;
      }
      if (!late && odd != 0) clear(lds + last, odd);
      if (saw) products(yes, no, lds + last, lds + last);
      if (!late) wait_lds_barrier();
    }
  } else {
    if (c0 < c1) copy_stage(c0, 0);
    for (int c = c0; c < c1; ++c) {
      const int at = ((c - c0) & 1) * S::kStageB;
      char* buf = lds + at;
      arrive(c, buf);
      wait_lds_barrier();
      if (c + 1 < c1) copy_stage(c + 1, S::kStageB - at);
      const bool skip = unseen(c);
      if (!skip) {
        products(no, yes, buf, buf);
        mask(c);
        softmax();
      }
      const uint64_t odd = scan(c, buf);
      if (odd != 0) {
        if (!skip) add_odd(c, buf, odd);
        clear(buf, odd);
      }
      if (!skip) products(yes, no, buf, buf);
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
// With 128 features a token costs 1.5 times as much in a tile of 64 as in one of 256 (12 prompts of 1500 tokens behind 2000,
// 20 heads, window 1000: 645 us and 430 us), so tiles of 256 are taken where they are no emptier than that, counted by the
// mean request (16 of 37 tokens behind 1000, 128 heads: 304 us with tiles of 256, 96 us with 64), and where there are two a
// CU or parts of ten stages and more (one prompt of 2048 tokens, 16 heads: 78 us and 54 us; 512 tokens behind 7680:
// 94 us and 100 us).  With 64 features they gain less, and from 2048 tokens on (2048 behind 6144, 32 heads: 212 us and
// 262 us; four of 1000 behind 2000, 64 heads: 357 us and 254 us).
Choice choose(int64_t R, int64_t n_tokens, int64_t n_rows, int heads, int head_dim, int cus) {
  const int64_t some = R < n_tokens ? R : n_tokens, mean = (n_tokens + some - 1) / some, stages = n_rows / R / kTB;
  auto with = [&](int64_t M) {
    const int64_t tiles = (mean + M - 1) / M * some * heads;
    int64_t parts = tiles >= cus ? 1 : (2 * cus + tiles - 1) / tiles;
    parts = parts < stages / 4 ? parts : stages / 4;
    return Choice{M == 256, int(n_tokens / M + some), int(parts < 1 ? 1 : (parts > 32 ? 32 : parts))};
  };
  const int64_t room = (mean + 255) / 256 * 256;
  const Choice c = with(256);
  const bool full = head_dim == 128 ? 2 * room <= 3 * ((mean + 63) / 64 * 64) : mean >= 2048;
  if (full && (room / 256 * some * heads >= 2 * cus || stages >= 10 * c.parts)) return c;
  return with(64);
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
  const Choice c = choose(R, n_tokens, n_rows, heads, head_dim, cus);
  return c.parts > 1 ? int64_t(c.parts) * n_tokens * heads * (head_dim + 2) * 4 : 0;
}

// For all of 1 .. n_tokens tokens and 0 .. n_rows rows of any requests.  Parts are 32 at most, with four stages each at least,
// and (2 cus - 1) / tiles + 1 at most where there are fewer tiles than CUs; a call's rows (tokens times heads) are tiles of 256
// rows at most each.  So parts times rows are 256 (2 cus - 1 + tiles) at most, and tiles cus - 1.
int64_t expanded_workspace_bytes_up_to(int64_t n_tokens, int64_t n_rows, int heads, int head_dim, int cus) {
  int64_t parts = n_rows / kTB / 4;
  if (parts < 2) return 0;
  if (parts > 32) parts = 32;
  const int64_t rows = parts * n_tokens * heads, most = int64_t(256) * (3 * cus - 2);
  return (rows < most ? rows : most) * (head_dim + 2) * 4;
}

hipError_t launch_latent_expanded(ExpandedArgs a, int cus, hipStream_t stream) {
  const Choice c = choose(a.rq.R, a.rq.n_tokens, a.n_rows, a.heads, a.head_dim, cus);
  a.tiles = c.tiles;
  a.parts = c.parts;
  if (a.head_dim == 128) return c.large ? run<128, 8, 2>(a, stream) : run<128, 4, 1>(a, stream);
  return c.large ? run<64, 8, 2>(a, stream) : run<64, 4, 1>(a, stream);
}

}  // namespace engram
