// Absorbed latent attention over the pages: out = softmax(scale q (c, k)^T) c, one latent row c a position.
//
// A row of a tile is a (token, head) pair of one request, M = 16 MB rows to a tile; a tile goes over its
// positions in stages of 64 rows of the cache, which lie in LDS as bf16 (FP8 rows are converted on the way in,
// exactly), read twice: along the features for the scores, and transposed (ds_read_tr16) for the values.
//  scores   S^T = C Q^T: a wave takes 16 of the positions and keeps all queries in registers; a lane then holds 4
//           consecutive positions of one query.
//  softmax  running maximum and sum in the base 2; the waves share each stage's maxima through LDS; the
//           reference lies up to 2^16 above it, and moves when it is passed.
//  values   out^T += C^T P^T: a wave takes a quarter of the latent's features for every query; the weights
//           pass through LDS, rounded to bf16 for the product (their sum is of the unrounded ones), the order of
//           positions in the product being that of the score fragments.
//
// For 32 rows a request and fewer, where the cache's bytes are what costs: 128 requests of up to 8192 positions, 16 heads,
// BF16 rows of 512 + 64: 177 to 189 us by the device for 793 MB, 4.2 to 4.5 TB/s (62% of the waves' cycles wait, for
// memory: stages are copied one ahead).
//
// Work is shared out in units of one stage of one tile: workgroup w of G takes units [w U / G, (w + 1) U / G) of
// the step's U, whatever the requests' lengths, so every CU has the same share.  What a workgroup holds of a
// tile that it does not finish alone goes to the workspace (fp32 sums, maxima), and k_absorbed_join
// adds a tile's parts in order.
//
// Rows that take no part (outside the tile's positions, on a bad page) are zeros in LDS and their scores
// -infinity.  Where the tokens of a tile see different positions, a value that is not finite must not reach those that do
// not see it (0 times infinity): such stages are looked through, and rows with one added where they are seen, one by one.
#include "latent_units.h"

namespace engram {

namespace {

constexpr int kThreads = 256;
constexpr int kTB = 64;  // positions per stage

template <int DC, int MB>
struct Shape {
  static constexpr int M = 16 * MB;
  static constexpr int kChunks = (DC + 64) / 8, kRowB = kChunks * 16;  // of a row in LDS
  static constexpr int kKB = DC / 32;                                  // K blocks of the latent
  static constexpr int kFB = DC / 64;                                  // 16-feature blocks of a wave's quarter
  static constexpr int kStageB = kTB * kRowB;
  static constexpr int kP = 2 * kStageB;                               // offsets into LDS
  static constexpr int kMax = kP + M * kTB * 2;
  static constexpr int kSlots = kMax + 4 * M * 4;
  static constexpr int kAlive = kSlots + 4 * kTB * 8;
  static constexpr int kMisc = kAlive + 4 * 8;
  static constexpr int kBytes = kMisc + 64;
};

template <int DC, int MB, bool FP8>
__global__ __launch_bounds__(kThreads, DC == 128 ? 2 : 1) void k_absorbed(AbsorbedArgs a) {
  using S = Shape<DC, MB>;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int rkb = a.rope_dim / 32;
  const int row_b = latent_row_bytes(DC, a.rope_dim, FP8);
  int64_t* slots = reinterpret_cast<int64_t*>(lds + S::kSlots);
  uint64_t* alive = reinterpret_cast<uint64_t*>(lds + S::kAlive);
  float* smax = reinterpret_cast<float*>(lds + S::kMax);
  int64_t* misc = reinterpret_cast<int64_t*>(lds + S::kMisc);

  const PartSpace space = part_space(a.workspace, gridDim.x, S::M);
  // A chunk's place differs from row to row in the low three bits of its number only, so the reads of a stage take
  // two (keys) and four (values) addresses and constants.  (Rows start at multiples of 128 bytes.)
  const int key_at = (wv * 16 + i16) * S::kRowB + (g ^ latent_swizzle(i16)) * 16;
  const int vrow = 4 * g + (i16 >> 2);
  const int value_at = vrow * S::kRowB + ((wv * (DC / 32) + ((i16 & 3) >> 1)) ^ latent_swizzle(vrow)) * 16 + (i16 & 1) * 8;
  Units un;
  if (!my_units<kThreads, S::M, kTB>(a.rq, a.heads, space.parts, misc, &un)) return;

  while (un.u < un.u1) {
    const Segment t = segment_of<S::M, kTB>(a.rq, a.heads, un);
    const int c0 = t.c0, n = t.n;

    // ---- queries: fragments in registers, and the position of each row's token (-1: no row)
    u32x4 qf[MB][S::kKB + 2];
    int qpos[MB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const int row = t.row0 + mb * 16 + i16, at = row < t.rows ? row : t.rows - 1;  // (rows past the last repeat it)
      const int tok = at / a.heads, head = at - tok * a.heads;
      qpos[mb] = row < t.rows ? t.s.pos + tok : -1;
      const uint16_t* src = a.q + (t.s.first + tok) * a.q_stride + int64_t(head) * (DC + a.rope_dim) + 8 * g;
#pragma unroll
      for (int kb = 0; kb < S::kKB + 2; ++kb)
        qf[mb][kb] = *reinterpret_cast<const u32x4*>(src + 32 * (kb < S::kKB + rkb ? kb : 0)) ^ a.q_sign;
    }
    f32x4 acc[S::kFB][MB];
    float m_run[MB], l_own[MB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      m_run[mb] = -kInf;
#pragma unroll
      for (int fb = 0; fb < S::kFB; ++fb) acc[fb][mb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) l_own[mb] = 0.0f;

    // ---- staging
    auto find_slot = [&](int c) -> int64_t {  // (wave 0) slot of the lane's row of stage c
      const int pos = t.base + c * kTB + lane;
      if (c >= c0 + n || pos < t.lo || pos >= t.hi) return -1;
      const int64_t slot = slot_of(a.rq, un.r, pos);
      if (slot < 0 && pos >= t.fresh && a.err_count != nullptr) atomicAdd(a.err_count, 1);
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
        const int row = tid / kNP + k * (kThreads / kNP), sw = latent_swizzle(row);
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
          *reinterpret_cast<u32x4*>(buf + row * S::kRowB + ((DC / 8 + id % rp) ^ latent_swizzle(row)) * 16) =
              (on >> row) & 1 ? rope[k] : u32x4{0u, 0u, 0u, 0u};
      }
    };
    // BF16: straight into LDS, 16 bytes a lane in the order of the buffer
    auto copy_stage = [&](int c, char* buf) {
      const int64_t* sl = slots + (c & 3) * kTB;
#pragma unroll
      for (int k = 0; k < S::kChunks / 4; ++k) {
        const int id = (k * 4 + wv) * 64 + lane, row = id / S::kChunks;
        int ch = (id - row * S::kChunks) ^ latent_swizzle(row);
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
      f32x4 s[MB];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) s[mb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      {
        const char* kp[2] = {buf + key_at, buf + (key_at ^ 64)};
        auto key = [&](int kb) { return *reinterpret_cast<const u32x4*>(kp[kb & 1] + (kb >> 1) * 128); };
        constexpr int kDeep = 4;
        u32x4 kf[kDeep];
#pragma unroll
        for (int kb = 0; kb < kDeep - 1; ++kb) kf[kb] = key(kb);
#pragma unroll
        for (int kb = 0; kb < S::kKB + 2; ++kb) {
          if (kb + kDeep - 1 < S::kKB + 2) kf[(kb + kDeep - 1) % kDeep] = key(kb + kDeep - 1);
          if (kb == S::kKB + 1 && rkb == 1) continue;
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) s[mb] = mfma16x16x32(kf[kb % kDeep], qf[mb][kb], s[mb]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      const uint64_t on = alive[c & 3];
      const int j0 = t.base + c * kTB;
      const bool differ = t.p_min != t.p_max && (j0 + kTB - 1 > t.p_min || (a.rq.window > 0 && j0 <= t.p_max - a.rq.window));
      const bool edge = on != ~uint64_t(0) || differ;
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        float m = -kInf;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[mb][e] = rounded_product(s[mb][e], a.scale_log2);
          if (edge) {
            const int row = wv * 16 + 4 * g + e, pos = j0 + row;
            const bool seen = ((on >> row) & 1) && pos <= qpos[mb] && (a.rq.window <= 0 || pos > qpos[mb] - a.rq.window);
            s[mb][e] = seen ? s[mb][e] : -kInf;
          }
          m = fmaxf(m, s[mb][e]);
        }
        m = quad_max(m);
        if (g == 0) smax[wv * S::M + mb * 16 + i16] = m;
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
        for (int k = 1; k < 4; ++k) m = fmaxf(m, smax[k * S::M + mb * 16 + i16]);
        m_new[mb] = m;
        grow |= m > m_run[mb];
      }
      if (__any(grow)) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          const float m = moved_reference(m_run[mb], m_new[mb]);
          const float alpha = m == -kInf ? 1.0f : __builtin_amdgcn_exp2f(m_run[mb] - m);
          m_run[mb] = m;
#pragma unroll
          for (int fb = 0; fb < S::kFB; ++fb) acc[fb][mb] *= alpha;
          l_own[mb] *= alpha;
        }
      }
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const float ref = m_run[mb] == -kInf ? 0.0f : m_run[mb];
        const int row = mb * 16 + i16;
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = __builtin_amdgcn_exp2f(s[mb][e] - ref);
          l_own[mb] += p[e];
        }
        // (the wave's positions 16 wv + 4 g ..: half wv & 1 of K block wv / 2)
        *reinterpret_cast<u32x2*>(lds + S::kP + row * kTB * 2 + (((wv >> 1) * 4 + g) ^ ((row >> 1) & 7)) * 16 + (wv & 1) * 8) =
            u32x2{pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3])};
      }
      if constexpr (FP8) {
        if (j + 1 < n) store_stage(c + 1, next);
        if (j + 2 < n) load_stage(c + 2);
      }
      wait_lds_barrier();

      // ---- values that are not finite, where the tile's tokens see different positions: added row by row where they are
      // seen, and zeros for the product
      if (differ) {
        uint64_t odd = 0;
#pragma unroll 1
        for (int k = tid; k < kTB * DC / 8; k += kThreads) {
          const int row = k / (DC / 8);
          if (any_not_finite(*reinterpret_cast<const u32x4*>(buf + row * S::kRowB + k % (DC / 8) * 16))) odd |= uint64_t{1} << row;
        }
        odd = any_rows(odd, misc);
        if (__builtin_expect(odd != 0, 0)) {
#pragma unroll 1
          for (uint64_t left = odd; left != 0; left &= left - 1) {
            const int row = __builtin_ctzll(left), half = row >> 5, in = row & 31, pos = j0 + row;
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
              const int m = mb * 16 + i16, q = t.row0 + m, qp = q < t.rows ? t.s.pos + q / a.heads : -1;
              const bool seen = ((on >> row) & 1) && pos <= qp && (a.rq.window <= 0 || pos > qp - a.rq.window);
              const float w = bf16_lo(*reinterpret_cast<const uint16_t*>(
                  lds + S::kP + m * kTB * 2 + ((half * 4 + ((in >> 2) & 3)) ^ ((m >> 1) & 7)) * 16 + (in >> 4) * 8 + (in & 3) * 2));
#pragma unroll
              for (int fb = 0; fb < S::kFB; ++fb) {
                const int ch = wv * (DC / 32) + fb * 2 + (g >> 1);
                const u32x2 v = *reinterpret_cast<const u32x2*>(buf + row * S::kRowB + (ch ^ latent_swizzle(row)) * 16 + (g & 1) * 8);
                acc[fb][mb][0] += seen ? w * bf16_lo(v.x) : 0.0f;
                acc[fb][mb][1] += seen ? w * bf16_hi(v.x) : 0.0f;
                acc[fb][mb][2] += seen ? w * bf16_lo(v.y) : 0.0f;
                acc[fb][mb][3] += seen ? w * bf16_hi(v.y) : 0.0f;
              }
            }
          }
          wait_lds_barrier();
          for (int k = tid; k < kTB * DC / 8; k += kThreads)
            if ((odd >> (k / (DC / 8))) & 1) *reinterpret_cast<u32x4*>(buf + k / (DC / 8) * S::kRowB + k % (DC / 8) * 16) = u32x4{0u, 0u, 0u, 0u};
          wait_lds_barrier();
        }
      }

      // ---- values
      const char* vp[4] = {buf + value_at, buf + (value_at ^ 32), buf + (value_at ^ 64), buf + (value_at ^ 96)};
      auto value = [&](int k) {  // K block k / kFB, features k % kFB
        const int fb = k % S::kFB;
        const char* at = vp[fb & 3] + (fb >> 2) * 128 + k / S::kFB * 32 * S::kRowB;
        const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)at));
        const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)(at + 16 * S::kRowB)));
        return u32x4{lo.x, lo.y, hi.x, hi.y};
      };
      const char* pp = lds + S::kP + i16 * kTB * 2;
      const int p_at = (g ^ ((i16 >> 1) & 7)) * 16;  // (of the second K block: ^ 64)
      u32x4 p[2][MB];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) p[0][mb] = *reinterpret_cast<const u32x4*>(pp + mb * 16 * kTB * 2 + p_at);
      constexpr int kDeep = 4, kSteps = 2 * S::kFB;
      u32x4 vf[kDeep];
#pragma unroll
      for (int k = 0; k < kDeep - 1; ++k) vf[k] = value(k);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) p[1][mb] = *reinterpret_cast<const u32x4*>(pp + mb * 16 * kTB * 2 + (p_at ^ 64));
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        if (k + kDeep - 1 < kSteps) vf[(k + kDeep - 1) % kDeep] = value(k + kDeep - 1);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) acc[k % S::kFB][mb] = mfma16x16x32(vf[k % kDeep], p[k / S::kFB][mb], acc[k % S::kFB][mb]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }

    // ---- the sums of all positions, then the outputs or a part
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      const float l = quad_sum(l_own[mb]);
      if (g == 0) smax[wv * S::M + mb * 16 + i16] = l;
    }
    wait_lds_barrier();
    float l_all[MB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      l_all[mb] = smax[mb * 16 + i16];
#pragma unroll
      for (int k = 1; k < 4; ++k) l_all[mb] += smax[k * S::M + mb * 16 + i16];
    }
    if (c0 == 0 && n == t.stages) {
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
      const int64_t at = 2 * un.w + (c0 == 0 ? 1 : 0);
      f32x4* to = space.acc + at * (S::M * DC / 4) + wv * (S::kFB * MB * kWave) + lane;
#pragma unroll
      for (int fb = 0; fb < S::kFB; ++fb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) to[(fb * MB + mb) * kWave] = acc[fb][mb];
      if (wv == 0 && g == 0) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          space.ml[at * 2 * S::M + mb * 16 + i16] = m_run[mb];
          space.ml[at * 2 * S::M + S::M + mb * 16 + i16] = l_all[mb];
        }
      }
      if (tid == 0) space.parts[at] = Part{t.s.first, t.row0, t.rows, c0 == 0 ? un.owner(un.u + t.stages - 1) : 0};
    }

    // ---- on to the next request with work, if this one is done
    un.u += n;
    un.rem += n;
    if (un.u < un.u1 && un.rem == t.units) {
      un.rem = 0;
      un.r = next_request<kThreads>(a.rq, un.r, misc);
      if (un.r >= a.rq.R) break;  // (cannot be: the units say that there is one)
    }
  }
}

template <int DC, int MB>
__global__ __launch_bounds__(kThreads) void k_absorbed_join(AbsorbedArgs a, int G) {
  join_parts<DC, 16 * MB>(a, G, [](int blk, int fb) { return fb * MB + blk; });
}

template <int DC, int MB, bool FP8>
hipError_t run(const AbsorbedArgs& a, int G, hipStream_t stream) {
  using S = Shape<DC, MB>;
  static_assert(S::kBytes <= 160 * 1024, "LDS of a CU");
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_absorbed<DC, MB, FP8>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e != hipSuccess) return e;
  k_absorbed<DC, MB, FP8><<<dim3(G), dim3(kThreads), S::kBytes, stream>>>(a);
  k_absorbed_join<DC, MB><<<dim3(MB * G), dim3(kThreads), 0, stream>>>(a, G);
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
  int64_t tokens = (a.rq.n_tokens + a.rq.R / 2) / a.rq.R;
  if (tokens < 1) tokens = 1;
  if (a.rq.max_tokens > 0 && tokens > a.rq.max_tokens) tokens = a.rq.max_tokens;
  const int64_t rows = tokens * a.heads;
  if (rows <= 16) return run<DC, 1>(a, G, stream);
  if (rows <= 32) return run<DC, 2>(a, G, stream);
  // Tiles of 128 rows read LDS half as often, but leave parts of twice the size: they pay where workgroups go over many
  // stages each.  The lengths are not known here; at most, the requests fill the table.  (64 requests of up to 8192
  // positions, 128 heads: 174 us a pass, 204 us in tiles of 64 rows; 32 of up to 3001, 5 tokens of 32 heads: 51 us and 48;
  // one of 65,536, 128 heads: 69 us and 57.)
  const int64_t stages = (rows + 127) / 128 * a.rq.R * (int64_t(a.rq.max_blocks) * a.rq.block_size / 32);
  return launch_absorbed_rows(a, G, rows > 64 && stages >= 32 * int64_t(G), stream);
}

}  // namespace

int64_t absorbed_workspace_bytes(int latent_dim, int cus) {
  return part_space_bytes(latent_dim == 128 ? 2 * cus : cus, 128, latent_dim);
}

hipError_t launch_latent_absorbed(const AbsorbedArgs& a, int cus, hipStream_t stream) {
  if (a.latent_dim == 128) return run<128>(a, cus, stream);
  if (a.latent_dim == 256) return run<256>(a, cus, stream);
  return run<512>(a, cus, stream);
}

}  // namespace engram
