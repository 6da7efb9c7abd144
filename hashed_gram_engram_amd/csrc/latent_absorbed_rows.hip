// Absorbed latent attention for many rows a request (tokens times heads): tiles of M = 64 RB rows.
//
// Each of the four waves takes 16 RB rows of the tile and all of the latent: its queries and its accumulators
// (512 features: 144 and 256 registers a lane at RB 2, where the compiler keeps some 20 of the others in memory, outside
// the products) stay in registers, and a stage of 32 positions goes through LDS as bf16, read twice by every wave: along
// the features for the scores, transposed for the values.
// S^T = C Q^T leaves a lane with 4 consecutive positions of one query, which is an operand of out^T += C^T P^T
// as it stands if that product counts its positions in the same order; so weights, maxima and sums never leave a wave.
// (latent_absorbed.hip has the form for few rows, where the waves share the latent instead.)
//
// FP8 rows are copied to LDS as they are, three stages ahead, and converted one stage ahead by the lanes that
// copied them; BF16 rows are copied two stages ahead to where they are read.
//
// What bounds it: a wave has its SIMD to itself, and nothing issues while it waits.  64 requests of up to 8192 positions,
// 128 heads, 512 + 64 features in FP8: 172 us, 0.59 PFLOP/s; of a wave's cycles 30% are matrix instructions, 35% issue vector
// ones (conversion, softmax, addresses) and 23% wait.  Part of the waits is the compiler's: the rare branches end in
// loads into the accumulators, and where they meet the common path, at the start of the second product, it waits for all
// memory, the copies that the stage has just issued included.  One request of 65,536: 45 us (18% matrix, 21% vector, 33%
// waits; a workgroup has 16 stages); 32 of up to 3001, 5 tokens, 32 heads, 256 + 64 features, window 2000: 41 us (14%, 21%, 35%).
#include "latent_units.h"

namespace engram {

namespace {

constexpr int kThreads = 256;
constexpr int kTB = 32;  // positions per stage
constexpr int kRing = 8;      // stages whose pages are kept
constexpr int kSlotRing = 4;  // and their slots

template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// What is seldom done to the accumulators (scaling them, adding a single row) is done in memory, in the part of the
// workspace that the segment may write: done in registers it takes some from the loop over the stages (512 features, 128
// rows, FP8: 33 that go through memory there instead of 27).  One store or load of 16 bytes a lane for each block.
template <int N, int RB>
__device__ __forceinline__ void acc_to_memory(const f32x4 (&acc)[N][RB], char* to) {
  asm volatile("" : "+v"(to)::"memory");
#pragma unroll
  for (int mb = 0; mb < RB; ++mb)
#pragma unroll
    for (int fb = 0; fb < N; ++fb) {
      *reinterpret_cast<f32x4*>(to) = acc[fb][mb];
      to += kWave * 16;
    }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}
template <int N, int RB>
__device__ __forceinline__ void acc_from_memory(f32x4 (&acc)[N][RB], const char* from) {
  asm volatile("" : "+v"(from)::"memory");
#pragma unroll
  for (int mb = 0; mb < RB; ++mb)
#pragma unroll
    for (int fb = 0; fb < N; ++fb) {
      acc[fb][mb] = *reinterpret_cast<const f32x4*>(from);
      from += kWave * 16;
    }
}

template <int DC, int RB, bool FP8>
struct Shape {
  static constexpr int M = 64 * RB;
  static constexpr int kChunks = (DC + 64) / 8, kRowB = kChunks * 16;  // of a row in LDS
  static constexpr int kKB = DC / 32, kFB = DC / 16;
  static constexpr int kStageB = kTB * kRowB;
  static constexpr int kBufs = FP8 ? 2 : 3;
  // FP8 rows as they are in the cache: codes, rope parts, and the scales once for each wave
  static constexpr int kCodeB = kTB * DC, kRopeB = kTB * 128, kRawB = kCodeB + kRopeB + 4 * 1024, kRaws = 3;
  static constexpr int kCodeCopies = kCodeB / 16 / kThreads;
  static constexpr int kCopies = FP8 ? kCodeCopies + 2 : kTB * kChunks / kThreads;  // of a thread and stage
  static constexpr int kRaw = kBufs * kStageB;  // offsets into LDS
  // each wave's own: the pages of some stages' positions, their places in the pages, and their slots
  static constexpr int kPages = kRaw + (FP8 ? kRaws * kRawB : 0);
  static constexpr int kPlaces = kPages + 4 * kRing * 256;
  static constexpr int kSlots = kPlaces + 4 * kRing * kTB * 4;
  static constexpr int kMisc = kSlots + 4 * kSlotRing * kTB * 4;
  static constexpr int kBytes = kMisc + 64;
};

template <int DC, int RB, bool FP8>
__global__ __launch_bounds__(kThreads, DC == 128 ? 2 : 1) void k_absorbed_rows(AbsorbedArgs a) {
  using S = Shape<DC, RB, FP8>;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int i16 = lane & 15, g = lane >> 4;
  const int rkb = a.rope_dim / 32;
  const int row_b = latent_row_bytes(DC, a.rope_dim, FP8);
  int32_t* pages = reinterpret_cast<int32_t*>(lds + S::kPages) + wv * kRing * 64;
  int32_t* slots = reinterpret_cast<int32_t*>(lds + S::kSlots) + wv * kSlotRing * kTB;
  int32_t* places = reinterpret_cast<int32_t*>(lds + S::kPlaces) + wv * kRing * kTB;
  int64_t* misc = reinterpret_cast<int64_t*>(lds + S::kMisc);
  const uint32_t lds_at = lds_address(lds);
  const PartSpace space = part_space(a.workspace, gridDim.x, S::M);
  Units un;
  if (!my_units<kThreads, S::M, kTB>(a.rq, a.heads, space.parts, misc, &un)) return;

  constexpr int kHalf = DC / 16, kRows = 64 / kHalf;  // of the conversion: chunks in half a row, rows of codes in a copy

  // (Addresses in LDS and of copies are made from the lane's number where they are used: kept around the loop they
  // would take the registers that queries and accumulators leave, and go through memory, behind all copies in flight.)
  auto fresh = [&]() {
    int l = lane;
    asm volatile("" : "+v"(l));
    return l;
  };
  constexpr bool kLean = RB == 2 && DC != 256;
  auto lane_now = [&]() { return kLean ? fresh() : lane; };
  // A chunk's place differs from row to row in the low three bits of its number only, so the reads of a stage take
  // two addresses (keys) or four (values) and constants.  (Rows start at multiples of 128 bytes.)
  auto key_place = [&]() {
    const int l = lane_now(), i = l & 15;
    return i * S::kRowB + ((l >> 4) ^ latent_swizzle(i)) * 16;
  };
  auto value_place = [&]() {
    const int l = lane_now(), i = l & 15, row = (l >> 4) * 4 + (i >> 2);
    return row * S::kRowB + (((i & 3) >> 1) ^ latent_swizzle(row)) * 16 + (i & 1) * 8;
  };

  while (un.u < un.u1) {
    const Segment t = segment_of<S::M, kTB>(a.rq, a.heads, un);
    const int c0 = t.c0, n = t.n;
    const int w0 = t.row0 + wv * 16 * RB;  // the wave's first row

    f32x4 acc[S::kFB][RB];
    float m_run[RB], l_own[RB];
#pragma unroll
    for (int mb = 0; mb < RB; ++mb) {
      m_run[mb] = -kInf;
      l_own[mb] = 0.0f;
#pragma unroll
      for (int fb = 0; fb < S::kFB; ++fb) acc[fb][mb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    const bool whole = c0 == 0 && n == t.stages;
    const int64_t part_at = 2 * un.w + (c0 == 0 ? 1 : 0);  // (a whole tile's segment comes before the one that leaves this part)

    auto acc_memory = [&]() {
      uint32_t off = (wv * RB * S::kFB * kWave + lane) * 16;
      asm volatile("" : "+v"(off));  // (made where it is used)
      return reinterpret_cast<char*>(space.acc + part_at * (S::M * DC / 4)) + off;
    };

    // ---- staging
    // Lanes l and 32 + l look after row l of a stage.  Its page is copied to LDS some stages before its slot is made (by a
    // copy, like the rows: a load into a register would have to wait for all the copies before it), which is before
    // its row is copied.  Every wave does so for itself.  The page's entry and the place in it go on by 32 positions a
    // stage; entries past the table repeat its last one (those positions are not the request's).
    const int32_t* table = a.rq.block_table + int64_t(un.r) * a.rq.max_blocks;
    int entry = a.rq.page_of(t.base + c0 * kTB + (lane & 31)), place = t.base + c0 * kTB + (lane & 31) - entry * a.rq.block_size;
    auto copy_pages = [&](int c) {  // stages one after the other
      const int row = lane_now() & 31;
      const int e = entry < a.rq.max_blocks ? entry : a.rq.max_blocks - 1;
      copy_to_lds<4>(table + e, lds_at + S::kPages + (wv * kRing + (c & (kRing - 1))) * 256);
      places[(c & (kRing - 1)) * kTB + row] = place;
      entry += a.rq.stage_pages;
      place += a.rq.stage_rest;
      if (place >= a.rq.block_size) {
        place -= a.rq.block_size;
        ++entry;
      }
    };
    struct Page {
      int page, place;
    };
    auto read_page = [&](int c) {
      const int row = lane_now() & 31;
      return Page{pages[(c & (kRing - 1)) * 64 + row], places[(c & (kRing - 1)) * kTB + row]};
    };
    // Writes the slots of stage c, 0 for rows that take no part; returns those that do.
    auto make_slots = [&](int c, const Page& p) -> uint32_t {
      const bool good = uint32_t(p.page) < uint32_t(a.rq.n_blocks);
      slots[(c & (kSlotRing - 1)) * kTB + (lane_now() & 31)] = good ? p.page * a.rq.block_size + p.place : 0;
      const int j0 = t.base + c * kTB, from = t.lo - j0, to = c < c0 + n ? t.hi - j0 : 0;  // rows [from, to)
      const uint32_t below = to >= 32 ? ~0u : (to <= 0 ? 0u : (1u << to) - 1u), above = from <= 0 ? ~0u : (from >= 32 ? 0u : ~0u << from);
      const uint32_t in = below & above, on = in & uint32_t(__ballot(good));
      if (__builtin_expect(on != in, 0)) {
        const int old = t.fresh - j0;  // (rows that an earlier tile has counted)
        const uint32_t bad = (in ^ on) & (old <= 0 ? ~0u : (old >= 32 ? 0u : ~0u << old));
        if (wv == 0 && lane == 0 && bad != 0 && a.err_count != nullptr) atomicAdd(a.err_count, __builtin_popcount(bad));
      }
      return on;
    };
    uint32_t on_ring[5];  // rows that take part in stages c .. c + 4
    // (rows that take no part are copied from the first slot and cleared later; stages past the last too, so that
    // every wave has the same number of copies in flight)
    // A lane's part in the copies of a stage: where the slots of its rows stand, and what it takes of a row.
    struct Copies {
      const int32_t* code;
      const int32_t* rope;
      const int32_t* scale;
      const uint8_t* code_from;
      const uint8_t* rope_from;
    };
    auto copies_of = [&](int c) {
      const int l = lane_now(), tid = wv * kWave + l;
      const int32_t* sl = slots + (c & (kSlotRing - 1)) * kTB;
      return Copies{sl + wv * kRows + l / kHalf, sl + (rkb == 2 ? tid >> 3 : (tid >> 2) & 31), sl + (l & 31),
                    a.cache + l % kHalf * 16, a.cache + DC + 16 + (rkb == 2 ? tid & 7 : tid & 3) * 16};
    };
    auto row_slot = [&](const Copies& p, int c, int k) -> int {  // of which copy k takes 16 bytes
      if constexpr (FP8) return k < S::kCodeCopies ? p.code[k * 4 * kRows] : (k == S::kCodeCopies ? *p.rope : *p.scale);
      const int id = k * kThreads + wv * kWave + lane_now();
      return slots[(c & (kSlotRing - 1)) * kTB + id / S::kChunks];
    };
    auto copy = [&](const Copies& p, int c, int k, int slot) {
      const uint64_t at = uint64_t(uint32_t(slot)) * uint32_t(row_b);
      if constexpr (FP8) {
        const uint8_t* from = k < S::kCodeCopies ? p.code_from : (k == S::kCodeCopies ? p.rope_from : a.cache + DC);
        copy_to_lds<16>(from + at, lds_at + S::kRaw + (c % S::kRaws) * S::kRawB + (k * 4 + wv) * 1024);
      } else {
        const int id = k * kThreads + wv * kWave + lane_now(), r = id / S::kChunks;
        int ch = (id - r * S::kChunks) ^ latent_swizzle(r);
        ch = ch < DC / 8 + 4 * rkb ? ch : 0;  // (a place that is not read)
        copy_to_lds<16>(a.cache + at + ch * 16, lds_at + (c % S::kBufs) * S::kStageB + (k * 4 + wv) * 1024);
      }
    };
    auto copy_stage = [&](int c) {
      const Copies p = copies_of(c);
#pragma unroll
      for (int k = 0; k < S::kCopies; ++k) copy(p, c, k, row_slot(p, c, k));
    };
    // FP8: of what the wave's copy k brought (kRows rows of codes; the last one: rope parts), a lane's chunks are first
    // and first + half a row, so that a wave's writes fill all banks.  Row 4 kRows k + row0: its swizzle differs from row0's in
    // the bits that row / 8 has there.
    struct Places {
      const char* raw;
      const uint8_t* scale;
      int write;
      const char* rope;
      char* rope_write;
      int row0;
    };
    auto places_of = [&](int c) {
      const int l = lane_now(), row0 = wv * kRows + l / kHalf, tid = wv * kWave + l;
      const int rp = rkb == 2 ? tid & 7 : tid & 3, rr = rkb == 2 ? tid >> 3 : (tid >> 2) & 31;
      const char* raw = lds + S::kRaw + (c % S::kRaws) * S::kRawB;
      const char* buf = lds + (c & 1) * S::kStageB;
      return Places{raw + row0 * DC + l % kHalf * 8,
                    reinterpret_cast<const uint8_t*>(raw + S::kCodeB + S::kRopeB + wv * 1024 + row0 * 16 + l % kHalf / 4),
                    int(buf - lds) + row0 * S::kRowB + (l % kHalf ^ latent_swizzle(row0)) * 16, raw + S::kCodeB + tid * 16,
                    lds + (c & 1) * S::kStageB + rr * S::kRowB + ((DC / 8 + rp) ^ latent_swizzle(rr)) * 16, row0};
    };
    struct Raw {
      u32x4 v;
      uint32_t scale0, scale1;
    };
    constexpr int kStep = 4 * kRows;  // rows between a wave's copies
    auto read_raw = [&](const Places& p, int k) {
      Raw r = {};
      if (k == S::kCodeCopies) {
        r.v = *reinterpret_cast<const u32x4*>(p.rope);
      } else {
        const u32x2 lo = *reinterpret_cast<const u32x2*>(p.raw + k * kStep * DC), hi = *reinterpret_cast<const u32x2*>(p.raw + k * kStep * DC + kHalf * 8);
        r.v = u32x4{lo.x, lo.y, hi.x, hi.y};
        r.scale0 = p.scale[k * kStep * 16];
        r.scale1 = p.scale[k * kStep * 16 + kHalf / 4];
      }
      return r;
    };
    auto convert = [&](const Places& p, uint32_t on, int k, int half, const Raw& r) {  // the lane's first chunk, or its second
      if (k == S::kCodeCopies) {
        if (half == 0) *reinterpret_cast<u32x4*>(p.rope_write) = r.v;  // (only scores read it: no need to clear)
        return;
      }
      u32x4 o = latent8(half == 0 ? u32x2{r.v.x, r.v.y} : u32x2{r.v.z, r.v.w}, half == 0 ? r.scale0 : r.scale1);
      if (__builtin_expect(on != ~0u, 0))
        if (!((on >> (p.row0 + k * kStep)) & 1)) o = u32x4{0u, 0u, 0u, 0u};
      *reinterpret_cast<u32x4*>(lds + (p.write ^ (latent_swizzle(k * kStep) * 16)) + k * kStep * S::kRowB + half * kHalf * 16) = o;  // (kHalf: whole 8 chunks)
    };
    auto clear_dead = [&](int c) {  // BF16: of what this lane copied
      const uint32_t on = on_ring[0];
      if (on == ~0u) return;
      char* buf = lds + (c % S::kBufs) * S::kStageB;
#pragma unroll 1
      for (int k = 0; k < S::kCopies; ++k) {
        const int id = k * kThreads + tid;
        if (!((on >> (id / S::kChunks)) & 1)) *reinterpret_cast<u32x4*>(buf + id * 16) = u32x4{0u, 0u, 0u, 0u};
      }
    };

    constexpr int kCopyStage = FP8 ? 3 : 2;  // stages that rows are copied ahead
    wait_all_barrier();  // nobody reads LDS or copies into it any more
#pragma unroll
    for (int k = 0; k <= kCopyStage; ++k) copy_pages(c0 + k);

    // ---- queries, and the position of each row's token (-1: no row)
    u32x4 qf[RB][S::kKB + 2];
    int qpos[RB];
#pragma unroll
    for (int mb = 0; mb < RB; ++mb) {
      const int row = w0 + mb * 16 + i16, at = row < t.rows ? row : t.rows - 1;  // (rows past the last repeat it)
      const int tok = at / a.heads, head = at - tok * a.heads;
      qpos[mb] = row < t.rows ? t.s.pos + tok : -1;
      const uint16_t* src = a.q + (t.s.first + tok) * a.q_stride + int64_t(head) * (DC + a.rope_dim) + 8 * g;
#pragma unroll
      for (int kb = 0; kb < S::kKB + 2; ++kb)
        qf[mb][kb] = *reinterpret_cast<const u32x4*>(src + 32 * (kb < S::kKB + rkb ? kb : 0)) ^ a.q_sign;
    }
    wait_copies<0>();
    {
      Page page[kCopyStage + 1];
#pragma unroll
      for (int k = 0; k <= kCopyStage; ++k) page[k] = read_page(c0 + k);
#pragma unroll
      for (int k = 0; k <= kCopyStage; ++k) on_ring[k] = make_slots(c0 + k, page[k]);
    }
#pragma unroll
    for (int k = 0; k < kCopyStage; ++k) {
      copy_stage(c0 + k);
      if (k >= kCopyStage - 2) copy_pages(c0 + k + 3);
    }
    if constexpr (FP8) {
      wait_copies<2 * S::kCopies + 2>();
      const Places at = places_of(c0);
      Raw raw[S::kCodeCopies + 1];
#pragma unroll
      for (int k = 0; k <= S::kCodeCopies; ++k) raw[k] = read_raw(at, k);
#pragma unroll
      for (int k = 0; k <= S::kCodeCopies; ++k) {
        convert(at, on_ring[0], k, 0, raw[k]);
        convert(at, on_ring[0], k, 1, raw[k]);
      }
    }

    for (int j = 0; j < n; ++j) {
      const int c = c0 + j;
      wait_copies<S::kCopies + 1>();  // FP8: of stage c + 1, BF16: of stage c, are there, and the pages of stage c + kCopyStage + 1
      if constexpr (!FP8) clear_dead(c);
      wait_lds_barrier();
      char* buf = lds + (FP8 ? (c & 1) : c % S::kBufs) * S::kStageB;

      f32x4 s[2][RB];
      u32x4 p[RB];
      const uint32_t on = on_ring[0], on_next = on_ring[1];
      const int j0 = t.base + c * kTB;
      const bool differ = t.p_min != t.p_max && (j0 + kTB - 1 > t.p_min || (a.rq.window > 0 && j0 <= t.p_max - a.rq.window));
      {
        // ---- scores, and (FP8) the next stage's conversion between them
        const int key_at = key_place();
        const char* kp[2] = {buf + key_at, buf + (key_at ^ 64)};
        auto key = [&](int kb, int tb) { return *reinterpret_cast<const u32x4*>(kp[kb & 1] + tb * 16 * S::kRowB + (kb >> 1) * 128); };
        constexpr int kDeep = RB == 2 ? 3 : 5;
        u32x4 kf[kDeep][2];
#pragma unroll
        for (int kb = 0; kb < kDeep - 1; ++kb) {
          kf[kb][0] = key(kb, 0);
          kf[kb][1] = key(kb, 1);
        }
        constexpr int kSteps = S::kKB + 2;
        int from[2];
        const Copies cp = copies_of(c + kCopyStage);
        // beside each step's products: the keys of a later step, and a row copied (its slot read two steps before)
        auto side = [&](int kb) {
          if (kb >= 2 && kb - 2 < S::kCopies) copy(cp, c + kCopyStage, kb - 2, from[kb & 1]);
          if (kb < S::kCopies) from[kb & 1] = row_slot(cp, c + kCopyStage, kb);
        };
#pragma unroll
        for (int kb = 0; kb < kSteps; ++kb) {
          if (kb + kDeep - 1 < kSteps) {
            kf[(kb + kDeep - 1) % kDeep][0] = key(kb + kDeep - 1, 0);
            kf[(kb + kDeep - 1) % kDeep][1] = key(kb + kDeep - 1, 1);
          }
          side(kb);
          if (kb < S::kKB + 1 || rkb == 2) {
#pragma unroll
            for (int tb = 0; tb < 2; ++tb)
#pragma unroll
              for (int mb = 0; mb < RB; ++mb)
                s[tb][mb] = mfma16x16x32(kf[kb % kDeep][tb], qf[mb][kb], kb == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : s[tb][mb]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int kb = kSteps; kb < S::kCopies + 2; ++kb) side(kb);  // what small latents leave
      }
      copy_pages(c + kCopyStage + 3);

      // ---- softmax
      if (on != ~0u || differ) {
#pragma unroll
        for (int tb = 0; tb < 2; ++tb)
#pragma unroll
          for (int mb = 0; mb < RB; ++mb)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int row = tb * 16 + 4 * g + e, pos = j0 + row;
              const bool seen = ((on >> row) & 1) && pos <= qpos[mb] && (a.rq.window <= 0 || pos > qpos[mb] - a.rq.window);
              s[tb][mb][e] = seen ? s[tb][mb][e] : -kInf;
            }
      }
      float m_new[RB];
      bool grow = false;
#pragma unroll
      for (int mb = 0; mb < RB; ++mb) {
        float m = fmaxf(fmaxf(fmaxf(s[0][mb][0], s[0][mb][1]), fmaxf(s[0][mb][2], s[0][mb][3])),
                        fmaxf(fmaxf(s[1][mb][0], s[1][mb][1]), fmaxf(s[1][mb][2], s[1][mb][3])));
        m_new[mb] = rounded_product(quad_max(m), a.scale_log2);  // (the scale is positive: its sign is in the queries)
        if (m_run[mb] == -kInf) m_run[mb] = m_new[mb] + kGrow;  // (nothing is summed yet)
        grow |= m_new[mb] > m_run[mb];
      }
      if (__any(grow)) {
        char* mem = acc_memory();
        acc_to_memory(acc, mem);
#pragma unroll
        for (int mb = 0; mb < RB; ++mb) {
          const float m = moved_reference(m_run[mb], m_new[mb]);
          const float alpha = m == -kInf ? 1.0f : __builtin_amdgcn_exp2f(m_run[mb] - m);
          m_run[mb] = m;
          l_own[mb] *= alpha;
#pragma unroll 1
          for (int fb = 0; fb < S::kFB; fb += 8) {
            f32x4* at = reinterpret_cast<f32x4*>(mem + (mb * S::kFB + fb) * (kWave * 16));
            f32x4 v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = at[e * kWave];
#pragma unroll
            for (int e = 0; e < 8; ++e) at[e * kWave] = v[e] * alpha;
          }
        }
        acc_from_memory(acc, mem);
      }
      float scale = a.scale_log2;
      bool big = false;
#pragma unroll
      for (int mb = 0; mb < RB; ++mb) big |= m_run[mb] != -kInf && !(__builtin_fabsf(m_run[mb]) < kBigScore);
      if (__builtin_expect(__any(big), 0)) {
#pragma unroll
        for (int mb = 0; mb < RB; ++mb)
#pragma unroll
          for (int tb = 0; tb < 2; ++tb)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[tb][mb][e] = rounded_product(s[tb][mb][e], scale);
        scale = 1.0f;
      }
#pragma unroll
      for (int mb = 0; mb < RB; ++mb) {
        const float ref = m_run[mb] == -kInf ? 0.0f : m_run[mb];
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[tb][mb][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[tb][mb][e], scale, -ref));
            l_own[mb] += s[tb][mb][e];
          }
          p[mb][2 * tb] = pack_bf16x2(s[tb][mb][0], s[tb][mb][1]);
          p[mb][2 * tb + 1] = pack_bf16x2(s[tb][mb][2], s[tb][mb][3]);
        }
      }

      // ---- values that are not finite, where the tile's tokens see different positions: added row by row where they are
      // seen, and zeros for the product
      if (differ) {
        uint32_t odd = 0;
#pragma unroll 1
        for (int k = tid; k < kTB * DC / 8; k += kThreads) {
          const int row = k / (DC / 8);
          const u32x4 v = *reinterpret_cast<const u32x4*>(buf + row * S::kRowB + k % (DC / 8) * 16);
          if (any_not_finite(v)) odd |= 1u << row;
        }
        odd = uint32_t(any_rows(odd, misc));
        if (__builtin_expect(odd != 0, 0)) {
          char* mem = acc_memory();
          acc_to_memory(acc, mem);
#pragma unroll 1
          for (uint32_t left = odd; left != 0; left &= left - 1) {
            const int row = __builtin_ctz(left), pos = j0 + row;
#pragma unroll
            for (int mb = 0; mb < RB; ++mb) {
              float w = 0.0f;
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if ((row >> 4) * 4 + (row & 3) == k) w = s[k >> 2][mb][k & 3];
              w = __shfl(w, ((row >> 2) & 3) * 16 + i16, kWave);
              if (!((on >> row) & 1) || pos > qpos[mb] || (a.rq.window > 0 && pos <= qpos[mb] - a.rq.window)) continue;
#pragma unroll 1
              for (int fb = 0; fb < S::kFB; ++fb) {
                const u32x2 v = *reinterpret_cast<const u32x2*>(buf + row * S::kRowB + ((fb * 2 + (g >> 1)) ^ latent_swizzle(row)) * 16 + (g & 1) * 8);
                f32x4* to = reinterpret_cast<f32x4*>(mem + (mb * S::kFB + fb) * (kWave * 16));
                *to += f32x4{w * bf16_lo(v.x), w * bf16_hi(v.x), w * bf16_lo(v.y), w * bf16_hi(v.y)};
              }
            }
          }
          acc_from_memory(acc, mem);
          wait_lds_barrier();
          for (int k = tid; k < kTB * DC / 8; k += kThreads)
            if ((odd >> (k / (DC / 8))) & 1)
              *reinterpret_cast<u32x4*>(buf + k / (DC / 8) * S::kRowB + k % (DC / 8) * 16) = u32x4{0u, 0u, 0u, 0u};
          wait_lds_barrier();
        }
      }

      // ---- values
      const int value_at = value_place();
      const char* vp[4] = {buf + value_at, buf + (value_at ^ 32), buf + (value_at ^ 64), buf + (value_at ^ 96)};
      auto value = [&](int fb) {
        const char* from = vp[fb & 3] + (fb >> 2) * 128;
        const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)from));
        const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)(from + 16 * S::kRowB)));
        return u32x4{lo.x, lo.y, hi.x, hi.y};
      };
      const Places at = places_of(c + 1);
      Raw raw;
      Page page;
      constexpr int kDeep = FP8 || RB == 1 ? 6 : 5;
      u32x4 vf[kDeep];
#pragma unroll
      for (int fb = 0; fb < kDeep - 1; ++fb) vf[fb] = value(fb);
#pragma unroll
      for (int fb = 0; fb < S::kFB; ++fb) {
        if (fb + kDeep - 1 < S::kFB) vf[(fb + kDeep - 1) % kDeep] = value(fb + kDeep - 1);
        if constexpr (FP8) {  // and beside them the next stage's conversion
          constexpr int kEvery = S::kFB / (S::kCodeCopies + 1);
          const int k = fb / kEvery, in = fb % kEvery;
          if (k <= S::kCodeCopies && in == kEvery - 2) convert(at, on_next, k, 0, raw);
          if (k <= S::kCodeCopies && in == kEvery - 1) convert(at, on_next, k, 1, raw);
          if (k <= S::kCodeCopies && in == 0) raw = read_raw(at, k);
        }
        if (fb == 1) page = read_page(c + kCopyStage + 1);
        if (fb == S::kFB / 2) on_ring[kCopyStage + 1] = make_slots(c + kCopyStage + 1, page);
#pragma unroll
        for (int mb = 0; mb < RB; ++mb) acc[fb][mb] = mfma16x16x32(vf[fb % kDeep], p[mb], acc[fb][mb]);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int k = 0; k <= kCopyStage; ++k) on_ring[k] = on_ring[k + 1];
    }
    wait_copies<0>();  // (none is in flight when LDS goes to another workgroup)

    // ---- the outputs, or a part
#pragma unroll
    for (int mb = 0; mb < RB; ++mb) {
      const float l = quad_sum(l_own[mb]);
      const int row = w0 + mb * 16 + i16;
      if (whole) {
        if (row >= t.rows) continue;
        const int tok = row / a.heads, head = row - tok * a.heads;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t* out = a.out + (t.s.first + tok) * a.out_stride + int64_t(head) * DC + 4 * g;
#pragma unroll
        for (int fb = 0; fb < S::kFB; ++fb)
          *reinterpret_cast<u32x2*>(out + fb * 16) = u32x2{pack_bf16x2(acc[fb][mb][0] * inv, acc[fb][mb][1] * inv),
                                                           pack_bf16x2(acc[fb][mb][2] * inv, acc[fb][mb][3] * inv)};
        if (a.lse != nullptr && g == 0)
          a.lse[int64_t(t.s.first + tok) * a.heads + head] =
              l == 0.0f ? -kInf : (m_run[mb] + __builtin_amdgcn_logf(l)) * 0.69314718f;
      } else {
        f32x4* to = space.acc + part_at * (S::M * DC / 4) + (wv * RB + mb) * (S::kFB * kWave) + lane;
#pragma unroll
        for (int fb = 0; fb < S::kFB; ++fb) to[fb * kWave] = acc[fb][mb];
        if (g == 0) {
          space.ml[part_at * 2 * S::M + (wv * RB + mb) * 16 + i16] = m_run[mb];
          space.ml[part_at * 2 * S::M + S::M + (wv * RB + mb) * 16 + i16] = l;
        }
      }
    }
    if (!whole && tid == 0) space.parts[part_at] = Part{t.s.first, t.row0, t.rows, c0 == 0 ? un.owner(un.u + t.stages - 1) : 0};

    un.u += n;
    un.rem += n;
    if (un.u < un.u1 && un.rem == t.units) {
      un.rem = 0;
      un.r = next_request<kThreads>(a.rq, un.r, misc);
      if (un.r >= a.rq.R) break;  // (cannot be: the units say that there is one)
    }
  }
}

template <int DC, int M>
__global__ __launch_bounds__(kThreads) void k_absorbed_rows_join(AbsorbedArgs a, int G) {
  join_parts<DC, M>(a, G, [](int blk, int fb) { return blk * (DC / 16) + fb; });
}

template <int DC, int RB, bool FP8>
hipError_t run(const AbsorbedArgs& a, int G, hipStream_t stream) {
  using S = Shape<DC, RB, FP8>;
  static_assert(S::kBytes <= 160 * 1024, "LDS of a CU");
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k_absorbed_rows<DC, RB, FP8>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e != hipSuccess) return e;
  k_absorbed_rows<DC, RB, FP8><<<dim3(G), dim3(kThreads), S::kBytes, stream>>>(a);
  k_absorbed_rows_join<DC, S::M><<<dim3(4 * G), dim3(kThreads), 0, stream>>>(a, G);
  return hipGetLastError();
}

template <int DC>
hipError_t run(const AbsorbedArgs& a, int G, bool wide, hipStream_t stream) {
  if (wide) return a.fp8 ? run<DC, 2, true>(a, G, stream) : run<DC, 2, false>(a, G, stream);
  return a.fp8 ? run<DC, 1, true>(a, G, stream) : run<DC, 1, false>(a, G, stream);
}

}  // namespace

hipError_t launch_absorbed_rows(const AbsorbedArgs& a, int G, bool wide, hipStream_t stream) {
  if (a.latent_dim == 128) return run<128>(a, G, wide, stream);
  if (a.latent_dim == 256) return run<256>(a, G, wide, stream);
  return run<512>(a, G, wide, stream);
}

}  // namespace engram
