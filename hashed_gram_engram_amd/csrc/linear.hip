// Matrix product with bias, activation (plain or gated) and residual: out = residual + act(x w^T + bias).
//
// Three kernels, by a modelled choice (choose() in linear_choice.h):
//  k_linear      a tile of BM tokens x BN weight rows by 1..8 waves, for most shapes;
//  k_linear_big  256 x 256 by two groups of waves that take turns at the matrix units, for large ones;
//  k_linear_few  16 x 16 with K shared by the waves of a workgroup, for up to 16 tokens.
// K is taken in stages of 64 features, copied global -> LDS (16 bytes per lane, rows of 128 bytes) into a
// ring of slots; a wave multiplies blocks of v_mfma_f32_16x16x32_bf16 with weight rows as A and tokens as
// B, so that a lane holds 4 consecutive weight rows of one token.  Where there are few tiles K is split
// over workgroups: they leave fp32 blocks in the caller's workspace and k_linear_join adds them in order.
//
// Gated: the weight has the N gate rows, then the N value rows.  A block of 16 rows takes 8 rows of the
// gate and the same 8 of the value, so both factors of an output meet in one wave's epilogue.
//
// Edges: weight rows past N and tokens past M repeat the last one and are not stored; the features past the
// last whole stage (K is a multiple of 8) are read straight into fragments, zeros past K.
//
// What bounds it.  Up to 64 tokens, the weight's bytes: 1 token x 6144 x 25,600 takes 54 us (5.8 TB/s), 64
// tokens 63 us.  That needs every column of tiles to start at another stage of K: rows are 2 K bytes apart,
// so workgroups in step ask the same memory channel (64 tokens: 81 us without, 66 us with).  A few hundred
// tokens: the copies, 12-16 TB/s out of the L2s and about 66 KB per us into a CU, hence the largest tile
// that still fills the device (301 x 5120 x 20,480: 77 us with 160 x 160, 97 us with 128 x 128).  Thousands:
// the matrix units (busy 68% of the cycles, at 1.8-1.9 GHz): 8192 x 6144 x 25,600 without activation
// 1.82-1.91 ms, 1.35-1.42 PFLOP/s; with GELU 1.86-2.0 ms.  Short K: the first copies and the epilogue of a tile, which
// overlap nothing where one workgroup fills a CU (6192 x 616 x 23,984: 277 us; its output alone takes 62 us).
#include "common.h"
#include "linear_choice.h"
#include "serving.h"

namespace engram {

namespace {

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// ---------------------------------------------------------------- epilogue
// act(z) of 8 values; one branch for all of them.  exp is the hardware's 2^x of a rounded product (within
// |z| 2^-23 of exp(z), relative, where the result is small against z) and 1 / v within one unit in the last
// place: with the library's expf, erff and division the epilogue of an 8192 x 6144 x 25,600 product took
// 140 us longer for GELU.  Phi(-|z|) is formula 7.1.26 of Abramowitz and Stegun, Handbook of Mathematical
// Functions (|error of erf| <= 1.5e-7).
__device__ __forceinline__ float rcp(float v) { return __builtin_amdgcn_rcpf(v); }
__device__ __forceinline__ void activate8(float (&z)[8], int act) {
  if (act == 0) return;
  if (act == 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = z[e] < 0.0f ? 0.0f : z[e];  // a NaN stays one
  } else if (act == 2) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = fabsf(z[e]) * 0.70710678f, t = rcp(1.0f + 0.3275911f * x);
      const float p = t * (0.254829592f + t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
      const float q = 0.5f * p * __expf(-x * x);  // Phi(-|z|)
      z[e] *= z[e] > 0.0f ? 1.0f - q : q;
    }
  } else if (act == 3) {
    // (1 + tanh v) / 2 = 1 / (1 + exp(-2 v)) with 2 v = 2 sqrt(2 / pi) (z + 0.044715 z^3)
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] *= rcp(1.0f + __expf(-z[e] * (1.5957691216057308f + 0.071354816272f * z[e] * z[e])));
  } else if (act == 4) {  // (tanh-GELU's expression with no cubic term would make 0 times an infinite z a NaN)
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] *= rcp(1.0f + __expf(-z[e]));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = rcp(1.0f + __expf(-z[e]));
  }
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = a[e];
    v[4 + e] = b[e];
  }
}

// bias[row .. row + 7] (`valid` of them are the weight's; the others, and all without a bias, 0).
__device__ __forceinline__ void load_bias(const float* bias, int64_t row, int valid, float (&b)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) b[e] = 0.0f;
  if (bias == nullptr) return;
  if (valid >= 8 && (row & 3) == 0) {
    load8(bias + row, b);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < valid) b[e] = bias[row + e];
}

// Output features n .. n + 7 of token m (those below N): v plus the residual, rounded once.
__device__ __forceinline__ void store8(const LinearArgs& a, int64_t m, int n, float (&v)[8], bool vec) {
  const int64_t o = m * a.out_stride + n, q = m * a.residual_stride + n;
  const bool whole = vec && n + 8 <= a.N;
  if (a.fp32) {
    float* out = static_cast<float*>(a.out) + o;
    const float* res = static_cast<const float*>(a.residual) + q;
    if (whole) {
      f32x4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
      if (a.residual != nullptr) {
        lo += *reinterpret_cast<const f32x4*>(res);
        hi += *reinterpret_cast<const f32x4*>(res + 4);
      }
      __builtin_nontemporal_store(lo, reinterpret_cast<f32x4*>(out));
      __builtin_nontemporal_store(hi, reinterpret_cast<f32x4*>(out + 4));
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (n + e < a.N) out[e] = v[e] + (a.residual != nullptr ? res[e] : 0.0f);
    return;
  }
  uint16_t* out = static_cast<uint16_t*>(a.out) + o;
  const uint16_t* res = static_cast<const uint16_t*>(a.residual) + q;
  if (whole) {
    if (a.residual != nullptr) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(res);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] += bf16_lo(w[e]);
        v[2 * e + 1] += bf16_hi(w[e]);
      }
    }
    __builtin_nontemporal_store(
        u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])},
        reinterpret_cast<u32x4*>(out));
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (n + e < a.N)
      out[e] = uint16_t(pack_bf16x2(v[e] + (a.residual != nullptr ? bf16_lo(res[e]) : 0.0f), 0.0f));
}

// Rows of 16-byte stores: every row of out (and of the residual) starts at a multiple of 16 bytes.
__device__ __forceinline__ bool vector_rows(const LinearArgs& a) {
  const int per = a.fp32 ? 4 : 8;
  return a.out_stride % per == 0 && (a.residual == nullptr || a.residual_stride % per == 0);
}

// The wave's LDS accesses before and after stay in order (other lanes' writes among them; the LDS
// unit takes one wave's accesses in order, so only the compiler is held).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Floats of a row of a wave's epilogue buffer (16 bytes of padding: rows start on other banks).
template <int TN>
constexpr int epilogue_row() { return TN * 16 + 4; }
template <int TN>
constexpr int epilogue_bytes() { return 16 * epilogue_row<TN>() * 4; }

// A wave's part of the tile: TN x TM blocks of 16 weight rows x 16 tokens, block (i, j) holding rows
// 16 i + 4 (l >> 4) + 0..3 of token 16 j + (l & 15).  16 tokens at a time pass through the wave's own
// piece of LDS, so that a lane gets 8 consecutive output features of a token (with GLU: a block's 8 gate
// rows and its 8 value rows) and stores are whole row segments.
template <int TN, int TM, bool GLU>
__device__ __forceinline__ void epilogue(const LinearArgs& a, const f32x4 (&acc)[TN][TM], char* lds, int64_t m0, int n0,
                                         int lane) {
  constexpr int kRow = epilogue_row<TN>();
  constexpr int kLanes = GLU ? TN : 2 * TN;     // of 8 output features each
  constexpr bool kFixed = kWave % kLanes == 0;     // a lane's features are the same in every pass
  float* buf = reinterpret_cast<float*>(lds);
  const bool vec = vector_rows(a);
  float b[8], bu[8];
  auto biases = [&](int n) {
    load_bias(a.bias, n, a.N - n, b);
    if constexpr (GLU) load_bias(a.bias, int64_t(a.N) + n, a.N - n, bu);
  };
  if constexpr (kFixed) biases(n0 + 8 * (lane % kLanes));
#pragma unroll 1
  for (int jj = 0; jj < TM; ++jj) {
#pragma unroll
    for (int j = 0; j < TM; ++j)
      if (j == jj) {  // (registers have no index)
#pragma unroll
        for (int i = 0; i < TN; ++i)
          *reinterpret_cast<f32x4*>(buf + (lane & 15) * kRow + 16 * i + 4 * (lane >> 4)) = acc[i][j];
      }
    wave_lds_fence();
#pragma unroll 1
    for (int e = lane; e < 16 * kLanes; e += kWave) {
      const int t = e / kLanes, c = 8 * (e - t * kLanes);
      const int64_t m = m0 + 16 * jj + t;
      const int n = n0 + c;
      if (m >= a.M || n >= a.N) continue;
      if constexpr (!kFixed) biases(n);
      float z[8];
      const float* p = buf + t * kRow + (GLU ? 2 * c : c);
      load8(p, z);
#pragma unroll
      for (int k = 0; k < 8; ++k) z[k] += b[k];
      activate8(z, a.act);
      if constexpr (GLU) {
        float u[8];
        load8(p + 8, u);
#pragma unroll
        for (int k = 0; k < 8; ++k) z[k] *= u[k] + bu[k];
      }
      store8(a, m, n, z, vec);
    }
    wave_lds_fence();
  }
}

// ---------------------------------------------------------------- K loop
template <int N>
__device__ __forceinline__ void wait_copies() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// Every LDS read of the wave has returned.  (The builtin, not inline assembly: the compiler then knows
// that the fragments are there and puts no wait of its own behind the next reads.)
__device__ __forceinline__ void wait_reads() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void group_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The weight row that row r of a tile holds (clamped into the weight).
template <bool GLU>
__device__ __forceinline__ int64_t weight_row(const LinearArgs& a, int64_t n0, int r) {
  if constexpr (!GLU) return n0 + r < a.N ? n0 + r : int64_t(a.N) - 1;
  int64_t n = n0 + (r >> 4) * 8 + (r & 7);
  n = n < a.N ? n : int64_t(a.N) - 1;
  return n + ((r >> 3) & 1) * int64_t(a.N);
}

// The tile of workgroup b of `tiles`: workgroups are dealt to the 8 XCDs round robin, so each XCD
// takes a run of consecutive tiles, token blocks fastest: a weight panel is read by one XCD, once.
__device__ __forceinline__ uint32_t xcd_tile(uint32_t b, uint32_t tiles) {
  const uint32_t q = tiles >> 3, rem = tiles & 7, x = b & 7;
  return x * q + (x < rem ? x : rem) + (b >> 3);
}

// 16-byte chunk c of row r of a stage lies at position c ^ swizzle(r): the 16 rows of a fragment read
// cover all 64 banks once.
__device__ __forceinline__ int swizzle(int r) { return (r >> 1) & 7; }

// Tiles in order: groups of 8 token blocks, and in a group token blocks fastest, so that the tiles that
// run on an XCD at one time share token panels as well as weight panels in its L2.
// (Tiles are counted in 32 bits: a 64-bit division is some 100 instructions before the first copy.)
__device__ __forceinline__ void tile_of(uint32_t tile, uint32_t tbs, uint32_t cbs, uint32_t* tb, uint32_t* cb) {
  constexpr uint32_t kGroup = 8;
  const uint32_t g = tbs <= kGroup ? 0 : tile / (kGroup * cbs), in = tile - g * kGroup * cbs;
  const uint32_t size = tbs - g * kGroup < kGroup ? tbs - g * kGroup : kGroup;
  *cb = in / size;
  *tb = g * kGroup + in - *cb * size;
}

// What a workgroup computes: a tile, and of its K the whole stages [first, first + stages) and, in the
// last part, the features past the last whole stage.  Split over K, part 0 of every tile comes first:
// the workgroups of an XCD then share panels as without a split.
struct Share {
  uint32_t tile, tb, cb;
  int part, first, stages;
  bool tail;
};
__device__ __forceinline__ Share share_of(const LinearArgs& a, uint32_t tbs, uint32_t cbs) {
  Share s;
  const uint32_t tiles = tbs * cbs, at = xcd_tile(blockIdx.x, gridDim.x);
  const int S = a.K / kBK;
  s.part = a.parts > 1 ? int(at / tiles) : 0;
  s.tile = at - s.part * tiles;
  tile_of(s.tile, tbs, cbs, &s.tb, &s.cb);
  s.first = a.parts > 1 ? S * s.part / a.parts : 0;  // (S < 2^14)
  s.stages = a.parts > 1 ? S * (s.part + 1) / a.parts - s.first : S;
  s.tail = s.part == a.parts - 1 && a.K % kBK != 0;
  return s;
}

// The features past the last whole stage: fragments straight from memory, zeros past K.  r0: the wave's
// first row of the tile, m0: its first token.
template <int TN, int TM, bool GLU>
__device__ __forceinline__ void tail(const LinearArgs& a, f32x4 (&acc)[TN][TM], int64_t n0, int r0, int64_t m0, int lane) {
  const int r16 = lane & 15, g = lane >> 4;
#pragma unroll 1
  for (int k0 = a.K / kBK * kBK; k0 < a.K; k0 += 32) {
    const int k = k0 + 8 * g;
    u32x4 x[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int64_t m = m0 + j * 16 + r16;
      x[j] = k < a.K ? *reinterpret_cast<const u32x4*>(a.x + (m < a.M ? m : a.M - 1) * a.x_stride + k)
                     : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      const u32x4 w = k < a.K ? *reinterpret_cast<const u32x4*>(a.w + weight_row<GLU>(a, n0, r0 + i * 16 + r16) * a.K + k)
                              : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = mfma16x16x32(w, x[j], acc[i][j]);
    }
  }
}

// Split over K: a wave's fp32 blocks in the order it holds them, 1 KB a block, at wave slot `at` of the
// workspace.
template <int TN, int TM>
__device__ __forceinline__ void store_partial(const LinearArgs& a, const f32x4 (&acc)[TN][TM], int64_t at, int lane) {
  f32x4* p = reinterpret_cast<f32x4*>(a.partials) + at * (TN * TM * kWave) + lane;
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) p[(i * TM + j) * kWave] = acc[i][j];
}

// Adds the parts of 16 tokens of a wave's blocks in order and finishes them; one wave per workgroup (with
// all of a wave's tokens in one, 1000 x 10,240 x 5120 in three parts took 28 us, and 19 us like this).
template <int BM, int BN, int WM, int WN, bool GLU>
__global__ __launch_bounds__(kWave) void k_linear_join(LinearArgs a) {
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16, kOutCols = GLU ? BN / 2 : BN;
  __shared__ __attribute__((aligned(16))) char lds[epilogue_bytes<TN>()];
  const int lane = threadIdx.x;
  const uint32_t tbs = uint32_t((a.M + BM - 1) / BM), cbs = uint32_t((a.N + kOutCols - 1) / kOutCols);
  const int64_t slots = int64_t(tbs) * cbs * WM * WN;
  const int j = int(blockIdx.x % TM);
  const uint32_t at = blockIdx.x / TM;
  const int wv = int(at % (WM * WN));
  uint32_t tb, cb;
  tile_of(at / (WM * WN), tbs, cbs, &tb, &cb);
  // which part of the tile a wave holds: as in k_linear_big (the 256 x 256 tile) and k_linear
  constexpr bool kGroups = BM == 256 && BN == 256;
  const int wm = kGroups ? wv % WM : wv / WN, wn = kGroups ? wv / WM : wv % WN;
  const int64_t m0 = int64_t(tb) * BM + (wm * TM + j) * 16;
  if (m0 >= a.M) return;
  const f32x4* p = reinterpret_cast<const f32x4*>(a.partials) + int64_t(at) * (TN * TM * kWave) + j * kWave + lane;
  f32x4 acc[TN][1];
#pragma unroll
  for (int i = 0; i < TN; ++i) acc[i][0] = p[i * TM * kWave];
  for (int part = 1; part < a.parts; ++part) {
    p += slots * (TN * TM * kWave);
#pragma unroll
    for (int i = 0; i < TN; ++i) acc[i][0] += p[i * TM * kWave];
  }
  epilogue<TN, 1, GLU>(a, acc, lds, m0, int(cb * kOutCols) + wn * TN * (GLU ? 8 : 16), lane);
}

// ---------------------------------------------------------------- tiles of BM x BN
// The waves share the tile as WM x WN parts of TM x TN blocks.  A stage of the ring (ST slots) holds BN weight
// rows, then BM token rows.  While a wave multiplies one half of a stage (32 features) it reads the next
// half's fragments; one barrier per stage, between its halves, hands the slot on.  (The wait counts hold
// only if nothing else is in flight: a spilled register would break them; none of these kernels has one.)
template <int BM, int BN, int WM, int WN, int ST, bool GLU>
__global__ __launch_bounds__(WM* WN* kWave, 2) void k_linear(LinearArgs a) {
  constexpr int kWaves = WM * WN;
  constexpr int kRowsT = BM + BN;                 // rows of a stage: the weight's, then the tokens'
  constexpr int kSlot = kRowsT * kRowB;
  constexpr int kAll = kRowsT / 8;                // copy instructions of a stage
  constexpr int kCopies = kAll / kWaves;          // of one wave
  constexpr int kFirst = kCopies / 2;             // of these, issued in the second half of a stage
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
  constexpr int kOutCols = GLU ? BN / 2 : BN;
  static_assert(kAll % kWaves == 0 && BN % 16 == 0, "tile");
  constexpr int kEpi = epilogue_bytes<TN>();
  static_assert(kEpi * kWaves <= ST * kSlot, "epilogue buffer");
  extern __shared__ __attribute__((aligned(16))) char lds[];

  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tbs = uint32_t((a.M + BM - 1) / BM), cbs = uint32_t((a.N + kOutCols - 1) / kOutCols);
  const Share sh = share_of(a, tbs, cbs);
  const int64_t m0 = int64_t(sh.tb) * BM, n0 = int64_t(sh.cb) * kOutCols;
  const int S = sh.stages;
  // the stages are taken from this one on, and round (see above: memory channels)
  const int turned = S > 0 ? int(sh.cb % uint32_t(S)) : 0;

  // lane l of copy q fills bytes 16 l of 1 KB: row 8 q + l / 8, position l % 8.  Its 8 rows start at
  // a wave-uniform address; the lane's part is a 32-bit offset.
  const char* base[kCopies];
  uint32_t off[kCopies];
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    const int r = (wv * kCopies + i) * 8;
    const uint32_t at = 16 * ((lane & 7) ^ swizzle(r + (lane >> 3)));
    if (r < BN) {
      const int64_t first = weight_row<GLU>(a, n0, r);
      base[i] = reinterpret_cast<const char*>(a.w + first * a.K);
      off[i] = uint32_t(weight_row<GLU>(a, n0, r + (lane >> 3)) - first) * uint32_t(a.K) * 2 + at;
    } else {
      const int64_t last = a.M - 1, m = m0 + r - BN, first = m < last ? m : last;
      base[i] = reinterpret_cast<const char*>(a.x + first * a.x_stride);
      const int64_t mine = m + (lane >> 3) < last ? m + (lane >> 3) : last;
      off[i] = uint32_t(mine - first) * uint32_t(a.x_stride) * 2 + at;
    }
  }
  // copies i0 .. i1 - 1 of stage t; stages past the last repeat it (into a slot that nobody reads any
  // more), so that every turn has issued the same number of copies
  auto copy = [&](int t, int slot, int i0, int i1) {
    char* dst = lds + slot * kSlot + wv * kCopies * 1024;
    int k = (t < S ? t : S - 1) + turned;
    k = k < S ? k : k - S;
    const size_t at = size_t(sh.first + k) * kRowB;
#pragma unroll
    for (int i = i0; i < i1; ++i)
      __builtin_amdgcn_global_load_lds((const void*)(base[i] + at + off[i]), (lds_ptr_t)(dst + i * 1024), 16, 0, 0);
  };

  f32x4 acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int wn = wv % WN, wm = wv / WN;
  const int r16 = lane & 15, g = lane >> 4;
  struct Frags {
    u32x4 w[TN], x[TM];
  };
  const int w_off = (wn * TN * 16 + r16) * kRowB, x_off = (BN + wm * TM * 16 + r16) * kRowB;
  // fragment q of a half stage: weight rows, then tokens
  auto read = [&](Frags& f, const char* b, int q) {
    if (q < TN) f.w[q] = *reinterpret_cast<const u32x4*>(b + w_off + q * 16 * kRowB);
    else f.x[q - TN] = *reinterpret_cast<const u32x4*>(b + x_off + (q - TN) * 16 * kRowB);
  };
  auto half_of = [&](int slot, int hh) { return lds + slot * kSlot + 16 * ((4 * hh + g) ^ swizzle(r16)); };
  // Multiplies one half stage, in this order: the reads of the next one's fragments over the first three
  // quarters of the MFMAs, copies i0 .. i1 - 1 of stage t over all of them.  A copy instruction occupies
  // the CU's address unit for 16 cycles, an MFMA its matrix unit for 16: a burst of either stalls the wave
  // that the other needs.
  auto half = [&](const Frags& now, Frags& next, const char* from, int t, int slot, int i0, int i1) {
    constexpr int R = TN + TM, M = TN * TM;
    const int C = i1 - i0;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int r0 = m * R * 4 / (3 * M), r1 = (m + 1) * R * 4 / (3 * M);
#pragma unroll
      for (int q = r0; q < (m == M - 1 ? R : r1); ++q)
        if (q < R) read(next, from, q);
      acc[m / TM][m % TM] = mfma16x16x32(now.w[m / TM], now.x[m % TM], acc[m / TM][m % TM]);
      __builtin_amdgcn_sched_barrier(0);
      copy(t, slot, i0 + m * C / M, i0 + (m + 1) * C / M);
    }
  };
  if (S > 0) {
#pragma unroll
    for (int t = 0; t < ST - 1; ++t) copy(t, t, 0, kCopies);
    copy(ST - 1, ST - 1, 0, kFirst);
    wait_copies<(ST - 2) * kCopies + kFirst>();
    group_barrier();
    Frags f0, f1;
#pragma unroll
    for (int q = 0; q < TN + TM; ++q) read(f0, half_of(0, 0), q);
    int slot = 0, before = ST - 1;
    for (int t = 0; t < S; ++t) {
      const int next = slot + 1 == ST ? 0 : slot + 1;
      wait_reads();
      // first half; the rest of stage t - 1 + ST goes into stage t - 1's slot
      half(f0, f1, half_of(slot, 1), t - 1 + ST, before, kFirst, kCopies);
      // Stage t + 1 is in LDS for everyone once only the copies of stages t + 2 .. t + ST - 1 are in
      // flight, and nobody reads stage t's slot any more once every wave has its last fragments.
      wait_copies<(ST - 2) * kCopies>();
      wait_reads();
      group_barrier();
      // second half; stage t + ST starts into stage t's slot (past the last stage the fragments read are
      // a repeat's, not used)
      half(f1, f0, half_of(next, 0), t + ST, slot, 0, kFirst);
      before = slot;
      slot = next;
    }
    wait_copies<0>();
  }
  if (sh.tail) {
    tail<TN, TM, GLU>(a, acc, n0, wn * TN * 16, m0 + wm * TM * 16, lane);
  }
  if (a.parts > 1) {
    store_partial<TN, TM>(a, acc, (int64_t(sh.part) * tbs * cbs + sh.tile) * kWaves + wv, lane);
    return;
  }
  __syncthreads();  // the ring is free
  epilogue<TN, TM, GLU>(a, acc, lds + wv * kEpi, m0 + wm * TM * 16, int(n0) + wn * TN * (GLU ? 8 : 16), lane);
}

// ---------------------------------------------------------------- tiles of 256 x 256
// Eight waves, two per SIMD.  Waves 0-3 (group 0) own weight rows 0-127 of the tile, waves 4-7
// (group 1) rows 128-255; in a group, wave w & 3 owns tokens 64 (w & 3) .. + 63, so a wave holds 8 x 4
// blocks.  The groups alternate: while one group's wave of a SIMD issues the 32 MFMAs of half a
// stage, the other's reads the fragments of its half; a barrier separates the phases, four to a stage.
//
// Weight stages have a ring of three slots and are copied two stages ahead, token stages a ring of two
// (5 x 32 KB).  Stage J is multiplied in phases 4 J .. 4 J + 3 and its last fragments are read in phase
// 4 J + 2.  Every wave issues 2 copies in every phase: the tokens of stage J + 1 in phases 4 J - 1 and
// 4 J, the weight rows of stage J + 2 in 4 J + 1 and 4 J + 2 (both slots held stage J - 1).  At the end
// of phase 4 J + 2 a wave waits until only its 4 weight copies of stage J + 2 are in flight: stage
// J + 1 is then there for its first reader (group 0, phase 4 J + 3).  Copies past the last stage
// repeat it, so that the counts hold.  (The 64 copies of a stage take the CU's memory path about 1600
// cycles, its 4 phases of MFMAs 2048: copies in one phase would make that phase three times as long.)
constexpr int kOpB = kBig * kRowB;  // one operand of one stage: weight slots 0..2, token slots 3, 4 of kBigLds
typedef f32x4 BigAcc[8][4];

struct BigPipe {
  const char* w_base[4];
  const char* x_base[4];
  uint32_t w_off[4], x_off[4];
  uint32_t frag[2];  // per-lane byte offset of a fragment read (half 0, 1)
  int wv, w_row, x_row;  // wave; byte offsets of its first weight and token row
};

__device__ __forceinline__ void big_copy(const char* const (&base)[4], const uint32_t (&off)[4], char* slot, int wv,
                                         int t, int i) {
  __builtin_amdgcn_global_load_lds((const void*)(base[i] + size_t(t) * kRowB + off[i]),
                                   (lds_ptr_t)(slot + (4 * wv + i) * 1024), 16, 0, 0);
}
__device__ __forceinline__ void big_read(u32x4 (&F)[12], const BigPipe& p, const char* W, const char* X, int hh) {
#pragma unroll
  for (int i = 0; i < 8; ++i) F[i] = *reinterpret_cast<const u32x4*>(W + p.w_row + p.frag[hh] + i * 16 * kRowB);
#pragma unroll
  for (int j = 0; j < 4; ++j) F[8 + j] = *reinterpret_cast<const u32x4*>(X + p.x_row + p.frag[hh] + j * 16 * kRowB);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}
__device__ __forceinline__ void big_mma(BigAcc& acc, const u32x4 (&F)[12], int i0, int i1) {
#pragma unroll
  for (int i = i0; i < i1; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = mfma16x16x32(F[i], F[8 + j], acc[i][j]);
  __builtin_amdgcn_sched_barrier(0);
}

template <int G>
__device__ __forceinline__ void big_loop(BigAcc& acc, const BigPipe& p, char* lds, int s0, int S, int turned) {
  u32x4 F[12];
  auto stage = [&](int t) {
    const int k = (t < S ? t : S - 1) + turned;
    return s0 + (k < S ? k : k - S);
  };
  // the two copies of a phase: tokens (weight rows) i, i + 1 of stage t
  auto tokens = [&](int t, int i) {
    big_copy(p.x_base, p.x_off, lds + (3 + (t & 1)) * kOpB, p.wv, stage(t), i);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto weights = [&](int t, int slot, int i) {
    big_copy(p.w_base, p.w_off, lds + slot * kOpB, p.wv, stage(t), i);
    __builtin_amdgcn_sched_barrier(0);
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) weights(0, 0, i);
#pragma unroll
  for (int i = 0; i < 4; ++i) tokens(0, i);
#pragma unroll
  for (int i = 0; i < 4; ++i) weights(1, 1, i);
  tokens(1, 0);
  tokens(1, 1);
  wait_copies<6>();
  group_barrier();
  if constexpr (G == 0) big_read(F, p, lds, lds + 3 * kOpB, 0);
  group_barrier();
  int w0 = 0;  // weight slot of stage J
  for (int J = 0; J < S; ++J) {
    const int w1 = w0 == 2 ? 0 : w0 + 1, w2 = w1 == 2 ? 0 : w1 + 1;
    const char* W = lds + w0 * kOpB;
    const char* X = lds + (3 + (J & 1)) * kOpB;
    if constexpr (G == 0) {
      big_mma(acc, F, 0, 3);  // 4 J: half 0
      tokens(J + 1, 2);
      big_mma(acc, F, 3, 6);
      tokens(J + 1, 3);
      big_mma(acc, F, 6, 8);
      group_barrier();
      weights(J + 2, w2, 0);  // 4 J + 1: read half 1
      weights(J + 2, w2, 1);
      big_read(F, p, W, X, 1);
      group_barrier();
      big_mma(acc, F, 0, 3);  // 4 J + 2: half 1
      weights(J + 2, w2, 2);
      big_mma(acc, F, 3, 6);
      weights(J + 2, w2, 3);
      big_mma(acc, F, 6, 8);
      wait_copies<4>();
      group_barrier();
      tokens(J + 2, 0);  // 4 J + 3: read half 0 of stage J + 1
      tokens(J + 2, 1);
      big_read(F, p, lds + w1 * kOpB, lds + (3 + ((J + 1) & 1)) * kOpB, 0);
      group_barrier();
    } else {
      tokens(J + 1, 2);  // 4 J: read half 0
      tokens(J + 1, 3);
      big_read(F, p, W, X, 0);
      group_barrier();
      big_mma(acc, F, 0, 3);  // 4 J + 1: half 0
      weights(J + 2, w2, 0);
      big_mma(acc, F, 3, 6);
      weights(J + 2, w2, 1);
      big_mma(acc, F, 6, 8);
      group_barrier();
      weights(J + 2, w2, 2);  // 4 J + 2: read half 1
      weights(J + 2, w2, 3);
      big_read(F, p, W, X, 1);
      wait_copies<4>();
      group_barrier();
      big_mma(acc, F, 0, 3);  // 4 J + 3: half 1
      tokens(J + 2, 0);
      big_mma(acc, F, 3, 6);
      tokens(J + 2, 1);
      big_mma(acc, F, 6, 8);
      group_barrier();
    }
    w0 = w1;
  }
  wait_copies<0>();
  group_barrier();
}

template <bool GLU>
__global__ __launch_bounds__(512, 2) void k_linear_big(LinearArgs a) {
  constexpr int kOut = GLU ? kBig / 2 : kBig;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t tbs = uint32_t((a.M + kBig - 1) / kBig), cbs = uint32_t((a.N + kOut - 1) / kOut);
  const Share sh = share_of(a, tbs, cbs);
  const int64_t m0 = int64_t(sh.tb) * kBig, n0 = int64_t(sh.cb) * kOut;
  BigPipe p;
  p.wv = wv;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (4 * wv + i) * 8, mine = r + (lane >> 3);
    const uint32_t at = 16 * ((lane & 7) ^ swizzle(mine));
    const int64_t row = weight_row<GLU>(a, n0, r);
    p.w_base[i] = reinterpret_cast<const char*>(a.w + row * a.K);
    p.w_off[i] = uint32_t(weight_row<GLU>(a, n0, mine) - row) * uint32_t(a.K) * 2 + at;
    const int64_t last = a.M - 1, first = m0 + r < last ? m0 + r : last, m = m0 + mine < last ? m0 + mine : last;
    p.x_base[i] = reinterpret_cast<const char*>(a.x + first * a.x_stride);
    p.x_off[i] = uint32_t(m - first) * uint32_t(a.x_stride) * 2 + at;
  }
  const int r16 = lane & 15, g = lane >> 4;
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) p.frag[hh] = uint32_t(r16 * kRowB + 16 * ((4 * hh + g) ^ swizzle(r16)));
  p.w_row = (wv >> 2) * 128 * kRowB;
  p.x_row = (wv & 3) * 64 * kRowB;
  BigAcc acc;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (sh.stages > 0) {
    const int turned = int(sh.cb % uint32_t(sh.stages));
    if (wv < 4) big_loop<0>(acc, p, lds, sh.first, sh.stages, turned);
    else big_loop<1>(acc, p, lds, sh.first, sh.stages, turned);
  }
  if (sh.tail) tail<8, 4, GLU>(a, acc, n0, (wv >> 2) * 128, m0 + (wv & 3) * 64, lane);
  if (a.parts > 1) {
    store_partial<8, 4>(a, acc, (int64_t(sh.part) * tbs * cbs + sh.tile) * 8 + wv, lane);
    return;
  }
  constexpr int kEpi = epilogue_bytes<8>();
  epilogue<8, 4, GLU>(a, acc, lds + wv * kEpi, m0 + (wv & 3) * 64, int(n0) + (wv >> 2) * 128 / (GLU ? 2 : 1), lane);
}

// ---------------------------------------------------------------- up to 16 tokens
// A tile of 16 tokens x 16 weight rows whose K is shared by the W waves of the workgroup: wave w
// takes stages w, w + W, ...  A wave has a ring of ST slots of its own (its weight rows, then XR token rows;
// with XR = 8 the fragments of tokens 8..15 read those of 0..7 and are dropped) and waits only for its own
// copies, so the waves run free of each other until they add up their sums.
template <int W, int ST, int XR, bool GLU>
__global__ __launch_bounds__(W* kWave) void k_linear_few(LinearArgs a) {
  constexpr int kCopies = 2 + XR / 8, kSlot = kCopies * 1024;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  static_assert(W * 1024 <= W * ST * kSlot && epilogue_bytes<1>() <= W * ST * kSlot, "sums and epilogue");
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int64_t n0 = int64_t(blockIdx.x) * (GLU ? 8 : 16);
  const int S = a.K / kBK, count = (S - wv + W - 1) / W;  // stages, this wave's
  const int turned = S > 0 ? int(blockIdx.x % unsigned(S)) : 0;
  char* ring = lds + wv * ST * kSlot;
  const char* base[kCopies];
  uint32_t off[kCopies];
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    const int r = 8 * (i < 2 ? i : i - 2), mine = r + (lane >> 3);
    const uint32_t at = 16 * ((lane & 7) ^ swizzle(mine));
    if (i < 2) {
      const int64_t row = weight_row<GLU>(a, n0, r);
      base[i] = reinterpret_cast<const char*>(a.w + row * a.K);
      off[i] = uint32_t(weight_row<GLU>(a, n0, mine) - row) * uint32_t(a.K) * 2 + at;
    } else {
      const int64_t last = a.M - 1, first = r < last ? r : last, m = mine < last ? mine : last;
      base[i] = reinterpret_cast<const char*>(a.x + first * a.x_stride);
      off[i] = uint32_t(m - first) * uint32_t(a.x_stride) * 2 + at;
    }
  }
  auto copy = [&](int i, int slot) {  // stages past the wave's last repeat it
    int t = wv + W * (i < count ? i : count - 1) + turned;
    t = t < S ? t : t - S;
    const size_t at = size_t(t) * kRowB;
#pragma unroll
    for (int c = 0; c < kCopies; ++c)
      __builtin_amdgcn_global_load_lds((const void*)(base[c] + at + off[c]), (lds_ptr_t)(ring + slot * kSlot + c * 1024), 16,
                                       0, 0);
  };
  f32x4 acc[1][1] = {{f32x4{0.f, 0.f, 0.f, 0.f}}};
  if (count > 0) {
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) copy(i, i);
    int slot = 0;
    for (int i = 0; i < count; ++i) {
      wait_copies<(ST - 2) * kCopies>();  // this stage is there
      const char* p = ring + slot * kSlot;
      u32x4 fw[2], fx[2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int c = 16 * ((4 * hh + g) ^ swizzle(r16));
        fw[hh] = *reinterpret_cast<const u32x4*>(p + r16 * kRowB + c);
        const int t = r16 & (XR - 1);
        fx[hh] = *reinterpret_cast<const u32x4*>(p + (16 + t) * kRowB + 16 * ((4 * hh + g) ^ swizzle(t)));
      }
      // the slot of the stage before: its fragments went into the last pass's MFMAs
      copy(i + ST - 1, slot == 0 ? ST - 1 : slot - 1);
      wait_reads();
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) acc[0][0] = mfma16x16x32(fw[hh], fx[hh], acc[0][0]);
      slot = slot + 1 == ST ? 0 : slot + 1;
    }
    wait_copies<0>();
  }
  if (wv == W - 1 && a.K % kBK != 0) tail<1, 1, GLU>(a, acc, n0, 0, 0, lane);
  __syncthreads();  // nobody copies into LDS any more
  f32x4* sums = reinterpret_cast<f32x4*>(lds);
  sums[wv * kWave + lane] = acc[0][0];
  __syncthreads();
  if (wv != 0) return;
  acc[0][0] = sums[lane];
#pragma unroll
  for (int v = 1; v < W; ++v) acc[0][0] += sums[v * kWave + lane];
  wave_lds_fence();
  epilogue<1, 1, GLU>(a, acc, lds, 0, int(n0), lane);
}

template <int W, int ST, int XR, bool GLU>
hipError_t launch_few(const LinearArgs& a, hipStream_t stream) {
  constexpr int kBytes = W * ST * (2 + XR / 8) * 1024;
  static_assert(kBytes <= 160 * 1024, "LDS");
  const int64_t tiles = ((GLU ? 2 : 1) * int64_t(a.N) + 15) / 16;
  if (tiles > 0x7FFFFFFF || a.M > XR) return hipErrorInvalidValue;
  const void* fn = reinterpret_cast<const void*>(&k_linear_few<W, ST, XR, GLU>);
  if constexpr (kBytes > 65536) {
    const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != hipSuccess) return e;
  }
  LinearArgs args = a;
  void* params[] = {&args};
  return hipLaunchKernel(fn, dim3(unsigned(tiles)), dim3(W * kWave), params, kBytes, stream);
}

// Launches `fn` over `tiles` tiles times a.parts parts, then the kernel that joins the parts
// (`joins` workgroups per tile: its waves times their blocks of 16 tokens).
hipError_t launch_parts(const LinearArgs& a, const void* fn, int bytes, int waves, const void* join, int joins,
                        int64_t tiles, hipStream_t stream) {
  if (a.parts < 1 || tiles > 0x7FFFFFFF / a.parts || (a.parts > 1 && tiles * joins > 0x7FFFFFFF))
    return hipErrorInvalidValue;
  hipError_t e = bytes > 65536 ? hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, bytes) : hipSuccess;
  if (e != hipSuccess) return e;
  LinearArgs args = a;
  void* params[] = {&args};
  e = hipLaunchKernel(fn, dim3(unsigned(tiles * a.parts)), dim3(waves * kWave), params, bytes, stream);
  if (e != hipSuccess || a.parts == 1) return e;
  return hipLaunchKernel(join, dim3(unsigned(tiles * joins)), dim3(kWave), params, 0, stream);
}

template <bool GLU>
hipError_t launch_big(const LinearArgs& a, hipStream_t stream) {
  constexpr int kOut = GLU ? kBig / 2 : kBig;
  const int64_t tiles = (a.M + kBig - 1) / kBig * ((int64_t(a.N) + kOut - 1) / kOut);
  return launch_parts(a, reinterpret_cast<const void*>(&k_linear_big<GLU>), kBigLds, 8,
                      reinterpret_cast<const void*>(&k_linear_join<kBig, kBig, 4, 2, GLU>), 8 * 4, tiles, stream);
}

template <int BM, int BN, int WM, int WN, int ST, bool GLU>
hipError_t launch_tile(const LinearArgs& a, hipStream_t stream) {
  constexpr int kOut = GLU ? BN / 2 : BN;
  constexpr int kBytes = ST * (BM + BN) * kRowB;
  static_assert(kBytes <= 160 * 1024, "LDS");
  const int64_t tiles = (a.M + BM - 1) / BM * ((int64_t(a.N) + kOut - 1) / kOut);
  return launch_parts(a, reinterpret_cast<const void*>(&k_linear<BM, BN, WM, WN, ST, GLU>), kBytes, WM * WN,
                      reinterpret_cast<const void*>(&k_linear_join<BM, BN, WM, WN, GLU>), WN * BM / 16, tiles, stream);
}

// ---------------------------------------------------------------- launch of the chosen tile (linear_choice.h)
template <bool GLU>
hipError_t launch_shape(int tile, const LinearArgs& a, hipStream_t stream) {
  switch (tile) {
    case kFew8: return launch_few<4, 4, 8, GLU>(a, stream);
    case kFew16: return launch_few<4, 5, 16, GLU>(a, stream);
    case 0: return launch_big<GLU>(a, stream);
    case 1: return launch_tile<128, 256, 4, 2, 3, GLU>(a, stream);
    case 2: return launch_tile<256, 128, 4, 2, 3, GLU>(a, stream);
    case 3: return launch_tile<160, 160, 2, 2, 4, GLU>(a, stream);
    case 4: return launch_tile<128, 160, 2, 2, 4, GLU>(a, stream);
    case 5: return launch_tile<192, 128, 2, 2, 4, GLU>(a, stream);
    case 6: return launch_tile<128, 128, 2, 2, 4, GLU>(a, stream);
    case 7: return launch_tile<128, 128, 2, 2, 2, GLU>(a, stream);
    case 8: return launch_tile<64, 256, 2, 4, 4, GLU>(a, stream);
    case 9: return launch_tile<64, 128, 2, 4, 6, GLU>(a, stream);
    case 10: return launch_tile<64, 64, 2, 2, 4, GLU>(a, stream);
    case 11: return launch_tile<32, 128, 1, 4, 6, GLU>(a, stream);
    case 12: return launch_tile<32, 64, 1, 4, 8, GLU>(a, stream);
    case 13: return launch_tile<32, 32, 1, 2, 8, GLU>(a, stream);
    case 14: return launch_tile<16, 16, 1, 1, 12, GLU>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

int64_t linear_workspace_bytes(int64_t M, int K, int N, bool glu, int cus) {
  return M > 0 ? choose(M, K, N, glu, cus).bytes : 0;
}

int64_t linear_workspace_bytes_up_to(int64_t M, int K, int N, bool glu, int cus) {
  return most_bytes_up_to(M, K, N, glu, cus);
}

hipError_t launch_linear(const LinearArgs& a, int cus, hipStream_t stream) {
  if (a.M <= 0) return hipSuccess;
  const LinearChoice c = choose(a.M, a.K, a.N, a.glu != 0, cus);
  LinearArgs args = a;
  args.parts = c.parts;
  return a.glu ? launch_shape<true>(c.tile, args, stream) : launch_shape<false>(c.tile, args, stream);
}

}  // namespace engram
