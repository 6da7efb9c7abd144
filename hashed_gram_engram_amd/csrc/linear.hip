// Matrix product with bias, activation (plain or gated) and residual: out = residual + act(x w^T + bias).
//
// A workgroup computes a tile of BM tokens x BN weight rows over all of K, in stages of 64 features.
// A stage holds BN weight rows, then BM token rows, of 128 bytes each in LDS, 16-byte chunk c of row r
// at position c ^ (r & 7) (conflict-free for the fragment reads); ST slots form a ring that global ->
// LDS copies of 16 bytes per lane fill ST - 1 stages ahead, one workgroup barrier per stage.  The
// waves share the tile as WM x WN parts; a wave multiplies its part as blocks of
// v_mfma_f32_16x16x32_bf16 (weight rows as A, tokens as B: a lane then holds 4 consecutive output
// features of one token).
//
// Gated: the weight has the N gate rows, then the N value rows.  A tile takes 16 rows of the gate, the
// same 16 of the value, and so on, so a lane holds both factors of an output and the epilogue needs no
// exchange.
//
// Features past K (K is a multiple of 8) are copied from 16 zero bytes; weight rows past N and tokens
// past M repeat the last one and are not stored.
#include "common.h"
#include "serving.h"

namespace engram {

namespace {

typedef __attribute__((address_space(3))) void* lds_ptr_t;

__device__ const u32x4 kZero16 = {0u, 0u, 0u, 0u};

constexpr int kStageB = 128;  // bytes of a row's stage: 64 features

// ---------------------------------------------------------------- epilogue
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case 1: return fmaxf(z, 0.0f);
    case 2: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
    case 3: return z / (1.0f + expf(-1.5957691216057308f * (z + 0.044715f * z * z * z)));
    case 4: return z / (1.0f + expf(-z));
    case 5: return 1.0f / (1.0f + expf(-z));
    default: return z;
  }
}

// Columns c .. c + 3 of z, plus the bias of weight rows r .. r + 3 (rows past the last repeat it).
__device__ __forceinline__ f32x4 add_bias(f32x4 z, const float* bias, int64_t row, int64_t last) {
  if (bias == nullptr) return z;
#pragma unroll
  for (int e = 0; e < 4; ++e) z[e] += bias[row + e < last ? row + e : last];
  return z;
}

// One row segment of 8 output features, fp32 -> out, with the residual.
__device__ __forceinline__ void store8(const LinearArgs& a, int64_t m, int n, f32x4 lo, f32x4 hi, bool vec) {
  float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  const int64_t o = m * a.out_stride + n, q = m * a.residual_stride + n;
  if (a.fp32) {
    float* out = static_cast<float*>(a.out) + o;
    const float* res = static_cast<const float*>(a.residual) + q;
    if (vec && n + 8 <= a.N) {
      if (a.residual != nullptr) {
        lo += *reinterpret_cast<const f32x4*>(res);
        hi += *reinterpret_cast<const f32x4*>(res + 4);
      }
      *reinterpret_cast<f32x4*>(out) = lo;
      *reinterpret_cast<f32x4*>(out + 4) = hi;
      return;
    }
    for (int e = 0; e < 8; ++e)
      if (n + e < a.N) out[e] = v[e] + (a.residual != nullptr ? res[e] : 0.0f);
    return;
  }
  uint16_t* out = static_cast<uint16_t*>(a.out) + o;
  const uint16_t* res = static_cast<const uint16_t*>(a.residual) + q;
  if (vec && n + 8 <= a.N) {
    if (a.residual != nullptr) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(res);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] += bf16_lo(w[e]);
        v[2 * e + 1] += bf16_hi(w[e]);
      }
    }
    *reinterpret_cast<u32x4*>(out) =
        u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    return;
  }
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

// A wave's part of the tile: TN x TM blocks of 16 weight rows x 16 tokens, block (i, j) holding rows
// 16 i + 4 (l >> 4) + 0..3 of token 16 j + (l & 15).  16 tokens at a time pass through the wave's own
// piece of LDS (rows of W floats, 16 bytes of padding), so that stores are whole row segments.
template <int TN, int TM, bool GLU>
__device__ __forceinline__ void epilogue(const LinearArgs& a, const f32x4 (&acc)[TN][TM], char* lds, int64_t m0, int n0,
                                         int lane) {
  constexpr int kBlocks = GLU ? TN / 2 : TN;
  constexpr int kCols = kBlocks * 16;           // output features of the wave
  constexpr int kRow = kCols + 4;               // floats per LDS row
  constexpr int kLanes = kCols / 8;             // lanes per row when read back
  constexpr int kRows = kWave / kLanes;         // rows per pass
  float* buf = reinterpret_cast<float*>(lds);
  const bool vec = vector_rows(a);
  const int64_t last = int64_t(a.N) - 1;
#pragma unroll
  for (int j = 0; j < TM; ++j) {
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      const int c = 16 * i + 4 * (lane >> 4);
      f32x4 z;
      if constexpr (GLU) {
        z = add_bias(acc[2 * i][j], a.bias, n0 + c, last);
        const f32x4 u = add_bias(acc[2 * i + 1][j], a.bias, int64_t(a.N) + n0 + c, last + a.N);
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = activate(z[e], a.act) * u[e];
      } else {
        z = add_bias(acc[i][j], a.bias, n0 + c, last);
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = activate(z[e], a.act);
      }
      *reinterpret_cast<f32x4*>(buf + (lane & 15) * kRow + c) = z;
    }
    wave_lds_fence();
#pragma unroll
    for (int p = 0; p < 16; p += kRows) {
      const int t = p + lane / kLanes, c = 8 * (lane % kLanes);
      const int64_t m = m0 + 16 * j + t;
      if ((kRows <= 16 || t < 16) && m < a.M && n0 + c < a.N)
        store8(a, m, n0 + c, *reinterpret_cast<const f32x4*>(buf + t * kRow + c),
               *reinterpret_cast<const f32x4*>(buf + t * kRow + c + 4), vec);
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
__device__ __forceinline__ void group_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The weight row that row r of a tile holds (clamped into the weight).
template <bool GLU>
__device__ __forceinline__ int64_t weight_row(const LinearArgs& a, int64_t n0, int r) {
  if constexpr (!GLU) return n0 + r < a.N ? n0 + r : int64_t(a.N) - 1;
  int64_t n = n0 + (r >> 5) * 16 + (r & 15);
  n = n < a.N ? n : int64_t(a.N) - 1;
  return n + ((r >> 4) & 1) * int64_t(a.N);
}

// The tile of workgroup b of `tiles`: workgroups are dealt to the 8 XCDs round robin, so each XCD
// takes a run of consecutive tiles, token blocks fastest: a weight panel is read by one XCD, once.
__device__ __forceinline__ int64_t xcd_tile(int64_t b, int64_t tiles) {
  const int64_t q = tiles >> 3, rem = tiles & 7, x = b & 7;
  return x * q + (x < rem ? x : rem) + (b >> 3);
}

template <int BM, int BN, int WM, int WN, int ST, bool GLU>
__global__ __launch_bounds__(WM* WN* kWave) void k_linear(LinearArgs a) {
  constexpr int kWaves = WM * WN;
  constexpr int kRowsT = BM + BN;                 // rows of a stage
  constexpr int kSlot = kRowsT * kStageB;
  constexpr int kCopies = kRowsT / 8 / kWaves;    // copy instructions per wave and stage, 8 rows each
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
  constexpr int kOutCols = GLU ? BN / 2 : BN;
  static_assert(kRowsT % (8 * kWaves) == 0 && (!GLU || TN % 2 == 0), "tile");
  constexpr int kEpi = 16 * ((GLU ? TN / 2 : TN) * 16 + 4) * 4;  // bytes of a wave's epilogue buffer
  static_assert(kEpi * kWaves <= ST * kSlot, "epilogue buffer");
  extern __shared__ __attribute__((aligned(16))) char lds[];

  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tbs = (a.M + BM - 1) / BM;
  const int64_t tile = xcd_tile(blockIdx.x, gridDim.x);
  const int64_t m0 = (tile % tbs) * BM;
  const int64_t n0 = (tile / tbs) * kOutCols;
  const int S = (a.K + 63) / 64;

  // lane l of a copy fills bytes 16 l of 1 KB: row 8 q + (l >> 3), position l & 7, chunk (l & 7) ^ (l >> 3)
  const int rr = lane >> 3, chunk = (lane & 7) ^ rr;
  const char* src[kCopies];
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    const int r = (wv * kCopies + i) * 8 + rr;
    if (r < BN) {
      src[i] = reinterpret_cast<const char*>(a.w + weight_row<GLU>(a, n0, r) * a.K) + 16 * chunk;
    } else {
      int64_t m = m0 + r - BN;
      m = m < a.M ? m : a.M - 1;
      src[i] = reinterpret_cast<const char*>(a.x + m * a.x_stride) + 16 * chunk;
    }
  }
  auto copy_stage = [&](int t) {
    char* dst = lds + (t % ST) * kSlot;
    const bool past = t * 64 + 8 * chunk >= a.K;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const char* s = past ? reinterpret_cast<const char*>(&kZero16) : src[i] + size_t(t) * kStageB;
      __builtin_amdgcn_global_load_lds((const void*)s, (lds_ptr_t)(dst + (wv * kCopies + i) * 1024), 16, 0, 0);
    }
  };

  f32x4 acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int wn = wv % WN, wm = wv / WN;
  const int r16 = lane & 15, g = lane >> 4;
  for (int t = 0; t < ST - 1 && t < S; ++t) copy_stage(t);
  for (int t = 0; t < S; ++t) {
    // stage t has landed when only the copies of the ST - 2 stages behind it are in flight
    if (S - 1 - t >= ST - 2) wait_copies<(ST - 2) * kCopies>();
    else wait_copies<0>();
    group_barrier();  // everyone's copies of stage t; everyone is done with stage t - 1
    if (t + ST - 1 < S) copy_stage(t + ST - 1);
    const char* W = lds + (t % ST) * kSlot + wn * TN * 16 * kStageB;
    const char* X = lds + (t % ST) * kSlot + (BN + wm * TM * 16) * kStageB;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int off = r16 * kStageB + 16 * ((4 * hh + g) ^ (r16 & 7));
      u32x4 fw[TN], fx[TM];
#pragma unroll
      for (int i = 0; i < TN; ++i) fw[i] = *reinterpret_cast<const u32x4*>(W + i * 16 * kStageB + off);
#pragma unroll
      for (int j = 0; j < TM; ++j) fx[j] = *reinterpret_cast<const u32x4*>(X + j * 16 * kStageB + off);
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = mfma16x16x32(fw[i], fx[j], acc[i][j]);
    }
  }
  __syncthreads();  // the ring is free
  epilogue<TN, TM, GLU>(a, acc, lds + wv * kEpi, m0 + wm * TM * 16, int(n0) + wn * (GLU ? TN * 8 : TN * 16), lane);
}

template <int BM, int BN, int WM, int WN, int ST, bool GLU>
hipError_t launch_tile(const LinearArgs& a, hipStream_t stream) {
  constexpr int kOut = GLU ? BN / 2 : BN;
  constexpr int kBytes = ST * (BM + BN) * kStageB;
  const int64_t tiles = (a.M + BM - 1) / BM * ((int64_t(a.N) + kOut - 1) / kOut);
  if (tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  const void* fn = reinterpret_cast<const void*>(&k_linear<BM, BN, WM, WN, ST, GLU>);
  if constexpr (kBytes > 65536) {
    const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != hipSuccess) return e;
  }
  LinearArgs args = a;
  void* params[] = {&args};
  return hipLaunchKernel(fn, dim3(unsigned(tiles)), dim3(WM * WN * kWave), params, kBytes, stream);
}

template <bool GLU>
hipError_t launch_any(const LinearArgs& a, hipStream_t stream) {
  if (a.M <= 16) return launch_tile<32, 64, 2, 2, 4, GLU>(a, stream);
  if (a.M <= 64) return launch_tile<64, 64, 2, 2, 3, GLU>(a, stream);
  return launch_tile<128, 128, 2, 2, 2, GLU>(a, stream);
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, int num_cus, hipStream_t stream) {
  (void)num_cus;
  if (a.M <= 0) return hipSuccess;
  return a.glu ? launch_any<true>(a, stream) : launch_any<false>(a, stream);
}

}  // namespace engram
