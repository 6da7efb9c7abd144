// Norms behind and before a block, with its gate and residual scale, in one pass over the streams.
//
// Per (token, stream) row, all in fp32:
//   n = y rsqrt(mean(y^2) + eps) w_post,  r = alpha x + beta g n,  h = r rsqrt(mean(r^2) + eps') w_pre
// T threads take a row, NV vectors of 8 features each, and keep it in registers from the first load
// to the last store: x, y and a gate per feature are read once, r and h written once.  The two sums
// are fp32: NV * 8 squares in a thread, then a tree over the T threads.
//
// What bounds it: HBM for long inputs (x and y read, r and h written: 8192 tokens x 4 streams x 5120 with a
// shared y move 1.09 GB in 231 us, 4.7 TB/s, where a large copy reaches 4.8); launch and a chain of memory
// round trips for a decode step (64 such tokens 4.7 us).  r and h are stored past the caches (nothing of
// this launch reads them again): 244 -> 231 us.
#include "common.h"
#include "launch.h"
#include "serving.h"

namespace engram {

namespace {

__device__ __forceinline__ void unpack8(u32x4 w, float (&v)[8]) {
  v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
  v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}
// The bf16 bits that unpack8 took (a rounding would change a NaN's).
__device__ __forceinline__ u32x4 bits8(const float (&v)[8]) {
  u32x4 w;
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = (__float_as_uint(v[2 * e]) >> 16) | (__float_as_uint(v[2 * e + 1]) & 0xFFFF0000u);
  return w;
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = a[e];
    v[4 + e] = b[e];
  }
}

// Sum over the T threads of a row.
template <int T>
__device__ __forceinline__ float row_sum(float v, float* tmp) {
  v = wave_sum(v);
  if constexpr (T > kWave) {
    const int wv = threadIdx.x >> 6;
    __syncthreads();  // the previous sum's readers are done
    if ((threadIdx.x & 63) == 0) tmp[wv] = v;
    __syncthreads();
    const int w0 = (wv / (T / kWave)) * (T / kWave);
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < T / kWave; ++w) v += tmp[w0 + w];
  }
  return v;
}

// 1 / sqrt(m) of a mean square.  The hardware's root takes a denormal for 0 (rows below 1e-19 with an epsilon
// of 0 came out infinite), so a small m is scaled by 2^60 first.
__device__ __forceinline__ float rstd_of(float m) {
  const bool small = m < 0x1p-100f;
  const float r = __frsqrt_rn(small ? m * 0x1p60f : m);
  return small ? r * 0x1p30f : r;
}

// T threads per row, NV vectors of 8 features per thread (dim <= T * NV * 8), FP32 streams or bf16.
template <int T, int NV, bool FP32>
__global__ __launch_bounds__(T < 256 ? 256 : T) void k_residual_norm(NormArgs a) {
  constexpr int kThreads = T < 256 ? 256 : T;
  constexpr int kRows = kThreads / T;  // rows of a workgroup
  __shared__ float tmp[kThreads / kWave];
  const int lane = threadIdx.x % T;
  // (rows are fewer than 2^31: 32-bit divisions)
  const uint32_t rows = uint32_t(a.M * a.hc), row_raw = blockIdx.x * uint32_t(kRows) + threadIdx.x / T;
  const bool in = row_raw < rows;
  const int64_t row = in ? row_raw : rows - 1;  // rows past the last repeat it and store nothing
  const int64_t m = uint32_t(row) / uint32_t(a.hc);
  const int s = int(uint32_t(row) - uint32_t(m) * uint32_t(a.hc));
  const int ys = a.y_streams == 1 ? 0 : s;
  const int nvec = a.dim >> 3;
  const bool has_y = a.y != nullptr;
  const bool open = has_y && (a.token_mask == nullptr || a.token_mask[m] != 0);

  float r[NV][8];
  u32x4 yv[NV];
  // every load of the row is in flight before the first use
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int v = lane + k * T;
    const bool ok = v < nvec;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[k][e] = 0.0f;
    yv[k] = u32x4{0u, 0u, 0u, 0u};
    if (ok) {
      if constexpr (FP32) load8(static_cast<const float*>(a.x) + row * a.dim + 8 * v, r[k]);
      else unpack8(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.x) + row * a.dim + 8 * v), r[k]);
      if (open) yv[k] = *reinterpret_cast<const u32x4*>(a.y + m * a.y_stride + int64_t(ys) * a.dim + 8 * v);
    }
  }
  // with few vectors a thread (short inputs: the time is a chain of memory round trips) the weights are
  // fetched along with them
  constexpr bool kEarly = NV <= 2;
  float wp[kEarly ? NV : 1][8], wh[kEarly ? NV : 1][8];
  auto weight = [&](const float* w, int k, float (&to)[8]) {
    const int v = lane + k * T;
#pragma unroll
    for (int e = 0; e < 8; ++e) to[e] = 1.0f;
    if (w != nullptr && v < nvec) load8(w + int64_t(s) * a.dim + 8 * v, to);
  };
  if constexpr (kEarly) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (open) weight(a.post_weight, k, wp[k]);
      if (a.h != nullptr) weight(a.pre_weight, k, wh[k]);
    }
  }
  float scale = a.beta;
  if (a.gate_kind == 1 && open) scale *= static_cast<const float*>(a.gate)[row];
  if (a.post_norm && has_y) {
    float q = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float y[8];
      unpack8(yv[k], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) q += y[e] * y[e];
    }
    q = row_sum<T>(q, tmp);
    scale *= rstd_of(q / float(a.dim) + a.post_eps);
  }
  if (open) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = lane + k * T;
      if (v >= nvec) continue;
      float n[8];
      unpack8(yv[k], n);
      if (a.post_weight != nullptr) {
        float w[8];
        if constexpr (!kEarly) weight(a.post_weight, k, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] *= kEarly ? wp[kEarly ? k : 0][e] : w[e];
      }
      if (a.gate_kind == 2) {
        float z[8];
        unpack8(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.gate) + m * a.gate_stride +
                                                int64_t(ys) * a.dim + 8 * v), z);
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] /= 1.0f + expf(-z[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) r[k][e] = a.alpha * r[k][e] + scale * n[e];
    }
  }
  if (in && has_y && (open || a.out != a.x)) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = lane + k * T;
      if (v >= nvec) continue;
      if constexpr (FP32) {
        float* o = static_cast<float*>(a.out) + row * a.dim + 8 * v;
        __builtin_nontemporal_store(f32x4{r[k][0], r[k][1], r[k][2], r[k][3]}, reinterpret_cast<f32x4*>(o));
        __builtin_nontemporal_store(f32x4{r[k][4], r[k][5], r[k][6], r[k][7]}, reinterpret_cast<f32x4*>(o + 4));
      } else {
        const u32x4 w = open ? pack8(r[k]) : bits8(r[k]);
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + row * a.dim + 8 * v));
      }
    }
  }
  if (a.h != nullptr) {
    float q = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) q += r[k][e] * r[k][e];
    q = row_sum<T>(q, tmp);
    const float rstd = rstd_of(q / float(a.dim) + a.pre_eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = lane + k * T;
      if (v >= nvec || !in) continue;
      float n[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] = r[k][e] * rstd;
      if (a.pre_weight != nullptr) {
        float w[8];
        if constexpr (!kEarly) weight(a.pre_weight, k, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] *= kEarly ? wh[kEarly ? k : 0][e] : w[e];
      }
      __builtin_nontemporal_store(pack8(n), reinterpret_cast<u32x4*>(a.h + row * a.dim + 8 * v));
    }
  }
}

template <int T, int NV>
hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  constexpr int kRows = (T < 256 ? 256 : T) / T;
  const int64_t grid = (a.M * a.hc + kRows - 1) / kRows;
  if (!launch_fits(grid, T < 256 ? 256 : T)) return hipErrorInvalidValue;
  NormArgs args = a;
  void* params[] = {&args};
  const void* fn = a.fp32 ? reinterpret_cast<const void*>(&k_residual_norm<T, NV, true>)
                          : reinterpret_cast<const void*>(&k_residual_norm<T, NV, false>);
  return hipLaunchKernel(fn, dim3(unsigned(grid)), dim3(T < 256 ? 256 : T), params, 0, stream);
}

template <int T>
hipError_t launch_threads(const NormArgs& a, hipStream_t stream) {
  const int nv = ((a.dim >> 3) + T - 1) / T;
  if (nv <= 1) return launch_norm<T, 1>(a, stream);
  if (nv <= 2) return launch_norm<T, 2>(a, stream);
  if (nv <= 3) return launch_norm<T, 3>(a, stream);
  if (nv <= 4) return launch_norm<T, 4>(a, stream);
  if (nv <= 5) return launch_norm<T, 5>(a, stream);
  return hipErrorInvalidValue;
}

}  // namespace

// Threads of a row: as few as hold it in 5 vectors each, so that a long input's waves have many loads in
// flight and sum with few barriers; while the rows leave threads of the device idle (2048 fit a compute
// unit) twice as many, up to one vector each.  Measured at dim 5120: 32,768 rows 231 us with 128 threads
// a row, 328 us with 512; 256 rows 6.9 us with 128, 4.7 us with 512.
hipError_t launch_residual_norm(const NormArgs& a, int cus, hipStream_t stream) {
  const int nvec = a.dim >> 3;
  int t = 64;
  while (t < 1024 && nvec > 5 * t) t *= 2;
  while (t < 1024 && 2 * t <= nvec && a.M * a.hc * 2 * t <= int64_t(2048) * cus) t *= 2;
  switch (t) {
    case 64: return launch_threads<64>(a, stream);
    case 128: return launch_threads<128>(a, stream);
    case 256: return launch_threads<256>(a, stream);
    case 512: return launch_threads<512>(a, stream);
    default: return launch_threads<1024>(a, stream);
  }
}

}  // namespace engram
