// Norms behind and before a block, with its gate and residual scale, in one pass over the streams.
//
// Per (token, stream) row, all in fp32:
//   n = y rsqrt(mean(y^2) + eps) w_post,  r = alpha x + beta g n,  h = r rsqrt(mean(r^2) + eps') w_pre
// T threads take a row, NV vectors of 8 features each, and keep it in registers from the first load
// to the last store: x, y and a gate per feature are read once, r and h written once.  The two sums
// are fp32: NV * 8 squares in a thread, then a tree over the T threads.
//
// What bounds it: HBM for long inputs (x and y read, r and h written); launch and one memory round
// trip for a decode step.
#include "common.h"
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

// T threads per row, NV vectors of 8 features per thread (dim <= T * NV * 8), FP32 streams or bf16.
template <int T, int NV, bool FP32>
__global__ __launch_bounds__(T < 256 ? 256 : T) void k_residual_norm(NormArgs a) {
  constexpr int kThreads = T < 256 ? 256 : T;
  constexpr int kRows = kThreads / T;  // rows of a workgroup
  __shared__ float tmp[kThreads / kWave];
  const int lane = threadIdx.x % T;
  const int64_t rows = a.M * a.hc;
  const int64_t row_raw = int64_t(blockIdx.x) * kRows + threadIdx.x / T;
  const bool in = row_raw < rows;
  const int64_t row = in ? row_raw : rows - 1;  // rows past the last repeat it and store nothing
  const int64_t m = row / a.hc;
  const int s = int(row - m * a.hc);
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
    scale *= __frsqrt_rn(q / float(a.dim) + a.post_eps);
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
        load8(a.post_weight + int64_t(s) * a.dim + 8 * v, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] *= w[e];
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
        *reinterpret_cast<f32x4*>(o) = f32x4{r[k][0], r[k][1], r[k][2], r[k][3]};
        *reinterpret_cast<f32x4*>(o + 4) = f32x4{r[k][4], r[k][5], r[k][6], r[k][7]};
      } else {
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.out) + row * a.dim + 8 * v) = pack8(r[k]);
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
    const float rstd = __frsqrt_rn(q / float(a.dim) + a.pre_eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int v = lane + k * T;
      if (v >= nvec || !in) continue;
      float n[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] = r[k][e] * rstd;
      if (a.pre_weight != nullptr) {
        float w[8];
        load8(a.pre_weight + int64_t(s) * a.dim + 8 * v, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] *= w[e];
      }
      *reinterpret_cast<u32x4*>(a.h + row * a.dim + 8 * v) = pack8(n);
    }
  }
}

template <int T, int NV>
hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
  constexpr int kRows = (T < 256 ? 256 : T) / T;
  const int64_t grid = (a.M * a.hc + kRows - 1) / kRows;
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  NormArgs args = a;
  void* params[] = {&args};
  const void* fn = a.fp32 ? reinterpret_cast<const void*>(&k_residual_norm<T, NV, true>)
                          : reinterpret_cast<const void*>(&k_residual_norm<T, NV, false>);
  return hipLaunchKernel(fn, dim3(unsigned(grid)), dim3(T < 256 ? 256 : T), params, 0, stream);
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs& a, hipStream_t stream) {
  const int nvec = a.dim >> 3;
  if (nvec <= 64) return launch_norm<64, 1>(a, stream);
  if (nvec <= 128) return launch_norm<64, 2>(a, stream);
  if (nvec <= 256) return launch_norm<128, 2>(a, stream);
  if (nvec <= 512) return launch_norm<128, 4>(a, stream);
  if (nvec <= 640) return launch_norm<128, 5>(a, stream);
  if (nvec <= 1024) return launch_norm<256, 4>(a, stream);
  if (nvec <= 2048) return launch_norm<256, 8>(a, stream);
  if (nvec <= 4096) return launch_norm<1024, 4>(a, stream);
  if (nvec <= 8192) return launch_norm<1024, 8>(a, stream);
  return hipErrorInvalidValue;
}

}  // namespace engram
