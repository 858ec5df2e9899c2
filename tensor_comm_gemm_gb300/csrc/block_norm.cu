// Layer norm and its gradient, first form: one thread block per row, one
// thread per column for the weights' gradients.

#include <cuda_bf16.h>

#include <type_traits>

#include "block.h"

namespace tpo {

namespace {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ float block_sum(float v) {
  __shared__ float part[8];
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < 8; ++w) s += part[w];
  return s;
}

template <class T, class W>
__global__ void __launch_bounds__(256) norm_kernel(const NormArgs a) {
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  T* y = static_cast<T*>(a.y) + row * a.ldy;
  const W *gamma = static_cast<const W*>(a.gamma), *beta = static_cast<const W*>(a.beta);
  float s = 0.0f;
  for (int64_t j = threadIdx.x; j < a.k; j += 256) s += to_f(x[j]);
  const float mean = block_sum(s) / a.k;
  s = 0.0f;
  for (int64_t j = threadIdx.x; j < a.k; j += 256) {
    const float d = to_f(x[j]) - mean;
    s += d * d;
  }
  const float rstd = 1.0f / sqrtf(block_sum(s) / a.k + a.eps);
  for (int64_t j = threadIdx.x; j < a.k; j += 256)
    put(&y[j], (to_f(x[j]) - mean) * rstd * (gamma ? to_f(gamma[j]) : 1.0f) + (beta ? to_f(beta[j]) : 0.0f));
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

template <class T, class W>
__global__ void __launch_bounds__(256) norm_dx_kernel(const NormArgs a) {
  const int64_t row = blockIdx.x;
  const T *x = static_cast<const T*>(a.x) + row * a.ldx, *dy = static_cast<const T*>(a.dy) + row * a.lddy;
  const T* dres = a.dres ? static_cast<const T*>(a.dres) + row * a.lddres : nullptr;
  T* dx = static_cast<T*>(a.y) + row * a.ldy;
  const W* gamma = static_cast<const W*>(a.gamma);
  const float mean = a.mean[row], rstd = a.rstd[row];
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t j = threadIdx.x; j < a.k; j += 256) {
    const float v = to_f(dy[j]) * (gamma ? to_f(gamma[j]) : 1.0f);
    s1 += v;
    s2 += v * ((to_f(x[j]) - mean) * rstd);
  }
  s1 = block_sum(s1) / a.k;
  s2 = block_sum(s2) / a.k;
  for (int64_t j = threadIdx.x; j < a.k; j += 256) {
    const float v = to_f(dy[j]) * (gamma ? to_f(gamma[j]) : 1.0f);
    const float xhat = (to_f(x[j]) - mean) * rstd;
    put(&dx[j], rstd * (v - s1 - xhat * s2) + (dres ? to_f(dres[j]) : 0.0f));
  }
}

template <class T, class W>
__global__ void __launch_bounds__(128) norm_dw_kernel(const NormArgs a) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  if (j >= a.k) return;
  float dg = 0.0f, db = 0.0f;
  for (int64_t i = 0; i < a.n; ++i) {
    const float d = to_f(static_cast<const T*>(a.dy)[i * a.lddy + j]);
    dg += d * ((to_f(static_cast<const T*>(a.x)[i * a.ldx + j]) - a.mean[i]) * a.rstd[i]);
    db += d;
  }
  if (a.dgamma) put(static_cast<W*>(a.dgamma) + j, dg);
  if (a.dbeta) put(static_cast<W*>(a.dbeta) + j, db);
}

template <class F>
cudaError_t with_types(int dtype, int wdtype, F f) {
  if (dtype == TPO_F32) return wdtype == TPO_F32 ? f(float(), float()) : f(float(), bf16());
  return wdtype == TPO_F32 ? f(bf16(), float()) : f(bf16(), bf16());
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int dtype, int wdtype, cudaStream_t s) {
  return with_types(dtype, wdtype, [&](auto t, auto w) {
    norm_kernel<decltype(t), decltype(w)><<<static_cast<unsigned>(a.n), 256, 0, s>>>(a);
    return cudaGetLastError();
  });
}

cudaError_t launch_norm_bwd(const NormArgs& a, int dtype, int wdtype, cudaStream_t s) {
  return with_types(dtype, wdtype, [&](auto t, auto w) {
    // the weights' gradients first: dx may overwrite dy
    if (a.dgamma || a.dbeta)
      norm_dw_kernel<decltype(t), decltype(w)><<<static_cast<unsigned>((a.k + 127) / 128), 128, 0, s>>>(a);
    if (a.y && a.n > 0) norm_dx_kernel<decltype(t), decltype(w)><<<static_cast<unsigned>(a.n), 256, 0, s>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace tpo
