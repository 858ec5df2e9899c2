// Layer norm and its gradient (sm_103a).
//
// Both are bound by memory: each reads and writes every row once, so a row
// lives in the registers of the threads that share it.  `tpr` threads (a power
// of two; part of a warp, or whole warps of one block) hold a row as NV vectors
// of VEC elements each, thread l the vectors l, l + tpr, ...; rows whose
// address or pitch is no multiple of 16 bytes, or whose length is no multiple
// of the vector, take VEC = 1.  Rows too long for that are walked by one block
// in several passes.
//
// Backward, a block takes rows g, g + G, ... and keeps the sums over its rows
// of dy xhat and dy for the columns its threads own in fp32 registers; they go
// to the workspace once, and a second kernel adds the blocks' sums in a fixed
// order.

#include <algorithm>

#include <cuda_bf16.h>

#include <type_traits>

#include "block.h"
#include "pdl.h"
#include "ptx.h"

namespace tpo {

namespace {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16* p, float v) { *p = __float2bfloat16_rn(v); }

// VEC consecutive elements as they lie in memory (16 bytes of x's type, or one element).
template <class T, int VEC>
struct alignas(VEC * sizeof(T) > 16 ? 16 : VEC * sizeof(T)) Vec {
  T e[VEC];
};
template <class T, int VEC>
__device__ __forceinline__ Vec<T, VEC> load(const T* p) {
  return *reinterpret_cast<const Vec<T, VEC>*>(p);
}

// Sums of two values over the `tpr` threads of a row, the same bits in each of
// them; `red` holds two floats per warp and is free for the next call after
// the one that follows (the callers alternate between two).
__device__ __forceinline__ float2 row_sum(float a, float b, int tpr, float2* red) {
#pragma unroll
  for (int d = 16; d; d >>= 1)
    if (d < tpr) {
      a += __shfl_xor_sync(0xffffffffu, a, d);
      b += __shfl_xor_sync(0xffffffffu, b, d);
    }
  if (tpr > 32) {
    const int warp = threadIdx.x >> 5, per = tpr >> 5, first = warp & ~(per - 1);
    if ((threadIdx.x & 31) == 0) red[warp] = make_float2(a, b);
    __syncthreads();
    a = b = 0.0f;
    for (int w = 0; w < per; ++w) {
      const float2 v = red[first + w];
      a += v.x;
      b += v.y;
    }
  }
  return make_float2(a, b);
}

template <class T, class W, int VEC, int NV>
__global__ void __launch_bounds__(512) norm_kernel(const NormArgs a, int tpr) {
  __shared__ float2 red[2][32];
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & (tpr - 1);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  const bool live = row < a.n;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  Vec<T, VEC> v[NV];
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lane + i * tpr) * VEC;
    if (live && c < a.k) v[i] = load<T, VEC>(x + c);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (live && (lane + i * tpr) * VEC < a.k)
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += to_f(v[i].e[j]);
  const float inv_k = 1.0f / static_cast<float>(a.k);
  const float mean = row_sum(s, 0.0f, tpr, red[0]).x * inv_k;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (live && (lane + i * tpr) * VEC < a.k)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float d = to_f(v[i].e[j]) - mean;
        s += d * d;
      }
  const float rstd = 1.0f / sqrtf(row_sum(s, 0.0f, tpr, red[1]).x * inv_k + a.eps);
  if (!live) return;
  const W *gamma = static_cast<const W*>(a.gamma), *beta = static_cast<const W*>(a.beta);
  T* y = static_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lane + i * tpr) * VEC;
    if (c >= a.k) continue;
    Vec<T, VEC> o;
    Vec<W, VEC> g, b;
    if (gamma) g = load<W, VEC>(gamma + c);
    if (beta) b = load<W, VEC>(beta + c);
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      put(&o.e[j], (to_f(v[i].e[j]) - mean) * rstd * (gamma ? to_f(g.e[j]) : 1.0f) + (beta ? to_f(b.e[j]) : 0.0f));
    *reinterpret_cast<Vec<T, VEC>*>(y + c) = o;
  }
  if (lane == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// The gradient: block g takes the row sets g, g + gridDim.x, ... of blockDim.x
// / tpr rows each; the next set's loads are in flight while a set is summed.
// part: [gridDim.x][2][k] fp32, this block's sums (NULL: not wanted).
template <class T, class W, int VEC, int NV>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormArgs a, int tpr, float* part) {
  __shared__ float2 red[2][32];
  extern __shared__ float sums[];  // one row of columns, to add the block's row groups
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = blockDim.x / tpr;
  const W* gamma = static_cast<const W*>(a.gamma);
  Vec<T, VEC> x[NV], dy[NV], xn[NV], dyn[NV];
  float dg[NV][VEC] = {}, db[NV][VEC] = {};
  float mean = 0.0f, rstd = 0.0f, mean_n = 0.0f, rstd_n = 0.0f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t row = static_cast<int64_t>(blockIdx.x) * groups + group;
  const int64_t sets = (a.n + groups - 1) / groups;  // row sets in all
  auto fetch = [&](int64_t r, Vec<T, VEC>(&px)[NV], Vec<T, VEC>(&pd)[NV], float& m, float& q) {
    if (r >= a.n) return;
    const T *sx = static_cast<const T*>(a.x) + r * a.ldx, *sd = static_cast<const T*>(a.dy) + r * a.lddy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * tpr) * VEC;
      if (c < a.k) {
        px[i] = load<T, VEC>(sx + c);
        pd[i] = load<T, VEC>(sd + c);
      }
    }
    m = a.mean[r];
    q = a.rstd[r];
  };
  fetch(row, x, dy, mean, rstd);
  const float inv_k = 1.0f / static_cast<float>(a.k);
  int buf = 0;
  for (int64_t set = blockIdx.x; set < sets; set += gridDim.x, row += step, buf ^= 1) {
    const bool live = row < a.n;
    fetch(row + step, xn, dyn, mean_n, rstd_n);
    float s1 = 0.0f, s2 = 0.0f;
    if (live)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * tpr) * VEC;
        if (c >= a.k) continue;
        Vec<W, VEC> g;
        if (gamma) g = load<W, VEC>(gamma + c);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float d = to_f(dy[i].e[j]), h = (to_f(x[i].e[j]) - mean) * rstd;
          const float w = gamma ? d * to_f(g.e[j]) : d;
          s1 += w;
          s2 += w * h;
          dg[i][j] += d * h;
          db[i][j] += d;
        }
      }
    if (a.y) {
      const float2 t = row_sum(s1, s2, tpr, red[buf]);
      const float m1 = t.x * inv_k, m2 = t.y * inv_k;
      if (live) {
        T* o = static_cast<T*>(a.y) + row * a.ldy;
        const T* dres = a.dres ? static_cast<const T*>(a.dres) + row * a.lddres : nullptr;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (lane + i * tpr) * VEC;
          if (c >= a.k) continue;
          Vec<W, VEC> g;
          if (gamma) g = load<W, VEC>(gamma + c);
          Vec<T, VEC> r, e;
          if (dres) e = load<T, VEC>(dres + c);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float d = to_f(dy[i].e[j]), h = (to_f(x[i].e[j]) - mean) * rstd;
            const float w = gamma ? d * to_f(g.e[j]) : d;
            put(&r.e[j], rstd * (w - m1 - h * m2) + (dres ? to_f(e.e[j]) : 0.0f));
          }
          *reinterpret_cast<Vec<T, VEC>*>(o + c) = r;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] = xn[i];
      dy[i] = dyn[i];
    }
    mean = mean_n;
    rstd = rstd_n;
  }
  if (!part) return;
  float* out = part + static_cast<int64_t>(blockIdx.x) * 2 * a.k;
  // the block's row groups one after another: a fixed order of additions
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    for (int q = 0; q < groups; ++q) {
      if (groups > 1) __syncthreads();
      if (q != group) continue;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int c = (lane + i * tpr) * VEC + j;
          if (c >= a.k) continue;
          float v = which ? db[i][j] : dg[i][j];
          if (q > 0) v += sums[c];
          if (q + 1 < groups)
            sums[c] = v;
          else
            out[which * a.k + c] = v;
        }
    }
  }
}

// ------------------------------------------------------------------ long rows

__device__ float block_sum(float v, float* part) {
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < 32; ++w) s += part[w];
  return s;
}

// One block per row, three passes (the later two mostly from L2).
template <class T, class W>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormArgs a) {
  __shared__ float red[32];
  grid_dep_launch();
  grid_dep_wait();
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  T* y = static_cast<T*>(a.y) + row * a.ldy;
  const W *gamma = static_cast<const W*>(a.gamma), *beta = static_cast<const W*>(a.beta);
  float s = 0.0f;
  for (int64_t j = threadIdx.x; j < a.k; j += 1024) s += to_f(x[j]);
  const float mean = block_sum(s, red) / a.k;
  s = 0.0f;
  for (int64_t j = threadIdx.x; j < a.k; j += 1024) {
    const float d = to_f(x[j]) - mean;
    s += d * d;
  }
  const float rstd = 1.0f / sqrtf(block_sum(s, red) / a.k + a.eps);
  for (int64_t j = threadIdx.x; j < a.k; j += 1024)
    put(&y[j], (to_f(x[j]) - mean) * rstd * (gamma ? to_f(gamma[j]) : 1.0f) + (beta ? to_f(beta[j]) : 0.0f));
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

template <class T, class W>
__global__ void __launch_bounds__(1024) norm_long_dx_kernel(const NormArgs a) {
  __shared__ float red[32];
  grid_dep_launch();
  grid_dep_wait();
  const int64_t row = blockIdx.x;
  const T *x = static_cast<const T*>(a.x) + row * a.ldx, *dy = static_cast<const T*>(a.dy) + row * a.lddy;
  const T* dres = a.dres ? static_cast<const T*>(a.dres) + row * a.lddres : nullptr;
  T* dx = static_cast<T*>(a.y) + row * a.ldy;
  const W* gamma = static_cast<const W*>(a.gamma);
  const float mean = a.mean[row], rstd = a.rstd[row];
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t j = threadIdx.x; j < a.k; j += 1024) {
    const float v = to_f(dy[j]) * (gamma ? to_f(gamma[j]) : 1.0f);
    s1 += v;
    s2 += v * ((to_f(x[j]) - mean) * rstd);
  }
  s1 = block_sum(s1, red) / a.k;
  s2 = block_sum(s2, red) / a.k;
  for (int64_t j = threadIdx.x; j < a.k; j += 1024) {
    const float v = to_f(dy[j]) * (gamma ? to_f(gamma[j]) : 1.0f);
    const float xhat = (to_f(x[j]) - mean) * rstd;
    put(&dx[j], rstd * (v - s1 - xhat * s2) + (dres ? to_f(dres[j]) : 0.0f));
  }
}

// Sums over the rows g, g + gridDim.y, ... of dy xhat and dy, one thread per column.
template <class T>
__global__ void __launch_bounds__(256) norm_long_dw_kernel(const NormArgs a, float* part) {
  grid_dep_launch();
  grid_dep_wait();
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (j >= a.k) return;
  float dg = 0.0f, db = 0.0f;
#pragma unroll 4
  for (int64_t i = blockIdx.y; i < a.n; i += gridDim.y) {
    const float d = to_f(static_cast<const T*>(a.dy)[i * a.lddy + j]);
    dg += d * ((to_f(static_cast<const T*>(a.x)[i * a.ldx + j]) - a.mean[i]) * a.rstd[i]);
    db += d;
  }
  part[static_cast<int64_t>(blockIdx.y) * 2 * a.k + j] = dg;
  part[static_cast<int64_t>(blockIdx.y) * 2 * a.k + a.k + j] = db;
}

// ------------------------------------------------------------------ host side

template <class F>
cudaError_t with_types(int dtype, int wdtype, F f) {
  if (dtype == TPO_F32) return wdtype == TPO_F32 ? f(float(), float()) : f(float(), bf16());
  return wdtype == TPO_F32 ? f(bf16(), float()) : f(bf16(), bf16());
}
template <class F>
cudaError_t with_nv(int nv, F f) {
  switch (nv) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    case 8: return f(std::integral_constant<int, 8>());
    default: return f(std::integral_constant<int, 16>());
  }
}

bool vec_ok(const void* p, int64_t ld, int64_t rows, int elem) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld * elem % 16 == 0);
}

// How a row is shared: vectors per thread and threads per row; tpr = 0 when it is too long.
struct Share {
  int nv, tpr;
};
Share share(int64_t vecs, int nv, int most_nv, int most_tpr) {
  Share s{nv, 1};
  while (static_cast<int64_t>(s.tpr) * s.nv < vecs) {
    if (s.tpr < most_tpr)
      s.tpr *= 2;
    else if (s.nv < most_nv)
      s.nv *= 2;
    else
      return {0, 0};
  }
  return s;
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int dtype, int wdtype, cudaStream_t s) {
  return with_types(dtype, wdtype, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    constexpr int V = 16 / sizeof(T);
    const bool vec = a.k % V == 0 && vec_ok(a.x, a.ldx, a.n, sizeof(T)) && vec_ok(a.y, a.ldy, a.n, sizeof(T)) &&
                     vec_ok(a.gamma, 0, 1, 4) && vec_ok(a.beta, 0, 1, 4);
    // few rows: as many threads per row as there are vectors; many: four vectors a thread
    const Share h = share(vec ? a.k / V : a.k, a.n >= 608 ? 4 : 1, 8, 512);
    if (!h.tpr) return launch_pdl(norm_long_kernel<T, W>, dim3(static_cast<unsigned>(a.n)), dim3(1024), 0, s, a);
    const int threads = std::max(h.tpr, 128), rows = threads / h.tpr;
    const dim3 grid(static_cast<unsigned>((a.n + rows - 1) / rows));
    return with_nv(h.nv, [&](auto nv) {
      constexpr int NV = decltype(nv)::value <= 8 ? decltype(nv)::value : 8;
      if (vec) return launch_pdl(norm_kernel<T, W, V, NV>, grid, dim3(threads), 0, s, a, h.tpr);
      return launch_pdl(norm_kernel<T, W, 1, NV>, grid, dim3(threads), 0, s, a, h.tpr);
    });
  });
}

cudaError_t launch_norm_bwd(const NormArgs& a, int dtype, int wdtype, float* part, cudaStream_t s) {
  return with_types(dtype, wdtype, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    constexpr int V = 16 / sizeof(T);
    const bool wants = a.dgamma || a.dbeta;
    const bool vec = a.k % V == 0 && vec_ok(a.x, a.ldx, a.n, sizeof(T)) && vec_ok(a.dy, a.lddy, a.n, sizeof(T)) &&
                     vec_ok(a.dres, a.lddres, a.n, sizeof(T)) && vec_ok(a.y, a.ldy, a.n, sizeof(T)) &&
                     vec_ok(a.gamma, 0, 1, 4);
    const Share h = share(vec ? a.k / V : a.k, 1, vec ? 2 : 16, 512);
    if (!wants) part = nullptr;
    int parts = 0;
    cudaError_t e = cudaSuccess;
    if (h.tpr && a.n > 0) {
      const int threads = std::max(h.tpr, 256), rows = threads / h.tpr;
      parts = static_cast<int>(std::min<int64_t>((a.n + rows - 1) / rows, NORM_PARTS));
      const size_t smem = rows > 1 ? static_cast<size_t>(a.k) * 4 : 0;
      e = with_nv(h.nv, [&](auto nv) {
        constexpr int NV = decltype(nv)::value;
        constexpr int NW = NV <= 2 ? NV : 2;
        if (vec) return launch_pdl(norm_bwd_kernel<T, W, V, NW>, dim3(parts), dim3(threads), smem, s, a, h.tpr, part);
        return launch_pdl(norm_bwd_kernel<T, W, 1, NV>, dim3(parts), dim3(threads), smem, s, a, h.tpr, part);
      });
    } else if (a.n > 0) {
      // the weights' gradients first: dx may overwrite dy
      parts = static_cast<int>(std::min<int64_t>(a.n, 32));
      if (wants)
        e = launch_pdl(norm_long_dw_kernel<T>, dim3(static_cast<unsigned>((a.k + 255) / 256), parts), dim3(256), 0, s,
                       a, part);
      if (e == cudaSuccess && a.y)
        e = launch_pdl(norm_long_dx_kernel<T, W>, dim3(static_cast<unsigned>(a.n)), dim3(1024), 0, s, a);
    }
    if (e == cudaSuccess && wants)
      e = launch_column_sums(part, parts, 2, a.k, a.dgamma, a.dbeta, wdtype, s);
    return e;
  });
}

}  // namespace tpo
