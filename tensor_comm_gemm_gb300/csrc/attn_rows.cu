// Gradient of attention, one warp a row (sm_103a).

#include <cuda_bf16.h>

#include <cmath>

#include "attn.h"
#include "pdl.h"
#include "ptx.h"

namespace tpo {

namespace {

using bf16 = __nv_bfloat16;
constexpr int WARPS = 8;
constexpr int PER_LANE = 4;  // elements of a head a lane holds: lane, lane + 32, ...

__device__ __forceinline__ const bf16* row_of(const Heads& x, int64_t row, int64_t head) {
  return static_cast<const bf16*>(x.p) + row * x.ld + head * x.hs;
}
__device__ __forceinline__ void load(const bf16* p, int lane, int dim, float (&v)[PER_LANE]) {
#pragma unroll
  for (int j = 0; j < PER_LANE; ++j) v[j] = lane + 32 * j < dim ? __bfloat162float(p[lane + 32 * j]) : 0.0f;
}
__device__ __forceinline__ void store(bf16* p, int lane, int dim, const float (&v)[PER_LANE]) {
#pragma unroll
  for (int j = 0; j < PER_LANE; ++j)
    if (lane + 32 * j < dim) p[lane + 32 * j] = __float2bfloat16_rn(v[j]);
}
__device__ __forceinline__ float dot(const float (&a)[PER_LANE], const float (&b)[PER_LANE]) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < PER_LANE; ++j) s += a[j] * b[j];
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

__global__ void __launch_bounds__(32 * WARPS) rows_dq_kernel(AttnArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, dim = static_cast<int>(a.dim);
  const int64_t h = blockIdx.y, kv = h / (a.heads / a.kv_heads);
  for (int64_t i = blockIdx.z; i < a.seq.batch; i += gridDim.z) {
    const Seq q = sequence(a.seq, i);
    for (int64_t t = blockIdx.x * WARPS + (threadIdx.x >> 5); t < q.nq; t += gridDim.x * WARPS) {
      float x[PER_LANE], dy[PER_LANE], y[PER_LANE], g[PER_LANE] = {};
      load(row_of(a.q, q.q0 + t, h), lane, dim, x);
      load(row_of(a.out, q.q0 + t, h), lane, dim, y);
      load(row_of(a.dout, q.q0 + t, h), lane, dim, dy);
      const float delta = dot(y, dy), lse = a.lse[(q.q0 + t) * a.heads + h];
      const int64_t end = keys_seen(q, static_cast<int>(t), a.causal);
      for (int64_t j = 0; j < end; ++j) {
        load(row_of(a.v, q.k0 + j, kv), lane, dim, y);
        const float dp = dot(dy, y);
        load(row_of(a.k, q.k0 + j, kv), lane, dim, y);
        const float ds = expf(dot(x, y) * a.scale - lse) * (dp - delta);
#pragma unroll
        for (int e = 0; e < PER_LANE; ++e) g[e] += ds * y[e];
      }
#pragma unroll
      for (int e = 0; e < PER_LANE; ++e) g[e] *= a.scale;
      store(const_cast<bf16*>(row_of(a.dq, q.q0 + t, h)), lane, dim, g);
    }
  }
}

__global__ void __launch_bounds__(32 * WARPS) rows_dkv_kernel(AttnArgs a) {
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, dim = static_cast<int>(a.dim);
  const int64_t kv = blockIdx.y, group = a.heads / a.kv_heads;
  for (int64_t i = blockIdx.z; i < a.seq.batch; i += gridDim.z) {
    const Seq q = sequence(a.seq, i);
    for (int64_t j = blockIdx.x * WARPS + (threadIdx.x >> 5); j < q.nk; j += gridDim.x * WARPS) {
      float x[PER_LANE], v[PER_LANE], y[PER_LANE], dy[PER_LANE], gk[PER_LANE] = {}, gv[PER_LANE] = {};
      load(row_of(a.k, q.k0 + j, kv), lane, dim, x);
      load(row_of(a.v, q.k0 + j, kv), lane, dim, v);
      const int64_t first = a.causal && j > q.nk - q.nq ? j - (q.nk - q.nq) : 0;
      for (int64_t h = kv * group; h < (kv + 1) * group; ++h)
        for (int64_t t = first; t < q.nq; ++t) {
          load(row_of(a.out, q.q0 + t, h), lane, dim, y);
          load(row_of(a.dout, q.q0 + t, h), lane, dim, dy);
          const float delta = dot(y, dy), dp = dot(v, dy);
          load(row_of(a.q, q.q0 + t, h), lane, dim, y);
          const float p = expf(dot(x, y) * a.scale - a.lse[(q.q0 + t) * a.heads + h]);
          const float ds = p * (dp - delta);
#pragma unroll
          for (int e = 0; e < PER_LANE; ++e) gk[e] += ds * y[e], gv[e] += p * dy[e];
        }
#pragma unroll
      for (int e = 0; e < PER_LANE; ++e) gk[e] *= a.scale;
      store(const_cast<bf16*>(row_of(a.dk, q.k0 + j, kv)), lane, dim, gk);
      store(const_cast<bf16*>(row_of(a.dv, q.k0 + j, kv)), lane, dim, gv);
    }
  }
}

// Blocks along the rows of a sequence, and along the sequences.
dim3 grid_of(int64_t rows, int64_t heads, int64_t batch) {
  const int64_t x = (rows + WARPS - 1) / WARPS, z = batch < 64 ? batch : 64;
  return dim3(static_cast<unsigned>(x < 4096 ? x : 4096), static_cast<unsigned>(heads), static_cast<unsigned>(z));
}

}  // namespace

int64_t need_attention_bwd(int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_attention_bwd(const Machine&, const AttnArgs& a, const Watch&, uint32_t*, void*, cudaStream_t s) {
  if (a.seq.n > 0) {
    const cudaError_t e =
        launch_pdl(rows_dq_kernel, grid_of(a.seq.n, a.heads, a.seq.batch), dim3(32 * WARPS), 0, s, a);
    if (e != cudaSuccess) return e;
  }
  return a.seq.nk > 0 ? launch_pdl(rows_dkv_kernel, grid_of(a.seq.nk, a.kv_heads, a.seq.batch), dim3(32 * WARPS), 0, s, a)
                      : cudaSuccess;
}

}  // namespace tpo
