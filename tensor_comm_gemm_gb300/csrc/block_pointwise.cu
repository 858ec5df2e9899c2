// Pointwise parts of the backward passes (sm_103a): the gradient of the
// pre-activations, with the bias gradient's column sums, and the addition of
// per-block column sums.
//
// All are bound by memory: a thread takes eight consecutive columns (16 bytes
// of bf16) of a row at a time.

#include <algorithm>

#include <cuda_bf16.h>

#include <type_traits>

#include "act.h"
#include "block.h"
#include "pdl.h"
#include "ptx.h"

namespace tpo {

namespace {

using bf16 = __nv_bfloat16;

// Columns [c, c + 8) of a row of m elements as they lie in memory (0 past its end); p is 16-byte aligned.
__device__ __forceinline__ uint4 raw8(const bf16* p, int64_t c, int64_t m) {
  if (c + 8 <= m) return *reinterpret_cast<const uint4*>(p + c);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = c + 2 * j < m ? __bfloat16_as_ushort(p[c + 2 * j]) : 0;
    const uint32_t hi = c + 2 * j + 1 < m ? __bfloat16_as_ushort(p[c + 2 * j + 1]) : 0;
    w[j] = lo | hi << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void widen8(const uint4& h, float (&v)[8]) {
  const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
// Rounds eight values to bf16 into a workspace row, whose pitch covers whole groups of eight.
__device__ __forceinline__ void store8(bf16* p, const float (&v)[8]) {
  uint32_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    h[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(h[0], h[1], h[2], h[3]);
}

// Eight columns from c on of some rows: dz from dy and z, stored if wanted, and
// added to the sums.  WHOLE: all eight exist.
template <int ACT, bool WHOLE>
__device__ __forceinline__ void act_bwd_rows(int64_t first, int64_t n, int64_t step, int64_t c, int64_t m,
                                             const bf16* dy, int64_t lddy, const bf16* z, int64_t ldz, bf16* dz,
                                             int64_t ldo, float (&sum)[8]) {
  constexpr int R = 2;  // rows whose loads are in flight together
  for (int64_t i0 = first; i0 < n; i0 += R * step) {
    uint4 hd[R], hz[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t i = i0 + r * step < n ? i0 + r * step : i0;
      hd[r] = raw8(dy + i * lddy, c, WHOLE ? c + 8 : m);
      if constexpr (ACT != TPO_ACT_NONE) hz[r] = raw8(z + i * ldz, c, WHOLE ? c + 8 : m);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (i0 + r * step >= n) break;
      float d[8], v[8];
      widen8(hd[r], d);
      if constexpr (ACT != TPO_ACT_NONE) {
        widen8(hz[r], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] *= act_grad_f<ACT>(v[j]);
      }
      if (dz) store8(dz + (i0 + r * step) * ldo + c, d);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += d[j];
    }
  }
}

// Block (x, y): columns [256 x, 256 x + 256) of the rows 8 y + w + 8 i gridDim.y,
// warp w.  With `part`, the sums over the block's rows (fp32, before dz is
// rounded) go to part[y][m].  No atomics: the sums come out the same every time.
// 4096 x 4096 with GELU's tanh form and db: 18 us with them (67 MB read; with
// dz written too 100 MB).  64 registers, four blocks per SM: with two of them
// and four rows in flight, 26 us.
template <int ACT>
__global__ void __launch_bounds__(256, 4) act_bwd_kernel(int64_t n, int64_t m, const bf16* dy, int64_t lddy,
                                                      const bf16* z, int64_t ldz, bf16* dz, int64_t ldo,
                                                      float* part) {
  __shared__ float red[8][256];
  grid_dep_launch();
  grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + lane * 8;
  const int64_t first = static_cast<int64_t>(blockIdx.y) * 8 + warp, step = static_cast<int64_t>(gridDim.y) * 8;
  float sum[8] = {};
  if (c + 8 <= m)
    act_bwd_rows<ACT, true>(first, n, step, c, m, dy, lddy, z, ldz, dz, ldo, sum);
  else if (c < m)
    act_bwd_rows<ACT, false>(first, n, step, c, m, dy, lddy, z, ldz, dz, ldo, sum);
  if (!part) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) red[warp][lane * 8 + j] = sum[j];
  __syncthreads();
  const int64_t o = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (o >= m) return;
  float v = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) v += red[w][threadIdx.x];
  part[static_cast<int64_t>(blockIdx.y) * m + o] = v;
}

// A thread per eight columns: 8192 x 3584, five matrices of 59 MB, in
// 39 us (7.5 TB/s, the last of the stores still in L2).
template <int ACT>
__global__ void __launch_bounds__(256) gated_act_bwd_kernel(int64_t n, int64_t m, const bf16* dh, int64_t lddh,
                                                            const bf16* g, int64_t ldg, const bf16* u, int64_t ldu,
                                                            bf16* dg, bf16* du, int64_t ldo) {
  grid_dep_launch();
  grid_dep_wait();
  const int64_t per_row = (m + 7) / 8, idx = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (idx >= n * per_row) return;
  const int64_t i = idx / per_row, c = (idx - i * per_row) * 8;
  float d[8], gv[8], uv[8], og[8], ou[8];
  widen8(raw8(dh + i * lddh, c, m), d);
  widen8(raw8(g + i * ldg, c, m), gv);
  widen8(raw8(u + i * ldu, c, m), uv);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    og[j] = d[j] * uv[j] * act_grad_f<ACT>(gv[j]);
    ou[j] = d[j] * act_f<ACT>(gv[j]);
  }
  store8(dg + i * ldo + c, og);
  store8(du + i * ldo + c, ou);
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16* p, float v) { *p = __float2bfloat16_rn(v); }

// out_y[c] = sum over p of part[p][y][c], y = blockIdx.y of gridDim.y vectors of
// `cols`: 32 columns a block, one of 32 slices of p a warp, joined by shuffles
// in a fixed order.  152 parts of 2 x 4096 columns (5 MB, from L2) in 6 us with
// cold caches, most of it latency, so a thread's loads are all in flight.
template <class W>
__global__ void __launch_bounds__(1024) column_sums_kernel(const float* part, int parts, int64_t cols, W* out0,
                                                           W* out1) {
  __shared__ float s[32][33];
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  W* out = blockIdx.y ? out1 : out0;
  if (!out) return;
  float v = 0.0f;
  // five loads in flight: all that a slice of the most parts (152) has
  const int64_t vectors = gridDim.y;
  for (int p = slice; c < cols && p < parts; p += 32 * 5) {
    float w[5];
#pragma unroll
    for (int j = 0; j < 5; ++j)
      w[j] = p + 32 * j < parts ? part[((p + 32 * j) * vectors + blockIdx.y) * cols + c] : 0.0f;
#pragma unroll
    for (int j = 0; j < 5; ++j) v += w[j];
  }
  s[slice][lane] = v;
  __syncthreads();
  v = s[lane][slice];
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int64_t o = static_cast<int64_t>(blockIdx.x) * 32 + slice;
  if (lane == 0 && o < cols) put(out + o, v);
}

}  // namespace

cudaError_t launch_column_sums(const float* part, int parts, int vectors, int64_t cols, void* out0, void* out1,
                               int dtype, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((cols + 31) / 32), vectors);
  if (dtype == TPO_F32)
    return launch_pdl(column_sums_kernel<float>, grid, dim3(1024), 0, s, part, parts, cols, static_cast<float*>(out0),
                      static_cast<float*>(out1));
  return launch_pdl(column_sums_kernel<bf16>, grid, dim3(1024), 0, s, part, parts, cols, static_cast<bf16*>(out0),
                    static_cast<bf16*>(out1));
}

cudaError_t launch_act_bwd(int64_t n, int64_t m, int act, const void* dy, int64_t lddy, const void* z, int64_t ldz,
                           void* dz, int64_t ldo, float* part, void* db, cudaStream_t s) {
  // about eight blocks per SM in all, at most ACT_PARTS over the rows, and two rows for each warp
  const int64_t cols = (m + 255) / 256;
  const int64_t want = std::max<int64_t>(1, 1216 / cols);
  const int parts = static_cast<int>(std::min(want, act_parts(n)));
  cudaError_t e = with_act(act, [&](auto a) {
    return launch_pdl(act_bwd_kernel<decltype(a)::value>, dim3(static_cast<unsigned>(cols), parts), dim3(256), 0, s, n,
                      m, static_cast<const bf16*>(dy), lddy, static_cast<const bf16*>(z), ldz, static_cast<bf16*>(dz),
                      ldo, db ? part : nullptr);
  });
  if (e == cudaSuccess && db) e = launch_column_sums(part, parts, 1, m, db, nullptr, TPO_BF16, s);
  return e;
}

cudaError_t launch_gated_act_bwd(int64_t n, int64_t m, int act, const void* dh, int64_t lddh, const void* g,
                                 int64_t ldg, const void* u, int64_t ldu, void* dg, void* du, int64_t ldo,
                                 cudaStream_t s) {
  return with_act(act, [&](auto a) {
    return launch_pdl(gated_act_bwd_kernel<decltype(a)::value>,
                      dim3(static_cast<unsigned>((n * ((m + 7) / 8) + 255) / 256)), dim3(256), 0, s, n, m,
                      static_cast<const bf16*>(dh), lddh, static_cast<const bf16*>(g), ldg,
                      static_cast<const bf16*>(u), ldu, static_cast<bf16*>(dg), static_cast<bf16*>(du), ldo);
  });
}

}  // namespace tpo
