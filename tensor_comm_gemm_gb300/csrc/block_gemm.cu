// Matrix products of the block operators, first form: one thread block per
// 64 x 64 output tile, operands staged through shared memory, fp32 sums on the
// CUDA cores.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "block.h"
#include "act.h"

namespace tpo {

namespace {

constexpr int T = 64, KT = 16;

struct GemmArgs {
  View a[2], b[2];
  int terms;
  int64_t M, N, K;
  Epi e;
};

template <bool FP8>
__device__ float load_elem(const View& v, int64_t i, int64_t j) {
  if constexpr (FP8)
    return static_cast<float>(static_cast<const __nv_fp8_e4m3*>(v.p)[i * v.row + j * v.col]);
  else
    return __bfloat162float(static_cast<const __nv_bfloat16*>(v.p)[i * v.row + j * v.col]);
}

template <bool FP8, int NB>
__device__ void product(const GemmArgs& g, const View* b, int64_t i0, int64_t j0, float (&acc)[4][4]) {
  __shared__ float sa[KT][T + 1], sb[KT][T + 1];
  const int tid = threadIdx.x, ti = tid / 16, tj = tid % 16;
  for (int t = 0; t < NB; ++t)
    for (int64_t k0 = 0; k0 < g.K; k0 += KT) {
      for (int x = tid; x < T * KT; x += 256) {
        // neighbouring threads walk the operand's contiguous dimension
        const int ka = g.a[t].col == 1 ? x % KT : x / T, ia = g.a[t].col == 1 ? x / KT : x % T;
        const int kb = b[t].col == 1 ? x % KT : x / T, ib = b[t].col == 1 ? x / KT : x % T;
        sa[ka][ia] = i0 + ia < g.M && k0 + ka < g.K ? load_elem<FP8>(g.a[t], i0 + ia, k0 + ka) : 0.0f;
        sb[kb][ib] = j0 + ib < g.N && k0 + kb < g.K ? load_elem<FP8>(b[t], j0 + ib, k0 + kb) : 0.0f;
      }
      __syncthreads();
      for (int kk = 0; kk < KT; ++kk) {
        float x[4], y[4];
        for (int q = 0; q < 4; ++q) x[q] = sa[kk][ti * 4 + q], y[q] = sb[kk][tj * 4 + q];
        for (int q = 0; q < 4; ++q)
          for (int r = 0; r < 4; ++r) acc[q][r] += x[q] * y[r];
      }
      __syncthreads();
    }
}

__device__ void put(void* out, int64_t ld, int64_t i, int64_t j, float v) {
  if (out) static_cast<__nv_bfloat16*>(out)[i * ld + j] = __float2bfloat16_rn(v);
}

template <bool FP8, int KIND, int ACT>
__global__ void __launch_bounds__(256) simple_gemm(const GemmArgs g) {
  const int64_t i0 = static_cast<int64_t>(blockIdx.y) * T, j0 = static_cast<int64_t>(blockIdx.x) * T;
  float acc[4][4] = {}, up[4][4] = {};
  if constexpr (KIND == EPI_GATED) {
    product<FP8, 1>(g, g.b, i0, j0, acc);
    product<FP8, 1>(g, g.b + 1, i0, j0, up);
  } else if (g.terms == 2) {
    product<FP8, 2>(g, g.b, i0, j0, acc);
  } else {
    product<FP8, 1>(g, g.b, i0, j0, acc);
  }
  const Epi& e = g.e;
  const float s0 = e.sx ? *e.sx * *e.sw0 : 1.0f, s1 = e.sx && e.sw1 ? *e.sx * *e.sw1 : 1.0f;
  const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
  for (int q = 0; q < 4; ++q)
    for (int r = 0; r < 4; ++r) {
      const int64_t i = i0 + ti * 4 + q, j = j0 + tj * 4 + r;
      if (i >= g.M || j >= g.N) continue;
      float z = acc[q][r] * s0;
      if constexpr (KIND == EPI_PLAIN) put(e.out0, e.ld0, i, j, z);
      if constexpr (KIND == EPI_LINEAR) {
        if (e.bias) z += __bfloat162float(static_cast<const __nv_bfloat16*>(e.bias)[j]);
        put(e.out1, e.ld1, i, j, z);
        float y = act_f<ACT>(z);
        if (e.residual) y += __bfloat162float(static_cast<const __nv_bfloat16*>(e.residual)[i * e.ldr + j]);
        put(e.out0, e.ld0, i, j, y);
      }
      if constexpr (KIND == EPI_GATED) {
        const float u = up[q][r] * s1;
        put(e.out1, e.ld1, i, j, z);
        put(e.out2, e.ld2, i, j, u);
        put(e.out0, e.ld0, i, j, act_f<ACT>(z) * u);
      }
    }
}

}  // namespace

cudaError_t launch_simple_gemm(const View* a, const View* b, int terms, int64_t M, int64_t N, int64_t K, bool fp8,
                               const Epi& e, cudaStream_t s) {
  GemmArgs g{};
  g.terms = terms;
  g.M = M, g.N = N, g.K = K, g.e = e;
  for (int t = 0; t < terms; ++t) g.a[t] = a[t], g.b[t] = b[t];
  if (e.kind == EPI_GATED) g.b[1] = b[1];
  const dim3 grid(static_cast<unsigned>((N + T - 1) / T), static_cast<unsigned>((M + T - 1) / T));
  return with_act(e.act, [&](auto act) {
    constexpr int A = decltype(act)::value;
    if (e.kind == EPI_PLAIN)
      simple_gemm<false, EPI_PLAIN, TPO_ACT_NONE><<<grid, 256, 0, s>>>(g);
    else if (e.kind == EPI_LINEAR && fp8)
      simple_gemm<true, EPI_LINEAR, A><<<grid, 256, 0, s>>>(g);
    else if (e.kind == EPI_LINEAR)
      simple_gemm<false, EPI_LINEAR, A><<<grid, 256, 0, s>>>(g);
    else if (fp8)
      simple_gemm<true, EPI_GATED, A><<<grid, 256, 0, s>>>(g);
    else
      simple_gemm<false, EPI_GATED, A><<<grid, 256, 0, s>>>(g);
    return cudaGetLastError();
  });
}

}  // namespace tpo
