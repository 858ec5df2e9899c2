// Pointwise parts of the backward passes: the gradient of the pre-activations
// and its column sums, first form.

#include <cuda_bf16.h>

#include <type_traits>

#include "block.h"
#include "act.h"

namespace tpo {

namespace {

using bf16 = __nv_bfloat16;

// One thread per column, rows in order: the bias gradient's sum is fp32, before dz is rounded.
template <int ACT>
__global__ void act_bwd_kernel(int64_t n, int64_t m, const bf16* dy, int64_t lddy, const bf16* z, int64_t ldz,
                               bf16* dz, int64_t ldo, bf16* db) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (j >= m) return;
  float sum = 0.0f;
  for (int64_t i = 0; i < n; ++i) {
    float v = __bfloat162float(dy[i * lddy + j]);
    if constexpr (ACT != TPO_ACT_NONE) v *= act_grad_f<ACT>(__bfloat162float(z[i * ldz + j]));
    if (dz) dz[i * ldo + j] = __float2bfloat16_rn(v);
    sum += v;
  }
  if (db) db[j] = __float2bfloat16_rn(sum);
}

template <int ACT>
__global__ void gated_act_bwd_kernel(int64_t n, int64_t m, const bf16* dh, int64_t lddh, const bf16* g, int64_t ldg,
                                     const bf16* u, int64_t ldu, bf16* dg, bf16* du, int64_t ldo) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t i = blockIdx.y;
  if (j >= m) return;
  const float d = __bfloat162float(dh[i * lddh + j]), gv = __bfloat162float(g[i * ldg + j]),
              uv = __bfloat162float(u[i * ldu + j]);
  dg[i * ldo + j] = __float2bfloat16_rn(d * uv * act_grad_f<ACT>(gv));
  du[i * ldo + j] = __float2bfloat16_rn(d * act_f<ACT>(gv));
}

}  // namespace

cudaError_t launch_act_bwd(int64_t n, int64_t m, int act, const void* dy, int64_t lddy, const void* z, int64_t ldz,
                           void* dz, int64_t ldo, void* db, cudaStream_t s) {
  return with_act(act, [&](auto a) {
    act_bwd_kernel<decltype(a)::value><<<static_cast<unsigned>((m + 127) / 128), 128, 0, s>>>(
        n, m, static_cast<const bf16*>(dy), lddy, static_cast<const bf16*>(z), ldz, static_cast<bf16*>(dz), ldo,
        static_cast<bf16*>(db));
    return cudaGetLastError();
  });
}

cudaError_t launch_gated_act_bwd(int64_t n, int64_t m, int act, const void* dh, int64_t lddh, const void* g,
                                 int64_t ldg, const void* u, int64_t ldu, void* dg, void* du, int64_t ldo,
                                 cudaStream_t s) {
  return with_act(act, [&](auto a) {
    for (int64_t i0 = 0; i0 < n; i0 += 65535) {  // grid.y holds 65535 rows
      const int64_t rows = n - i0 < 65535 ? n - i0 : 65535;
      gated_act_bwd_kernel<decltype(a)::value>
          <<<dim3(static_cast<unsigned>((m + 127) / 128), static_cast<unsigned>(rows)), 128, 0, s>>>(
              rows, m, static_cast<const bf16*>(dh) + i0 * lddh, lddh, static_cast<const bf16*>(g) + i0 * ldg, ldg,
              static_cast<const bf16*>(u) + i0 * ldu, ldu, static_cast<bf16*>(dg) + i0 * ldo,
              static_cast<bf16*>(du) + i0 * ldo, ldo);
    }
    return cudaGetLastError();
  });
}

}  // namespace tpo
