// Shared by the host side (block.cu) and the kernels of the block operators
// (layer norm, linear with epilogue, gated projections).  Private to
// libtpoverlap; include/tpoverlap.h has the contract.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tpoverlap.h"

namespace tpo {

// A matrix operand as the simple kernels address it: element (i, j) at
// p + i * row + j * col, in elements.
struct View {
  const void* p;
  int64_t row, col;
};

// One product C[M, N] = sum over terms of A_t[M, K] . B_t[N, K]^T.
enum EpiKind : int {
  EPI_PLAIN = 0,   // out0 = C
  EPI_LINEAR = 1,  // out1 = C + bias (if wanted), out0 = act(C + bias) + residual
  EPI_GATED = 2,   // out1 = A.B0^T, out2 = A.B1^T (if wanted), out0 = act(out1) * out2, unrounded
};
struct Epi {
  int kind = EPI_PLAIN;
  int act = TPO_ACT_NONE;
  const void* bias = nullptr;      // bf16 [N]
  const void* residual = nullptr;  // bf16 [M, N]
  int64_t ldr = 0;
  void *out0 = nullptr, *out1 = nullptr, *out2 = nullptr;  // bf16
  int64_t ld0 = 0, ld1 = 0, ld2 = 0;
  const float *sx = nullptr, *sw0 = nullptr, *sw1 = nullptr;  // e4m3 scales or NULL
};

struct NormArgs {
  int64_t n, k;
  const void *x, *dy, *dres, *gamma, *beta;
  int64_t ldx, lddy, lddres, ldy;  // ldy: pitch of y or dx
  void *y;                         // y or dx
  float *mean, *rstd;              // forward: written; backward: read
  void *dgamma, *dbeta;
  float eps;
};

cudaError_t launch_simple_gemm(const View* a, const View* b, int terms, int64_t M, int64_t N, int64_t K, bool fp8,
                               const Epi& e, cudaStream_t s);
// dz = dy act'(z) as bf16 [n, m] with pitch ldo (NULL: not written) and db = column sums (NULL: not wanted).
cudaError_t launch_act_bwd(int64_t n, int64_t m, int act, const void* dy, int64_t lddy, const void* z, int64_t ldz,
                           void* dz, int64_t ldo, void* db, cudaStream_t s);
// dg = dh u act'(g), du = dh act(g), bf16 with pitch ldo.
cudaError_t launch_gated_act_bwd(int64_t n, int64_t m, int act, const void* dh, int64_t lddh, const void* g,
                                 int64_t ldg, const void* u, int64_t ldu, void* dg, void* du, int64_t ldo,
                                 cudaStream_t s);
cudaError_t launch_norm(const NormArgs& a, int dtype, int wdtype, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormArgs& a, int dtype, int wdtype, cudaStream_t s);

void set_last_error(const char* msg);  // ctx.cu: the message tpo_last_error returns

}  // namespace tpo
