// Shared by the host side (block.cu) and the kernels of the block operators
// (layer norm, linear with epilogue, gated projections).  Private to
// libtpoverlap; include/tpoverlap.h has the contract.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tpoverlap.h"

namespace tpo {

// One matrix product C[M, N] = sum over `terms` of A_t[M, K] . B_t[N, K]^T.  An
// operand is K-major (the contraction index contiguous: element (i, j) at
// p + i * ld + j) or MN-major (p + j * ld + i).
struct Operand {
  const void* p;
  int64_t ld;
  bool mn_major;
};
struct Product {
  Operand a[2], b[2];
  int terms;
  int64_t M, N, K;
  void* out;  // bf16 [M, N]
  int64_t ldo;
};

enum EpiKind : int {
  EPI_PLAIN = 0,   // out = C
  EPI_LINEAR = 1,  // out1 = C + bias (if wanted), out = act(C + bias) + residual
  EPI_GATED = 2,   // out1 = A.B0^T, out2 = A.B1^T (if wanted), out = act(out1) * out2 from the unrounded two
};
struct Epi {
  int kind = EPI_PLAIN;
  int act = TPO_ACT_NONE;
  const void* bias = nullptr;      // bf16 [N]
  const void* residual = nullptr;  // bf16 [M, N]
  int64_t ldr = 0;
  void *out1 = nullptr, *out2 = nullptr;  // bf16
  int64_t ld1 = 0, ld2 = 0;
  const float *sx = nullptr, *sw0 = nullptr, *sw1 = nullptr;  // e4m3 scales or NULL
};

// A launch's error word, and how long a wait of its kernels may last.
struct Watch {
  uint32_t* err;
  unsigned long long limit_ns;
};

// What the current device holds at a time.
constexpr int MAX_SPLIT = 8;  // CTAs of a cluster that cuts a contraction
struct Machine {
  int sms, pairs;                    // CTA pairs of the product kernel
  int clusters[2][MAX_SPLIT + 1];    // clusters of s CTAs, with one or two CTAs per SM
};
// Also set the kernels' attributes.
cudaError_t configure_products(Machine* m);
// The column tiles' width of each product of a launch (all after the first are
// of one shape), and the launch's modelled time.  Narrower tiles than the
// widest cost more per column, so they are taken where they fill a last round
// or spread few tiles over the pairs (in rows of calls: 4096^3 without an
// epilogue 86.3 us with 224 columns, 87.5 with 256, 90.2 with 192;
// 1777x4096x2*14336 249 us with 256, 260 with 192).
void plan_width(const Machine& mc, const Product* q, int count, bool fp8, bool gated, int* widths, double* us);
// Runs `count` (1 to 3) products in one launch; more than one take EPI_PLAIN.
cudaError_t launch_products(const Machine& mc, const Product* q, int count, bool fp8, const Epi& e, const Watch& w,
                            cudaStream_t s);

// The same for one product with few rows (M tokens): S CTAs of a cluster cut the contraction.
struct SplitPlan {
  int nt = 0;       // tokens of a tile
  int split = 1;    // CTAs of a cluster
  int stages = 0;
};
cudaError_t configure_split(Machine* m);
// Whether the product takes that form (path 0: by rule, 1: never, 2: always; split 0: by rule), and its plan.
bool use_split(const Machine& mc, const Product& q, bool fp8, bool gated, int64_t path, int64_t split, SplitPlan* plan);
// Its plan and modelled time for a bf16 product without an epilogue; false if path or the device rule it out.
bool split_cost(const Machine& mc, const Product& q, int64_t path, int64_t split, SplitPlan* plan, double* us);
cudaError_t launch_split(const Product& q, const SplitPlan& plan, bool fp8, const Epi& e, const Watch& w,
                         cudaStream_t s);

struct NormArgs {
  int64_t n, k;
  const void *x, *dy, *dres, *gamma, *beta;
  int64_t ldx, lddy, lddres, ldy;  // ldy: pitch of y or dx
  void *y;                         // y or dx
  float *mean, *rstd;              // forward: written; backward: read
  void *dgamma, *dbeta;
  float eps;
};

// out0 and out1 (of TPO_BF16 or TPO_F32, NULL: not wanted) from per-block sums part[parts][vectors][cols].
cudaError_t launch_column_sums(const float* part, int parts, int vectors, int64_t cols, void* out0, void* out1,
                               int dtype, cudaStream_t s);
// dz = dy act'(z) as bf16 [n, m] with pitch ldo (NULL: not written) and db = column sums (NULL: not wanted; part:
// workspace of act_parts(n) x m floats).
constexpr int ACT_PARTS = 152;
inline int64_t act_parts(int64_t n) { return (n + 15) / 16 < ACT_PARTS ? (n + 15) / 16 : ACT_PARTS; }
cudaError_t launch_act_bwd(int64_t n, int64_t m, int act, const void* dy, int64_t lddy, const void* z, int64_t ldz,
                           void* dz, int64_t ldo, float* part, void* db, cudaStream_t s);
// dg = dh u act'(g), du = dh act(g), bf16 with pitch ldo.
cudaError_t launch_gated_act_bwd(int64_t n, int64_t m, int act, const void* dh, int64_t lddh, const void* g,
                                 int64_t ldg, const void* u, int64_t ldu, void* dg, void* du, int64_t ldo,
                                 cudaStream_t s);
cudaError_t launch_norm(const Machine& mc, const NormArgs& a, int dtype, int wdtype, cudaStream_t s);
// part: workspace of min(n, NORM_PARTS) x 2 x k floats, the blocks' sums for dgamma and dbeta.
constexpr int NORM_PARTS = 152;
cudaError_t launch_norm_bwd(const Machine& mc, const NormArgs& a, int dtype, int wdtype, float* part, cudaStream_t s);

void set_last_error(const char* msg);  // ctx.cu: the message tpo_last_error returns

}  // namespace tpo
