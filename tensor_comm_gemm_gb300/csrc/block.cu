// Host side of the block operators: the handle, argument checks and the
// launches of each call.  See include/tpoverlap.h for the contract.

#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <new>

#include "block.h"

namespace {

tpo_status fail(tpo_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  tpo::set_last_error(buf);
  return s;
}

tpo_status cuda_fail(cudaError_t e, const char* what) {
  return fail(TPO_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

constexpr int64_t kMaxSize = 1ll << 30;
constexpr size_t kErrBytes = 256;  // the error words ahead of the workspace

int64_t round_up(int64_t v, int64_t q) { return (v + q - 1) / q * q; }

// Pitch of a bf16 workspace matrix: whole 128-byte lines.
int64_t ws_pitch(int64_t m) { return round_up(m, 64); }

}  // namespace

struct tpo_block {
  int device = 0;
  uint8_t* mem = nullptr;  // error words, then the workspace
  int64_t ws_bytes = 0;
  tpo::Machine machine{};
  int64_t path = 0, split = 0, wait_timeout_ms = 2000;  // options
  uint32_t* err() const { return reinterpret_cast<uint32_t*>(mem); }
  tpo::Watch watch() const { return {err(), static_cast<unsigned long long>(wait_timeout_ms) * 1000000ull}; }
  uint8_t* ws() const { return mem + kErrBytes; }
};

namespace {

struct Option {
  const char* key;
  int64_t tpo_block::*field;
  int64_t lo, hi;
};
const Option* find_option(const char* key) {
  static const Option options[] = {{"path", &tpo_block::path, 0, 2},
                                   {"split", &tpo_block::split, 0, tpo::MAX_SPLIT},
                                   {"wait_timeout_ms", &tpo_block::wait_timeout_ms, 1, 600000}};
  for (const Option& o : options)
    if (std::strcmp(key, o.key) == 0) return &o;
  return nullptr;
}

// A matrix argument: `rows` x `cols` elements of `elem` bytes, `ld` elements apart.
struct Mat {
  const char* name;
  const void* p;
  int64_t rows, cols, ld;
  int elem;
};

// Checks one matrix of a product (16-byte rows) and replaces the pitch of a
// single row, which has none, by a whole one.
tpo_status check_mat(Mat& a) {
  if (a.rows == 0) return TPO_OK;
  if (!a.p || (reinterpret_cast<uintptr_t>(a.p) & 15u))
    return fail(TPO_ERR_INVALID_ARG, "%s must be non-NULL and 16-byte aligned", a.name);
  const int unit = 16 / a.elem;
  if (a.rows == 1) {
    a.ld = round_up(a.cols, unit);
    return TPO_OK;
  }
  if (a.ld < a.cols || a.ld > (1ll << 34))
    return fail(TPO_ERR_INVALID_ARG, "%s: row pitch %lld is outside [%lld, 2^34]", a.name, (long long)a.ld,
                (long long)a.cols);
  if (a.ld % unit)
    return fail(TPO_ERR_UNSUPPORTED, "%s: row pitch %lld must be a multiple of %d elements (16-byte rows)", a.name,
                (long long)a.ld, unit);
  return TPO_OK;
}

// A matrix of the norms: any pitch, element alignment.
tpo_status check_rows(const Mat& a) {
  if (a.rows == 0) return TPO_OK;
  if (!a.p || reinterpret_cast<uintptr_t>(a.p) % static_cast<uintptr_t>(a.elem))
    return fail(TPO_ERR_INVALID_ARG, "%s must be non-NULL and aligned to its elements", a.name);
  if (a.rows > 1 && (a.ld < a.cols || a.ld > (1ll << 34)))
    return fail(TPO_ERR_INVALID_ARG, "%s: row pitch %lld is outside [%lld, 2^34]", a.name, (long long)a.ld,
                (long long)a.cols);
  return TPO_OK;
}

tpo_status check_vec(const char* name, const void* p, int elem) {
  if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(elem))
    return fail(TPO_ERR_INVALID_ARG, "%s must be aligned to its elements", name);
  return TPO_OK;
}

tpo_status check_sizes(int64_t n, int64_t k, int64_t m) {
  if (n < 0 || n > kMaxSize || k < 1 || k > kMaxSize || m < 1 || m > kMaxSize)
    return fail(TPO_ERR_INVALID_ARG, "sizes out of range: n=%lld in [0, 2^30], k=%lld and m=%lld in [1, 2^30]",
                (long long)n, (long long)k, (long long)m);
  return TPO_OK;
}

tpo_status check_act(int act) {
  if (act < TPO_ACT_NONE || act > TPO_ACT_SILU) return fail(TPO_ERR_INVALID_ARG, "act=%d is not a tpo_act", act);
  return TPO_OK;
}

tpo_status check_types(int dtype, const float* const* scales, int count) {
  if (dtype != TPO_BF16 && dtype != TPO_FP8_E4M3)
    return fail(TPO_ERR_INVALID_ARG, "dtype=%d is neither TPO_BF16 (0) nor TPO_FP8_E4M3 (1)", dtype);
  for (int i = 0; i < count; ++i) {
    if (dtype == TPO_FP8_E4M3 && !scales[i])
      return fail(TPO_ERR_INVALID_ARG, "e4m3 inputs need every scale_inv device pointer");
    if (dtype == TPO_BF16 && scales[i])
      return fail(TPO_ERR_INVALID_ARG, "bf16 inputs take no scale_inv pointers (pass NULL)");
    if (tpo_status st = check_vec("a scale_inv pointer", scales[i], 4)) return st;
  }
  return TPO_OK;
}

// The handle, checked last so that the other argument errors need no GPU.
tpo_status check_block(const tpo_block* b, int64_t need) {
  if (!b) return fail(TPO_ERR_INVALID_ARG, "NULL block handle");
  if (need > b->ws_bytes)
    return fail(TPO_ERR_INVALID_ARG, "the call needs %lld bytes of workspace, the handle has %lld", (long long)need,
                (long long)b->ws_bytes);
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "no usable CUDA device");
  if (dev != b->device)
    return fail(TPO_ERR_INVALID_ARG, "the handle is of device %d, the current device is %d", b->device, dev);
  return TPO_OK;
}

// One product on CTA pairs or, with few rows, on clusters that cut the contraction.
cudaError_t run_product(tpo_block* b, const tpo::Product& q, bool fp8, const tpo::Epi& e, cudaStream_t s) {
  tpo::SplitPlan plan;
  if (tpo::use_split(b->machine, q, fp8, e.kind == tpo::EPI_GATED, b->path, b->split, &plan))
    return tpo::launch_split(q, plan, fp8, e, b->watch(), s);
  return tpo::launch_products(b->machine, &q, 1, fp8, e, b->watch(), s);
}

// The gradients' products: dx (if wanted) first, then the weights' gradients,
// which are of one shape.  Each of the two kinds runs on clusters by itself or
// on CTA pairs, there all in one launch: whichever the models add up to least.
cudaError_t run_products(tpo_block* b, const tpo::Product* q, int count, int dx, cudaStream_t s) {
  tpo::SplitPlan plans[3];
  double alone[3] = {};
  bool can[3] = {};
  for (int i = 0; i < count; ++i)
    can[i] = tpo::split_cost(b->machine, q[i], b->path, b->split, &plans[i], &alone[i]);
  int best = 0;
  double best_us = 0;
  for (int choice = 0; choice < 4; ++choice) {  // bit 0: dx on clusters, bit 1: the weights' gradients
    tpo::Product rest[3];
    int left = 0;
    double us = 0;
    bool ok = true;
    for (int i = 0; i < count; ++i) {
      if (choice >> (i < dx ? 0 : 1) & 1) {
        ok = ok && can[i];
        us += alone[i];
      } else {
        rest[left++] = q[i];
      }
    }
    if (!ok || ((choice & 1) && dx == 0) || ((choice & 2) && dx == count)) continue;
    double pairs_us = 0;
    int widths[3];
    if (left) tpo::plan_width(b->machine, rest, left, false, false, widths, &pairs_us);
    us += pairs_us;
    if (b->path == 2) us = -choice;  // every product on clusters
    if (choice == 0 || us < best_us) best = choice, best_us = us;
  }
  tpo::Product rest[3];
  int left = 0;
  for (int i = 0; i < count; ++i) {
    if (!(best >> (i < dx ? 0 : 1) & 1)) {
      rest[left++] = q[i];
      continue;
    }
    const cudaError_t e = tpo::launch_split(q[i], plans[i], false, tpo::Epi(), b->watch(), s);
    if (e != cudaSuccess) return e;
  }
  return left ? tpo::launch_products(b->machine, rest, left, false, tpo::Epi(), b->watch(), s) : cudaSuccess;
}

tpo_status launched(cudaError_t e) { return e == cudaSuccess ? TPO_OK : cuda_fail(e, "kernel launch"); }

// dz, then the bias gradient's per-block sums.  dz, dg and du are kept in bf16: they are operands of the products that
// follow, which the tensor cores take in that type.  It is one rounding more than those of the results (the gradients'
// error against 64 bits is 0.0023 of their size, 0.0017 without it); keeping them whole would take two products for one.
int64_t dz_bytes(int64_t n, int64_t m) { return n * ws_pitch(m) * 2; }
int64_t need_linear_bwd(int64_t n, int64_t m) { return dz_bytes(n, m) + tpo::act_parts(n) * m * 4; }
int64_t need_gated_bwd(int64_t n, int64_t m) { return 2 * n * ws_pitch(m) * 2; }
int64_t need_norm_bwd(int64_t n, int64_t k) { return (n < tpo::NORM_PARTS ? n : tpo::NORM_PARTS) * 8 * k; }

tpo_status zero_rows(void* p, int64_t ld, int64_t rows, int64_t cols, cudaStream_t s) {
  if (!p) return TPO_OK;
  const cudaError_t e = cudaMemset2DAsync(p, static_cast<size_t>(ld) * 2, 0, static_cast<size_t>(cols) * 2,
                                          static_cast<size_t>(rows), s);
  return e == cudaSuccess ? TPO_OK : cuda_fail(e, "zero gradient of an empty batch");
}

}  // namespace

extern "C" {

int64_t tpo_block_workspace(int op, int64_t n, int64_t k, int64_t m) {
  const bool norm = op == TPO_OP_LAYER_NORM || op == TPO_OP_LAYER_NORM_BWD;
  if (check_sizes(n, k, norm ? 1 : m) != TPO_OK) return -1;
  switch (op) {
    case TPO_OP_LAYER_NORM:
    case TPO_OP_LINEAR:
    case TPO_OP_GATED: return 0;
    case TPO_OP_LAYER_NORM_BWD: return need_norm_bwd(n, k);
    case TPO_OP_LINEAR_BWD: return need_linear_bwd(n, m);
    case TPO_OP_GATED_BWD: return need_gated_bwd(n, m);
    default: fail(TPO_ERR_INVALID_ARG, "op=%d is not a tpo_block_op", op); return -1;
  }
}

tpo_block* tpo_block_create(int64_t workspace_bytes) {
  if (workspace_bytes < 0) {
    fail(TPO_ERR_INVALID_ARG, "workspace_bytes=%lld is negative", (long long)workspace_bytes);
    return nullptr;
  }
  tpo_block* b = new (std::nothrow) tpo_block();
  if (!b) {
    fail(TPO_ERR_OOM, "no host memory for a handle");
    return nullptr;
  }
  int major = 0, minor = 0;
  cudaError_t e = cudaGetDevice(&b->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, b->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, b->device);
  if (e != cudaSuccess) {
    cuda_fail(e, "no usable CUDA device");
    delete b;
    return nullptr;
  }
  if (major != 10 || minor != 3) {
    fail(TPO_ERR_UNSUPPORTED, "libtpoverlap is compiled for sm_103a only; device is sm_%d%d", major, minor);
    delete b;
    return nullptr;
  }
  e = tpo::configure_products(&b->machine);
  if (e == cudaSuccess) e = tpo::configure_split(&b->machine);
  if (e != cudaSuccess) {
    cuda_fail(e, "kernel configuration");
    delete b;
    return nullptr;
  }
  b->ws_bytes = workspace_bytes;
  e = cudaMalloc(&b->mem, kErrBytes + static_cast<size_t>(workspace_bytes));
  if (e != cudaSuccess) {
    fail(TPO_ERR_OOM, "workspace of %lld bytes: %s", (long long)workspace_bytes, cudaGetErrorString(e));
    cudaGetLastError();
    delete b;
    return nullptr;
  }
  e = cudaMemset(b->mem, 0, kErrBytes);
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
  if (e != cudaSuccess) {
    cuda_fail(e, "block set-up");
    cudaFree(b->mem);
    delete b;
    return nullptr;
  }
  return b;
}

tpo_status tpo_block_destroy(tpo_block* b) {
  if (!b) return TPO_OK;
  cudaFree(b->mem);  // waits for the device's pending work
  delete b;
  return TPO_OK;
}

tpo_status tpo_block_set_opt(tpo_block* b, const char* key, int64_t value) {
  if (!key) return fail(TPO_ERR_INVALID_ARG, "NULL option key");
  const Option* o = find_option(key);
  if (!o) return fail(TPO_ERR_INVALID_ARG, "unknown option '%s'", key);
  if (value < o->lo || value > o->hi)
    return fail(TPO_ERR_INVALID_ARG, "option '%s'=%lld outside [%lld, %lld]", key, (long long)value, (long long)o->lo,
                (long long)o->hi);
  if (!b) return fail(TPO_ERR_INVALID_ARG, "NULL block handle");
  b->*(o->field) = value;
  return TPO_OK;
}

tpo_status tpo_block_get_opt(tpo_block* b, const char* key, int64_t* value) {
  if (!key || !value) return fail(TPO_ERR_INVALID_ARG, "NULL option key or value");
  const Option* o = find_option(key);
  if (!o) return fail(TPO_ERR_INVALID_ARG, "unknown option '%s'", key);
  if (!b) return fail(TPO_ERR_INVALID_ARG, "NULL block handle");
  *value = b->*(o->field);
  return TPO_OK;
}

tpo_status tpo_block_sync_status(tpo_block* b, void* stream) {
  if (!b) return fail(TPO_ERR_INVALID_ARG, "NULL block handle");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t err[4] = {};
  cudaError_t e = cudaMemcpyAsync(err, b->err(), sizeof(err), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "synchronise");
  if (err[0] == 0) return TPO_OK;
  e = cudaMemsetAsync(b->mem, 0, kErrBytes, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "reset after device failure");
  return fail(TPO_ERR_TIMEOUT, "device wait timed out (site %u, block %u)", err[1], err[2]);
}

tpo_status tpo_layer_norm(tpo_block* b, int64_t n, int64_t k, int dtype, int wdtype, const void* x, int64_t ldx,
                          const void* gamma, const void* beta, float eps, void* y, int64_t ldy, float* mean,
                          float* rstd, void* stream) {
  if (tpo_status st = check_sizes(n, k, 1)) return st;
  if ((dtype != TPO_BF16 && dtype != TPO_F32) || (wdtype != TPO_BF16 && wdtype != TPO_F32))
    return fail(TPO_ERR_INVALID_ARG, "layer norm types are TPO_BF16 (0) or TPO_F32 (2): dtype=%d wdtype=%d", dtype,
                wdtype);
  if (!(eps >= 0.0f)) return fail(TPO_ERR_INVALID_ARG, "eps must be at least 0");
  const int elem = dtype == TPO_F32 ? 4 : 2, welem = wdtype == TPO_F32 ? 4 : 2;
  if (tpo_status st = check_rows({"x", x, n, k, ldx, elem})) return st;
  if (tpo_status st = check_rows({"y", y, n, k, ldy, elem})) return st;
  if (tpo_status st = check_vec("gamma", gamma, welem)) return st;
  if (tpo_status st = check_vec("beta", beta, welem)) return st;
  if (tpo_status st = check_vec("mean", mean, 4)) return st;
  if (tpo_status st = check_vec("rstd", rstd, 4)) return st;
  if (tpo_status st = check_block(b, 0)) return st;
  if (n == 0) return TPO_OK;
  tpo::NormArgs a{};
  a.n = n, a.k = k, a.x = x, a.ldx = ldx, a.gamma = gamma, a.beta = beta, a.eps = eps;
  a.y = y, a.ldy = ldy, a.mean = mean, a.rstd = rstd;
  return launched(tpo::launch_norm(b->machine, a, dtype, wdtype, static_cast<cudaStream_t>(stream)));
}

tpo_status tpo_layer_norm_bwd(tpo_block* b, int64_t n, int64_t k, int dtype, int wdtype, const void* dy,
                              int64_t lddy, const void* x, int64_t ldx, const void* gamma, const float* mean,
                              const float* rstd, const void* dres, int64_t lddres, void* dx, int64_t lddx,
                              void* dgamma, void* dbeta, void* stream) {
  if (tpo_status st = check_sizes(n, k, 1)) return st;
  if ((dtype != TPO_BF16 && dtype != TPO_F32) || (wdtype != TPO_BF16 && wdtype != TPO_F32))
    return fail(TPO_ERR_INVALID_ARG, "layer norm types are TPO_BF16 (0) or TPO_F32 (2): dtype=%d wdtype=%d", dtype,
                wdtype);
  const int elem = dtype == TPO_F32 ? 4 : 2, welem = wdtype == TPO_F32 ? 4 : 2;
  if (tpo_status st = check_rows({"dy", dy, n, k, lddy, elem})) return st;
  if (tpo_status st = check_rows({"x", x, n, k, ldx, elem})) return st;
  if (dres)
    if (tpo_status st = check_rows({"dres", dres, n, k, lddres, elem})) return st;
  if (dx)
    if (tpo_status st = check_rows({"dx", dx, n, k, lddx, elem})) return st;
  if (n > 0 && (!mean || !rstd)) return fail(TPO_ERR_INVALID_ARG, "mean and rstd of the forward call are needed");
  const void* vecs[] = {gamma, dgamma, dbeta};
  for (const void* v : vecs)
    if (tpo_status st = check_vec("gamma, dgamma and dbeta", v, welem)) return st;
  if (tpo_status st = check_vec("mean", mean, 4)) return st;
  if (tpo_status st = check_vec("rstd", rstd, 4)) return st;
  if (tpo_status st = check_block(b, dgamma || dbeta ? need_norm_bwd(n, k) : 0)) return st;
  tpo::NormArgs a{};
  a.n = n, a.k = k, a.x = x, a.ldx = ldx, a.dy = dy, a.lddy = lddy, a.gamma = gamma, a.dres = dres;
  a.lddres = lddres, a.y = n > 0 ? dx : nullptr, a.ldy = lddx, a.dgamma = dgamma, a.dbeta = dbeta;
  a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
  return launched(tpo::launch_norm_bwd(b->machine, a, dtype, wdtype, reinterpret_cast<float*>(b->ws()),
                                       static_cast<cudaStream_t>(stream)));
}

tpo_status tpo_linear(tpo_block* b, int64_t n, int64_t k, int64_t m, int dtype, const void* x, int64_t ldx,
                      const void* w, int64_t ldw, const void* bias, int act, const void* residual, int64_t ldr,
                      void* z, int64_t ldz, void* y, int64_t ldy, const float* d_scale_inv_x,
                      const float* d_scale_inv_w, void* stream) {
  if (tpo_status st = check_sizes(n, k, m)) return st;
  if (tpo_status st = check_act(act)) return st;
  const float* scales[] = {d_scale_inv_x, d_scale_inv_w};
  if (tpo_status st = check_types(dtype, scales, 2)) return st;
  const int elem = dtype == TPO_FP8_E4M3 ? 1 : 2;
  Mat mx{"x", x, n, k, ldx, elem}, mw{"w", w, m, k, ldw, elem}, my{"y", y, n, m, ldy, 2},
      mr{"residual", residual, n, m, ldr, 2}, mz{"z", z, n, m, ldz, 2};
  if (tpo_status st = check_mat(mx)) return st;
  if (tpo_status st = check_mat(mw)) return st;
  if (tpo_status st = check_mat(my)) return st;
  if (residual)
    if (tpo_status st = check_mat(mr)) return st;
  if (z)
    if (tpo_status st = check_mat(mz)) return st;
  if (tpo_status st = check_vec("bias", bias, 2)) return st;
  if (tpo_status st = check_block(b, 0)) return st;
  if (n == 0) return TPO_OK;
  tpo::Epi e;
  e.kind = tpo::EPI_LINEAR, e.act = act, e.bias = bias, e.residual = residual, e.ldr = mr.ld;
  e.out1 = z, e.ld1 = mz.ld, e.sx = d_scale_inv_x, e.sw0 = d_scale_inv_w;
  const tpo::Product q{{{x, mx.ld, false}}, {{w, mw.ld, false}}, 1, n, m, k, y, my.ld};
  return launched(run_product(b, q, dtype == TPO_FP8_E4M3, e, static_cast<cudaStream_t>(stream)));
}

tpo_status tpo_linear_bwd(tpo_block* b, int64_t n, int64_t k, int64_t m, int act, const void* dy, int64_t lddy,
                          const void* z, int64_t ldz, const void* x, int64_t ldx, const void* w, int64_t ldw,
                          void* dx, int64_t lddx, void* dw, int64_t lddw, void* db, void* stream) {
  if (tpo_status st = check_sizes(n, k, m)) return st;
  if (tpo_status st = check_act(act)) return st;
  Mat mdy{"dy", dy, n, m, lddy, 2}, mz{"z", z, n, m, ldz, 2}, mx{"x", x, n, k, ldx, 2}, mw{"w", w, m, k, ldw, 2},
      mdx{"dx", dx, n, k, lddx, 2}, mdw{"dw", dw, m, k, lddw, 2};
  if (tpo_status st = check_mat(mdy)) return st;
  if (act == TPO_ACT_NONE ? z != nullptr : !z && n > 0)
    return fail(TPO_ERR_INVALID_ARG, "z is needed with an activation, and only then");
  if (z)
    if (tpo_status st = check_mat(mz)) return st;
  if (dx) {
    if (tpo_status st = check_mat(mdx)) return st;
    if (tpo_status st = check_mat(mw)) return st;
  }
  if (dw) {
    if (tpo_status st = check_mat(mdw)) return st;
    if (tpo_status st = check_mat(mx)) return st;
  }
  if (tpo_status st = check_vec("db", db, 2)) return st;
  const bool make_dz = act != TPO_ACT_NONE && (dx || dw);
  if (tpo_status st = check_block(b, make_dz || db ? need_linear_bwd(n, m) : 0)) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n == 0) {
    if (tpo_status st = zero_rows(dw, mdw.ld, m, k, s)) return st;
    return zero_rows(db, m, 1, m, s);
  }
  const void* dz = dy;
  int64_t lddz = mdy.ld;
  if (make_dz || db) {
    void* out = make_dz ? b->ws() : nullptr;
    const cudaError_t e = tpo::launch_act_bwd(n, m, act, dy, mdy.ld, z, mz.ld, out, ws_pitch(m),
                                              reinterpret_cast<float*>(b->ws() + dz_bytes(n, m)), db, s);
    if (e != cudaSuccess) return launched(e);
    if (make_dz) dz = out, lddz = ws_pitch(m);
  }
  tpo::Product q[2];
  int count = 0;
  if (dx) q[count++] = {{{dz, lddz, false}}, {{w, mw.ld, true}}, 1, n, k, m, dx, mdx.ld};
  if (dw) q[count++] = {{{dz, lddz, true}}, {{x, mx.ld, true}}, 1, m, k, n, dw, mdw.ld};
  return launched(run_products(b, q, count, dx ? 1 : 0, s));
}

tpo_status tpo_gated(tpo_block* b, int64_t n, int64_t k, int64_t m, int dtype, const void* x, int64_t ldx,
                     const void* wg, int64_t ldwg, const void* wu, int64_t ldwu, int act, void* g, int64_t ldg,
                     void* u, int64_t ldu, void* h, int64_t ldh, const float* d_scale_inv_x,
                     const float* d_scale_inv_wg, const float* d_scale_inv_wu, void* stream) {
  if (tpo_status st = check_sizes(n, k, m)) return st;
  if (tpo_status st = check_act(act)) return st;
  const float* scales[] = {d_scale_inv_x, d_scale_inv_wg, d_scale_inv_wu};
  if (tpo_status st = check_types(dtype, scales, 3)) return st;
  const int elem = dtype == TPO_FP8_E4M3 ? 1 : 2;
  Mat mx{"x", x, n, k, ldx, elem}, mg{"wg", wg, m, k, ldwg, elem}, mu{"wu", wu, m, k, ldwu, elem},
      mh{"h", h, n, m, ldh, 2}, mog{"g", g, n, m, ldg, 2}, mou{"u", u, n, m, ldu, 2};
  Mat* need[] = {&mx, &mg, &mu, &mh};
  for (Mat* a : need)
    if (tpo_status st = check_mat(*a)) return st;
  if (n > 0 && !g != !u) return fail(TPO_ERR_INVALID_ARG, "g and u are stored together or not at all");
  if (g) {
    if (tpo_status st = check_mat(mog)) return st;
    if (tpo_status st = check_mat(mou)) return st;
  }
  if (tpo_status st = check_block(b, 0)) return st;
  if (n == 0) return TPO_OK;
  tpo::Epi e;
  e.kind = tpo::EPI_GATED, e.act = act, e.out1 = g, e.ld1 = mog.ld, e.out2 = u, e.ld2 = mou.ld;
  e.sx = d_scale_inv_x, e.sw0 = d_scale_inv_wg, e.sw1 = d_scale_inv_wu;
  const tpo::Product q{{{x, mx.ld, false}}, {{wg, mg.ld, false}, {wu, mu.ld, false}}, 1, n, m, k, h, mh.ld};
  return launched(run_product(b, q, dtype == TPO_FP8_E4M3, e, static_cast<cudaStream_t>(stream)));
}

tpo_status tpo_gated_bwd(tpo_block* b, int64_t n, int64_t k, int64_t m, int act, const void* dh, int64_t lddh,
                         const void* g, int64_t ldg, const void* u, int64_t ldu, const void* x, int64_t ldx,
                         const void* wg, int64_t ldwg, const void* wu, int64_t ldwu, void* dx, int64_t lddx,
                         void* dwg, int64_t lddwg, void* dwu, int64_t lddwu, void* stream) {
  if (tpo_status st = check_sizes(n, k, m)) return st;
  if (tpo_status st = check_act(act)) return st;
  Mat mdh{"dh", dh, n, m, lddh, 2}, mg{"g", g, n, m, ldg, 2}, mu{"u", u, n, m, ldu, 2}, mx{"x", x, n, k, ldx, 2},
      mwg{"wg", wg, m, k, ldwg, 2}, mwu{"wu", wu, m, k, ldwu, 2}, mdx{"dx", dx, n, k, lddx, 2},
      mdwg{"dwg", dwg, m, k, lddwg, 2}, mdwu{"dwu", dwu, m, k, lddwu, 2};
  Mat* need[] = {&mdh, &mg, &mu};
  for (Mat* a : need)
    if (tpo_status st = check_mat(*a)) return st;
  if (!dwg != !dwu) return fail(TPO_ERR_INVALID_ARG, "dwg and dwu are computed together or not at all");
  if (dx) {
    Mat* ms[] = {&mdx, &mwg, &mwu};
    for (Mat* a : ms)
      if (tpo_status st = check_mat(*a)) return st;
  }
  if (dwg) {
    Mat* ms[] = {&mx, &mdwg, &mdwu};
    for (Mat* a : ms)
      if (tpo_status st = check_mat(*a)) return st;
  }
  if (tpo_status st = check_block(b, need_gated_bwd(n, m))) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n == 0) {
    if (tpo_status st = zero_rows(dwg, mdwg.ld, m, k, s)) return st;
    return zero_rows(dwu, mdwu.ld, m, k, s);
  }
  if (!dx && !dwg) return TPO_OK;
  const int64_t ld = ws_pitch(m);
  uint8_t* dg = b->ws();
  uint8_t* du = dg + n * ld * 2;
  cudaError_t ce = tpo::launch_gated_act_bwd(n, m, act, dh, mdh.ld, g, mg.ld, u, mu.ld, dg, du, ld, s);
  if (ce != cudaSuccess) return launched(ce);
  tpo::Product q[3];
  int count = 0;
  if (dx)
    q[count++] = {{{dg, ld, false}, {du, ld, false}}, {{wg, mwg.ld, true}, {wu, mwu.ld, true}}, 2, n, k, m, dx, mdx.ld};
  if (dwg) {
    q[count++] = {{{dg, ld, true}}, {{x, mx.ld, true}}, 1, m, k, n, dwg, mdwg.ld};
    q[count++] = {{{du, ld, true}}, {{x, mx.ld, true}}, 1, m, k, n, dwu, mdwu.ld};
  }
  return launched(run_products(b, q, count, dx ? 1 : 0, s));
}

}  // extern "C"
