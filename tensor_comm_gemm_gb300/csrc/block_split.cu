// Matrix products of the block operators with few rows (sm_103a): decoding
// steps and short prompts.
//
// Bound by reading the weights once, so the roles are swapped: a tile is 128
// output features (the MMA's M: rows of w; for the gated form 64 rows of wg
// and 64 of wu) by up to 256 tokens (its N), and the contraction is cut among
// the S CTAs of a cluster, so that every SM streams weights even when the
// output is small.  Each CTA runs a TMA -> tcgen05.mma pipeline over its K
// blocks; then the fp32 accumulators go to shared memory as [token][feature],
// and after one cluster barrier every CTA adds its share of the outputs over
// the cluster's shared memories, in the order of the ranks, and runs the
// epilogue on it.
//
// One token through 4096 x 4096 takes 8.8 us in a row of calls replayed from a
// graph (4.9 for the weights at the copy rate), four through gate and up of
// 3584 x 8192 21.2 (17.4), 48 through 8192 x 3584 14.3 (8.9): the rest is the
// launch, the first loads' latency and the cluster's additions, 4 to 5 us that a
// call this short cannot hide.  Two CTAs share an SM where their stages fit, so that one's
// additions run beside the other's loads.

#include <algorithm>
#include <cstring>

#include "act.h"
#include "block.h"
#include "block_dev.h"
#include "ptx.h"

namespace tpo {

namespace {

constexpr int FT = 128;                // accumulator rows of a tile
constexpr int A_BYTES = FT * KB;       // weights of one K block
constexpr int MAX_STAGES = 8;
constexpr int THREADS = 256;           // warp 0 TMA, warp 1 MMA, warps 4-7 drain; all add
constexpr int SMEM_TAIL = 8 * (2 * MAX_STAGES + 2) + 16 + 1024;  // barriers, tensor memory slot, slack to align
constexpr int SMEM_ONE = 232448;       // one CTA per SM
constexpr int SMEM_TWO = 114688;       // two

struct Args {
  CUtensorMap a[2], b[2];
  int M, N;             // features and tokens
  int tiles_f;          // feature tiles
  int nt;               // tokens of a tile (16 .. 256, a multiple of 16)
  int kb_seg, kb;       // K blocks per term and in all
  int a_mn, b_mn;
  int b_bytes;          // a stage's tokens: nt rows of a K block, or blocks of 64 tokens by 64 rows
  int stages, tmem_cols;
  int act;
  const __nv_bfloat16 *bias, *residual;
  int bias_vec;                      // the bias is 8-byte aligned
  __nv_bfloat16 *out, *out1, *out2;  // [tokens, features]
  int64_t ldr, ldo, ld1, ld2;
  const float *sx, *sw0, *sw1;
  Watch watch;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ float act_any(int act, float z) {
  switch (act) {
    case TPO_ACT_RELU: return act_f<TPO_ACT_RELU>(z);
    case TPO_ACT_GELU: return act_f<TPO_ACT_GELU>(z);
    case TPO_ACT_GELU_TANH: return act_f<TPO_ACT_GELU_TANH>(z);
    case TPO_ACT_SILU: return act_f<TPO_ACT_SILU>(z);
    default: return z;
  }
}

// Four consecutive features of one token; p is 8-byte aligned, `count` of them exist.
__device__ __forceinline__ void put4(__nv_bfloat16* p, const float (&v)[4], int count) {
  if (count >= 4) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    for (int j = 0; j < count; ++j) p[j] = __float2bfloat16_rn(v[j]);
  }
}
// Four consecutive bf16 values (0 past `count`), as they lie in memory; `vec`: p is 8-byte aligned.
__device__ __forceinline__ uint2 get4(const __nv_bfloat16* p, int count, bool vec) {
  if (vec && count >= 4) return *reinterpret_cast<const uint2*>(p);
  uint32_t h[4] = {};
  for (int j = 0; j < 4; ++j)
    if (j < count) h[j] = __bfloat16_as_ushort(p[j]);
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}
__device__ __forceinline__ void add4(uint2 h, float (&v)[4]) {
  v[0] += __uint_as_float(h.x << 16);
  v[1] += __uint_as_float(h.x & 0xffff0000u);
  v[2] += __uint_as_float(h.y << 16);
  v[3] += __uint_as_float(h.y & 0xffff0000u);
}

// Grid: tiles x S CTAs, a cluster of S per tile.
template <int KIND, bool FP8>
__global__ void __launch_bounds__(THREADS, 2) split_kernel(const __grid_constant__ Args p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
  grid_dep_launch();
  constexpr int KEL = FP8 ? KB : KB / 2;
  constexpr int FEATURES = KIND == EPI_GATED ? FT / 2 : FT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t stage_bytes = A_BYTES + static_cast<uint32_t>(p.b_bytes);
  const uint32_t full0 = sbase + stage_bytes * p.stages, empty0 = full0 + 8 * MAX_STAGES,
                 tfull = empty0 + 8 * MAX_STAGES, slot = tfull + 16;
  const int S = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int tile = static_cast<int>(blockIdx.x) / S;
  const int f0 = tile % p.tiles_f * FEATURES, t0 = tile / p.tiles_f * p.nt;
  const int lo = static_cast<int>(static_cast<int64_t>(p.kb) * rank / S),
            hi = static_cast<int>(static_cast<int64_t>(p.kb) * (rank + 1) / S);
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    mbar_init(tfull, 1);
    fence_barrier_init();
    for (int t = 0; t < 2; ++t) {
      tma_prefetch_map(&p.a[t]);
      tma_prefetch_map(&p.b[t]);
    }
  }
  if (warp == 1) {
    tmem_alloc_cg<1>(slot, p.tmem_cols);
    tmem_relinquish_cg<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ld_shared_u32(slot);
  grid_dep_wait();
  // the bias and residual of this thread's first outputs, in flight beside the product
  constexpr int QUADS = FEATURES / 4;  // groups of four features of a token
  const int tokens = min(p.nt, p.N - t0);
  const int first = rank * THREADS + static_cast<int>(threadIdx.x);
  uint2 pre_b = make_uint2(0, 0), pre_r = pre_b;
  auto fetch = [&](int i) {
    const int col = f0 + i % QUADS * 4, count = p.M - col;
    if (KIND != EPI_LINEAR || i >= tokens * QUADS || count <= 0) return;
    if (p.bias) pre_b = get4(p.bias + col, count, p.bias_vec);
    if (p.residual) pre_r = get4(p.residual + (t0 + i / QUADS) * p.ldr + col, count, true);
  };
  fetch(first);
  if (warp == 0) {
    // the load warp, converged
    const uint32_t stages = static_cast<uint32_t>(p.stages), kb_seg = static_cast<uint32_t>(p.kb_seg);
    uint32_t stage = 0, phase = 0, armed = 0;
    // `boxes` issues the loads of one stage at `sa`, K offset kx of term seg
    auto run = [&](auto boxes) {
      int seg = lo >= static_cast<int>(kb_seg) ? 1 : 0, kk = lo - seg * static_cast<int>(kb_seg);
      for (int i = lo; i < hi; ++i) {
        if (!wait_bar_warp(p.watch, empty0 + 8u * stage, phase ^ 1u, S_EMPTY)) return;
        const uint32_t fb = full0 + 8u * stage;
        boxes(fb, sbase + stage * stage_bytes, seg, kk * KEL);
        ++armed;
        if (++kk == static_cast<int>(kb_seg)) kk = 0, ++seg;
        if (++stage == stages) stage = 0, phase ^= 1u;
      }
    };
    const uint64_t ma = reinterpret_cast<uint64_t>(&p.a[0]), mb = reinterpret_cast<uint64_t>(&p.b[0]);
    constexpr uint64_t kMap = sizeof(CUtensorMap);
    if (KIND == EPI_GATED)
      run([&](uint32_t fb, uint32_t sa, int, int kx) {
        const Box x[3] = {{sa, ma, kx, f0}, {sa + A_BYTES / 2, ma + kMap, kx, f0}, {sa + A_BYTES, mb, kx, t0}};
        stage_loads<1>(1u, fb, stage_bytes, fb, x);
      });
    else if (p.b_mn && p.nt > 64)
      run([&](uint32_t fb, uint32_t sa, int seg, int kx) {
        const Box x[4] = {{sa, ma + seg * kMap, f0, kx}, {sa + A_BYTES / 2, ma + seg * kMap, f0 + 64, kx},
                          {sa + A_BYTES, mb + seg * kMap, t0, kx}, {sa + A_BYTES + 8192u, mb + seg * kMap, t0 + 64, kx}};
        stage_loads<1>(1u, fb, stage_bytes, fb, x);
      });
    else if (p.b_mn)
      run([&](uint32_t fb, uint32_t sa, int seg, int kx) {
        const Box x[3] = {{sa, ma + seg * kMap, f0, kx}, {sa + A_BYTES / 2, ma + seg * kMap, f0 + 64, kx},
                          {sa + A_BYTES, mb + seg * kMap, t0, kx}};
        stage_loads<1>(1u, fb, stage_bytes, fb, x);
      });
    else if (p.a_mn)
      run([&](uint32_t fb, uint32_t sa, int seg, int kx) {
        const Box x[3] = {{sa, ma + seg * kMap, f0, kx}, {sa + A_BYTES / 2, ma + seg * kMap, f0 + 64, kx},
                          {sa + A_BYTES, mb + seg * kMap, kx, t0}};
        stage_loads<1>(1u, fb, stage_bytes, fb, x);
      });
    else
      run([&](uint32_t fb, uint32_t sa, int seg, int kx) {
        const Box x[2] = {{sa, ma + seg * kMap, kx, f0}, {sa + A_BYTES, mb + seg * kMap, kx, t0}};
        stage_loads<1>(1u, fb, stage_bytes, fb, x);
      });
    // whatever became of the MMAs, the loads must land before the CTA gives up its shared memory
    if (lane == 0)
      for (uint32_t j = armed > stages ? armed - stages : 0u; j < armed; ++j)
        wait_bar(p.watch, full0 + 8u * (j % stages), (j / stages) & 1u, S_DRAIN, false);
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = idesc_n(make_idesc(FP8, FT), p.nt) | (p.a_mn ? 1u << 15 : 0u) | (p.b_mn ? 1u << 16 : 0u);
    const uint64_t da0 = p.a_mn ? desc_mn(sbase) : smem_desc_sw128(sbase);
    const uint64_t db0 = p.b_mn ? desc_mn(sbase + A_BYTES) : smem_desc_sw128(sbase + A_BYTES);
    const uint64_t step_a = p.a_mn ? 128u : 2u, step_b = p.b_mn ? 128u : 2u;
    uint32_t stage = 0, phase = 0;
    for (int i = lo; i < hi; ++i) {
      if (!wait_bar_warp(p.watch, full0 + 8u * stage, phase, S_FULL)) break;
      tc_fence_after();
      const uint64_t off = static_cast<uint64_t>(stage_bytes >> 4) * stage;
      mma_kblock<1, FP8>(tmem, da0 + off, db0 + off, idesc, i > lo ? 1u : 0u, step_a, step_b);
      mma_commit_cg<1>(empty0 + 8u * stage);
      if (++stage == static_cast<uint32_t>(p.stages)) stage = 0, phase ^= 1u;
    }
    // also after a failure: every MMA issued must complete before tensor memory is freed
    mma_commit_cg<1>(tfull);
    if (!wait_bar_warp(p.watch, tfull, 0, S_TFULL) && lane == 0) wait_bar(p.watch, tfull, 0, S_DRAIN, false);
    __syncwarp();
  }
  // ---- the accumulator, [token][feature] in fp32, over the pipeline's memory
  if (warp >= 4) {
    if (wait_bar_warp(p.watch, tfull, 0, S_TFULL)) {
      tc_fence_after();
      const int quad = warp & 3;
      for (int c = 0; c < tokens; c += 32) {
        uint32_t r[32];
        tmem_ld32_sync(tmem + (static_cast<uint32_t>(quad * 32) << 16) + c, r);
        const uint32_t at = sbase + static_cast<uint32_t>(c * FT + quad * 32 + lane) * 4u;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c + j < tokens) st_shared_u32(at + static_cast<uint32_t>(j * FT) * 4u, r[j]);
      }
      tc_fence_before();
    }
  }
  __syncwarp();
  cluster_sync();  // every thread of the cluster
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<1>(tmem, p.tmem_cols);
  }
  // ---- sums over the cluster and the epilogue: four features of one token at a time
  const float s0 = FP8 ? __ldg(p.sx) * __ldg(p.sw0) : 1.0f;
  const float s1 = FP8 && KIND == EPI_GATED ? __ldg(p.sx) * __ldg(p.sw1) : 1.0f;
  const bool good = *reinterpret_cast<volatile uint32_t*>(p.watch.err) == 0u;
  for (int i = first; good && i < tokens * QUADS; i += S * THREADS) {
    const int tok = i / QUADS, fq = i % QUADS * 4;
    const int64_t row = t0 + tok;
    const int col = f0 + fq, count = p.M - col;
    if (count <= 0) continue;
    if (i != first) fetch(i);
    const uint32_t at = sbase + static_cast<uint32_t>(tok * FT + fq) * 4u;
    float4 x[MAX_SPLIT], y[MAX_SPLIT];  // all in flight before the first is added
#pragma unroll
    for (int s = 0; s < MAX_SPLIT; ++s) {
      if (s >= S) break;
      const uint32_t peer = map_to_rank(at, s);
      x[s] = ld_cluster_f4(peer);
      if constexpr (KIND == EPI_GATED) y[s] = ld_cluster_f4(peer + FT / 2 * 4);
    }
    float v[4] = {}, u[4] = {};
#pragma unroll
    for (int s = 0; s < MAX_SPLIT; ++s) {
      if (s >= S) break;
      v[0] += x[s].x, v[1] += x[s].y, v[2] += x[s].z, v[3] += x[s].w;
      if constexpr (KIND == EPI_GATED) u[0] += y[s].x, u[1] += y[s].y, u[2] += y[s].z, u[3] += y[s].w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= s0, u[j] *= s1;
    if constexpr (KIND == EPI_LINEAR) {
      if (p.bias) add4(pre_b, v);
      if (p.out1) put4(p.out1 + row * p.ld1 + col, v, count);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = act_any(p.act, v[j]);
      if (p.residual) add4(pre_r, v);
    }
    if constexpr (KIND == EPI_GATED) {
      if (p.out1) {
        put4(p.out1 + row * p.ld1 + col, v, count);
        put4(p.out2 + row * p.ld2 + col, u, count);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = act_any(p.act, v[j]) * u[j];
    }
    put4(p.out + row * p.ldo + col, v, count);
  }
  __syncwarp();
  cluster_sync_relaxed();  // no CTA leaves while a peer reads its shared memory
}

template <int KIND, bool FP8>
cudaError_t launch_split_as(const Args& p, int tiles, int S, int smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * S));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(S);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, split_kernel<KIND, FP8>, p);
}

}  // namespace

cudaError_t configure_split(Machine* m) {
  const void* fns[] = {reinterpret_cast<const void*>(split_kernel<EPI_PLAIN, false>),
                       reinterpret_cast<const void*>(split_kernel<EPI_LINEAR, false>),
                       reinterpret_cast<const void*>(split_kernel<EPI_LINEAR, true>),
                       reinterpret_cast<const void*>(split_kernel<EPI_GATED, false>),
                       reinterpret_cast<const void*>(split_kernel<EPI_GATED, true>)};
  for (const void* f : fns) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_ONE);
    if (e != cudaSuccess) return e;
  }
  // The occupancy query counts a kernel that allocates tensor memory as one CTA
  // per SM.  Two do run together when shared memory and tensor memory allow it
  // (304 CTAs of 64 columns each were seen to start within 0.4 us).
  for (int s = 1; s <= MAX_SPLIT; ++s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(s));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_ONE;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(s);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&m->clusters[0][s], split_kernel<EPI_GATED, false>, &cfg);
    if (e != cudaSuccess) return e;
    m->clusters[1][s] = 2 * m->clusters[0][s];
  }
  return cudaSuccess;
}

// Bytes of a stage's tokens.
static int token_bytes(int nt, bool b_mn) { return b_mn ? (nt + 63) / 64 * 8192 : nt * KB; }

// Tokens of a tile, stages and the cluster size: the largest with which all
// tiles are resident at once (a second round of clusters costs more than
// longer slices) and a CTA still has four K blocks (below that the cluster's
// additions cost more than the slices save).  False if not all tiles are.
static bool plan_split(const Machine& mc, const Product& q, bool fp8, bool gated, int64_t split, SplitPlan* plan,
                       double* us) {
  SplitPlan& o = *plan;
  const bool b_mn = q.a[0].mn_major;
  const int kb = ceil_div(q.K, fp8 ? KB : KB / 2) * q.terms;
  const int tiles_t = ceil_div(q.M, b_mn ? 128 : 256);
  o.nt = ceil_div(ceil_div(q.M, tiles_t), 16) * 16;
  const int64_t tiles = static_cast<int64_t>(tiles_t) * ceil_div(q.N, gated ? FT / 2 : FT);
  const int stage = A_BYTES + token_bytes(o.nt, b_mn);
  // two CTAs per SM while they hold at least three stages each
  const int per_sm = (SMEM_TWO - SMEM_TAIL) / stage >= 3 ? 2 : 1;
  o.stages = std::min(MAX_STAGES, ((per_sm == 2 ? SMEM_TWO : SMEM_ONE) - SMEM_TAIL) / stage);
  o.split = 1;
  for (int s = 2; s <= MAX_SPLIT && s * 4 <= kb; ++s)
    if (tiles <= mc.clusters[per_sm - 1][s]) o.split = s;
  if (split > 0) o.split = static_cast<int>(std::min<int64_t>(split, kb));
  // measured: 9.6 us and 0.31 us a K block with 128 tokens, two CTAs per SM; one per SM, 8.0 and 0.32 with 192, 9.1
  // and 0.39 with 256
  const int64_t places = std::max(1, mc.clusters[per_sm - 1][o.split]);
  const int64_t blocks = (tiles + places - 1) / places * ((kb + o.split - 1) / o.split);
  *us = per_sm == 2 ? 6.0 + 0.028 * o.nt + static_cast<double>(blocks) * (0.2 + 0.0009 * o.nt)
                    : 4.5 + 0.018 * o.nt + static_cast<double>(blocks) * (0.13 + 0.001 * o.nt);
  return tiles <= places;
}

// By rule: up to 128 tokens always (128 tokens: level with the pairs on
// 14336x4096, 26.6 us and 26.3, and 5000x1000, 10.3 and 9.6; ahead on 1024x1024,
// 6.3 and 6.9, 4096x4096, 13.9 and 16.6, and 3584x8192, 18.0 and 27.5), otherwise
// where all tiles are resident and the models say so (512 tokens, 1000x5000:
// 15.7 us, 21.9 on pairs; 4096x4096: 22.2 us, 18.2 on pairs).  A weight's
// gradient has the weight's rows for tokens and the tokens for its contraction:
// few tiles of a small weight, long ones of a long batch.
bool use_split(const Machine& mc, const Product& q, bool fp8, bool gated, int64_t path, int64_t split,
               SplitPlan* plan) {
  if (path == 1) return false;
  double split_us = 0, pairs_us = 0;
  const bool fits = plan_split(mc, q, fp8, gated, split, plan, &split_us);
  if (path == 2 || q.M <= 128) return true;
  if (!fits) return false;
  int width;
  plan_width(mc, &q, 1, fp8, gated, &width, &pairs_us);
  return split_us < pairs_us;
}

bool split_cost(const Machine& mc, const Product& q, int64_t path, int64_t split, SplitPlan* plan, double* us) {
  const bool fits = plan_split(mc, q, false, false, split, plan, us);
  return path == 2 || (path == 0 && fits);
}

cudaError_t launch_split(const Product& c, const SplitPlan& plan, bool fp8, const Epi& e, const Watch& w,
                         cudaStream_t s) {
  const bool gated = e.kind == EPI_GATED;
  // The forms of operands that the kernel has: features may be MN-major by themselves, tokens only with them, and
  // the gated form has both K-major.
  for (int t = 0; t < (gated ? 2 : c.terms); ++t)
    if (c.b[t].mn_major != c.b[0].mn_major || (t < c.terms && c.a[t].mn_major != c.a[0].mn_major))
      return cudaErrorInvalidValue;
  if ((c.a[0].mn_major && !c.b[0].mn_major) || (c.b[0].mn_major && (gated || fp8)) || (gated && c.terms != 1))
    return cudaErrorInvalidValue;
  Args p;
  std::memset(&p, 0, sizeof(p));
  // the roles are swapped: B's rows (features) are the MMA's M, A's rows (tokens) its N
  p.M = static_cast<int>(c.N), p.N = static_cast<int>(c.M);
  p.tiles_f = ceil_div(c.N, gated ? FT / 2 : FT);
  p.nt = plan.nt;
  p.kb_seg = ceil_div(c.K, fp8 ? KB : KB / 2);
  p.kb = p.kb_seg * c.terms;
  p.a_mn = c.b[0].mn_major;
  p.b_mn = c.a[0].mn_major;
  p.b_bytes = token_bytes(plan.nt, p.b_mn);
  p.stages = plan.stages;
  p.tmem_cols = 32;
  while (p.tmem_cols < p.nt) p.tmem_cols *= 2;
  bool ok = true;
  for (int t = 0; t < c.terms && ok; ++t)
    ok = encode_operand(&p.a[t], c.b[t], fp8, c.N, c.K, gated ? FT / 2 : FT) &&
         encode_operand(&p.b[t], c.a[t], fp8, c.M, c.K, p.nt);
  if (ok && gated) ok = encode_operand(&p.a[1], c.b[1], fp8, c.N, c.K, FT / 2);
  if (!ok) return cudaErrorInvalidValue;
  p.act = e.act;
  p.bias = static_cast<const __nv_bfloat16*>(e.bias);
  p.bias_vec = reinterpret_cast<uintptr_t>(e.bias) % 8 == 0;  // callers may slice it from a packed vector
  p.residual = static_cast<const __nv_bfloat16*>(e.residual);
  p.out = static_cast<__nv_bfloat16*>(c.out);
  p.out1 = static_cast<__nv_bfloat16*>(e.out1);
  p.out2 = static_cast<__nv_bfloat16*>(e.out2);
  p.ldr = e.ldr, p.ldo = c.ldo, p.ld1 = e.ld1, p.ld2 = e.ld2;
  p.sx = e.sx, p.sw0 = e.sw0, p.sw1 = e.sw1;
  p.watch = w;
  const int tiles = p.tiles_f * ceil_div(c.M, p.nt);
  const int smem = p.stages * (A_BYTES + p.b_bytes) + SMEM_TAIL;
  switch (e.kind) {
    case EPI_LINEAR: return fp8 ? launch_split_as<EPI_LINEAR, true>(p, tiles, plan.split, smem, s)
                                : launch_split_as<EPI_LINEAR, false>(p, tiles, plan.split, smem, s);
    case EPI_GATED: return fp8 ? launch_split_as<EPI_GATED, true>(p, tiles, plan.split, smem, s)
                               : launch_split_as<EPI_GATED, false>(p, tiles, plan.split, smem, s);
    default: return launch_split_as<EPI_PLAIN, false>(p, tiles, plan.split, smem, s);
  }
}

}  // namespace tpo
