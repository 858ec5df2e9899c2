// Gradient of attention (sm_103a).  With p = exp(scale q k^T - lse) and
// ds = p (dout v^T - delta):  dv = p^T dout,  dk = scale ds^T q,  dq = scale ds k.
//
// Two kernels of one form, so that no sum depends on the order in which blocks
// come: one holds a tile of 128 keys and walks over the queries that see it, the
// other holds 128 query rows and walks over their keys.  Both recompute p, seven
// products for the five of a single pass whose dq would be added up in memory.
// (The rows of a query tile are the heads that share a key head, token by token,
// as in the forward pass.)
//
//   keys:     S^T = K Q^T, dP^T = V dO^T;  dV += P^T dO, dK += dS^T Q
//   queries:  S = Q K^T,   dP = dO V^T;    dQ += dS K
//
// The first two are taken from shared memory; P and dS (bf16) go back to tensor
// memory over S and dP, as operands of the others, so they never pass through
// shared memory.  The products are ordered so that the tensor core has one to
// work on while the threads are at the other half of a step.
//
// Roles: warp 0 loads (TMA), warp 1 issues the MMAs, warps 2 and 3 bring the
// rows' statistics and clear rows that belong to no query (or key) of the
// sequence, warps 4-7 and 8-11 compute, each group half of a step's columns.

#include <algorithm>
#include <cstring>

#include <cuda_bf16.h>

#include "attn_dev.h"
#include "pdl.h"

namespace tpo {

namespace {

using bf16 = __nv_bfloat16;
constexpr int THREADS = 384;
constexpr int COMPUTE = 256;  // threads of the two computing groups

struct Args {
  CUtensorMap q, dout, k, v;
  Sequences seq;
  int heads, kv_heads, group, tokens;  // tokens: of a query tile
  int dim, causal;
  float scale, c;       // c: scale log2(e)
  const float2* stats;  // [n, heads]: -lse log2(e), -delta
  bf16 *out0, *out1;    // dv and dk, or dq
  int64_t ld0, h0, ld1, h1;
  float* part;
  uint32_t* arrivals;
  Watch watch;
};

// KEYS: tiles of keys, steps of queries; otherwise the other way round.
template <bool KEYS>
struct Tiles {
  int kv_heads, tokens, causal;
  __device__ __forceinline__ int tiles(const Seq& s) const {
    return KEYS ? (s.nk + BLK - 1) / BLK : (s.nq + tokens - 1) / tokens;
  }
  __device__ __forceinline__ void range(const Seq& s, int tile, int* lo, int* hi) const {
    if constexpr (KEYS) {
      *lo = causal ? max(0, tile * BLK - s.nk + s.nq) / tokens : 0;
      *hi = max((s.nq + tokens - 1) / tokens, *lo + 1);  // a step of none where there are no queries
    } else {
      const int limit = keys_seen(s, min(s.nq, (tile + 1) * tokens) - 1, causal);
      *lo = 0;
      *hi = limit <= BLK ? 1 : (limit + BLK - 1) / BLK;
    }
  }
};

template <int DP>
struct Layout {
  static constexpr int TILE = BLK * DP * 2;
  static constexpr int STAGES = DP == 128 ? 2 : 4;  // of each ring
  static constexpr int F1 = TILE, R0 = 2 * TILE, R1 = R0 + STAGES * TILE;  // the tile's two matrices, the rings
  static constexpr int STATS = R1 + STAGES * TILE;  // [stage][2][128]: -lse log2(e), -delta
  static constexpr int BARS = STATS + STAGES * 1024;
  static constexpr int N_BARS = 6 * STAGES + 9;
  static constexpr int SLOT = BARS + 8 * N_BARS, LAST = SLOT + 4;
  static constexpr int STAGE = (SLOT + 8 + 15) / 16 * 16;  // a staging box for each computing warp
  static constexpr int PLAN = STAGE + 8 * 2048;
  static constexpr int SMEM = PLAN + static_cast<int>(sizeof(PlanScratch)) + 1024;
  static_assert(SMEM <= 232448, "shared memory of one block");
};

template <int DP>
struct Bars {
  uint32_t full0, full1, empty0, empty1, fix, free, ffull, fempty, sfull, pfull, dpfull, dsfull, accfull, drain;
  __device__ explicit Bars(uint32_t sbase) {
    uint32_t b = sbase + Layout<DP>::BARS;
    auto next = [&](int n) {
      const uint32_t r = b;
      b += 8 * n;
      return r;
    };
    constexpr int S = Layout<DP>::STAGES;
    full0 = next(S), full1 = next(S), empty0 = next(S), empty1 = next(S), fix = next(S), free = next(S);
    ffull = next(1), fempty = next(1), sfull = next(2), pfull = next(1), dpfull = next(1), dsfull = next(1);
    accfull = next(1), drain = next(1);
  }
};

__device__ __forceinline__ void bar_compute() { asm volatile("bar.sync 1, %0;" ::"n"(COMPUTE) : "memory"); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

template <int DP, bool KEYS>
__device__ void load_role(const Args& a, const Tiles<KEYS>& tiles, const Shares& sh, uint32_t sbase) {
  using L = Layout<DP>;
  const Bars<DP> b(sbase);
  const bool lead = (threadIdx.x & 31) == 0;
  const uint32_t qbytes = static_cast<uint32_t>(a.group * a.tokens) * 128u * (DP / 64), kbytes = L::TILE;
  const CUtensorMap *f0 = KEYS ? &a.k : &a.q, *f1 = KEYS ? &a.v : &a.dout, *r0 = KEYS ? &a.q : &a.k,
                    *r1 = KEYS ? &a.dout : &a.v;
  uint32_t n = 0, n1 = 0, fn = 0;  // loads so far
  bool ok = true;
  Walk w;
  for (walk_begin(tiles, sh, w); ok && walk_has(w); walk_next(tiles, a.seq, w)) {
    const Part p = walk_part(w);
    const int qh = w.head * a.group, kh = w.head;
    auto load = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, int head, int row) {
      for (int d = 0; d < DP / 64; ++d) tma_load_3d(dst + d * 16384, map, bar, d * 64, head, row);
    };
    if (!(ok = wait_warp(a.watch, b.fempty, (fn & 1u) ^ 1u, S_EMPTY))) break;
    if (lead) {
      const int head = KEYS ? kh : qh, row = KEYS ? w.s.k0 + w.tile * BLK : w.s.q0 + w.tile * a.tokens;
      mbar_expect_tx(b.ffull, 2 * (KEYS ? kbytes : qbytes));
      load(sbase, f0, b.ffull, head, row);
      load(sbase + L::F1, f1, b.ffull, head, row);
    }
    __syncwarp();
    ++fn;
    for (int j = p.lo; j < p.hi; ++j) {
      const int head = KEYS ? qh : kh, row = KEYS ? w.s.q0 + j * a.tokens : w.s.k0 + j * BLK;
      const uint32_t st = n % L::STAGES, ph = n / L::STAGES & 1u;
      if (!(ok = wait_warp(a.watch, b.empty0 + 8 * st, ph ^ 1u, S_EMPTY))) break;
      if (lead) {
        mbar_expect_tx(b.full0 + 8 * st, KEYS ? qbytes : kbytes);
        load(sbase + L::R0 + st * L::TILE, r0, b.full0 + 8 * st, head, row);
      }
      __syncwarp();
      ++n;
      if (!(ok = wait_warp(a.watch, b.empty1 + 8 * st, ph ^ 1u, S_EMPTY))) break;
      if (lead) {
        mbar_expect_tx(b.full1 + 8 * st, KEYS ? qbytes : kbytes);
        load(sbase + L::R1 + st * L::TILE, r1, b.full1 + 8 * st, head, row);
      }
      __syncwarp();
      ++n1;
    }
  }
  if (!ok && lead) {  // what is in flight must land before the block gives up its shared memory
    for (uint32_t j = n > L::STAGES ? n - L::STAGES : 0u; j < n; ++j)
      wait_bar(a.watch, b.full0 + 8 * (j % L::STAGES), j / L::STAGES & 1u, S_DRAIN, false);
    for (uint32_t j = n1 > L::STAGES ? n1 - L::STAGES : 0u; j < n1; ++j)
      wait_bar(a.watch, b.full1 + 8 * (j % L::STAGES), j / L::STAGES & 1u, S_DRAIN, false);
    if (fn) wait_bar(a.watch, b.ffull, (fn - 1) & 1u, S_DRAIN, false);
  }
  __syncwarp();
}

// Tensor memory: KEYS S, dP, dV and dK; otherwise S of even steps, dP, dQ and S of odd steps.
template <int DP, bool KEYS>
__device__ void mma_role(const Args& a, const Tiles<KEYS>& tiles, const Shares& sh, uint32_t sbase, uint32_t tmem) {
  using L = Layout<DP>;
  const Bars<DP> b(sbase);
  const int ksteps = (a.dim + 15) / 16;
  const uint32_t idesc_s = idesc_n(make_idesc(false, BLK), BLK);
  const uint32_t idesc_o = idesc_n(make_idesc(false, BLK), ksteps * 16) | 1u << 16;
  const uint64_t f0 = smem_desc_sw128(sbase), f1 = smem_desc_sw128(sbase + L::F1),
                 r0 = smem_desc_sw128(sbase + L::R0), r1 = smem_desc_sw128(sbase + L::R1),
                 t0 = desc_rows(sbase + L::R0), t1 = desc_rows(sbase + L::R1);
  const uint32_t dp = tmem + BLK, acc0 = tmem + 2 * BLK, acc1 = tmem + 3 * BLK;
  uint32_t n = 0, fn = 0;  // steps and parts so far
  bool ok = true;
  Walk w;
  for (walk_begin(tiles, sh, w); ok && walk_has(w); walk_next(tiles, a.seq, w), ++fn) {
    const Part p = walk_part(w);
    const int steps = p.hi - p.lo;
    auto stage = [&](uint32_t s) { return static_cast<uint64_t>(s % L::STAGES) * (L::TILE >> 4); };
    // step s of the launch: S and dP from shared memory
    auto scores = [&](uint32_t s) {
      if (!wait_warp(a.watch, b.full0 + 8 * (s % L::STAGES), s / L::STAGES & 1u, S_FULL)) return false;
      tc_fence_after();
      const uint32_t d = KEYS || !(s & 1u) ? tmem : acc1;
      mma_head<DP>(d, f0, r0 + stage(s), idesc_s);
      mma_commit_cg<1>(b.sfull + 8 * (s & 1u));  // two: the threads may still be at the step before
      return true;
    };
    auto dots = [&](uint32_t s) {
      if (!wait_warp(a.watch, b.full1 + 8 * (s % L::STAGES), s / L::STAGES & 1u, S_FULL)) return false;
      tc_fence_after();
      mma_head<DP>(dp, f1, r1 + stage(s), idesc_s);
      mma_commit_cg<1>(b.dpfull);
      return true;
    };
    // an accumulator += bf16 columns at `from` (64 and 64 columns apart) . rows of a ring's stage
    auto add = [&](uint32_t acc, uint32_t from, uint64_t rows, bool fresh) {
      tc_fence_after();
      mma4_ts(acc, from, rows, idesc_o, !fresh);
      mma4_ts(acc, from + 64, rows + 512, idesc_o, 1u);
    };
    if (!(ok = wait_warp(a.watch, b.ffull, fn & 1u, S_FULL))) break;
    ok = scores(n) && dots(n);
    for (int i = 0; ok && i < steps; ++i, ++n) {
      const uint32_t st = n % L::STAGES;
      if constexpr (KEYS) {
        if (!(ok = wait_warp(a.watch, b.pfull, n & 1u, S_TFULL))) break;
        add(acc0, tmem, t1 + stage(n), i == 0);  // dV
        mma_commit_cg<1>(b.empty1 + 8 * st);
        if (i + 1 < steps && !(ok = scores(n + 1))) break;
        if (!(ok = wait_warp(a.watch, b.dsfull, n & 1u, S_TFULL))) break;
        add(acc1, dp, t0 + stage(n), i == 0);  // dK
        mma_commit_cg<1>(b.empty0 + 8 * st);
      } else {
        if (i + 1 < steps && !(ok = scores(n + 1))) break;
        if (!(ok = wait_warp(a.watch, b.dsfull, n & 1u, S_TFULL))) break;
        mma_commit_cg<1>(b.empty1 + 8 * st);  // V: dP of this step is done
        add(acc0, dp, t0 + stage(n), i == 0);  // dQ
        mma_commit_cg<1>(b.empty0 + 8 * st);
      }
      if (i + 1 < steps && !(ok = dots(n + 1))) break;
    }
    if (!ok) break;
    mma_commit_cg<1>(b.fempty);
    mma_commit_cg<1>(b.accfull);
  }
  // also after a failure: every MMA issued must complete before tensor memory is freed
  mma_commit_cg<1>(b.drain);
  if ((threadIdx.x & 31) == 0) wait_bar(a.watch, b.drain, 0u, S_DRAIN, false);
  __syncwarp();
}

// Statistics of a step's query rows (KEYS), and rows of the rings that belong to
// no query or key of the sequence cleared, since they are operands of the products
// with P and dS.
template <int DP, bool KEYS>
__device__ void aux_role(const Args& a, const Tiles<KEYS>& tiles, const Shares& sh, uint32_t sbase, uint8_t* smem) {
  using L = Layout<DP>;
  const Bars<DP> b(sbase);
  const int lane = threadIdx.x & 31, me = threadIdx.x - 64;
  const int used = a.group * a.tokens;
  uint32_t n = 0;
  Walk w;
  for (walk_begin(tiles, sh, w); walk_has(w); walk_next(tiles, a.seq, w)) {
    const Part p = walk_part(w);
    for (int j = p.lo; j < p.hi; ++j, ++n) {
      const uint32_t st = n % L::STAGES, ph = n / L::STAGES & 1u;
      const int left = KEYS ? min(a.tokens, w.s.nq - j * a.tokens) * a.group : w.s.nk - j * BLK;  // rows in use
      if constexpr (KEYS) {
        if (!wait_warp(a.watch, b.free + 8 * st, ph ^ 1u, S_EMPTY)) return;
        float* stats = reinterpret_cast<float*>(smem + L::STATS) + st * 256;
#pragma unroll
        for (int r = me; r < BLK; r += 64) {
          float2 v = make_float2(-INFINITY, 0.0f);  // a weight of 0
          if (r < left) {
            const int tok = r / a.group;
            v = a.stats[(static_cast<int64_t>(w.s.q0) + j * a.tokens + tok) * a.heads + w.head * a.group +
                        (r - tok * a.group)];
          }
          stats[r] = v.x;
          stats[BLK + r] = v.y;
        }
      }
      if (!wait_warp(a.watch, b.full0 + 8 * st, ph, S_FULL)) return;
      if (KEYS && !wait_warp(a.watch, b.full1 + 8 * st, ph, S_FULL)) return;
      if (left < (KEYS ? used : BLK)) {
        for (int r = me; r < BLK; r += 64) {
          if (r < left) continue;
#pragma unroll
          for (int d = 0; d < DP / 64; ++d)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t at = st * L::TILE + d * 16384 + r * 128 + ((i ^ (r & 7)) << 4);
              *reinterpret_cast<uint4*>(smem + L::R0 + at) = make_uint4(0, 0, 0, 0);
              if (KEYS) *reinterpret_cast<uint4*>(smem + L::R1 + at) = make_uint4(0, 0, 0, 0);
            }
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(b.fix + 8 * st);
    }
  }
}

template <int DP, bool KEYS>
__device__ void compute_role(const Args& a, const Tiles<KEYS>& tiles, const Shares& sh, uint32_t sbase, uint8_t* smem,
                             uint32_t tmem) {
  using L = Layout<DP>;
  const Bars<DP> b(sbase);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = warp & 3, half = (warp - 4) >> 2;
  const int row = quad * 32 + lane, me = threadIdx.x - 128;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16), mine = lanes + half * 64;
  const int dt = row / a.group, head_in = row - dt * a.group;
  const int chunks = (a.dim + 31) / 32;
  const float2 c2 = make_float2(a.c, a.c);
  uint32_t n = 0, fn = 0;
  bool ok = true;
  Walk w;
  for (walk_begin(tiles, sh, w); walk_has(w); walk_next(tiles, a.seq, w), ++fn) {
    const Part p = walk_part(w);
    // KEYS: this row's key, and the first token that sees it; otherwise the row's query and the keys that it sees
    const int tok = w.tile * a.tokens + dt;
    const bool valid = KEYS ? w.tile * BLK + row < w.s.nk : dt < a.tokens && tok < w.s.nq;
    const int seen = KEYS ? (a.causal ? w.tile * BLK + row - w.s.nk + w.s.nq : 0)
                          : (valid ? keys_seen(w.s, tok, a.causal) : 0);
    float2 nl = make_float2(0.0f, 0.0f), nd = nl;
    if (!KEYS && valid) {
      const float2 v = a.stats[(static_cast<int64_t>(w.s.q0) + tok) * a.heads + w.head * a.group + head_in];
      nl = make_float2(v.x, v.x), nd = make_float2(v.y, v.y);
    }
    for (int j = p.lo; j < p.hi; ++j, ++n) {
      const uint32_t st = n % L::STAGES, ph = n / L::STAGES & 1u;
      // columns [from, to) of the group's 64 that the row sees
      const int from = KEYS ? min(a.tokens, max(0, seen - j * a.tokens)) * a.group - half * 64 : 0;
      const int to = (KEYS ? min(a.tokens, w.s.nq - j * a.tokens) * a.group : seen - j * BLK) - half * 64;
      const bool all = __all_sync(0xffffffffu, from <= 0 && to >= 64);
      const float* stats = reinterpret_cast<const float*>(smem + L::STATS) + st * 256 + half * 64;
      float2 pr[32];
      if (ok) ok = wait_warp(a.watch, b.sfull + 8 * (n & 1u), n >> 1 & 1u, S_TFULL);
      if (KEYS && ok) ok = wait_warp(a.watch, b.fix + 8 * st, ph, S_FULL);
      if (ok) {
        tc_fence_after();
        uint32_t x[64];
        tmem_ld64_sync(mine + (KEYS || !(n & 1u) ? 0 : 3 * BLK), x);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float2 l0 = nl, l1 = nl;
          if constexpr (KEYS) {
            const float4 v = *reinterpret_cast<const float4*>(stats + 2 * e);
            l0 = make_float2(v.x, v.y), l1 = make_float2(v.z, v.w);
          }
          const float2 s0 = fma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), c2, l0);
          const float2 s1 = fma2(make_float2(__uint_as_float(x[2 * e + 2]), __uint_as_float(x[2 * e + 3])), c2, l1);
          pr[e] = make_float2(exp2_fast(s0.x), exp2_fast(s0.y));
          pr[e + 1] = make_float2(exp2_fast(s1.x), exp2_fast(s1.y));
        }
        if (!all) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            if (2 * e < from || 2 * e >= to) pr[e].x = 0.0f;
            if (2 * e + 1 < from || 2 * e + 1 >= to) pr[e].y = 0.0f;
          }
        }
        if constexpr (KEYS) {
          uint32_t h[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) h[e] = pack_bf16(pr[e].x, pr[e].y);
          tmem_st32(mine, h);
          tmem_wait_st();
        }
      }
      if constexpr (KEYS) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b.pfull);
      }
      if (ok) ok = wait_warp(a.watch, b.dpfull, n & 1u, S_TFULL);
      if (!KEYS && ok) ok = wait_warp(a.watch, b.fix + 8 * st, ph, S_FULL);
      if (ok) {
        tc_fence_after();
        uint32_t x[64], h[32];
        tmem_ld64_sync(mine + BLK, x);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float2 d0 = nd, d1 = nd;
          if constexpr (KEYS) {
            const float4 v = *reinterpret_cast<const float4*>(stats + BLK + 2 * e);
            d0 = make_float2(v.x, v.y), d1 = make_float2(v.z, v.w);
          }
          float2 g0 = mul2(pr[e], add2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), d0));
          float2 g1 = mul2(pr[e + 1], add2(make_float2(__uint_as_float(x[2 * e + 2]), __uint_as_float(x[2 * e + 3])), d1));
          if (!all) {  // what is not seen may be anything
            if (2 * e < from || 2 * e >= to) g0.x = 0.0f;
            if (2 * e + 1 < from || 2 * e + 1 >= to) g0.y = 0.0f;
            if (2 * e + 2 < from || 2 * e + 2 >= to) g1.x = 0.0f;
            if (2 * e + 3 < from || 2 * e + 3 >= to) g1.y = 0.0f;
          }
          h[e] = pack_bf16(g0.x, g0.y);
          h[e + 1] = pack_bf16(g1.x, g1.y);
        }
        tmem_st32(mine + BLK, h);
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(b.dsfull);
        mbar_arrive(b.free + 8 * st);
      }
    }
    // ---- the end of the part: one group writes dV, the other dK; or each its chunks of dQ
    if (ok) ok = wait_warp(a.watch, b.accfull, fn & 1u, S_TFULL);
    tc_fence_after();
    const bool second = KEYS && half == 1;
    const float scale = KEYS && !second ? 1.0f : a.scale;
    bf16* out = second ? a.out1 : a.out0;
    const int64_t ld = second ? a.ld1 : a.ld0, hs = second ? a.h1 : a.h0;
    const int64_t out_row = KEYS ? static_cast<int64_t>(w.s.k0) + w.tile * BLK + row : static_cast<int64_t>(w.s.q0) + tok;
    const int head = KEYS ? w.head : w.head * a.group + head_in;
    const int64_t slot = static_cast<int64_t>(KEYS ? 2 : 1) * BLK * a.dim;
    float* part = a.part + part_slot(w) * slot + static_cast<int64_t>(second ? BLK : 0) * a.dim;
    uint8_t* stage = smem + L::STAGE + (warp - 4) * 2048;
    const void* to_row = valid && p.whole ? out + out_row * ld + head * hs : nullptr;
#pragma unroll 1
    for (int c = KEYS ? 0 : half; ok && c < chunks; c += KEYS ? 1 : 2) {  // 32 columns
      uint32_t o[32];
      tmem_ld32_sync(lanes + (second ? 3 : 2) * BLK + c * 32, o);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(o[8 * g + e]) * scale;
        if (p.whole)
          stage_row<32>(stage, g, v);
        else if (valid)
          store_part(part, BLK, row, v, c * 32 + g * 8, a.dim);
      }
      if (p.whole) store_staged<32>(stage, to_row, c * 32, a.dim - c * 32);
    }
    tc_fence_before();
    if (p.whole) continue;
    // ---- a divided tile: whoever comes last adds its parts
    __threadfence();
    bar_compute();
    int first;
    const int shares = tile_shares(sh, tile_begin(sh, w), w.hi - w.lo, &first);
    volatile int* last = reinterpret_cast<volatile int*>(smem + L::LAST);
    if (me == 0) {
      const uint32_t before = atomicAdd(a.arrivals + first, ok ? 1u : 0u);
      *last = ok && before + 1 == static_cast<uint32_t>(shares);
      if (*last) a.arrivals[first] = 0;
    }
    bar_compute();
    if (*last) {
      __threadfence();
      // a matrix's rows side by side, eight columns at a time, and two such groups
      constexpr int U = 2;
      const int groups = (KEYS ? 2 : 1) * BLK * (a.dim / 8);
      for (int i0 = me; i0 < groups; i0 += U * COMPUTE) {
        float4 v[U][2];
        const float* src[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = min(i0 + u * COMPUTE, groups - 1);
          v[u][0] = v[u][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          src[u] = a.part + (static_cast<int64_t>(2 * (i >> 7)) * BLK + (i & (BLK - 1))) * 4;
        }
        auto add = [&](int s) {
          const int64_t at = tile_slot(first, s) * slot;
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float4 y = *reinterpret_cast<const float4*>(src[u] + at + j * BLK * 4);
              v[u][j].x += y.x, v[u][j].y += y.y, v[u][j].z += y.z, v[u][j].w += y.w;
            }
        };
        int s = 0;
#pragma unroll 1
        for (; s + 4 <= shares; s += 4) add(s), add(s + 1), add(s + 2), add(s + 3);
        if (s + 2 <= shares) add(s), add(s + 1), s += 2;
        if (s < shares) add(s);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * COMPUTE, in = i & (BLK - 1), g = i >> 7;
          if (i >= groups) continue;
          const bool two = KEYS && g >= a.dim / 8;  // the second matrix
          const int col = (g - (two ? a.dim / 8 : 0)) * 8;
          int64_t o_row;
          int h = w.head;
          if constexpr (KEYS) {
            if (w.tile * BLK + in >= w.s.nk) continue;
            o_row = static_cast<int64_t>(w.s.k0) + w.tile * BLK + in;
          } else {
            const int d = in / a.group;
            if (d >= a.tokens || w.tile * a.tokens + d >= w.s.nq) continue;
            o_row = static_cast<int64_t>(w.s.q0) + w.tile * a.tokens + d;
            h = w.head * a.group + in - d * a.group;
          }
          *reinterpret_cast<uint4*>((two ? a.out1 : a.out0) + o_row * (two ? a.ld1 : a.ld0) + h * (two ? a.h1 : a.h0) + col) =
              make_uint4(pack_bf16(v[u][0].x, v[u][0].y), pack_bf16(v[u][0].z, v[u][0].w),
                         pack_bf16(v[u][1].x, v[u][1].y), pack_bf16(v[u][1].z, v[u][1].w));
        }
      }
    }
    bar_compute();
  }
}

// Grid: one block per SM at most, each an equal share of the steps.
template <int DP, bool KEYS>
__global__ void __launch_bounds__(THREADS, 1) bwd_kernel(const __grid_constant__ Args a) {
  using L = Layout<DP>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  grid_dep_launch();
  const int warp = threadIdx.x >> 5;
  PlanScratch* plan = reinterpret_cast<PlanScratch*>(smem + L::PLAN);
  if (threadIdx.x == 0) {
    const Bars<DP> b(sbase);
    auto init = [&](uint32_t bar, int n, uint32_t count) {
      for (int i = 0; i < n; ++i) mbar_init(bar + 8 * i, count);
    };
    init(b.full0, 4 * L::STAGES, 1);  // and full1, empty0, empty1
    init(b.fix, L::STAGES, 2);
    init(b.free, L::STAGES, 8);
    init(b.ffull, 2, 1);  // and fempty
    init(b.sfull, 2, 1);
    init(b.pfull, 1, 8);
    init(b.dpfull, 1, 1);
    init(b.dsfull, 1, 8);
    init(b.accfull, 2, 1);  // and drain
    fence_barrier_init();
    tma_prefetch_map(&a.q);
    tma_prefetch_map(&a.dout);
    tma_prefetch_map(&a.k);
    tma_prefetch_map(&a.v);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc_cg<1>(sbase + L::SLOT, 512);
    tmem_relinquish_cg<1>();
  }
  if (KEYS) {  // rows of a query tile that no load writes are operands of the products too
    const int unused = BLK - a.group * a.tokens;
    for (int i = threadIdx.x; i < unused * 8 * (DP / 64) * 2 * L::STAGES; i += THREADS) {
      const int r = i / 8 % unused, block = i / 8 / unused;
      *reinterpret_cast<uint4*>(smem + L::R0 + block * 16384 + (BLK - 1 - r) * 128 + i % 8 * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ld_shared_u32(sbase + L::SLOT);
  grid_dep_wait();
  const Tiles<KEYS> tiles{a.kv_heads, a.tokens, a.causal};
  plan_shares<THREADS>(tiles, a.seq, plan);
  const Shares& sh = plan->shares;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;" : "+r"(sbase)::"memory");  // nothing of a role is computed ahead of it
    if (warp == 0) load_role<DP, KEYS>(a, tiles, sh, sbase);
    if (warp == 1) mma_role<DP, KEYS>(a, tiles, sh, sbase, tmem);
    if (warp >= 2) aux_role<DP, KEYS>(a, tiles, sh, sbase, smem);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;" : "+r"(sbase)::"memory");  // nothing of a role is computed ahead of it
    compute_role<DP, KEYS>(a, tiles, sh, sbase, smem, tmem);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<1>(tmem, 512);
  }
}

// -lse log2(e) and -delta of each row and head, sixteen lanes a head.  Bound by
// memory: out and dout are read once.
constexpr int STAT_THREADS = 256, STAT_ROWS = 4;  // rows of a group of lanes in flight together
__global__ void __launch_bounds__(STAT_THREADS) stats_kernel(int64_t rows, int heads, int dim, Heads out, Heads dout,
                                                            const float* lse, float2* stats) {
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 15;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (STAT_THREADS / 16);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (STAT_THREADS / 16) + (threadIdx.x >> 4);
  const int64_t rounds = (rows + step * STAT_ROWS - 1) / (step * STAT_ROWS);  // the same for every thread
  for (int64_t k = 0; k < rounds; ++k) {
    uint4 x[STAT_ROWS], y[STAT_ROWS];
#pragma unroll
    for (int r = 0; r < STAT_ROWS; ++r) {
      const int64_t i = first + (k * STAT_ROWS + r) * step, row = i / heads, h = i - row * heads;
      x[r] = y[r] = make_uint4(0, 0, 0, 0);
      if (i < rows && lane * 8 < dim) {
        x[r] = *reinterpret_cast<const uint4*>(static_cast<const bf16*>(out.p) + row * out.ld + h * out.hs + lane * 8);
        y[r] = *reinterpret_cast<const uint4*>(static_cast<const bf16*>(dout.p) + row * dout.ld + h * dout.hs + lane * 8);
      }
    }
#pragma unroll
    for (int r = 0; r < STAT_ROWS; ++r) {
      const uint32_t a[4] = {x[r].x, x[r].y, x[r].z, x[r].w}, b[4] = {y[r].x, y[r].y, y[r].z, y[r].w};
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s += __uint_as_float(a[j] << 16) * __uint_as_float(b[j] << 16);
        s += __uint_as_float(a[j] & 0xffff0000u) * __uint_as_float(b[j] & 0xffff0000u);
      }
      for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const int64_t i = first + (k * STAT_ROWS + r) * step;
      if (lane == 0 && i < rows) {
        const float l = lse[i];
        stats[i] = make_float2(l == -INFINITY ? 0.0f : -l * kLog2e, -s);
      }
    }
  }
}

int64_t stats_bytes(int64_t n, int64_t heads) { return (n * heads * 8 + 255) / 256 * 256; }

template <int DP, bool KEYS>
cudaError_t launch_as(const Args& a, int grid, cudaStream_t s) {
  return launch_pdl(bwd_kernel<DP, KEYS>, dim3(static_cast<unsigned>(grid)), dim3(THREADS), Layout<DP>::SMEM, s, a);
}
template <int DP, bool KEYS>
cudaError_t configure_as() {
  return cudaFuncSetAttribute(bwd_kernel<DP, KEYS>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<DP>::SMEM);
}

}  // namespace

cudaError_t configure_attention_bwd() {
  cudaError_t e = configure_as<64, false>();
  if (e == cudaSuccess) e = configure_as<64, true>();
  if (e == cudaSuccess) e = configure_as<128, false>();
  if (e == cudaSuccess) e = configure_as<128, true>();
  return e;
}

int64_t need_attention_bwd(int64_t n, int64_t, int64_t heads, int64_t, int64_t dim) {
  return stats_bytes(n, heads) + 2ll * MAX_SHARES * 2 * BLK * dim * 4;
}

cudaError_t launch_attention_bwd(const Machine& mc, const AttnArgs& x, const Watch& w, uint32_t* arrivals, void* ws,
                                 cudaStream_t s) {
  const int64_t n = x.seq.n, nk = x.seq.nk;
  Args a;
  std::memset(static_cast<void*>(&a), 0, sizeof(a));
  a.seq = x.seq;
  a.heads = static_cast<int>(x.heads), a.kv_heads = static_cast<int>(x.kv_heads);
  a.group = a.heads / a.kv_heads, a.tokens = BLK / a.group;
  a.dim = static_cast<int>(x.dim), a.causal = x.causal, a.scale = x.scale, a.c = x.scale * kLog2e;
  a.stats = static_cast<const float2*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + stats_bytes(n, x.heads));
  a.arrivals = arrivals, a.watch = w;
  // without keys (or queries) the loads go to the others, which no row sees
  const int64_t rq = n ? n : nk, hq = n ? x.heads : x.kv_heads, rk = nk ? nk : n, hk = nk ? x.kv_heads : x.heads;
  if (!encode_heads(&a.q, n ? x.q : x.k, rq, hq, x.dim, a.group, a.tokens) ||
      !encode_heads(&a.dout, n ? x.dout : x.k, rq, hq, x.dim, a.group, a.tokens) ||
      !encode_heads(&a.k, nk ? x.k : x.q, rk, hk, x.dim, 1, BLK) ||
      !encode_heads(&a.v, nk ? x.v : x.q, rk, hk, x.dim, 1, BLK))
    return cudaErrorInvalidValue;
  const int64_t sms = std::min(mc.sms, MAX_SHARES);
  auto grid = [&](int64_t tiles, int64_t steps) {  // no more blocks than the most steps that these sizes can have
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(sms, tiles * x.kv_heads * steps)));
  };
  const int64_t q_tiles = n / a.tokens + std::min(x.seq.batch, n), k_tiles = nk / BLK + std::min(x.seq.batch, nk);
  if (n > 0) {
    const int64_t rows = n * x.heads, per = STAT_THREADS / 16 * STAT_ROWS;
    cudaError_t e = launch_pdl(stats_kernel, dim3(static_cast<unsigned>(std::min((rows + per - 1) / per, sms * 8))),
                               dim3(STAT_THREADS), 0, s, rows, a.heads, a.dim, x.out, x.dout,
                               static_cast<const float*>(x.lse), static_cast<float2*>(ws));
    if (e != cudaSuccess) return e;
    a.out0 = static_cast<bf16*>(const_cast<void*>(x.dq.p)), a.ld0 = x.dq.ld, a.h0 = x.dq.hs;
    const int g = grid(q_tiles, nk / BLK + 1);
    e = x.dim <= 64 ? launch_as<64, false>(a, g, s) : launch_as<128, false>(a, g, s);
    if (e != cudaSuccess) return e;
  }
  if (nk == 0) return cudaSuccess;
  a.out0 = static_cast<bf16*>(const_cast<void*>(x.dv.p)), a.ld0 = x.dv.ld, a.h0 = x.dv.hs;
  a.out1 = static_cast<bf16*>(const_cast<void*>(x.dk.p)), a.ld1 = x.dk.ld, a.h1 = x.dk.hs;
  const int g = grid(k_tiles, n / a.tokens + 1);
  return x.dim <= 64 ? launch_as<64, true>(a, g, s) : launch_as<128, true>(a, g, s);
}

}  // namespace tpo
