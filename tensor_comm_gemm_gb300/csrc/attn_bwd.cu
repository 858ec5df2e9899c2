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
// Roles: warp 0 loads (TMA), warps 1 and 2 issue the MMAs (a wait or a commit
// delays the warp that makes it by 60 to 130 cycles, and the tensor core takes few
// instructions ahead of time), warp 3 brings the rows' statistics and clears rows
// that belong to no query (or key) of the sequence, warps 4-7 and 8-11 compute,
// each group half of a step's columns, and store.
//
// Measured (back-to-back calls with a flushed L2): two sequences of 4096 causal
// tokens, 32 heads of 128 over 8, 730 to 754 us, or 1.28 to 1.32 PFLOP/s of the seven
// products (65 to 67 % of the measured matrix rate; 910 to 940 TFLOP/s of the five that
// a single pass would need).  Bound by a step's chain of product, exponentials, product and
// store to tensor memory, with 512 columns of it all in use: sixteen computing
// warps of half the columns took 842 us, groups that take the steps in turns as
// long as these.  Odd sequences of 9 heads of 80 over 3: 72 us, bound by the five
// launches' starts and by filling the pipeline at each tile.

#include <algorithm>
#include <climits>
#include <cstring>

#include <cuda_bf16.h>

#include "attn_dev.h"
#include "pdl.h"

namespace tpo {

namespace {

using bf16 = __nv_bfloat16;
constexpr int THREADS = 384;

struct Args {
  CUtensorMap q, dout, k, v;
  Sequences seq;
  int heads, kv_heads, group, tokens;  // tokens: of a query tile
  int dim, causal;
  float scale, c;       // c: scale log2(e)
  const float2* stats;  // [n, heads]: -lse log2(e), -delta
  bf16 *out0, *out1;    // dv and dk, or dq
  int64_t ld0, h0, ld1, h1;
  Entry* begun;         // [MAX_SHARES]: the tile that a share begins and does not end
  float* part;          // its parts, two slots a share: matrices [dim / 4][128][4]
  Watch watch;
};

// KEYS: tiles of keys, steps of queries; otherwise the other way round.
template <bool KEYS>
struct Tiles {
  static constexpr int COST = BWD_TILE_COST;
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

// What a step takes from ring 0 is held from its first product to its last, and with two stages each step of the kernel of
// queries waited for its keys.  Where heads of 128 elements leave no memory for a third, it gets the place of the boxes
// through which rows are stored in whole lines (TIGHT): the long training case took 778 us without, 748 with it, and 762
// with a third stage in the kernel of keys too.
template <int DP, bool KEYS>
struct Layout {
  static constexpr bool TIGHT = DP == 128 && !KEYS;
  static constexpr int TILE = BLK * DP * 2;
  static constexpr int S0 = TIGHT ? 3 : DP == 128 ? 2 : 4, S1 = DP == 128 ? 2 : 4;
  static constexpr int F1 = TILE, R0 = 2 * TILE, R1 = R0 + S0 * TILE;  // the tile's two matrices, the rings
  static constexpr int STATS = R1 + S1 * TILE;  // KEYS: [stage][2][128]: -lse log2(e), -delta
  static constexpr int BARS = STATS + (KEYS ? S0 * 1024 : 0);
  static constexpr int N_BARS = 4 * S0 + 2 * S1 + RING + 13;
  static constexpr int SLOT = BARS + 8 * N_BARS;
  static constexpr int RING_AT = (SLOT + 8 + 15) / 16 * 16;
  static constexpr int SHARES = RING_AT + RING * static_cast<int>(sizeof(Entry));
  static constexpr int STAGE = (SHARES + static_cast<int>(sizeof(Shares)) + 15) / 16 * 16;
  static constexpr int END = STAGE + (TIGHT ? 0 : 8 * 2048);  // a staging box for each computing warp
  static constexpr int PLAN = TIGHT ? R0 : END;               // scratch, before the loads
  static constexpr int SMEM = (TIGHT ? END : END + static_cast<int>(sizeof(PlanScratch))) + 1024;
  static_assert(SMEM <= 232448, "shared memory of one block");
};

template <int DP, bool KEYS>
struct Bars {
  uint32_t full0, full1, empty0, empty1, fix, free, items, ffull, fempty, sfull, pfull, dpfull, dsfull, done, accfull, drain;
  __device__ explicit Bars(uint32_t sbase) {
    uint32_t b = sbase + Layout<DP, KEYS>::BARS;
    auto next = [&](int n) {
      const uint32_t r = b;
      b += 8 * n;
      return r;
    };
    constexpr int S0 = Layout<DP, KEYS>::S0, S1 = Layout<DP, KEYS>::S1;
    full0 = next(S0), full1 = next(S1), empty0 = next(S0), empty1 = next(S1), fix = next(S0), free = next(S0);
    items = next(RING), ffull = next(1), fempty = next(1), sfull = next(1), pfull = next(1), dpfull = next(2);
    dsfull = next(2), done = next(2), accfull = next(1), drain = next(2);
  }
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

template <int DP, bool KEYS>
__device__ void load_role(const Args& a, const Tiles<KEYS>& tiles, const Shares& sh, uint32_t sbase, uint8_t* smem) {
  using L = Layout<DP, KEYS>;
  const Bars<DP, KEYS> b(sbase);
  const bool lead = (threadIdx.x & 31) == 0;
  const uint32_t qbytes = static_cast<uint32_t>(a.group * a.tokens) * 128u * (DP / 64), kbytes = L::TILE;
  uint32_t n0 = 0, n1 = 0, fn = 0, fixed = 0;  // loads so far
  bool ok = true, open = false;
  Walk w{};
  walk_begin(tiles, sh, w);
  Entry e, next = put_item<Tiles<KEYS>>(sh, w, smem + L::RING_AT, b.items, 0, a.begun, &open);
  for (; ok && next.hi > next.lo; ++fn) {
    e = next;
    const int qh = e.head * a.group;
    // the rings' first, the tile itself as soon as the one before it is done with, then the rings in turns
    const int loads = 1 + 2 * (e.hi - e.lo);
#pragma unroll 1
    for (int i = 0; ok && i <= loads; ++i) {
      if (i == min(loads, 4)) {  // the next tile is looked up while this one's products run, not when its loads are due
        walk_next(tiles, a.seq, w);
        next = put_item<Tiles<KEYS>>(sh, w, smem + L::RING_AT, b.items, fn + 1, a.begun, &open);
      }
      if (i == loads) break;
      const bool tile = i == 1, second = i > 1 && !(i & 1);
      const uint32_t n = tile ? fn : second ? n1 : n0, ring = tile ? 1u : second ? L::S1 : L::S0, st = n % ring;
      const uint32_t full = tile ? b.ffull : (second ? b.full1 : b.full0) + 8 * st;
      const uint32_t empty = tile ? b.fempty : (second ? b.empty1 : b.empty0) + 8 * st;
      if (!(ok = wait_warp(a.watch, empty, (n / ring & 1u) ^ 1u, S_EMPTY))) break;
      if (lead) {
        const bool queries = KEYS != tile;  // or keys
        const int j = e.lo + (i == 0 ? 0 : second ? (i - 2) >> 1 : (i - 1) >> 1), at = tile ? e.tile : j;
        const int row = queries ? e.s.q0 + at * a.tokens : e.s.k0 + at * BLK;
        const uint32_t to = sbase + (tile ? 0u : (second ? L::R1 : L::R0) + st * L::TILE);
        mbar_expect_tx(full, (queries ? qbytes : kbytes) * (tile ? 2u : 1u));
#pragma unroll 1
        for (int m = second ? 1 : 0; m < (tile || second ? 2 : 1); ++m)  // q or k, dout or v
          for (int d = 0; d < DP / 64; ++d)
            tma_load_3d(to + (tile ? m * L::TILE : 0) + d * 16384, queries ? (m ? &a.dout : &a.q) : (m ? &a.v : &a.k), full,
                        d * 64, queries ? qh : e.head, row);
      }
      __syncwarp();
      if (tile)
        ++fixed;
      else if (second)
        ++n1;
      else
        ++n0;
    }
  }
  // What is in flight must land before the block gives up its shared memory, whichever role gave up: this one may have had
  // room for all of its loads, which nobody waits for then.  (After a call that went well all have landed.)
  if (lead) {
#pragma unroll 1
    for (uint32_t j = n0 > L::S0 ? n0 - L::S0 : 0u; j < n0; ++j)
      wait_bar(a.watch, b.full0 + 8 * (j % L::S0), j / L::S0 & 1u, S_DRAIN, false);
#pragma unroll 1
    for (uint32_t j = n1 > L::S1 ? n1 - L::S1 : 0u; j < n1; ++j)
      wait_bar(a.watch, b.full1 + 8 * (j % L::S1), j / L::S1 & 1u, S_DRAIN, false);
    if (fixed) wait_bar(a.watch, b.ffull, (fixed - 1) & 1u, S_DRAIN, false);
  }
  __syncwarp();
}

// KEYS: tensor memory S, dP, dV, dK.  One warp issues S and, from what overwrites it, dV = P^T dO, the other dP and dK.
template <int DP>
__device__ void mma_keys_role(const Args& a, uint32_t sbase, uint8_t* smem, uint32_t tmem, int second) {
  using L = Layout<DP, true>;
  const Bars<DP, true> b(sbase);
  const uint32_t idesc_s = idesc_n(make_idesc(false, BLK), BLK);
  const uint32_t idesc_o = idesc_n(make_idesc(false, BLK), (a.dim + 15) / 16 * 16) | 1u << 16;
  const uint64_t f = smem_desc_sw128(sbase + (second ? L::F1 : 0)), r = smem_desc_sw128(sbase + (second ? L::R1 : L::R0));
  // dV and dK read rows of the other warp's ring
  const uint64_t t = desc_rows(sbase + (second ? L::R0 : L::R1));
  const uint32_t full = second ? b.full1 : b.full0, empty = second ? b.empty1 : b.empty0;
  const uint32_t t_full = second ? b.full0 : b.full1, t_empty = second ? b.empty0 : b.empty1;
  const uint32_t from = tmem + (second ? BLK : 0), acc = tmem + (second ? 3 : 2) * BLK;
  uint32_t n = 0, fn = 0;  // steps and parts so far
  bool ok = true;
  auto await = [&](uint32_t bar, uint32_t parity, uint32_t site) {
    if (ok) ok = wait_warp(a.watch, bar, parity & 1u, site);
  };
  for (Entry e; ok && get_item(a.watch, smem + L::RING_AT, b.items, fn, &e); ++fn) {
    const int steps = e.hi - e.lo;
    auto scores = [&](uint32_t s) {  // S or dP of step s of the launch
      await(full + 8 * (s % L::S0), s / L::S0, S_FULL);
      if (!ok) return;
      tc_fence_after();
      mma_head<DP>(from, f, r + (s % L::S0) * (L::TILE >> 4), idesc_s);
      mma_commit_cg<1>(second ? b.dpfull + 8 * (s & 1u) : b.sfull);
    };
    await(b.ffull, fn, S_FULL);
    scores(n);
#pragma unroll 1
    for (int i = 0; ok && i < steps; ++i, ++n) {
      const uint32_t st = n % L::S0;
      await(t_full + 8 * st, n / L::S0, S_FULL);
      await(second ? b.dsfull + 8 * (n & 1u) : b.pfull, second ? n >> 1 : n, S_TFULL);
      if (!ok) break;
      tc_fence_after();
      const uint64_t rows = t + st * (L::TILE >> 4);
      mma4_ts(acc, from, rows, idesc_o, i > 0);
      mma4_ts(acc, from + 64, rows + 512, idesc_o, 1u);
      mma_commit_cg<1>(t_empty + 8 * st);
      mma_commit_cg<1>(empty + 8 * st);  // this step's S or dP is long done
      if (i + 1 < steps) scores(n + 1);
    }
    if (!ok) break;
    mma_commit_cg<1>(b.fempty);
    mma_commit_cg<1>(b.accfull);
  }
  // also after a failure: every MMA issued must complete before tensor memory is freed
  mma_commit_cg<1>(b.drain + 8 * second);
  if ((threadIdx.x & 31) == 0) wait_bar(a.watch, b.drain + 8 * second, 0u, S_DRAIN, false);
  __syncwarp();
}

// Otherwise: tensor memory S, dP of even steps, dQ, dP of odd steps.  One warp issues S as soon as the one before has been
// read, and dP, a step ahead of what the threads are at; the other dQ.
template <int DP>
__device__ void mma_queries_role(const Args& a, uint32_t sbase, uint8_t* smem, uint32_t tmem, int second) {
  using L = Layout<DP, false>;
  const Bars<DP, false> b(sbase);
  const uint32_t idesc_s = idesc_n(make_idesc(false, BLK), BLK);
  const uint32_t idesc_o = idesc_n(make_idesc(false, BLK), (a.dim + 15) / 16 * 16) | 1u << 16;
  const uint64_t f0 = smem_desc_sw128(sbase), f1 = smem_desc_sw128(sbase + L::F1), r0 = smem_desc_sw128(sbase + L::R0),
                 r1 = smem_desc_sw128(sbase + L::R1), t = desc_rows(sbase + L::R0);
  const uint32_t acc = tmem + 2 * BLK;
  uint32_t n = 0, fn = 0;  // steps and parts so far
  bool ok = true;
  auto await = [&](uint32_t bar, uint32_t parity, uint32_t site) {
    if (ok) ok = wait_warp(a.watch, bar, parity & 1u, site);
  };
  for (Entry e; ok && get_item(a.watch, smem + L::RING_AT, b.items, fn, &e); ++fn) {
    const int steps = e.hi - e.lo;
    if (!second) await(b.ffull, fn, S_FULL);
#pragma unroll 1
    for (int i = 0; ok && i < steps; ++i, ++n) {
      const uint32_t st = n % L::S0, at = st * (L::TILE >> 4), sv = n % L::S1, odd = n & 1u;
      const uint32_t dp = tmem + (odd ? 3 : 1) * BLK;
      if (!second) {
        await(b.full0 + 8 * st, n / L::S0, S_FULL);
        if (n >= 1) await(b.pfull, n - 1, S_TEMPTY);  // S has been read
        if (ok) {
          tc_fence_after();
          mma_head<DP>(tmem, f0, r0 + at, idesc_s);
          mma_commit_cg<1>(b.sfull);
          mma_commit_cg<1>(b.empty0 + 8 * st);
        }
        await(b.full1 + 8 * sv, n / L::S1, S_FULL);
        if (n >= 2) await(b.done + 8 * odd, n / 2 - 1, S_TEMPTY);  // dS over this dP has been used
        if (ok) {
          tc_fence_after();
          mma_head<DP>(dp, f1, r1 + sv * (L::TILE >> 4), idesc_s);
          mma_commit_cg<1>(b.dpfull + 8 * odd);
          mma_commit_cg<1>(b.empty1 + 8 * sv);
        }
      } else {
        await(b.full0 + 8 * st, n / L::S0, S_FULL);
        await(b.dsfull + 8 * odd, n >> 1, S_TFULL);
        if (ok) {
          tc_fence_after();
          mma4_ts(acc, dp, t + at, idesc_o, i > 0);
          mma4_ts(acc, dp + 64, t + at + 512, idesc_o, 1u);
          mma_commit_cg<1>(b.done + 8 * odd);
          mma_commit_cg<1>(b.empty0 + 8 * st);
        }
      }
    }
    if (ok) mma_commit_cg<1>(second ? b.accfull : b.fempty);
  }
  // also after a failure: every MMA issued must complete before tensor memory is freed
  mma_commit_cg<1>(b.drain + 8 * second);
  if ((threadIdx.x & 31) == 0) wait_bar(a.watch, b.drain + 8 * second, 0u, S_DRAIN, false);
  __syncwarp();
}

// Statistics of a step's query rows (KEYS), and rows of the rings that belong to
// no query or key of the sequence cleared, since they are operands of the products
// with P and dS.
template <int DP, bool KEYS>
__device__ void aux_role(const Args& a, uint32_t sbase, uint8_t* smem) {
  using L = Layout<DP, KEYS>;
  const Bars<DP, KEYS> b(sbase);
  const int lane = threadIdx.x & 31;
  const int used = a.group * a.tokens;
  uint32_t n = 0, fn = 0;
  for (Entry e; get_item(a.watch, smem + L::RING_AT, b.items, fn, &e); ++fn) {
#pragma unroll 1
    for (int j = e.lo; j < e.hi; ++j, ++n) {
      const uint32_t st = n % L::S0, ph = n / L::S0 & 1u;
      const int left = KEYS ? min(a.tokens, e.s.nq - j * a.tokens) * a.group : e.s.nk - j * BLK;  // rows in use
      if constexpr (KEYS) {
        if (!wait_warp(a.watch, b.free + 8 * st, ph ^ 1u, S_EMPTY)) return;
        float* stats = reinterpret_cast<float*>(smem + L::STATS) + st * 256;
        float2 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = lane + 32 * i, tok = r / a.group;
          v[i] = make_float2(-INFINITY, 0.0f);  // a weight of 0
          if (r < left)
            v[i] = a.stats[(static_cast<int64_t>(e.s.q0) + j * a.tokens + tok) * a.heads + e.head * a.group +
                           (r - tok * a.group)];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) stats[lane + 32 * i] = v[i].x, stats[BLK + lane + 32 * i] = v[i].y;
      }
      if (!wait_warp(a.watch, b.full0 + 8 * st, ph, S_FULL)) return;
      if (KEYS && !wait_warp(a.watch, b.full1 + 8 * st, ph, S_FULL)) return;
      if (left < (KEYS ? used : BLK)) {
#pragma unroll 1
        for (int r = lane; r < BLK; r += 32) {
          if (r < left) continue;
#pragma unroll 1
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
__device__ void compute_role(const Args& a, uint32_t sbase, uint8_t* smem, uint32_t tmem) {
  using L = Layout<DP, KEYS>;
  const Bars<DP, KEYS> b(sbase);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = warp & 3, half = (warp - 4) >> 2;
  const int row = quad * 32 + lane;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16), mine = lanes + half * 64;
  const int dt = row / a.group, head_in = row - dt * a.group;
  const int chunks = (a.dim + 31) / 32;
  const float2 c2 = make_float2(a.c, a.c);
  uint32_t n = 0, fn = 0;
  bool ok = true;
  for (Entry e; ok && get_item(a.watch, smem + L::RING_AT, b.items, fn, &e); ++fn) {
    // KEYS: this row's key, and the first token that sees it; otherwise the row's query and the keys that it sees
    const int tok = e.tile * a.tokens + dt;
    const bool valid = KEYS ? e.tile * BLK + row < e.s.nk : dt < a.tokens && tok < e.s.nq;
    const int seen = KEYS ? (a.causal ? e.tile * BLK + row - e.s.nk + e.s.nq : 0)
                          : (valid ? keys_seen(e.s, tok, a.causal) : INT_MAX);  // a row that is none may come to anything
    float2 nl = make_float2(0.0f, 0.0f), nd = nl;
    if (!KEYS && valid) {
      const float2 v = a.stats[(static_cast<int64_t>(e.s.q0) + tok) * a.heads + e.head * a.group + head_in];
      nl = make_float2(v.x, v.x), nd = make_float2(v.y, v.y);
    }
#pragma unroll 1
    for (int j = e.lo; j < e.hi; ++j, ++n) {
      const uint32_t st = n % L::S0, ph = n / L::S0 & 1u;
      // columns [from, to) of the group's 64 that the row sees
      const int from = KEYS ? min(a.tokens, max(0, seen - j * a.tokens)) * a.group - half * 64 : 0;
      const int to = (KEYS ? min(a.tokens, e.s.nq - j * a.tokens) * a.group : seen - j * BLK) - half * 64;
      const bool all = __all_sync(0xffffffffu, from <= 0 && to >= 64);
      const float* stats = reinterpret_cast<const float*>(smem + L::STATS) + st * 256 + half * 64;
      float2 pr[32];
      const uint32_t odd = n & 1u, dp = KEYS || !odd ? BLK : 3 * BLK;
      if (!(ok = wait_warp(a.watch, b.sfull, odd, S_TFULL))) break;
      if (KEYS && !(ok = wait_warp(a.watch, b.fix + 8 * st, ph, S_FULL))) break;
      {
        tc_fence_after();
        uint32_t x[64];
        tmem_ld64_sync(mine, x);
        if (!KEYS) {  // S is read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(b.pfull);
        }
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
          // p, and ds below, are operands of products with bf16 tensors, and take their type: the gradients are off by 0.0025
          // of their size, for 0.0018 with both in fp32
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
      if (!(ok = wait_warp(a.watch, b.dpfull + 8 * odd, n >> 1 & 1u, S_TFULL))) break;
      if (!KEYS && !(ok = wait_warp(a.watch, b.fix + 8 * st, ph, S_FULL))) break;
      {
        tc_fence_after();
        uint32_t x[64], h[32];
        tmem_ld64_sync(mine + dp, x);
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
        tmem_st32(mine + dp, h);
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(b.dsfull + 8 * odd);
        mbar_arrive(b.free + 8 * st);
      }
    }
    // ---- the end of the part: one group writes dV, the other dK; or each its columns of dQ
    if (!ok || !(ok = wait_warp(a.watch, b.accfull, fn & 1u, S_TFULL))) break;
    tc_fence_after();
    const bool second = KEYS && half == 1, whole = e.shares == 1;
    const float scale = KEYS && !second ? 1.0f : a.scale;
    bf16* out = second ? a.out1 : a.out0;
    const int64_t ld = second ? a.ld1 : a.ld0, hs = second ? a.h1 : a.h0;
    const int64_t out_row = KEYS ? static_cast<int64_t>(e.s.k0) + e.tile * BLK + row : static_cast<int64_t>(e.s.q0) + tok;
    const int head = KEYS ? e.head : e.head * a.group + head_in;
    float* part = a.part + static_cast<int64_t>(e.slot * (KEYS ? 2 : 1) + second) * BLK * a.dim;
    uint8_t* stage = smem + L::STAGE + (warp - 4) * 2048;
    const void* to_row = valid ? out + out_row * ld + head * hs : nullptr;
#pragma unroll 1
    for (int c = KEYS ? 0 : half; c < chunks; c += KEYS ? 1 : 2) {  // 32 columns
      uint32_t o[32];
      tmem_ld32_sync(lanes + (second ? 3 : 2) * BLK + c * 32, o);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(o[8 * g + i]) * scale;
        if (!whole) {
          if (valid) store_part(part, BLK, row, v, c * 32 + g * 8, a.dim);
        } else if (!L::TIGHT) {
          stage_row(stage, g, v);
        } else if (valid && c * 32 + g * 8 < a.dim) {
          *reinterpret_cast<uint4*>(out + out_row * ld + head * hs + c * 32 + g * 8) =
              make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
        }
      }
      if (whole && !L::TIGHT) store_staged(stage, to_row, c * 32, a.dim - c * 32);
    }
    tc_fence_before();
  }
}

// Grid: one block per SM at most, each an equal share of the steps.
template <int DP, bool KEYS>
__global__ void __launch_bounds__(THREADS, 1) bwd_kernel(const __grid_constant__ Args a) {
  using L = Layout<DP, KEYS>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  grid_dep_launch();
  const int warp = threadIdx.x >> 5;
  PlanScratch* plan = reinterpret_cast<PlanScratch*>(smem + L::PLAN);
  if (threadIdx.x == 0) {
    const Bars<DP, KEYS> b(sbase);
    auto init = [&](uint32_t bar, int n, uint32_t count) {
      for (int i = 0; i < n; ++i) mbar_init(bar + 8 * i, count);
    };
    init(b.full0, L::S0 + L::S1, 1);  // and full1
    init(b.empty0, L::S0, 2);     // both issuing warps
    init(b.empty1, L::S1, KEYS ? 2 : 1);
    init(b.fix, L::S0, 1);
    init(b.free, L::S0, 8);
    init(b.items, RING, 1);
    init(b.ffull, 1, 1);
    init(b.fempty, 1, KEYS ? 2 : 1);
    init(b.sfull, 1, 1);
    init(b.pfull, 1, 8);
    init(b.dpfull, 2, 1);
    init(b.dsfull, 2, 8);
    init(b.done, 2, 1);
    init(b.accfull, 1, KEYS ? 2 : 1);
    init(b.drain, 2, 1);
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
    for (int i = threadIdx.x; i < unused * 8 * (DP / 64) * 2 * L::S0; i += THREADS) {
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
  Shares& sh = *reinterpret_cast<Shares*>(smem + L::SHARES);
  plan_shares<THREADS>(tiles, a.seq, plan, &sh, a.watch.err);
  if (L::TIGHT) {  // loads follow where the scratch was
    fence_proxy_async_smem();
    __syncthreads();
  }
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;" : "+r"(sbase)::"memory");  // nothing of a role is computed ahead of it
    if (warp == 0) load_role<DP, KEYS>(a, tiles, sh, sbase, smem);
    if (warp == 1 || warp == 2) {
      if constexpr (KEYS)
        mma_keys_role<DP>(a, sbase, smem, tmem, warp - 1);
      else
        mma_queries_role<DP>(a, sbase, smem, tmem, warp - 1);
    }
    if (warp == 3) aux_role<DP, KEYS>(a, sbase, smem);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;" : "+r"(sbase)::"memory");  // nothing of a role is computed ahead of it
    compute_role<DP, KEYS>(a, sbase, smem, tmem);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<1>(tmem, 512);
  }
}

// Adds the parts of the tile that share blockIdx.x began and did not end, in the order of the shares; block y takes 16
// rows of a matrix (dq, or dv and then dk), eight columns a thread.
constexpr int JOIN_THREADS = 256, JOIN_ROWS = 16;
__global__ void __launch_bounds__(JOIN_THREADS) join_bwd_kernel(const __grid_constant__ Args a, int keys) {
  grid_dep_launch();
  grid_dep_wait();
  const Entry e = a.begun[blockIdx.x];
  if (*a.watch.err != 0u || !e.begins || e.hi <= e.lo) return;  // after a failure the entries may be an earlier call's
  const int y = blockIdx.y, second = y >= BLK / JOIN_ROWS, r = (y * JOIN_ROWS & (BLK - 1)) + (threadIdx.x & 15);
  const int c = threadIdx.x >> 4, matrices = keys ? 2 : 1;
  int64_t out_row;
  int head = e.head;
  if (keys) {
    if (e.tile * BLK + r >= e.s.nk) return;
    out_row = static_cast<int64_t>(e.s.k0) + e.tile * BLK + r;
  } else {
    const int dt = r / a.group, tok = e.tile * a.tokens + dt;
    if (dt >= a.tokens || tok >= e.s.nq) return;
    out_row = static_cast<int64_t>(e.s.q0) + tok;
    head = e.head * a.group + r - dt * a.group;
  }
  if (c * 8 >= a.dim) return;
  const int64_t slot = static_cast<int64_t>(matrices) * BLK * a.dim;
  const float* src = a.part + static_cast<int64_t>(second) * BLK * a.dim + (static_cast<int64_t>(2 * c) * BLK + r) * 4;
  float v[8] = {};
  some_parts(0, e.shares, [&](auto count, int s) {
    constexpr int U = decltype(count)::value;
    float4 lo[U], hi[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float* p = src + tile_slot(e.from, min(s + u, e.shares - 1)) * slot;
      lo[u] = *reinterpret_cast<const float4*>(p);
      hi[u] = *reinterpret_cast<const float4*>(p + BLK * 4);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s + u >= e.shares) break;
      v[0] += lo[u].x, v[1] += lo[u].y, v[2] += lo[u].z, v[3] += lo[u].w;
      v[4] += hi[u].x, v[5] += hi[u].y, v[6] += hi[u].z, v[7] += hi[u].w;
    }
  });
  bf16* out = second ? a.out1 : a.out0;
  *reinterpret_cast<uint4*>(out + out_row * (second ? a.ld1 : a.ld0) + head * (second ? a.h1 : a.h0) + c * 8) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// -lse log2(e) and -delta of each row and head, sixteen lanes a head.  Bound by
// memory: out and dout are read once, 135 MB in 25 us of a cold start (43 when
// blocks went round in a grid of eight an SM and lse came last).
constexpr int STAT_THREADS = 256, STAT_ROWS = 4;  // rows of a group of lanes in flight together
__global__ void __launch_bounds__(STAT_THREADS) stats_kernel(int64_t rows, int heads, int dim, Heads out, Heads dout,
                                                            const float* lse, float2* stats) {
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 15;
  constexpr int STEP = STAT_THREADS / 16;
  const int64_t each = static_cast<int64_t>(gridDim.x) * (STEP * STAT_ROWS);
  const int64_t rounds = (rows + each - 1) / each;  // the same for every thread
  for (int64_t k = 0; k < rounds; ++k) {
    const int64_t first = (k * gridDim.x + blockIdx.x) * (STEP * STAT_ROWS) + (threadIdx.x >> 4);
    uint4 x[STAT_ROWS], y[STAT_ROWS];
    float l[STAT_ROWS];
#pragma unroll
    for (int r = 0; r < STAT_ROWS; ++r) {
      const int64_t i = first + r * STEP;
      const int64_t row = i >> 32 ? i / heads : static_cast<uint32_t>(i) / static_cast<uint32_t>(heads), h = i - row * heads;
      x[r] = y[r] = make_uint4(0, 0, 0, 0);
      l[r] = 0.0f;
      if (i < rows && lane * 8 < dim) {
        x[r] = *reinterpret_cast<const uint4*>(static_cast<const bf16*>(out.p) + row * out.ld + h * out.hs + lane * 8);
        y[r] = *reinterpret_cast<const uint4*>(static_cast<const bf16*>(dout.p) + row * dout.ld + h * dout.hs + lane * 8);
        if (lane == 0) l[r] = lse[i];
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
      const int64_t i = first + r * STEP;
      if (lane == 0 && i < rows) stats[i] = make_float2(l[r] == -INFINITY ? 0.0f : -l[r] * kLog2e, -s);
    }
  }
}

int64_t stats_bytes(int64_t n, int64_t heads) { return (n * heads * 8 + 255) / 256 * 256; }

template <int DP, bool KEYS>
cudaError_t launch_as(const Args& a, int grid, cudaStream_t s) {
  return launch_pdl(bwd_kernel<DP, KEYS>, dim3(static_cast<unsigned>(grid)), dim3(THREADS), Layout<DP, KEYS>::SMEM, s, a);
}
// steps: the most that a tile can have; tiles of one are never divided
template <bool KEYS>
cudaError_t launch_both(const Args& a, int grid, int64_t steps, cudaStream_t s) {
  const cudaError_t e = a.dim <= 64 ? launch_as<64, KEYS>(a, grid, s) : launch_as<128, KEYS>(a, grid, s);
  if (e != cudaSuccess || steps <= 1) return e;
  return launch_pdl(join_bwd_kernel, dim3(static_cast<unsigned>(grid), (KEYS ? 2 : 1) * BLK / JOIN_ROWS), dim3(JOIN_THREADS),
                    0, s, a, KEYS ? 1 : 0);
}
template <int DP, bool KEYS>
cudaError_t configure_as() {
  return cudaFuncSetAttribute(bwd_kernel<DP, KEYS>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<DP, KEYS>::SMEM);
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
  return stats_bytes(n, heads) + BEGUN_BYTES + 2ll * MAX_SHARES * 2 * BLK * dim * 4;
}

cudaError_t launch_attention_bwd(const Machine& mc, const AttnArgs& x, const Watch& w, void* ws, cudaStream_t s) {
  const int64_t n = x.seq.n, nk = x.seq.nk;
  Args a;
  std::memset(static_cast<void*>(&a), 0, sizeof(a));
  a.seq = x.seq;
  a.heads = static_cast<int>(x.heads), a.kv_heads = static_cast<int>(x.kv_heads);
  a.group = a.heads / a.kv_heads, a.tokens = BLK / a.group;
  a.dim = static_cast<int>(x.dim), a.causal = x.causal, a.scale = x.scale, a.c = x.scale * kLog2e;
  a.stats = static_cast<const float2*>(ws);
  a.begun = reinterpret_cast<Entry*>(static_cast<uint8_t*>(ws) + stats_bytes(n, x.heads));
  a.part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(a.begun) + BEGUN_BYTES);
  a.watch = w;
  // without keys (or queries) the loads go to the others, which no row sees
  const int64_t rq = n ? n : nk, hq = n ? x.heads : x.kv_heads, rk = nk ? nk : n, hk = nk ? x.kv_heads : x.heads;
  if (!encode_heads(&a.q, n ? x.q : x.k, rq, hq, x.dim, a.group, a.tokens) ||
      !encode_heads(&a.dout, n ? x.dout : x.k, rq, hq, x.dim, a.group, a.tokens) ||
      !encode_heads(&a.k, nk ? x.k : x.q, rk, hk, x.dim, 1, BLK) ||
      !encode_heads(&a.v, nk ? x.v : x.q, rk, hk, x.dim, 1, BLK))
    return cudaErrorInvalidValue;
  const int64_t sms = std::min(mc.sms, MAX_SHARES);
  auto grid = [&](int64_t tiles, int64_t steps) {  // no more blocks than the most steps that these sizes can have
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(sms, std::min<int64_t>(tiles * x.kv_heads, MAX_SHARES) * steps)));
  };
  const int64_t q_tiles = n / a.tokens + std::min(x.seq.batch, n), k_tiles = nk / BLK + std::min(x.seq.batch, nk);
  if (n > 0) {
    const int64_t rows = n * x.heads, per = STAT_THREADS / 16 * STAT_ROWS;
    cudaError_t e = launch_pdl(stats_kernel, dim3(static_cast<unsigned>(std::min<int64_t>((rows + per - 1) / per, 1 << 20))),
                               dim3(STAT_THREADS), 0, s, rows, a.heads, a.dim, x.out, x.dout,
                               static_cast<const float*>(x.lse), static_cast<float2*>(ws));
    if (e != cudaSuccess) return e;
    a.out0 = static_cast<bf16*>(const_cast<void*>(x.dq.p)), a.ld0 = x.dq.ld, a.h0 = x.dq.hs;
    e = launch_both<false>(a, grid(q_tiles, nk / BLK + 1), (nk + BLK - 1) / BLK, s);
    if (e != cudaSuccess) return e;
  }
  if (nk == 0) return cudaSuccess;
  a.out0 = static_cast<bf16*>(const_cast<void*>(x.dv.p)), a.ld0 = x.dv.ld, a.h0 = x.dv.hs;
  a.out1 = static_cast<bf16*>(const_cast<void*>(x.dk.p)), a.ld1 = x.dk.ld, a.h1 = x.dk.hs;
  return launch_both<true>(a, grid(k_tiles, n / a.tokens + 1), (n + a.tokens - 1) / a.tokens, s);
}

}  // namespace tpo
