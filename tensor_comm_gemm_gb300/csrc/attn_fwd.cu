// Attention over packed sequences and caches (sm_103a): out = softmax(scale q
// k^T) v, in one pass over the keys with a running maximum and sum.
//
// Rows: the query heads that share a key head are rows of one tile, token by
// token, so that they read its keys once: a half of 128 rows holds
// floor(128 / group) tokens.  A tile has two halves with scores S and an output
// O of 128 columns each in tensor memory (all 512).  While one half's softmax
// runs, the tensor core works on the other:  S = Q K^T from shared memory, then
// P (bf16, over S) V into O.  A sequence with at most one half of queries has
// its steps taken by turns instead: both accumulators serve the same rows, and
// are joined at the end.
//
// A thread holds one row: 128 scores of a step in registers, its maximum and
// sum.  The maximum that is subtracted follows the true one only when that has
// grown by 2^8 (P then stays below 2^8, whose bf16 is as exact), so O is seldom
// rescaled.  Keys that a row does not see are taken out by selection, never by
// arithmetic with their values; the rows of V that no query of the tile sees are
// cleared in shared memory before the product, and a value that is not finite
// where only some rows see it is added to those rows alone at the end.
//
// Roles: warp 0 loads (TMA), warps 1 and 2 issue the two halves' MMAs, warp 3
// clears V, warps 4-7 and 8-11 are the two halves' softmax, warps 12-15 divide by
// the sums and store, beside the next tile's scores and weights.
//
// The tensor core takes about two instructions ahead of time, a wait costs the
// issuing warp 130 cycles even when there is nothing to wait for and a commit 60.
// One warp with all of them needed 1760 cycles for a half's products, which take
// 1033.  With two, one waits while the other issues; they issue the end of a step
// in turns, since otherwise both halves come to run in step, softmax against
// softmax (3950 cycles a step, now 2850, of which the tensor core works 2080).
//
// Measured (times of back-to-back calls with a flushed L2): 8192 causal tokens of
// 32 heads of 128 over 8 take 398 to 415 us, 1.33 to 1.38 PFLOP/s, 67 to 70 % of the
// measured matrix rate; bound by that step: a half's scores, softmax (about 1450 cycles, 512 of
// them exponentials at 32 a cycle) and P V follow one another, and two halves do
// not quite fill each other's gaps.  12 packed sequences of 8 heads over 1:
// 53 us, bound by filling the pipeline at the start and at each tile (about 6000
// cycles).  One token of 64 sequences over 8 heads of keys: 181 us, 89 % of the
// measured bandwidth.  One token over 32768 keys: 22 to 24 us, bound by latency (a
// cold load, two steps and the join of 130 parts).  A step of heads of 64 takes as
// long as one of 128, 2800 cycles (8192 tokens both ways, 16 heads: 303 us), though
// its products take half: so a token of 64 sequences over 8 heads of 64 takes 135 us,
// 4.0 TB/s.

#include <algorithm>
#include <climits>
#include <cstring>

#include <cuda_bf16.h>

#include "attn_dev.h"
#include "pdl.h"

namespace tpo {

namespace {

using bf16 = __nv_bfloat16;
constexpr int THREADS = 512;
constexpr float GROWTH = 8.0f;           // of the maximum, in powers of two, before O is rescaled
constexpr int BAD_SETS = 8, BAD_STEPS = 3;  // steps of a tile that only some of its rows see whole

struct Args {
  CUtensorMap q, k, v;
  Sequences seq;
  int heads, kv_heads, group, tokens;  // tokens: of a half
  int dim, causal;
  float c;                             // scale log2(e)
  const bf16* values;
  int64_t ldv, hv;
  bf16* out;
  int64_t ldo, ho;
  float* lse;
  Entry* begun;                        // [MAX_SHARES]: the tile that a share begins and does not end
  float* part;                         // its parts: two slots a share, [dim / 4][rows][4], then maxima and sums
  int part_rows;
  Watch watch;
};

struct Tiles {
  static constexpr int COST = FWD_TILE_COST;
  int kv_heads, tokens, causal;
  __device__ __forceinline__ int tiles(const Seq& s) const {
    return (s.nq + 2 * tokens - 1) / (2 * tokens);
  }
  __device__ __forceinline__ void range(const Seq& s, int tile, int* lo, int* hi) const {
    const int limit = keys_seen(s, min(s.nq, (tile + 1) * 2 * tokens) - 1, causal);
    *lo = 0;
    *hi = limit <= BLK ? 1 : (limit + BLK - 1) / BLK;
  }
};

template <int DP>
struct Layout {
  static constexpr int TILE = BLK * DP * 2;          // 128 rows of a head
  static constexpr int STAGES = DP == 128 ? 2 : 4;   // of K, and of V
  static constexpr int K0 = 2 * TILE, V0 = K0 + STAGES * TILE, BARS = V0 + STAGES * TILE;
  static constexpr int N_BARS = 5 * STAGES + RING + 20;
  static constexpr int SLOT = BARS + 8 * N_BARS;     // the address of tensor memory, then the issuing warps' turns
  static constexpr int RING_AT = (SLOT + 16 + 15) / 16 * 16;
  static constexpr int BAD = RING_AT + RING * static_cast<int>(sizeof(Entry));  // [BAD_SETS][BAD_STEPS][4] keys, a bit each
  static constexpr int ROWS = BAD + BAD_SETS * BAD_STEPS * 16;  // [2][2][128] floats: maxima and sums
  static constexpr int STAGE = ROWS + 2048;  // the storing warps' boxes
  static constexpr int PLAN = STAGE + 4 * 2048;
  static constexpr int SHARES = PLAN + static_cast<int>(sizeof(PlanScratch));
  static constexpr int SMEM = SHARES + static_cast<int>(sizeof(Shares)) + 1024;
  static_assert(SMEM <= 232448 && RING_AT % 16 == 0, "shared memory of one block");
};

template <int DP>
struct Bars {
  uint32_t kfull, kempty, vfull, vempty, vfix, items, qfull, qempty, sfull, pfull, ofull, ofree, lfull, lfree, drain;
  __device__ explicit Bars(uint32_t sbase) {
    uint32_t b = sbase + Layout<DP>::BARS;
    auto next = [&](int n) {
      const uint32_t r = b;
      b += 8 * n;
      return r;
    };
    constexpr int S = Layout<DP>::STAGES;
    kfull = next(S), kempty = next(S), vfull = next(S), vempty = next(S), vfix = next(S), items = next(RING);
    qfull = next(2), qempty = next(2), sfull = next(2), pfull = next(4), ofull = next(2), ofree = next(2);
    lfull = next(2), lfree = next(2), drain = next(2);
  }
};

// What the roles derive from an entry.
struct Item : Entry {
  int tok;    // first token of the tile, in the sequence
  int halves;
  int some;   // keys from here on are not seen by all queries
};
__device__ __forceinline__ void derive(const Args& a, Item& i) {
  i.tok = i.tile * 2 * a.tokens;
  i.halves = i.s.nq - i.tok <= a.tokens ? 1 : 2;
  i.some = keys_seen(i.s, i.tok, a.causal);
}
template <int DP>
__device__ __forceinline__ bool next_item(const Args& a, const Bars<DP>& b, const uint8_t* smem, uint32_t n, Item& i) {
  if (!get_item(a.watch, smem + Layout<DP>::RING_AT, b.items, n, &i)) return false;
  derive(a, i);
  return true;
}
__device__ __forceinline__ bool needs_fix(const Item& i, int j) { return (j + 1) * BLK > i.some; }

template <int DP>
__device__ void load_role(const Args& a, const Tiles& tiles, const Shares& sh, uint32_t sbase, uint8_t* smem) {
  using L = Layout<DP>;
  const Bars<DP> b(sbase);
  const bool lead = (threadIdx.x & 31) == 0;
  uint32_t kn = 0, vn = 0, q0 = 0, q1 = 0;  // loads so far; of Q by half
  bool ok = true, open = false;
  Walk w{};
  walk_begin(tiles, sh, w);
  Item it, next;
  static_cast<Entry&>(next) = put_item<Tiles>(sh, w, smem + L::RING_AT, b.items, 0, a.begun, &open);
  while (ok && next.hi > next.lo) {
    it = next;
    derive(a, it);
    // K one step ahead of V, as the products take them: K, Q, Q, K, V, K, V, .. V.  Each half (or turn) has its own Q,
    // which the next tile's replaces as soon as the half has made its last scores.
    const int loads = 2 + 2 * (it.hi - it.lo);
#pragma unroll 1
    for (int i = 0; ok && i <= loads; ++i) {
      if (i == min(loads, 5)) {  // the next tile is looked up while this one's products run, not when its loads are due
        walk_next(tiles, a.seq, w);
        static_cast<Entry&>(next) = put_item<Tiles>(sh, w, smem + L::RING_AT, b.items, q1, a.begun, &open);
      }
      if (i == loads) break;
      const bool q = i == 1 || i == 2, v = !q && i > 0 && (i == loads - 1 || !(i & 1));
      const uint32_t n = q ? (i == 1 ? q0 : q1) : v ? vn : kn, ring = q ? 1u : static_cast<uint32_t>(L::STAGES), st = n % ring;
      const uint32_t full = q ? b.qfull + 8 * (i - 1) : (v ? b.vfull : b.kfull) + 8 * st;
      const uint32_t empty = q ? b.qempty + 8 * (i - 1) : (v ? b.vempty : b.kempty) + 8 * st;
      if (!(ok = wait_warp(a.watch, empty, (n / ring & 1u) ^ 1u, S_EMPTY))) break;
      if (lead) {
        const CUtensorMap* map = q ? &a.q : v ? &a.v : &a.k;
        const uint32_t to = sbase + (q ? (i - 1) * L::TILE : (v ? L::V0 : L::K0) + st * L::TILE);
        const int j = it.lo + (i == 0 ? 0 : v ? (i - 3) >> 1 : (i - 1) >> 1);
        const int row = q ? it.s.q0 + it.tok + (it.halves == 2 ? i - 1 : 0) * a.tokens : it.s.k0 + j * BLK;
        mbar_expect_tx(full, q ? static_cast<uint32_t>(a.group * a.tokens) * 128u * (DP / 64) : L::TILE);
        for (int d = 0; d < DP / 64; ++d)
          tma_load_3d(to + d * 16384, map, full, d * 64, q ? it.head * a.group : it.head, row);
      }
      __syncwarp();
      if (i == 1)
        ++q0;
      else if (i == 2)
        ++q1;
      else if (v)
        ++vn;
      else
        ++kn;
    }
  }
  // What is in flight must land before the block gives up its shared memory, whichever role gave up: this one may have had
  // room for all of its loads, which nobody waits for then.  (After a call that went well all have landed.)
  if (lead) {
#pragma unroll 1
    for (uint32_t j = kn > L::STAGES ? kn - L::STAGES : 0u; j < kn; ++j)
      wait_bar(a.watch, b.kfull + 8 * (j % L::STAGES), j / L::STAGES & 1u, S_DRAIN, false);
#pragma unroll 1
    for (uint32_t j = vn > L::STAGES ? vn - L::STAGES : 0u; j < vn; ++j)
      wait_bar(a.watch, b.vfull + 8 * (j % L::STAGES), j / L::STAGES & 1u, S_DRAIN, false);
    if (q0) wait_bar(a.watch, b.qfull, (q0 - 1) & 1u, S_DRAIN, false);
    if (q1) wait_bar(a.watch, b.qfull + 8, (q1 - 1) & 1u, S_DRAIN, false);
  }
  __syncwarp();
}

// The products of one half.  Where a tile has one half only, the warps (and accumulators) take its steps by turns, and
// pass over the other's: both release a stage.
template <int DP>
__device__ void mma_role(const Args& a, uint32_t sbase, uint8_t* smem, uint32_t tmem, int half) {
  using L = Layout<DP>;
  const Bars<DP> b(sbase);
  const bool lead = (threadIdx.x & 31) == 0;
  const uint32_t idesc_s = idesc_n(make_idesc(false, BLK), BLK);
  const uint32_t idesc_o = idesc_n(make_idesc(false, BLK), (a.dim + 15) / 16 * 16) | 1u << 16;
  const uint64_t dk = smem_desc_sw128(sbase + L::K0), dv = desc_rows(sbase + L::V0);
  const uint32_t s = tmem + half * BLK, o = tmem + 2 * BLK + half * BLK;
  uint32_t kn = 0, vn = 0, qn = 0, pn = 0, on = 0, turn = 0;
  uint32_t fixed = 0;  // parity of each stage's next clearing
  volatile uint32_t* turns = reinterpret_cast<volatile uint32_t*>(smem + L::SLOT + 4);  // taken by each warp
  bool ok = true;
  auto await = [&](uint32_t bar, uint32_t parity) {
    if (ok) ok = wait_warp(a.watch, bar, parity & 1u, S_FULL);
  };
  for (Item it; ok && next_item(a, b, smem, qn, it); ++qn) {
    const int steps = it.hi - it.lo;
    int two = it.halves - 1;
    const uint64_t dq = smem_desc_sw128(sbase + half * L::TILE);
    await(b.qfull + 8 * half, qn);
    // The next scores: of step i, if it is this warp's.  With one half the other turn's are only released.
    auto scores = [&](int i) {
      const uint32_t st = kn % L::STAGES;
      const bool mine = two || (i & 1) == half;
      await(b.kfull + 8 * st, kn / L::STAGES);
      if (ok && mine) {
        tc_fence_after();
        mma_head<DP>(s, dq, dk + st * (L::TILE >> 4), idesc_s);
        mma_commit_cg<1>(b.sfull + 8 * half);
      }
    };
    auto free_k = [&](int i) {
      const uint32_t st = kn % L::STAGES;
      if (ok && (two || (i & 1) == half))
        mma_commit_cg<1>(b.kempty + 8 * st);
      else if (lead)
        mbar_arrive(b.kempty + 8 * st);
      ++kn;
    };
    int k = 0;  // steps whose scores are made
#pragma unroll 1
    while (k < steps && k <= (two ? 0 : half)) {
      anew(two);
      scores(k);
      free_k(k);
      if (++k == steps && ok) mma_commit_cg<1>(b.qempty + 8 * half);
    }
    // the accumulator is free once the last part that used it has been stored
    if (two || half < steps) {
      if (on > 0) await(b.ofree + 8 * half, on - 1);
      ++on;
    }
#pragma unroll 1
    for (int i = 0; ok && i < steps; ++i) {
      anew(two);
      const uint32_t st = vn % L::STAGES;
      const bool mine = two || (i & 1) == half;
      await(b.vfull + 8 * st, vn / L::STAGES);
      if (needs_fix(it, it.lo + i)) {
        if (mine) await(b.vfix + 8 * st, fixed >> st);
        fixed ^= 1u << st;
      }
      if (mine) {
        const uint64_t vd = dv + st * (L::TILE >> 4);
        // with two halves the next keys are long there: no wait between this product and their scores
        if (two && k < steps) await(b.kfull + 8 * (kn % L::STAGES), kn / L::STAGES);
        await(b.pfull + 16 * half, pn);
        if (ok) {
          tc_fence_after();
          mma4_ts(o, s, vd, idesc_o, i > (two ? 0 : half) ? 1u : 0u);
        }
        await(b.pfull + 16 * half + 8, pn++);
        if (two) {  // half 0's nth turn comes after half 1's one before, half 1's nth after half 0's nth
          const uint32_t due = turn + half;
          uint32_t tries = 0;
          unsigned long long t0 = 0;
#pragma unroll 1
          while (ok && !__all_sync(0xffffffffu, static_cast<int32_t>(turns[1 - half] - due) >= 0)) {
            if (++tries == 256u) t0 = gtime();
            if (tries > 256u && !(tries & 255u)) ok = !waited_long(t0, a.watch.limit_ns, a.watch.err, S_EMPTY);
          }
        }
        if (ok) {
          tc_fence_after();
          mma4_ts(o, s + 64, vd + 512, idesc_o, 1u);
          if (two && k < steps) {
            mma_head<DP>(s, dq, dk + (kn % L::STAGES) * (L::TILE >> 4), idesc_s);
            mma_commit_cg<1>(b.sfull + 8 * half);
          }
        }
        if (two) {
          ++turn;
          if (lead) turns[half] = turn;
          __syncwarp();
        }
        if (ok) mma_commit_cg<1>(b.vempty + 8 * st);
        if (ok && i + (two ? 1 : 2) >= steps) mma_commit_cg<1>(b.ofull + 8 * half);
      } else if (lead) {
        mbar_arrive(b.vempty + 8 * st);
      }
      ++vn;
      if (k < steps) {
        if (!two) scores(k);
        free_k(k);
        if (++k == steps && ok) mma_commit_cg<1>(b.qempty + 8 * half);
      }
    }
  }
  // also after a failure: every MMA issued must complete before tensor memory is freed
  mma_commit_cg<1>(b.drain + 8 * half);
  if (lead) wait_bar(a.watch, b.drain + 8 * half, 0u, S_DRAIN, false);
  __syncwarp();
}

// Clears the rows of V behind the last key, and takes values that are not finite
// out of rows that only some queries see, noting their keys.
template <int DP>
__device__ void fix_role(const Args& a, uint32_t sbase, uint8_t* smem) {
  using L = Layout<DP>;
  const Bars<DP> b(sbase);
  const int lane = threadIdx.x & 31;
  uint32_t vn = 0, item = 0;
  for (Item it; next_item(a, b, smem, item, it); ++item) {
    uint32_t* bad = reinterpret_cast<uint32_t*>(smem + L::BAD) + item % BAD_SETS * BAD_STEPS * 4;
    if (lane < 4 * BAD_STEPS) bad[lane] = 0;
    __syncwarp();
#pragma unroll 1
    for (int j = it.lo; j < it.hi; ++j, ++vn) {
      const uint32_t st = vn % L::STAGES;
      if (!wait_warp(a.watch, b.vfull + 8 * st, vn / L::STAGES & 1u, S_FULL)) return;
      if (needs_fix(it, j)) {
        uint8_t* v = smem + L::V0 + st * L::TILE;
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {
          const int r = 32 * g + lane, key = j * BLK + r;
          uint32_t top = 0;  // the row's largest magnitudes, as a pair of bf16
#pragma unroll 1
          for (int d = 0; d < DP / 64; ++d)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint4* x = reinterpret_cast<uint4*>(v + d * 16384 + r * 128 + ((i ^ (r & 7)) << 4));
              if (key >= it.s.nk) {
                *x = make_uint4(0, 0, 0, 0);
              } else if (key >= it.some) {
                const uint32_t y[4] = {x->x, x->y, x->z, x->w};
#pragma unroll
                for (int k = 0; k < 4; ++k) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(y[k] & 0x7fff7fffu));
              }
            }
          const bool found = (top & 0x7f80u) == 0x7f80u || (top & 0x7f800000u) == 0x7f800000u;
          const uint32_t all = __ballot_sync(0xffffffffu, found);
          if (!all) continue;
          if (found) {
#pragma unroll 1
            for (int i = 0; i < DP; ++i) {
              uint16_t* x = reinterpret_cast<uint16_t*>(v + (i >> 6) * 16384 + r * 128) + (i & 63);
              if ((*x & 0x7f80u) == 0x7f80u) *x = 0;
            }
          }
          if (lane == 0) bad[(j - it.some / BLK) * 4 + g] = all;  // from the step that holds key `some` on
          __syncwarp();
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b.vfix + 8 * st);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(b.vempty + 8 * st);
    }
  }
}

// A thread's row of a tile.
struct Row {
  int t, limit;  // its token, the keys that it sees
  bool valid;
};
__device__ __forceinline__ Row row_of(const Args& a, const Item& it, int half, int dt) {
  Row r;
  r.t = it.tok + (it.halves == 2 ? half * a.tokens : 0) + dt;
  r.valid = dt < a.tokens && r.t < it.s.nq;
  r.limit = r.valid ? keys_seen(it.s, r.t, a.causal) : 0;
  return r;
}

template <int DP>
__device__ void softmax_role(const Args& a, uint32_t sbase, uint8_t* smem, uint32_t tmem, int half) {
  using L = Layout<DP>;
  const Bars<DP> b(sbase);
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, row = quad * 32 + lane;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  const uint32_t ts = lanes + half * BLK, to = lanes + 2 * BLK + half * BLK;
  const int dt = row / a.group, chunks = (a.dim + 15) / 16;
  float* stats = reinterpret_cast<float*>(smem + L::ROWS) + half * 256;
  const float2 c2 = make_float2(a.c, a.c);
  uint32_t sn = 0, item = 0;
  bool ok = true;
  auto arrive = [&](uint32_t bar) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  for (Item it; ok && next_item(a, b, smem, item, it); ++item) {
    const int steps = it.hi - it.lo;
    const Row r = row_of(a, it, half, dt);
    const bool idle = __all_sync(0xffffffffu, r.limit == 0);
    const int limit = r.valid ? r.limit : INT_MAX;  // a row that is none may come to anything
    float m = -INFINITY, l = 0.0f;  // the maximum that is subtracted (in powers of two), the sum
    const int first = it.halves == 2 ? 0 : half, by = it.halves == 2 ? 1 : 2;
#pragma unroll 1
    for (int i = first; i < steps; i += by, ++sn) {
      if (!(ok = wait_warp(a.watch, b.sfull + 8 * half, sn & 1u, S_TFULL))) break;
      if (idle) {
        arrive(b.pfull + 16 * half);
        arrive(b.pfull + 16 * half + 8);
        continue;
      }
      // all of the row's scores in registers
      uint32_t x[64], y[64];
      const int left = limit - (it.lo + i) * BLK;
      tc_fence_after();
      tmem_ld128_sync(ts, x, y);
      const int least = __reduce_min_sync(0xffffffffu, left);
      if (least < BLK) {  // only the columns that some row does not see
        auto mask = [&](uint32_t(&z)[64], int from) {
#pragma unroll
          for (int g = 0; g < 4; ++g)
            if (from + 16 * g + 16 > least) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (from + 16 * g + e >= left) z[16 * g + e] = 0xff800000u;
            }
        };
        mask(x, 0);
        mask(y, 64);
      }
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < 64; e += 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) top[k] = max3(top[k], __uint_as_float(x[e + k]), __uint_as_float(y[e + k]));
      }
      const float peak = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.c;
      const bool grow = r.valid && peak > m + GROWTH;
      if (__any_sync(0xffffffffu, grow)) {
        const float f = grow ? exp2_fast(m - peak) : 1.0f;  // from -infinity: 0
        if (grow) m = peak;
        l *= f;
        if (i != first) {  // the products before this step's scores are done
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            uint32_t o[16];
            tmem_ld16_sync(to + c * 16, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(to + c * 16, o);
          }
        }
      }
      const float sub = m == -INFINITY ? 0.0f : -m;
      const float2 sub2 = make_float2(sub, sub);
      float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
      // 64 keys' weights, over their own columns; the product with the first 64 runs beside the others.  They are rounded to
      // bf16, since the matrix instruction takes both operands in V's type: out is off by 0.0018 to 0.0024 of its size, where
      // weights in fp32 would give 0.0015 to 0.0017.  Their sum is taken before that.
      auto weights = [&](uint32_t(&z)[64], uint32_t at, uint32_t bar) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int k = 16 * g + 2 * e;
            const float2 s = fma2(make_float2(__uint_as_float(z[k]), __uint_as_float(z[k + 1])), c2, sub2);
            const float2 p = make_float2(exp2_fast(s.x), exp2_fast(s.y));
            sum[e & 1] = add2(sum[e & 1], p);
            h[e] = pack_bf16(p.x, p.y);
          }
          tmem_st8(at + 8 * g, h);
        }
        tmem_wait_st();
        arrive(bar);
      };
      weights(x, ts, b.pfull + 16 * half);
      weights(y, ts + 64, b.pfull + 16 * half + 8);
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
    }
    if (ok && item > 0) ok = wait_warp(a.watch, b.lfree + 8 * half, (item - 1) & 1u, S_TEMPTY);
    stats[row] = m;
    stats[128 + row] = l;
    __syncwarp();
    if (lane == 0) mbar_arrive(b.lfull + 8 * half);
  }
}

// Divides by the sums and stores; parts of divided tiles as they are, with their maxima and sums.
template <int DP>
__device__ void store_role(const Args& a, uint32_t sbase, uint8_t* smem, uint32_t tmem) {
  using L = Layout<DP>;
  const Bars<DP> b(sbase);
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, row = quad * 32 + lane;
  const uint32_t to = tmem + (static_cast<uint32_t>(quad * 32) << 16) + 2 * BLK;
  const int dt = row / a.group, head_in = row - dt * a.group;  // the row's token in its half, its head in the group
  const float* stats = reinterpret_cast<const float*>(smem + L::ROWS);
  uint8_t* stage = smem + L::STAGE + quad * 2048;
  const int64_t ml_at = static_cast<int64_t>(a.part_rows) * a.dim;
  uint32_t item = 0, on0 = 0, on1 = 0;
  bool ok = true;
  for (Item it; ok && next_item(a, b, smem, item, it); ++item) {
    const int steps = it.hi - it.lo, head = it.head * a.group + head_in;
    const bool both = it.halves == 1;  // the two accumulators are of the same rows
    const bool two = both && steps > 1, whole = it.shares == 1;
#pragma unroll 1
    for (int half = 0; ok && half < it.halves; ++half) {
      const Row r = row_of(a, it, half, dt);
      const bool idle = __all_sync(0xffffffffu, r.limit == 0);
      float m = -INFINITY, l = 0.0f, f0 = 1.0f, f1 = 0.0f;
#pragma unroll 1
      for (int h = half; ok && h < (both ? 2 : half + 1); ++h) {  // h: the accumulator
        ok = wait_warp(a.watch, b.lfull + 8 * h, item & 1u, S_TFULL);
        const float mh = stats[h * 256 + row], lh = stats[h * 256 + 128 + row];
        __syncwarp();
        if (lane == 0) mbar_arrive(b.lfree + 8 * h);
        if (ok && (!both || h < steps)) ok = wait_warp(a.watch, b.ofull + 8 * h, (h ? on1++ : on0++) & 1u, S_TFULL);
        if (h == half) {
          m = mh, l = lh;
        } else {
          const float top = fmaxf(m, mh);
          f0 = m == -INFINITY ? 0.0f : exp2_fast(m - top);
          f1 = mh == -INFINITY ? 0.0f : exp2_fast(mh - top);
          m = top, l = l * f0 + lh * f1;
        }
      }
      if (!ok) break;
      tc_fence_after();
      const uint32_t* bad = reinterpret_cast<const uint32_t*>(smem + L::BAD) + item % BAD_SETS * BAD_STEPS * 4;
      const bool any_bad = __any_sync(0xffffffffu, a.causal && lane < BAD_STEPS * 4 && bad[lane] != 0);
      const int64_t q_row = static_cast<int64_t>(it.s.q0) + r.t;
      float* part = a.part + it.slot * (ml_at + 2 * a.part_rows) + (half * BLK + row) * 4;
      if (whole) {
        const float inv = l == 0.0f ? (r.limit > 0 ? __uint_as_float(0x7fc00000u) : 0.0f) : 1.0f / l;
        f0 *= inv, f1 *= inv;
        if (r.valid && a.lse) a.lse[q_row * a.heads + head] = r.limit > 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
      } else if (r.valid) {
        float* ml = part - 3 * (half * BLK + row) + ml_at;
        ml[0] = m;
        ml[a.part_rows] = l;
      }
      const void* to_row = r.valid ? a.out + q_row * a.ldo + head * a.ho : nullptr;
#pragma unroll 1
      for (int c = 0; c < a.dim; c += 32) {  // few at a time: the code is fetched for each tile anew
        uint32_t o[32];
        if (idle) {  // no product: the accumulator may hold anything
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        } else {
          tmem_ld32_sync(to + half * BLK + c, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f0);
          if (two) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              uint32_t x[16];
              tmem_ld16_sync(to + BLK + c + g * 16, x);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                o[16 * g + e] = __float_as_uint(fmaf(__uint_as_float(x[e]), f1, __uint_as_float(o[16 * g + e])));
            }
          }
        }
        auto v = [&](int e) { return __uint_as_float(o[e]); };
        if (c + 32 >= a.dim) {  // the accumulator is read: the next tile's products may begin
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(b.ofree + 8 * half);
            if (two) mbar_arrive(b.ofree + 8);
          }
        }
        if (any_bad) {  // the noted values, for a row that sees their keys
#pragma unroll 1
          for (int i = 0; i < BAD_STEPS * 128; ++i) {
            const int key = it.some / BLK * BLK + i;
            if (!(bad[i >> 5] >> (i & 31) & 1u) || key >= r.limit) continue;
            const bf16* x = a.values + (static_cast<int64_t>(it.s.k0) + key) * a.ldv + it.head * a.hv + c;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float y = c + e < a.dim ? __bfloat162float(x[e]) : 0.0f;
              if (!isfinite(y)) o[e] = __float_as_uint(v(e) + y);
            }
          }
        }
        if (whole) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float z[8] = {v(8 * g),     v(8 * g + 1), v(8 * g + 2), v(8 * g + 3),
                                v(8 * g + 4), v(8 * g + 5), v(8 * g + 6), v(8 * g + 7)};
            stage_row(stage, g, z);
          }
          store_staged(stage, to_row, c, a.dim - c);
        } else if (r.valid) {
#pragma unroll
          for (int g = 0; g < 8; ++g)
            if (c + 4 * g < a.dim)
              *reinterpret_cast<float4*>(part + static_cast<int64_t>((c >> 2) + g) * a.part_rows * 4) =
                  make_float4(v(4 * g), v(4 * g + 1), v(4 * g + 2), v(4 * g + 3));
        }
      }
    }
  }
}

// Grid: one block per SM at most, each an equal share of the steps.
template <int DP>
__global__ void __launch_bounds__(THREADS, 1) fwd_kernel(const __grid_constant__ Args a) {
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
    init(b.kfull, L::STAGES, 1);
    init(b.kempty, L::STAGES, 2);  // both halves' products
    init(b.vfull, L::STAGES, 1);
    init(b.vempty, L::STAGES, 3);  // and the clearing warp
    init(b.vfix, L::STAGES, 1);
    init(b.items, RING, 1);
    init(b.qfull, 4, 1);           // and qempty
    init(b.sfull, 2, 1);
    init(b.pfull, 4, 4);           // a half's warps, 64 keys at a time
    init(b.ofull, 2, 1);
    init(b.ofree, 2, 4);
    init(b.lfull, 2, 4);
    init(b.lfree, 2, 4);
    init(b.drain, 2, 1);
    st_shared_u32(sbase + L::SLOT + 4, 0u);
    st_shared_u32(sbase + L::SLOT + 8, 0u);
    fence_barrier_init();
    tma_prefetch_map(&a.q);
    tma_prefetch_map(&a.k);
    tma_prefetch_map(&a.v);
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc_cg<1>(sbase + L::SLOT, 512);
    tmem_relinquish_cg<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ld_shared_u32(sbase + L::SLOT);
  grid_dep_wait();
  const Tiles tiles{a.kv_heads, a.tokens, a.causal};
  Shares& sh = *reinterpret_cast<Shares*>(smem + L::SHARES);
  plan_shares<THREADS>(tiles, a.seq, plan, &sh, a.watch.err);
  // registers: 128 a thread at launch, 65536 in all, shared out as the roles need them
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;" : "+r"(sbase)::"memory");  // nothing of a role is computed ahead of it
    if (warp == 0) load_role<DP>(a, tiles, sh, sbase, smem);
    if (warp == 1 || warp == 2) mma_role<DP>(a, sbase, smem, tmem, warp - 1);
    if (warp == 3) fix_role<DP>(a, sbase, smem);
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;" : "+r"(sbase)::"memory");
    softmax_role<DP>(a, sbase, smem, tmem, (warp - 4) >> 2);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;" : "+r"(sbase)::"memory");
    store_role<DP>(a, sbase, smem, tmem);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<1>(tmem, 512);
  }
}

// Joins the parts of the tile that share blockIdx.x began and did not end, in the
// order of the shares; block y takes its rows y, y + ROW_BLOCKS, ...  A row at a
// time: its weights by all threads, then eight columns a thread, over a slice of
// the parts where there are more than a few.  With few parts 16 rows at a time.
// Bound by latency: a kernel of its own adds 3 to 5 us to a call, where joining at
// the end of the main kernel held its blocks for 24000 to 54000 cycles.
constexpr int JOIN_THREADS = 256, ROW_BLOCKS = 16;
struct JoinArgs {
  const Entry* begun;
  const float* part;
  int part_rows, heads, group, tokens, dim, causal;
  bf16* out;
  int64_t ldo, ho;
  float* lse;
  const uint32_t* err;
};
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(JoinArgs a) {
  __shared__ float weight[MAX_SHARES * 16];
  __shared__ float sums[JOIN_THREADS][8];
  grid_dep_launch();
  grid_dep_wait();
  const Entry e = a.begun[blockIdx.x];
  if (*a.err != 0u || !e.begins || e.hi <= e.lo) return;  // after a failure the entries may be an earlier call's
  const int me = threadIdx.x, shares = e.shares, columns = a.dim / 8;
  const int tok0 = e.tile * 2 * a.tokens, left = e.s.nq - tok0;
  const int64_t slot = static_cast<int64_t>(a.part_rows) * (a.dim + 2), ml_at = static_cast<int64_t>(a.part_rows) * a.dim;
  const int halves = left <= a.tokens ? 1 : 2;
  // rows at a time, and slices of the parts, so that there is about a thread for each row's eight columns and slice
  const int used = a.tokens * a.group, rows = left <= a.tokens ? left * a.group : 2 * BLK;
  const int slices = shares <= 8 || rows > 2 * ROW_BLOCKS ? 1 : min(JOIN_THREADS / columns, (shares + 7) / 8);
  const int at_once = slices == 1 ? 16 : 1;
  for (int first = blockIdx.y * at_once; first < halves * BLK; first += ROW_BLOCKS * at_once) {
    auto place = [&](int r, int64_t* q_row, int* h, int* limit) {  // of row r of the tile
      const int in = r & (BLK - 1), dtok = in / a.group, t = tok0 + (r >> 7) * a.tokens + dtok;
      *q_row = static_cast<int64_t>(e.s.q0) + t;
      *h = e.head * a.group + in - dtok * a.group;
      *limit = keys_seen(e.s, t, a.causal);
      return in < used && t < e.s.nq;
    };
    int64_t q_row;
    int h, limit;
    if (at_once == 1 && !place(first, &q_row, &h, &limit)) continue;  // the same for all threads
    // ---- the weights: sixteen lanes a row
    const int wr = me >> 4, wl = me & 15;
    if (wr < at_once) {
      const float* ml = a.part + ml_at + first + wr;
      float top = -INFINITY, sum = 0.0f;
      for (int s = wl; s < shares; s += 16) top = fmaxf(top, ml[tile_slot(e.from, s) * slot]);
      for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffu << (me & 16), top, o));
      const float base = top == -INFINITY ? 0.0f : top;
      for (int s = wl; s < shares; s += 16) {
        const float* p = ml + tile_slot(e.from, s) * slot;
        const float f = exp2_fast(p[0] - base);
        weight[wr * MAX_SHARES + s] = f;
        sum += p[a.part_rows] * f;
      }
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffu << (me & 16), sum, o);
      const bool there = place(first + wr, &q_row, &h, &limit);
      const float inv = sum == 0.0f ? (limit > 0 ? __uint_as_float(0x7fc00000u) : 0.0f) : 1.0f / sum;
      for (int s = wl; s < shares; s += 16) weight[wr * MAX_SHARES + s] *= inv;
      if (there && a.lse && wl == 0) a.lse[q_row * a.heads + h] = limit > 0 ? (top + log2f(sum)) * kLn2 : -INFINITY;
    }
    __syncthreads();
    // ---- the sums
    const int r = at_once == 1 ? 0 : me & 15, c = at_once == 1 ? me % columns : me >> 4, slice = at_once == 1 ? me / columns : 0;
    const bool mine = c < columns && slice < slices && place(first + r, &q_row, &h, &limit);
    float v[8] = {};
    if (mine) {
      const int each = (shares + slices - 1) / slices, end = min(shares, (slice + 1) * each);
      const float* src = a.part + (static_cast<int64_t>(2 * c) * a.part_rows + first + r) * 4;
      const float* f = weight + r * MAX_SHARES;
      some_parts(slice * each, end, [&](auto count, int s) {
        constexpr int U = decltype(count)::value;
        float4 lo[U], hi[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float* p = src + tile_slot(e.from, min(s + u, end - 1)) * slot;
          lo[u] = *reinterpret_cast<const float4*>(p);
          hi[u] = *reinterpret_cast<const float4*>(p + static_cast<int64_t>(a.part_rows) * 4);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (s + u >= end) break;
          const float k = f[s + u];
          v[0] = fmaf(lo[u].x, k, v[0]), v[1] = fmaf(lo[u].y, k, v[1]), v[2] = fmaf(lo[u].z, k, v[2]), v[3] = fmaf(lo[u].w, k, v[3]);
          v[4] = fmaf(hi[u].x, k, v[4]), v[5] = fmaf(hi[u].y, k, v[5]), v[6] = fmaf(hi[u].z, k, v[6]), v[7] = fmaf(hi[u].w, k, v[7]);
        }
      });
    }
    if (slices > 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[me][i] = v[i];
      __syncthreads();
      for (int t = 1; slice == 0 && mine && t < slices; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += sums[t * columns + me][i];
    }
    if (mine && slice == 0)
      *reinterpret_cast<uint4*>(a.out + q_row * a.ldo + h * a.ho + c * 8) =
          make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    __syncthreads();
  }
}

int64_t part_rows(int64_t n, int64_t group) { return n <= BLK / group ? BLK : 2 * BLK; }

template <int DP>
cudaError_t launch_as(const Args& a, int grid, cudaStream_t s) {
  return launch_pdl(fwd_kernel<DP>, dim3(static_cast<unsigned>(grid)), dim3(THREADS), Layout<DP>::SMEM, s, a);
}

}  // namespace

cudaError_t configure_attention() {
  const cudaError_t e =
      cudaFuncSetAttribute(fwd_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<64>::SMEM);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(fwd_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<128>::SMEM);
}

int64_t need_attention(int64_t n, int64_t, int64_t heads, int64_t kv_heads, int64_t dim) {
  return BEGUN_BYTES + 2ll * MAX_SHARES * part_rows(n, heads / kv_heads) * (dim + 2) * 4;
}

cudaError_t launch_attention(const Machine& mc, const AttnArgs& x, const Watch& w, void* ws, cudaStream_t s) {
  Args a;
  std::memset(static_cast<void*>(&a), 0, sizeof(a));
  a.seq = x.seq;
  a.heads = static_cast<int>(x.heads), a.kv_heads = static_cast<int>(x.kv_heads);
  a.group = a.heads / a.kv_heads, a.tokens = BLK / a.group;
  a.dim = static_cast<int>(x.dim), a.causal = x.causal, a.c = x.scale * kLog2e;
  a.values = static_cast<const bf16*>(x.v.p), a.ldv = x.v.ld, a.hv = x.v.hs;
  a.out = static_cast<bf16*>(const_cast<void*>(x.out.p)), a.ldo = x.out.ld, a.ho = x.out.hs;
  a.lse = x.lse, a.watch = w;
  a.begun = static_cast<Entry*>(ws), a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + BEGUN_BYTES);
  a.part_rows = static_cast<int>(part_rows(x.seq.n, a.group));
  // without keys the loads go to the queries, which no row sees
  const bool keys = x.seq.nk > 0;
  const int64_t nk = keys ? x.seq.nk : x.seq.n, kv = keys ? x.kv_heads : x.heads;
  if (!encode_heads(&a.q, x.q, x.seq.n, x.heads, x.dim, a.group, a.tokens) ||
      !encode_heads(&a.k, keys ? x.k : x.q, nk, kv, x.dim, 1, BLK) ||
      !encode_heads(&a.v, keys ? x.v : x.q, nk, kv, x.dim, 1, BLK))
    return cudaErrorInvalidValue;
  // no more blocks than the most steps that these sizes can have
  const int64_t tiles = (x.seq.n / (2 * a.tokens) + std::min(x.seq.batch, x.seq.n)) * x.kv_heads;
  const int64_t most = std::min<int64_t>(tiles, MAX_SHARES) * (x.seq.nk / BLK + 1);
  const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min(mc.sms, MAX_SHARES), most)));
  const cudaError_t e = x.dim <= 64 ? launch_as<64>(a, grid, s) : launch_as<128>(a, grid, s);
  if (e != cudaSuccess || x.seq.nk <= BLK) return e;  // tiles of one step are never divided
  const JoinArgs j{a.begun, a.part, a.part_rows, a.heads, a.group, a.tokens, a.dim, a.causal, a.out, a.ldo, a.ho, a.lse, w.err};
  return launch_pdl(join_kernel, dim3(static_cast<unsigned>(grid), ROW_BLOCKS), dim3(JOIN_THREADS), 0, s, j);
}

}  // namespace tpo
