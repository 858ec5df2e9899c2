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
// softmax (3950 cycles a step).

#include <algorithm>
#include <cstring>

#include <cuda_bf16.h>

#include "attn_dev.h"
#include "pdl.h"

namespace tpo {

namespace {

using bf16 = __nv_bfloat16;
constexpr int THREADS = 512;
constexpr int STORE = 128;               // threads of the storing group
constexpr float GROWTH = 8.0f;           // of the maximum, in powers of two, before O is rescaled
constexpr int JOIN = 2048;               // parts of rows whose weights are in shared memory at a time
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
  float* part;
  int part_rows;
  uint32_t* arrivals;
  Watch watch;
};

struct Tiles {
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
  static constexpr int N_BARS = 5 * STAGES + 18;
  static constexpr int SLOT = BARS + 8 * N_BARS;
  static constexpr int LAST = SLOT + 4;
  static constexpr int BAD = SLOT + 8;               // [BAD_SETS][BAD_STEPS][4] keys, a bit each
  static constexpr int ROWS = (BAD + BAD_SETS * BAD_STEPS * 16 + 15) / 16 * 16;  // [2][2][128] floats: maxima and sums
  static constexpr int JOIN_AT = ROWS + 2048;        // [2][JOIN] floats, or the storing warps' staging boxes
  static constexpr int PLAN = JOIN_AT + 8 * JOIN;
  static_assert(JOIN_AT % 16 == 0 && 8 * JOIN >= 4 * 2048, "also a staging box for each warp");
  static constexpr int SMEM = PLAN + static_cast<int>(sizeof(PlanScratch)) + 1024;
  static_assert(SMEM <= 232448, "shared memory of one block");
};

template <int DP>
struct Bars {
  uint32_t kfull, kempty, vfull, vempty, vfix, qfull, qempty, sfull, pfull, ofull, ofree, lfull, lfree, drain;
  __device__ explicit Bars(uint32_t sbase) {
    uint32_t b = sbase + Layout<DP>::BARS;
    auto next = [&](int n) {
      const uint32_t r = b;
      b += 8 * n;
      return r;
    };
    constexpr int S = Layout<DP>::STAGES;
    kfull = next(S), kempty = next(S), vfull = next(S), vempty = next(S), vfix = next(S), qfull = next(1);
    qempty = next(1), sfull = next(2), pfull = next(4), ofull = next(2), ofree = next(2), lfull = next(2);
    lfree = next(2), drain = next(2);
  }
};

__device__ __forceinline__ void bar_store() { asm volatile("bar.sync 1, %0;" ::"n"(STORE) : "memory"); }

// What the roles derive from a part of a tile.
struct Item {
  Part p;
  int tok;    // first token of the tile, in the sequence
  int halves;
  int some;   // keys from here on are not seen by all queries
};
__device__ __forceinline__ Item item_of(const Args& a, const Walk& w) {
  Item i;
  i.p = walk_part(w);
  i.tok = w.tile * 2 * a.tokens;
  i.halves = w.s.nq - i.tok <= a.tokens ? 1 : 2;
  i.some = keys_seen(w.s, i.tok, a.causal);
  return i;
}
__device__ __forceinline__ bool needs_fix(const Item& i, int j) { return (j + 1) * BLK > i.some; }

template <int DP>
__device__ void load_role(const Args& a, const Tiles& tiles, const Shares& sh, uint32_t sbase) {
  using L = Layout<DP>;
  const Bars<DP> b(sbase);
  const bool lead = (threadIdx.x & 31) == 0;
  uint32_t kn = 0, vn = 0, qn = 0;  // loads so far
  bool ok = true;
  Walk w;
  for (walk_begin(tiles, sh, w); ok && walk_has(w); walk_next(tiles, a.seq, w)) {
    const Item it = item_of(a, w);
    if (!(ok = wait_warp(a.watch, b.qempty, (qn & 1u) ^ 1u, S_EMPTY))) break;
    if (lead) {
      mbar_expect_tx(b.qfull, static_cast<uint32_t>(a.group * a.tokens) * 128u * (DP / 64) * it.halves);
      for (int h = 0; h < it.halves; ++h)
        for (int d = 0; d < DP / 64; ++d)
          tma_load_3d(sbase + h * L::TILE + d * 16384, &a.q, b.qfull, d * 64, w.head * a.group,
                      w.s.q0 + it.tok + h * a.tokens);
    }
    __syncwarp();
    ++qn;
    auto load = [&](const CUtensorMap* map, uint32_t full, uint32_t empty, uint32_t base, uint32_t& n, int j) {
      const uint32_t st = n % L::STAGES, ph = n / L::STAGES & 1u;
      if (!wait_warp(a.watch, empty + 8 * st, ph ^ 1u, S_EMPTY)) return false;
      if (lead) {
        mbar_expect_tx(full + 8 * st, L::TILE);
        for (int d = 0; d < DP / 64; ++d)
          tma_load_3d(base + st * L::TILE + d * 16384, map, full + 8 * st, d * 64, w.head, w.s.k0 + j * BLK);
      }
      __syncwarp();
      ++n;
      return true;
    };
    // K one step ahead of V, as the products take them
    for (int j = it.p.lo; ok && j <= it.p.hi; ++j) {
      if (j < it.p.hi) ok = load(&a.k, b.kfull, b.kempty, sbase + L::K0, kn, j);
      if (ok && j > it.p.lo) ok = load(&a.v, b.vfull, b.vempty, sbase + L::V0, vn, j - 1);
    }
  }
  if (!ok && lead) {  // what is in flight must land before the block gives up its shared memory
    for (uint32_t j = kn > L::STAGES ? kn - L::STAGES : 0u; j < kn; ++j)
      wait_bar(a.watch, b.kfull + 8 * (j % L::STAGES), j / L::STAGES & 1u, S_DRAIN, false);
    for (uint32_t j = vn > L::STAGES ? vn - L::STAGES : 0u; j < vn; ++j)
      wait_bar(a.watch, b.vfull + 8 * (j % L::STAGES), j / L::STAGES & 1u, S_DRAIN, false);
    if (qn) wait_bar(a.watch, b.qfull, (qn - 1) & 1u, S_DRAIN, false);
  }
  __syncwarp();
}

// The turns of the two issuing warps, by named barriers: pass_turn lets the other's next take_turn through.
__device__ __forceinline__ void take_turn(int half) {
  if (half)
    asm volatile("bar.sync 2, 64;" ::: "memory");
  else
    asm volatile("bar.sync 3, 64;" ::: "memory");
}
__device__ __forceinline__ void pass_turn(int half) {
  if (half)
    asm volatile("bar.arrive 3, 64;" ::: "memory");
  else
    asm volatile("bar.arrive 2, 64;" ::: "memory");
}

// The products of one half.  Where a tile has one half only, the warps (and accumulators) take its steps by turns, and
// pass over the other's: both release a stage.
template <int DP>
__device__ void mma_role(const Args& a, const Tiles& tiles, const Shares& sh, uint32_t sbase, uint32_t tmem, int half) {
  using L = Layout<DP>;
  const Bars<DP> b(sbase);
  const bool lead = (threadIdx.x & 31) == 0;
  const uint32_t idesc_s = idesc_n(make_idesc(false, BLK), BLK);
  const uint32_t idesc_o = idesc_n(make_idesc(false, BLK), (a.dim + 15) / 16 * 16) | 1u << 16;
  const uint64_t dk = smem_desc_sw128(sbase + L::K0), dv = desc_rows(sbase + L::V0);
  const uint32_t s = tmem + half * BLK, o = tmem + 2 * BLK + half * BLK;
  uint32_t kn = 0, vn = 0, qn = 0, pn = 0;
  uint32_t fixed = 0;  // parity of each stage's next clearing
  bool ok = true;      // after a failure the turns go on, without waits and products
  bool turns = false;  // whether there was a turn: the first is half 0's without asking
  Walk w;
  for (walk_begin(tiles, sh, w); walk_has(w); walk_next(tiles, a.seq, w), ++qn) {
    const Item it = item_of(a, w);
    const int steps = it.p.hi - it.p.lo;
    const uint64_t dq = smem_desc_sw128(sbase + (it.halves == 2 ? half * L::TILE : 0));
    auto await = [&](uint32_t bar, uint32_t parity) {
      if (ok) ok = wait_warp(a.watch, bar, parity & 1u, S_FULL);
    };
    auto await_k = [&] { await(b.kfull + 8 * (kn % L::STAGES), kn / L::STAGES); };
    auto await_v = [&](int i) {
      const uint32_t st = vn % L::STAGES;
      await(b.vfull + 8 * st, vn / L::STAGES);
      if (needs_fix(it, it.p.lo + i)) {
        await(b.vfix + 8 * st, fixed >> st);
        fixed ^= 1u << st;
      }
    };
    auto scores = [&] {
      if (!ok) return;
      tc_fence_after();
      mma_head<DP>(s, dq, dk + (kn % L::STAGES) * (L::TILE >> 4), idesc_s);
      mma_commit_cg<1>(b.sfull + 8 * half);
    };
    auto free_k = [&] {
      if (ok) mma_commit_cg<1>(b.kempty + 8 * (kn % L::STAGES));
      ++kn;
    };
    auto free_v = [&] {
      if (ok) mma_commit_cg<1>(b.vempty + 8 * (vn % L::STAGES));
      ++vn;
    };
    auto product = [&](int part, bool fresh) {  // 64 keys
      if (!ok) return;
      tc_fence_after();
      mma4_ts(o, s + 64 * part, dv + (vn % L::STAGES) * (L::TILE >> 4) + 512 * part, idesc_o, fresh ? 0u : 1u);
    };
    await(b.qfull, qn);
    if (it.halves == 2) {
      await_k();
      scores();
      free_k();
      if (steps == 1 && ok) mma_commit_cg<1>(b.qempty);
      for (int i = 0; i < steps; ++i, ++pn) {
        const bool more = i + 1 < steps;
        // the accumulator is free once the part before has been stored
        if (i == 0 && qn > 0) await(b.ofree + 8 * half, qn - 1);
        await_v(i);
        if (more) await_k();
        await(b.pfull + 16 * half, pn);
        product(0, i == 0);
        await(b.pfull + 16 * half + 8, pn);
        if (half || turns) take_turn(half);
        turns = true;
        product(1, false);
        if (more)
          scores();
        else if (ok)
          mma_commit_cg<1>(b.ofull + 8 * half);
        pass_turn(half);
        free_v();
        if (more) free_k();
        if (i + 2 == steps && ok) mma_commit_cg<1>(b.qempty);
      }
    } else {
      auto skip_k = [&] {
        await_k();
        if (lead) mbar_arrive(b.kempty + 8 * (kn % L::STAGES));
        ++kn;
      };
      auto skip_v = [&](int i) {
        await(b.vfull + 8 * (vn % L::STAGES), vn / L::STAGES);
        if (needs_fix(it, it.p.lo + i)) fixed ^= 1u << (vn % L::STAGES);
        if (lead) mbar_arrive(b.vempty + 8 * (vn % L::STAGES));
        ++vn;
      };
      if (half) skip_k();
      if (half < steps) {
        await_k();
        scores();
        free_k();
      }
      if (qn > 0) await(b.ofree + 8 * half, qn - 1);
      if (half) skip_v(0);
      for (int i = half; i < steps; i += 2, ++pn) {
        await_v(i);
        await(b.pfull + 16 * half, pn);
        product(0, i < 2);
        await(b.pfull + 16 * half + 8, pn);
        product(1, false);
        free_v();
        if (i + 1 < steps) skip_k();
        if (i + 2 < steps) {
          await_k();
          scores();
          free_k();
        } else if (ok) {
          mma_commit_cg<1>(b.ofull + 8 * half);
        }
        if (i + 1 < steps) skip_v(i + 1);
      }
      if (ok) mma_commit_cg<1>(b.qempty);
    }
  }
  if (!half && turns) take_turn(half);  // the last one that was passed
  // also after a failure: every MMA issued must complete before tensor memory is freed
  mma_commit_cg<1>(b.drain + 8 * half);
  if (lead) wait_bar(a.watch, b.drain + 8 * half, 0u, S_DRAIN, false);
  __syncwarp();
}

// Clears the rows of V behind the last key, and takes values that are not finite
// out of rows that only some queries see, noting their keys.
template <int DP>
__device__ void fix_role(const Args& a, const Tiles& tiles, const Shares& sh, uint32_t sbase, uint8_t* smem) {
  using L = Layout<DP>;
  const Bars<DP> b(sbase);
  const int lane = threadIdx.x & 31;
  uint32_t vn = 0, item = 0;
  Walk w;
  for (walk_begin(tiles, sh, w); walk_has(w); walk_next(tiles, a.seq, w), ++item) {
    const Item it = item_of(a, w);
    uint32_t* bad = reinterpret_cast<uint32_t*>(smem + L::BAD) + item % BAD_SETS * BAD_STEPS * 4;
    if (lane < 4 * BAD_STEPS) bad[lane] = 0;
    __syncwarp();
    for (int j = it.p.lo; j < it.p.hi; ++j, ++vn) {
      const uint32_t st = vn % L::STAGES;
      if (!wait_warp(a.watch, b.vfull + 8 * st, vn / L::STAGES & 1u, S_FULL)) return;
      if (needs_fix(it, j)) {
        uint8_t* v = smem + L::V0 + st * L::TILE;
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {
          const int r = 32 * g + lane, key = j * BLK + r;
          uint32_t top = 0;  // the row's largest magnitudes, as a pair of bf16
          if (key >= w.s.nk) {
#pragma unroll
            for (int d = 0; d < DP / 64; ++d)
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4*>(v + d * 16384 + r * 128 + ((i ^ (r & 7)) << 4)) = make_uint4(0, 0, 0, 0);
          } else if (key >= it.some) {
            auto most = [&](uint32_t x) {
              asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(x & 0x7fff7fffu));
            };
#pragma unroll
            for (int d = 0; d < DP / 64; ++d)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint4 x = *reinterpret_cast<const uint4*>(v + d * 16384 + r * 128 + ((i ^ (r & 7)) << 4));
                most(x.x), most(x.y), most(x.z), most(x.w);
              }
          }
          const bool found = (top & 0x7f80u) == 0x7f80u || (top & 0x7f800000u) == 0x7f800000u;
          const uint32_t all = __ballot_sync(0xffffffffu, found);
          if (!all) continue;
          if (found)
            for (int d = 0; d < DP / 64; ++d)
              for (int i = 0; i < 64; ++i) {
                uint16_t* x = reinterpret_cast<uint16_t*>(v + d * 16384 + r * 128) + i;
                if ((*x & 0x7f80u) == 0x7f80u) *x = 0;
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
__device__ __forceinline__ Row row_of(const Args& a, const Walk& w, const Item& it, int half, int dt) {
  Row r;
  r.t = it.tok + (it.halves == 2 ? half * a.tokens : 0) + dt;
  r.valid = dt < a.tokens && r.t < w.s.nq;
  r.limit = r.valid ? keys_seen(w.s, r.t, a.causal) : 0;
  return r;
}

template <int DP>
__device__ void softmax_role(const Args& a, const Tiles& tiles, const Shares& sh, uint32_t sbase, uint8_t* smem,
                             uint32_t tmem, int half) {
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
  Walk w;
  for (walk_begin(tiles, sh, w); walk_has(w); walk_next(tiles, a.seq, w), ++item) {
    const Item it = item_of(a, w);
    const int steps = it.p.hi - it.p.lo;
    const int limit = row_of(a, w, it, half, dt).limit;
    const bool idle = __all_sync(0xffffffffu, limit == 0);
    float m = -INFINITY, l = 0.0f;  // the maximum that is subtracted (in powers of two), the sum
    const int first = it.halves == 2 ? 0 : half, by = it.halves == 2 ? 1 : 2;
    for (int i = first; i < steps; i += by, ++sn) {
      if (ok) ok = wait_warp(a.watch, b.sfull + 8 * half, sn & 1u, S_TFULL);
      if (!ok || idle) {
        arrive(b.pfull + 16 * half);
        arrive(b.pfull + 16 * half + 8);
        continue;
      }
      // all of the row's scores in registers
      uint32_t x[64], y[64];
      const int left = limit - (it.p.lo + i) * BLK;
      tc_fence_after();
      tmem_ld128_sync(ts, x, y);
      if (!__all_sync(0xffffffffu, left >= BLK)) {
#pragma unroll
        for (int e = 0; e < 64; ++e) {
          if (e >= left) x[e] = 0xff800000u;
          if (e + 64 >= left) y[e] = 0xff800000u;
        }
      }
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < 64; e += 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) top[k] = max3(top[k], __uint_as_float(x[e + k]), __uint_as_float(y[e + k]));
      }
      const float peak = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.c;
      const bool grow = peak > m + GROWTH;
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
      // 64 keys' weights, rounded, over their own columns; the product with the first 64 runs beside the others
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

// Divides by the sums and stores, and joins the parts of divided tiles.
template <int DP>
__device__ void store_role(const Args& a, const Tiles& tiles, const Shares& sh, uint32_t sbase, uint8_t* smem,
                           uint32_t tmem) {
  using L = Layout<DP>;
  const Bars<DP> b(sbase);
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, row = quad * 32 + lane, me = threadIdx.x - 384;
  const uint32_t to = tmem + (static_cast<uint32_t>(quad * 32) << 16) + 2 * BLK;
  const int dt = row / a.group, head_in = row - dt * a.group;  // the row's token in its half, its head in the group
  const int chunks = (a.dim + 31) / 32;
  const float* stats = reinterpret_cast<const float*>(smem + L::ROWS);
  uint8_t* stage = smem + L::JOIN_AT + quad * 2048;
  uint32_t item = 0, on[2] = {0, 0};
  bool ok = true;
  Walk w;
  for (walk_begin(tiles, sh, w); walk_has(w); walk_next(tiles, a.seq, w), ++item) {
    const Item it = item_of(a, w);
    const int steps = it.p.hi - it.p.lo, head = w.head * a.group + head_in;
    float* part = a.part + static_cast<int64_t>(part_slot(w)) * a.part_rows * (a.dim + 2);
    const bool both = it.halves == 1;  // the two accumulators are of the same rows
#pragma unroll 1
    for (int half = 0; half < it.halves; ++half) {
      const Row r = row_of(a, w, it, half, dt);
      const bool idle = __all_sync(0xffffffffu, r.limit == 0);
      float ms[2] = {-INFINITY, -INFINITY}, ls[2] = {0.0f, 0.0f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // h: the accumulator
        if (!both && h != half) continue;
        if (ok) ok = wait_warp(a.watch, b.lfull + 8 * h, item & 1u, S_TFULL);
        ms[h] = stats[h * 256 + row];
        ls[h] = stats[h * 256 + 128 + row];
        __syncwarp();
        if (lane == 0) mbar_arrive(b.lfree + 8 * h);
        if (!both || h < steps) {  // else it has no product
          if (ok) ok = wait_warp(a.watch, b.ofull + 8 * h, on[h] & 1u, S_TFULL);
          ++on[h];
        }
      }
      tc_fence_after();
      const float m = fmaxf(ms[0], ms[1]);
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) f[h] = ms[h] == -INFINITY ? 0.0f : exp2_fast(ms[h] - m);
      const float l = ls[0] * f[0] + ls[1] * f[1];
      const uint32_t* bad = reinterpret_cast<const uint32_t*>(smem + L::BAD) + item % BAD_SETS * BAD_STEPS * 4;
      uint32_t any_bad = 0;
      if (ok && a.causal && lane < BAD_STEPS * 4) any_bad = bad[lane];
      any_bad = __any_sync(0xffffffffu, any_bad != 0);
      const int64_t q_row = static_cast<int64_t>(w.s.q0) + r.t;
      const float scale = !it.p.whole ? 1.0f : l == 0.0f ? (r.limit > 0 ? __uint_as_float(0x7fc00000u) : 0.0f) : 1.0f / l;
      const float f0 = f[both ? 0 : half] * scale, f1 = f[1] * scale;
      const RowsOut to_rows = rows_out(r.valid && it.p.whole ? a.out + q_row * a.ldo + head * a.ho : nullptr);
#pragma unroll 1
      for (int c = 0; ok && c < chunks; ++c) {
        float v[32];
        if (idle) {  // no product: the accumulator may hold anything
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0.0f;
        } else {
          uint32_t o[32];
          tmem_ld32_sync(to + half * BLK + c * 32, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[e]) * f0;
          if (both && steps > 1) {
            tmem_ld32_sync(to + BLK + c * 32, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = fmaf(__uint_as_float(o[e]), f1, v[e]);
          }
        }
        if (any_bad)  // the noted values, for a row that sees their keys
          for (int i = 0; i < BAD_STEPS * 4; ++i)
            for (uint32_t left = bad[i]; left; left &= left - 1) {
              const int key = it.some / BLK * BLK + 32 * i + __ffs(left) - 1;
              if (key >= r.limit) continue;
              const bf16* x = a.values + (static_cast<int64_t>(w.s.k0) + key) * a.ldv + w.head * a.hv + c * 32;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float y = c * 32 + e < a.dim ? __bfloat162float(x[e]) : 0.0f;
                if (!isfinite(y)) v[e] += y;
              }
            }
        if (it.p.whole)
          store_rows(stage, v, to_rows, c * 32, a.dim - c * 32);
        else if (r.valid)
          store_part(part, a.part_rows, half * BLK + row, v, c * 32, a.dim);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(b.ofree + 8 * half);
        if (both) mbar_arrive(b.ofree + 8);
      }
      if (ok && r.valid) {
        if (!it.p.whole) {
          float* ml = part + static_cast<int64_t>(a.part_rows) * a.dim;
          ml[half * BLK + row] = m;
          ml[a.part_rows + half * BLK + row] = l;
        } else if (a.lse) {
          a.lse[q_row * a.heads + head] = r.limit > 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
        }
      }
    }
    if (it.p.whole) continue;
    // ---- a divided tile: whoever comes last joins its parts
    __threadfence();
    bar_store();
    int from;
    const int shares = tile_shares(sh, w, &from);
    volatile int* last = reinterpret_cast<volatile int*>(smem + L::LAST);
    if (me == 0) {
      const uint32_t before = atomicAdd(a.arrivals + from, ok ? 1u : 0u);
      *last = ok && before + 1 == static_cast<uint32_t>(shares);
      if (*last) a.arrivals[from] = 0;
    }
    bar_store();
    if (!*last) {
      bar_store();
      continue;
    }
    __threadfence();
    const int64_t slot = static_cast<int64_t>(a.part_rows) * (a.dim + 2), stats = static_cast<int64_t>(a.part_rows) * a.dim;
    auto place = [&](int r, int* tok, int* h) {  // of row r of the tile
      const int in = r & (BLK - 1), dtok = in / a.group;
      *tok = it.tok + (r >> 7) * a.tokens + dtok;
      *h = w.head * a.group + in - dtok * a.group;
      return dtok < a.tokens && *tok < w.s.nq;
    };
    // as many rows at a time as their parts' weights find room: a warp makes a row's weights, then every thread adds
    // four columns of some rows
    const int left = w.s.nq - it.tok;
    const int count = left <= a.tokens ? left * a.group : left < 2 * a.tokens ? BLK + (left - a.tokens) * a.group : 2 * BLK;
    const int batch = min(count, JOIN / shares);
    float* table = reinterpret_cast<float*>(smem + L::JOIN_AT);
    for (int r0 = 0; r0 < count; r0 += batch) {
      const int rows_now = min(batch, count - r0);
      for (int i = me; i < rows_now * shares; i += STORE) {
        const int s = i / rows_now, r = i - s * rows_now;
        const float* ml = a.part + tile_slot(from, s) * slot + stats + r0 + r;
        table[r * shares + s] = ml[0];
        table[JOIN + r * shares + s] = ml[a.part_rows];
      }
      bar_store();
      // as many lanes a row as it has parts, up to a warp
      int wide = 1;
      while (wide < shares && wide < 32) wide *= 2;
      const int in = me & (wide - 1);
#pragma unroll 1
      for (int r0w = 0; r0w < rows_now; r0w += STORE / wide) {
        const int r = r0w + me / wide;
        float* tm = table + min(r, rows_now - 1) * shares;
        float top = -INFINITY, sum = 0.0f;
        for (int s = in; s < shares; s += wide) top = fmaxf(top, tm[s]);
        for (int o = wide / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float base = top == -INFINITY ? 0.0f : top;
        for (int s = in; s < shares; s += wide) sum += tm[JOIN + s] * exp2_fast(tm[s] - base);
        for (int o = wide / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        int tok, h;
        const bool there = r < rows_now && place(r0 + r, &tok, &h);
        const int lim = there ? keys_seen(w.s, tok, a.causal) : 0;
        const float inv = lim == 0 ? 0.0f : sum == 0.0f ? __uint_as_float(0x7fc00000u) : 1.0f / sum;
        __syncwarp();  // rows past the last one read its entries
        if (r < rows_now)
          for (int s = in; s < shares; s += wide) tm[s] = exp2_fast(tm[s] - base) * inv;
        if (there && a.lse && in == 0)
          a.lse[(static_cast<int64_t>(w.s.q0) + tok) * a.heads + h] = lim > 0 ? (top + log2f(sum)) * kLn2 : -INFINITY;
      }
      bar_store();
      constexpr int U = 2;  // two groups of eight columns at a time
      const int groups = rows_now * (a.dim / 8);
      for (int i0 = me; i0 < groups; i0 += U * STORE) {
        float4 v[U][2];
        const float *src[U], *f[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = min(i0 + u * STORE, groups - 1), g = i / rows_now, r = i - g * rows_now;
          v[u][0] = v[u][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          f[u] = table + r * shares;
          src[u] = a.part + (static_cast<int64_t>(2 * g) * a.part_rows + r0 + r) * 4;
        }
        auto add = [&](int s) {
          const int64_t at = tile_slot(from, s) * slot;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float k = f[u][s];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float4 y = *reinterpret_cast<const float4*>(src[u] + at + static_cast<int64_t>(j) * a.part_rows * 4);
              v[u][j].x += y.x * k, v[u][j].y += y.y * k, v[u][j].z += y.z * k, v[u][j].w += y.w * k;
            }
          }
        };
        int s = 0;
#pragma unroll 1
        for (; s + 4 <= shares; s += 4) add(s), add(s + 1), add(s + 2), add(s + 3);
        if (s + 2 <= shares) add(s), add(s + 1), s += 2;
        if (s < shares) add(s);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * STORE, g = i / rows_now, r = i - g * rows_now;
          int tok, h;
          if (i < groups && place(r0 + r, &tok, &h))
            *reinterpret_cast<uint4*>(a.out + (static_cast<int64_t>(w.s.q0) + tok) * a.ldo + h * a.ho + g * 8) =
                make_uint4(pack_bf16(v[u][0].x, v[u][0].y), pack_bf16(v[u][0].z, v[u][0].w),
                           pack_bf16(v[u][1].x, v[u][1].y), pack_bf16(v[u][1].z, v[u][1].w));
        }
      }
      bar_store();
    }
    bar_store();
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
    init(b.qfull, 1, 1);
    init(b.qempty, 1, 2);
    init(b.sfull, 2, 1);
    init(b.pfull, 4, 4);           // a half's warps, 64 keys at a time
    init(b.ofull, 2, 1);
    init(b.ofree, 2, 4);
    init(b.lfull, 2, 4);
    init(b.lfree, 2, 4);
    init(b.drain, 2, 1);
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
  plan_shares<THREADS>(tiles, a.seq, plan);
  const Shares& sh = plan->shares;
  // registers: 128 a thread at launch, 65536 in all, shared out as the roles need them
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;" : "+r"(sbase)::"memory");  // nothing of a role is computed ahead of it
    if (warp == 0) load_role<DP>(a, tiles, sh, sbase);
    if (warp == 1 || warp == 2) mma_role<DP>(a, tiles, sh, sbase, tmem, warp - 1);
    if (warp == 3) fix_role<DP>(a, tiles, sh, sbase, smem);
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;" : "+r"(sbase)::"memory");  // nothing of a role is computed ahead of it
    softmax_role<DP>(a, tiles, sh, sbase, smem, tmem, (warp - 4) >> 2);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;" : "+r"(sbase)::"memory");  // nothing of a role is computed ahead of it
    store_role<DP>(a, tiles, sh, sbase, smem, tmem);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<1>(tmem, 512);
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
  return 2ll * MAX_SHARES * part_rows(n, heads / kv_heads) * (dim + 2) * 4;
}

cudaError_t launch_attention(const Machine& mc, const AttnArgs& x, const Watch& w, uint32_t* arrivals, void* ws,
                             cudaStream_t s) {
  Args a;
  std::memset(static_cast<void*>(&a), 0, sizeof(a));
  a.seq = x.seq;
  a.heads = static_cast<int>(x.heads), a.kv_heads = static_cast<int>(x.kv_heads);
  a.group = a.heads / a.kv_heads, a.tokens = BLK / a.group;
  a.dim = static_cast<int>(x.dim), a.causal = x.causal, a.c = x.scale * kLog2e;
  a.values = static_cast<const bf16*>(x.v.p), a.ldv = x.v.ld, a.hv = x.v.hs;
  a.out = static_cast<bf16*>(const_cast<void*>(x.out.p)), a.ldo = x.out.ld, a.ho = x.out.hs;
  a.lse = x.lse, a.part = static_cast<float*>(ws), a.arrivals = arrivals, a.watch = w;
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
  const int64_t most = tiles * (x.seq.nk / BLK + 1);
  const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min(mc.sms, MAX_SHARES), most)));
  return x.dim <= 64 ? launch_as<64>(a, grid, s) : launch_as<128>(a, grid, s);
}

}  // namespace tpo
