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
// Roles: warp 0 loads (TMA), warp 1 issues the MMAs, warps 2 and 3 clear V,
// warps 4-7 and 8-11 are the two halves' softmax.

#include <algorithm>
#include <cstring>

#include <cuda_bf16.h>

#include "attn_dev.h"
#include "pdl.h"

namespace tpo {

namespace {

using bf16 = __nv_bfloat16;
constexpr int THREADS = 384;
constexpr int SOFTMAX = 256;             // threads of the two softmax groups
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
  static constexpr int N_BARS = 5 * STAGES + 11;
  static constexpr int SLOT = BARS + 8 * N_BARS;
  static constexpr int LAST = SLOT + 4;
  static constexpr int BAD = SLOT + 8;               // [BAD_SETS][BAD_STEPS][4] keys, a bit each
  static constexpr int ROWS = (BAD + BAD_SETS * BAD_STEPS * 16 + 15) / 16 * 16;  // [2][256] floats: maxima and sums
  static constexpr int JOIN_AT = ROWS + 2048;        // [2][JOIN] floats
  static constexpr int PLAN = JOIN_AT + 8 * JOIN;
  static_assert(JOIN_AT % 16 == 0 && 8 * JOIN >= 8 * 2048, "also a staging box for each warp");
  static constexpr int SMEM = PLAN + static_cast<int>(sizeof(PlanScratch)) + 1024;
  static_assert(SMEM <= 232448, "shared memory of one block");
};

__device__ __forceinline__ void bar_softmax() { asm volatile("bar.sync 1, %0;" ::"n"(SOFTMAX) : "memory"); }

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
  const uint32_t kfull = sbase + L::BARS, kempty = kfull + 8 * L::STAGES, vfull = kempty + 8 * L::STAGES,
                 vempty = vfull + 8 * L::STAGES, qfull = vempty + 16 * L::STAGES, qempty = qfull + 8;
  const bool lead = (threadIdx.x & 31) == 0;
  uint32_t kn = 0, vn = 0, qn = 0;  // loads so far
  bool ok = true;
  Walk w;
  for (walk_begin(tiles, a.seq, sh, w); ok && walk_has(w); walk_next(tiles, a.seq, w)) {
    const Item it = item_of(a, w);
    const int q_head = w.head * a.group;
    if (!(ok = wait_warp(a.watch, qempty, (qn & 1u) ^ 1u, S_EMPTY))) break;
    if (lead) {
      const uint32_t box = static_cast<uint32_t>(a.group * a.tokens) * 128u;
      mbar_expect_tx(qfull, box * (DP / 64) * it.halves);
      for (int h = 0; h < it.halves; ++h)
        for (int d = 0; d < DP / 64; ++d)
          tma_load_3d(sbase + h * L::TILE + d * 16384, &a.q, qfull, d * 64, q_head,
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
          tma_load_3d(base + st * L::TILE + d * 16384, map, full + 8 * st, d * 64, w.head,
                      w.s.k0 + j * BLK);
      }
      __syncwarp();
      ++n;
      return true;
    };
    // K one step ahead of V, as the products take them
    ok = load(&a.k, kfull, kempty, sbase + L::K0, kn, it.p.lo);
    for (int j = it.p.lo; ok && j < it.p.hi; ++j) {
      if (j + 1 < it.p.hi) ok = load(&a.k, kfull, kempty, sbase + L::K0, kn, j + 1);
      if (ok) ok = load(&a.v, vfull, vempty, sbase + L::V0, vn, j);
    }
  }
  if (!ok && lead) {  // what is in flight must land before the block gives up its shared memory
    for (uint32_t j = kn > L::STAGES ? kn - L::STAGES : 0u; j < kn; ++j)
      wait_bar(a.watch, kfull + 8 * (j % L::STAGES), j / L::STAGES & 1u, S_DRAIN, false);
    for (uint32_t j = vn > L::STAGES ? vn - L::STAGES : 0u; j < vn; ++j)
      wait_bar(a.watch, vfull + 8 * (j % L::STAGES), j / L::STAGES & 1u, S_DRAIN, false);
    if (qn) wait_bar(a.watch, qfull, (qn - 1) & 1u, S_DRAIN, false);
  }
  __syncwarp();
}

template <int DP>
__device__ void mma_role(const Args& a, const Tiles& tiles, const Shares& sh, uint32_t sbase, uint32_t tmem) {
  using L = Layout<DP>;
  const uint32_t kfull = sbase + L::BARS, kempty = kfull + 8 * L::STAGES, vfull = kempty + 8 * L::STAGES,
                 vempty = vfull + 8 * L::STAGES, vfix = vempty + 8 * L::STAGES, qfull = vfix + 8 * L::STAGES,
                 qempty = qfull + 8, sfull = qempty + 8, pfull = sfull + 16, ofull = pfull + 32, drain = ofull + 16;
  const int ksteps = (a.dim + 15) / 16;
  const uint32_t idesc_s = idesc_n(make_idesc(false, BLK), BLK);
  const uint32_t idesc_o = idesc_n(make_idesc(false, BLK), ksteps * 16) | 1u << 16;
  const uint64_t dq = smem_desc_sw128(sbase), dk = smem_desc_sw128(sbase + L::K0), dv = desc_rows(sbase + L::V0);
  uint32_t kn = 0, vn = 0, qn = 0, pn0 = 0, pn1 = 0;
  uint32_t fixed[L::STAGES] = {};
  bool ok = true;
  Walk w;
  for (walk_begin(tiles, a.seq, sh, w); ok && walk_has(w); walk_next(tiles, a.seq, w)) {
    const Item it = item_of(a, w);
    const int steps = it.p.hi - it.p.lo, units = it.halves * steps;
    if (!(ok = wait_warp(a.watch, qfull, qn & 1u, S_FULL))) break;
    ++qn;
    // unit u: half (or turn) u & 1 of a step
    auto scores = [&](int u) {
      const bool first = it.halves == 1 || !(u & 1), last = it.halves == 1 || (u & 1);
      const uint32_t st = kn % L::STAGES;
      if (first && !wait_warp(a.watch, kfull + 8 * st, kn / L::STAGES & 1u, S_FULL)) return false;
      tc_fence_after();
      const uint32_t half = u & 1;
      const uint64_t qd = dq + (it.halves == 2 ? half * (L::TILE >> 4) : 0u), kd = dk + st * (L::TILE >> 4);
      mma_head<DP>(tmem + half * BLK, qd, kd, idesc_s, ksteps);
      mma_commit_cg<1>(sfull + 8 * half);
      if (last) mma_commit_cg<1>(kempty + 8 * st), ++kn;
      if (u == units - 1) mma_commit_cg<1>(qempty);
      return true;
    };
    ok = scores(0) && (units < 2 || scores(1));
    for (int u = 0; ok && u < units; ++u) {
      const uint32_t half = u & 1;
      const bool first = it.halves == 1 || !half, last = it.halves == 1 || half;
      const int j = it.p.lo + (it.halves == 1 ? u : u >> 1);
      const uint32_t st = vn % L::STAGES;
      const uint32_t turn = half ? pn1++ : pn0++;
      if (!(ok = wait_warp(a.watch, pfull + 16 * half, turn & 1u, S_FULL))) break;
      if (first) {
        if (!(ok = wait_warp(a.watch, vfull + 8 * st, vn / L::STAGES & 1u, S_FULL))) break;
        if (needs_fix(it, j)) {
          uint32_t n = 0;
#pragma unroll
          for (int i = 0; i < L::STAGES; ++i)
            if (i == static_cast<int>(st)) n = fixed[i]++;
          if (!(ok = wait_warp(a.watch, vfix + 8 * st, n & 1u, S_FULL))) break;
        }
      }
      tc_fence_after();
      const uint64_t vd = dv + st * (L::TILE >> 4);
      const uint32_t p = tmem + half * BLK, o = tmem + 2 * BLK + half * BLK;
      const bool fresh = u < 2;  // this half's first product of the part
      mma4_ts(o, p, vd, idesc_o, !fresh);
      if (!(ok = wait_warp(a.watch, pfull + 16 * half + 8, turn & 1u, S_FULL))) break;
      tc_fence_after();
      mma4_ts(o, p + 64, vd + 512, idesc_o, 1u);
      if (u >= units - 2) mma_commit_cg<1>(ofull + 8 * half);
      if (last) mma_commit_cg<1>(vempty + 8 * st), ++vn;
      if (u + 2 < units) ok = scores(u + 2);
    }
  }
  // also after a failure: every MMA issued must complete before tensor memory is freed
  mma_commit_cg<1>(drain);
  if ((threadIdx.x & 31) == 0) wait_bar(a.watch, drain, 0u, S_DRAIN, false);
  __syncwarp();
}

// Clears the rows of V behind the last key, and takes values that are not finite
// out of rows that only some queries see, noting their keys.
template <int DP>
__device__ void fix_role(const Args& a, const Tiles& tiles, const Shares& sh, uint32_t sbase, uint8_t* smem) {
  using L = Layout<DP>;
  const uint32_t vfull = sbase + L::BARS + 16 * L::STAGES, vempty = vfull + 8 * L::STAGES,
                 vfix = vempty + 8 * L::STAGES;
  const int lane = threadIdx.x & 31, mine = (threadIdx.x >> 5) - 2;  // this warp's rows: 32 mine, and 64 further on
  uint32_t vn = 0, item = 0;
  Walk w;
  for (walk_begin(tiles, a.seq, sh, w); walk_has(w); walk_next(tiles, a.seq, w), ++item) {
    const Item it = item_of(a, w);
    uint32_t* bad = reinterpret_cast<uint32_t*>(smem + L::BAD) + item % BAD_SETS * BAD_STEPS * 4;
    if (lane < 2 * BAD_STEPS) bad[2 * lane + mine] = 0;
    __syncwarp();
    for (int j = it.p.lo; j < it.p.hi; ++j, ++vn) {
      const uint32_t st = vn % L::STAGES;
      if (!wait_warp(a.watch, vfull + 8 * st, vn / L::STAGES & 1u, S_FULL)) return;
      if (needs_fix(it, j)) {
        uint8_t* v = smem + L::V0 + st * L::TILE;
#pragma unroll 1
        for (int g = mine; g < 4; g += 2) {
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
        if (lane == 0) mbar_arrive(vfix + 8 * st);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(vempty + 8 * st);
    }
  }
}

template <int DP>
__device__ void softmax_role(const Args& a, const Tiles& tiles, const Shares& sh, uint32_t sbase, uint8_t* smem,
                             uint32_t tmem) {
  using L = Layout<DP>;
  const uint32_t qempty = sbase + L::BARS + 40 * L::STAGES + 8, sfull = qempty + 8, pfull = sfull + 16,
                 ofull = pfull + 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = warp & 3, half = (warp - 4) >> 2;
  const int row = quad * 32 + lane, me = threadIdx.x - 128;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  const uint32_t ts = lanes + half * BLK, to = lanes + 2 * BLK + half * BLK;
  const int dt = row / a.group, head_in = row - dt * a.group;  // the row's token in its half, its head in the group
  const int chunks = (a.dim + 31) / 32;
  float* rows = reinterpret_cast<float*>(smem + L::ROWS);
  const float2 c2 = make_float2(a.c, a.c);
  uint32_t sn = 0, on = 0, item = 0;
  bool ok = true;
  Walk w;
  for (walk_begin(tiles, a.seq, sh, w); walk_has(w); walk_next(tiles, a.seq, w), ++item) {
    const Item it = item_of(a, w);
    const int steps = it.p.hi - it.p.lo;
    const int t = it.tok + (it.halves == 2 ? half * a.tokens : 0) + dt;
    const bool valid = dt < a.tokens && t < w.s.nq;
    const int limit = valid ? keys_seen(w.s, t, a.causal) : 0;
    const bool idle = __all_sync(0xffffffffu, limit == 0);
    float m = -INFINITY, l = 0.0f;  // the maximum that is subtracted (in powers of two), the sum
    const int first = it.halves == 2 ? 0 : half, by = it.halves == 2 ? 1 : 2;
    for (int i = first; i < steps; i += by, ++sn) {
      if (ok) ok = wait_warp(a.watch, sfull + 8 * half, sn & 1u, S_TFULL);
      auto arrive = [&](uint32_t bar) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      };
      if (!ok || idle) {
        arrive(pfull + 16 * half);
        arrive(pfull + 16 * half + 8);
        continue;
      }
      // Half of the scores at a time, each read twice, first for the maximum: a thread holds 64 of them and not 128, and
      // the code is short (its first pass runs at the speed of the instruction fetches).  A half's weights go over its
      // own columns, and the product with the first half's runs beside the second's.
      uint32_t x[64];
      const int left = limit - (it.p.lo + i) * BLK;
      const bool all = __all_sync(0xffffffffu, left >= BLK);
      auto read = [&](int from) {
        tmem_ld64_sync(ts + from, x);
        if (!all) {
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (from + e >= left) x[e] = 0xff800000u;
        }
      };
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      tc_fence_after();
#pragma unroll 1
      for (int from = 0; from < BLK; from += 64) {
        read(from);
#pragma unroll
        for (int e = 0; e < 64; e += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            top[k] = max3(top[k], __uint_as_float(x[e + 2 * k]), __uint_as_float(x[e + 2 * k + 1]));
      }
      const float peak = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.c;
      const bool grow = peak > m + GROWTH;
      if (__any_sync(0xffffffffu, grow)) {
        const float f = grow ? exp2_fast(m - peak) : 1.0f;  // from -infinity: 0
        if (grow) m = peak;
        l *= f;
        if (i != first) {  // the products before this step's scores are done
#pragma unroll 1
          for (int c = 0; c < 2 * chunks; ++c) {
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
#pragma unroll 1
      for (int from = 0; from < BLK; from += 64) {
        read(from);
        uint32_t h[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 s = fma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), c2, sub2);
          const float2 p = make_float2(exp2_fast(s.x), exp2_fast(s.y));
          sum[e & 1] = add2(sum[e & 1], p);
          h[e] = pack_bf16(p.x, p.y);
        }
        tmem_st32(ts + from, h);
        tmem_wait_st();
        arrive(pfull + 16 * half + from / 8);
      }
      l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
    }
    // ---- the end of the part
    if (steps > first) {
      if (ok) ok = wait_warp(a.watch, ofull + 8 * half, on & 1u, S_TFULL);
      ++on;
    }
    tc_fence_after();
    float w0 = 1.0f, w1 = 0.0f;  // weights of the two accumulators
    const bool two = it.halves == 1 && steps > 1;
    if (it.halves == 1) {  // both groups end with the joined maximum and sum
      rows[half * 256 + row] = m;
      rows[half * 256 + 128 + row] = l;
      bar_softmax();
      tc_fence_after();
      const float m0 = rows[row], l0 = rows[128 + row], m1 = rows[256 + row], l1 = rows[384 + row];
      m = fmaxf(m0, m1);
      w0 = m0 == -INFINITY ? 0.0f : exp2_fast(m0 - m);
      w1 = m1 == -INFINITY ? 0.0f : exp2_fast(m1 - m);
      l = l0 * w0 + l1 * w1;
    }
    const uint32_t* bad = reinterpret_cast<const uint32_t*>(smem + L::BAD) + item % BAD_SETS * BAD_STEPS * 4;
    uint32_t any_bad = 0;
    if (ok && a.causal)
      for (int i = 0; i < BAD_STEPS * 4; ++i) any_bad |= bad[i];
    const int64_t q_row = static_cast<int64_t>(w.s.q0) + t;
    const int head = w.head * a.group + head_in;
    const int prow = it.halves == 2 ? half * BLK + row : row;
    float* part = a.part + static_cast<int64_t>(part_slot(w)) * a.part_rows * (a.dim + 2);
    const float scale = !it.p.whole ? 1.0f : l == 0.0f ? (limit > 0 ? __uint_as_float(0x7fc00000u) : 0.0f) : 1.0f / l;
    uint8_t* stage = smem + L::JOIN_AT + (warp - 4) * 2048;
    const RowsOut to_rows = rows_out(valid && it.p.whole ? a.out + q_row * a.ldo + head * a.ho : nullptr);
    const float f0 = (it.halves == 1 ? w0 : 1.0f) * scale, f1 = w1 * scale;
#pragma unroll 1
    for (int c = it.halves == 1 ? half : 0; ok && c < chunks; c += by) {
      uint32_t o[32];
      float v[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = 0.0f;
      if (!idle) {  // an accumulator that does not count may hold anything
        tmem_ld32_sync((it.halves == 1 ? lanes + 2 * BLK : to) + c * 32, o);
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = f0 == 0.0f ? 0.0f : __uint_as_float(o[e]) * f0;
        if (two) {
          tmem_ld32_sync(lanes + 3 * BLK + c * 32, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] += f1 == 0.0f ? 0.0f : __uint_as_float(o[e]) * f1;
        }
      }
      if (any_bad)  // the noted values, for a row that sees their keys
        for (int i = 0; i < BAD_STEPS * 4; ++i)
          for (uint32_t left = bad[i]; left; left &= left - 1) {
            const int key = it.some / BLK * BLK + 32 * i + __ffs(left) - 1;
            if (key >= limit) continue;
            const bf16* x = a.values + (static_cast<int64_t>(w.s.k0) + key) * a.ldv + w.head * a.hv + c * 32;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float f = c * 32 + e < a.dim ? __bfloat162float(x[e]) : 0.0f;
              if (!isfinite(f)) v[e] += f;
            }
          }
      if (it.p.whole)
        store_rows(stage, v, to_rows, c * 32, a.dim - c * 32);
      else if (valid)
        store_part(part, a.part_rows, prow, v, c * 32, a.dim);
    }
    if (ok && valid && (it.halves == 2 || half == 0)) {
      if (!it.p.whole) {
        float* ml = part + static_cast<int64_t>(a.part_rows) * a.dim;
        ml[prow] = m;
        ml[a.part_rows + prow] = l;
      } else if (a.lse) {
        a.lse[q_row * a.heads + head] = limit > 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
      }
    }
    tc_fence_before();
    if (it.halves == 1) bar_softmax();  // both have read both accumulators, and the rows' sums
    if (it.p.whole) continue;
    // ---- a divided tile: whoever comes last joins its parts
    __threadfence();
    bar_softmax();
    const int from = share_of(sh, it.p.begin), shares = share_of(sh, it.p.end - 1) - from + 1;
    volatile int* last = reinterpret_cast<volatile int*>(smem + L::LAST);
    if (me == 0) {
      const uint32_t before = atomicAdd(a.arrivals + from, ok ? 1u : 0u);
      *last = ok && before + 1 == static_cast<uint32_t>(shares);
      if (*last) a.arrivals[from] = 0;
    }
    bar_softmax();
    if (!*last) {
      bar_softmax();
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
      for (int i = me; i < rows_now * shares; i += SOFTMAX) {
        const int s = i / rows_now, r = i - s * rows_now;
        const float* ml = a.part + tile_slot(from, s) * slot + stats + r0 + r;
        table[r * shares + s] = ml[0];
        table[JOIN + r * shares + s] = ml[a.part_rows];
      }
      bar_softmax();
      for (int r = warp - 4; r < rows_now; r += SOFTMAX / 32) {
        float* tm = table + r * shares;
        float top = -INFINITY, sum = 0.0f;
        for (int s = lane; s < shares; s += 32) top = fmaxf(top, tm[s]);
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float base = top == -INFINITY ? 0.0f : top;
        for (int s = lane; s < shares; s += 32) {
          const float f = exp2_fast(tm[s] - base);
          sum += tm[JOIN + s] * f;
          tm[s] = f;
        }
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        int tok, h;
        if (!place(r0 + r, &tok, &h)) continue;
        const int lim = keys_seen(w.s, tok, a.causal);
        const float inv = lim == 0 ? 0.0f : sum == 0.0f ? __uint_as_float(0x7fc00000u) : 1.0f / sum;
        for (int s = lane; s < shares; s += 32) tm[s] *= inv;
        if (a.lse && lane == 0)
          a.lse[(static_cast<int64_t>(w.s.q0) + tok) * a.heads + h] = lim > 0 ? (top + log2f(sum)) * kLn2 : -INFINITY;
      }
      bar_softmax();
      constexpr int U = 2;  // two groups of eight columns at a time
      const int groups = rows_now * (a.dim / 8);
      for (int i0 = me; i0 < groups; i0 += U * SOFTMAX) {
        float4 v[U][2];
        const float *src[U], *f[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = min(i0 + u * SOFTMAX, groups - 1), g = i / rows_now, r = i - g * rows_now;
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
          const int i = i0 + u * SOFTMAX, g = i / rows_now, r = i - g * rows_now;
          int tok, h;
          if (i < groups && place(r0 + r, &tok, &h))
            *reinterpret_cast<uint4*>(a.out + (static_cast<int64_t>(w.s.q0) + tok) * a.ldo + h * a.ho + g * 8) =
                make_uint4(pack_bf16(v[u][0].x, v[u][0].y), pack_bf16(v[u][0].z, v[u][0].w),
                           pack_bf16(v[u][1].x, v[u][1].y), pack_bf16(v[u][1].z, v[u][1].w));
        }
      }
      bar_softmax();
    }
    bar_softmax();
  }
}

// Grid: one block per SM at most, each an equal share of the steps.
template <int DP>
__global__ void __launch_bounds__(THREADS, 1) fwd_kernel(const __grid_constant__ Args a) {
  using L = Layout<DP>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  grid_dep_launch();
  const int warp = threadIdx.x >> 5;
  PlanScratch* plan = reinterpret_cast<PlanScratch*>(smem + L::PLAN);
  if (threadIdx.x == 0) {
    uint32_t bar = sbase + L::BARS;
    auto init = [&](int n, uint32_t count) {
      for (int i = 0; i < n; ++i, bar += 8) mbar_init(bar, count);
    };
    init(3 * L::STAGES, 1);  // kfull, kempty, vfull
    init(L::STAGES, 3);      // vempty: the products and the two clearing warps
    init(L::STAGES, 2);      // vfix
    init(2, 1);              // qfull, qempty
    init(2, 1);              // sfull
    init(4, 4);              // pfull: the half's warps, 64 keys at a time
    init(2, 1);              // ofull
    init(1, 1);              // drain
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
  const Shares sh = plan->shares;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 0) load_role<DP>(a, tiles, sh, sbase);
    if (warp == 1) mma_role<DP>(a, tiles, sh, sbase, tmem);
    if (warp >= 2) fix_role<DP>(a, tiles, sh, sbase, smem);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    softmax_role<DP>(a, tiles, sh, sbase, smem, tmem);
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
