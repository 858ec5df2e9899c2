// What the attention kernels share: how a launch's work is cut into equal
// shares, matrix instructions with an operand in tensor memory, and packed fp32
// arithmetic.
#pragma once

#include "attn.h"
#include "block_dev.h"
#include "ptx.h"

namespace tpo {

constexpr int BLK = 128;           // rows of a tile's half, and keys (or queries) of a step
constexpr int MAX_SHARES = 152;    // blocks of a launch
constexpr float kLog2e = 1.4426950408889634074f, kLn2 = 0.69314718055994530942f;

// ------------------------------------------------------------------ equal shares
//
// A launch's work is a list of tiles (outputs that one block can hold) by
// sequence, key head and position, each of some steps (what it contracts over,
// 128 at a time).  The lengths are known on the device only, and differ: so the
// list is cut by steps into as many equal shares as there are blocks, wherever
// the cuts fall.  (A tile counts T::COST more, ahead of its steps: a share of many
// short tiles took twice the time of one of a long tile.)  A tile that a cut
// divides is computed in parts, in fp32, which a second kernel joins in the
// shares' order.  At most one tile begins and does not end in a share, so that
// the share's number is the tile's in that kernel.

// A share's place in the list, tile by tile.
struct Walk {
  int done, left;   // of the share before this tile, and from here on
  int off;          // of the tile, that earlier shares have
  int seq, head, tile, tiles;
  Seq s;
  int lo, hi;       // the tile's steps, lo with its cost ahead of them
};
// The share's steps of a tile.
struct Part {
  int lo, hi;  // none where the share has but the tile's cost
  bool whole;
};

struct Shares {
  int total, each;      // steps (and tiles' costs) in all and of a share; the first `more` have one more
  int count, more;
  int at, end;          // this block's share
  int seq;              // where it begins: sequence,
  int before;           // steps ahead of the sequence,
  int a_head;           // and steps of one of its key heads
  Seq s;
};

__device__ __forceinline__ int share_begin(const Shares& p, int c) { return c * p.each + min(c, p.more); }
// The share that holds step x.
__device__ __forceinline__ int share_of(const Shares& p, int x) {
  const int longer = p.more * (p.each + 1);
  const bool in = x < longer;
  return (in ? 0 : p.more) + static_cast<int>(static_cast<uint32_t>(in ? x : x - longer) / static_cast<uint32_t>(p.each + (in ? 1 : 0)));
}

constexpr int PLAN_SEQS = 512;  // sequences at a time, at most as many as the block's threads
struct PlanScratch {
  int steps[32], tiles[32];  // of a warp's sequences
  int longer;                // sequences of more than one tile: their number, their lengths and then their steps
  int nq[PLAN_SEQS], nk[PLAN_SEQS];
};

// The sum of a warp's 32 values, none of them negative, held at 2^31.
__device__ __forceinline__ uint32_t sum_held(int v) {
  const uint32_t lo = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v) & 0xffffu);
  const uint32_t hi = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v) >> 16) + (lo >> 16);
  return hi >> 15 ? 1u << 31 : hi << 16 | (lo & 0xffffu);
}

// Steps of sequence i for one key head; every thread of the block calls it, with
// its own i (at or past `batch`: none).  Held at 2^31 - 1.  *s gets the sequence,
// *tiles the tiles' number.  A thread counts a single tile itself; those of longer
// sequences are counted by a warp each.
template <int THREADS, class T>
__device__ __forceinline__ int cost_of(const T& t, const Sequences& q, int64_t i, Seq* s, int* tiles, PlanScratch* sc) {
  static_assert(THREADS <= PLAN_SEQS, "a place for each thread's sequence");
  *s = Seq{0, 0, 0, 0};
  if (i < q.batch) *s = sequence(q, i);
  const int n = i < q.batch ? t.tiles(*s) : 0;
  int sum = 0, at = 0, lo, hi;
  if (threadIdx.x == 0) sc->longer = 0;
  __syncthreads();
  if (n == 1) t.range(*s, 0, &lo, &hi), sum = hi - lo + T::COST;
  if (n > 1) {
    at = atomicAdd(&sc->longer, 1);
    sc->nq[at] = s->nq, sc->nk[at] = s->nk;
  }
  __syncthreads();
#pragma unroll 1
  for (int k = threadIdx.x >> 5; k < sc->longer; k += THREADS / 32) {
    const Seq o{0, sc->nq[k], 0, sc->nk[k]};
    const int count = t.tiles(o);
    int64_t v = 0;
#pragma unroll 1
    for (int j = threadIdx.x & 31; j < count; j += 32) t.range(o, j, &lo, &hi), v += hi - lo + T::COST;
    const uint32_t held = sum_held(static_cast<int>(min(v, static_cast<int64_t>(INT_MAX))));
    if ((threadIdx.x & 31) == 0) sc->nq[k] = static_cast<int>(min(held, static_cast<uint32_t>(INT_MAX)));
  }
  __syncthreads();
  if (n > 1) sum = sc->nq[at];
  *tiles = n;
  return sum;
}

// Cuts the list; every thread of the block takes part.  At least MIN_STEPS a
// share, unless there are more tiles than such shares.  Steps are counted in 32
// bits: more than MAX_STEPS are found here, reported, and nothing is done.  The scratch
// is free at the end.
template <int THREADS, class T>
__device__ __forceinline__ void plan_shares(const T& t, const Sequences& q, PlanScratch* sc, Shares* shares, uint32_t* err) {
  constexpr int MIN_STEPS = 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, block = blockIdx.x;
  int mine = 0, upto = 0;  // steps of this thread's sequence, and with those of the block's threads before it
  Seq s;
  Shares p{};
  // first all steps and tiles; then, once the share is known, where it begins (another scan, if there are more
  // sequences than threads)
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    int ahead = 0, tiles = 0;
    bool over = false;
#pragma unroll 1
    for (int64_t base = 0; base < q.batch; base += THREADS) {
      int all = 0;
      if (pass == 0 || q.batch > THREADS) {
        int n;
        mine = cost_of<THREADS>(t, q, base + threadIdx.x, &s, &n, sc);
        n = __reduce_add_sync(0xffffffffu, n);
        upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const int u = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += u;
        }
        const uint32_t held = __any_sync(0xffffffffu, mine == INT_MAX) ? 1u << 31 : sum_held(mine);
        __syncthreads();
        if (lane == 31) sc->steps[warp] = held >> 31 ? -1 : upto, sc->tiles[warp] = n;
        __syncthreads();
        const int w_steps = lane < THREADS / 32 ? sc->steps[lane] : 0;
        over = over || __any_sync(0xffffffffu, w_steps < 0) ||
               ahead + static_cast<uint64_t>(sum_held(max(w_steps, 0))) * t.kv_heads > MAX_STEPS;
        upto += __reduce_add_sync(0xffffffffu, lane < warp ? w_steps : 0);
        all = __reduce_add_sync(0xffffffffu, w_steps);
        tiles += __reduce_add_sync(0xffffffffu, lane < THREADS / 32 ? sc->tiles[lane] : 0);
      }
      if (pass == 1) {
        const int from = ahead + (upto - mine) * t.kv_heads;
        if (from <= p.at && p.at < from + mine * t.kv_heads) {
          shares->seq = static_cast<int>(base + threadIdx.x);
          shares->before = from;
          shares->a_head = mine;
          shares->s = s;
        }
      }
      ahead += all * t.kv_heads;
    }
    if (pass == 0) {
      if (over) {
        ahead = 0;
        if (block == 0 && threadIdx.x == 0) give_up(err, S_STEPS);
      }
      p.total = ahead;
      tiles *= t.kv_heads;
      const int steps = ahead - tiles * T::COST;
      // where the tiles are long their costs have shares of their own, so that no other has more than MIN_STEPS
      const int most = (steps >= 8 * static_cast<int64_t>(tiles) ? ahead : steps) / MIN_STEPS;
      p.count = max(1, min(min(static_cast<int>(gridDim.x), steps), max(most, tiles)));
      p.each = p.total / p.count;
      p.more = p.total - p.each * p.count;
      if (block < p.count && p.total > 0) p.at = share_begin(p, block), p.end = share_begin(p, block + 1);
      if (threadIdx.x == 0) *shares = p;
    }
    __syncthreads();
    if (p.at >= p.end) return;
  }
}

// The first tile of this block's share, by a converged warp.
template <class T>
__device__ __forceinline__ void walk_begin(const T& t, const Shares& p, Walk& w) {
  w.done = 0;
  w.left = p.end - p.at;
  if (w.left <= 0) return;
  w.seq = p.seq;
  w.s = p.s;
  w.tiles = t.tiles(w.s);
  w.head = (p.at - p.before) / p.a_head;
  int ahead = p.before + p.a_head * w.head;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int base = 0; base < w.tiles; base += 32) {
    int lo = 0, hi = 0;
    if (base + lane < w.tiles) t.range(w.s, base + lane, &lo, &hi);
    if (hi > lo) lo -= T::COST;
    int v = hi - lo;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, ahead + v > p.at);
    if (past) {
      const int l = __ffs(past) - 1;
      w.tile = base + l;
      w.lo = __shfl_sync(0xffffffffu, lo, l);
      w.hi = __shfl_sync(0xffffffffu, hi, l);
      w.off = p.at - ahead - __shfl_sync(0xffffffffu, v, l) + (w.hi - w.lo);
      return;
    }
    ahead += __shfl_sync(0xffffffffu, v, 31);
  }
  w.left = 0;  // not reached: the tile exists
}
__device__ __forceinline__ bool walk_has(const Walk& w) { return w.left > 0; }
template <class T>
__device__ __forceinline__ Part walk_part(const Walk& w) {
  Part r;
  r.lo = w.lo + max(w.off, T::COST);
  r.hi = min(w.hi, w.lo + w.off + w.left);
  r.whole = w.off <= T::COST && r.hi == w.hi;
  return r;
}
// The next tile, by a converged warp.
template <class T>
__device__ __forceinline__ void walk_next(const T& t, const Sequences& q, Walk& w) {
  const int steps = w.hi - w.lo - w.off;
  w.done += steps;
  w.left -= steps;
  w.off = 0;
  if (w.left <= 0) return;
  if (++w.tile == w.tiles) {
    w.tile = 0;
    if (++w.head == t.kv_heads) {
      w.head = 0;
      // the next sequence with tiles, 32 at a time: a captured call's batch may be mostly slots without queries, and the
      // other roles' waits are running (one at a time a million of them took more than 100 ms)
      const int lane = threadIdx.x & 31;
      uint32_t some = 0;
#pragma unroll 1
      for (w.seq += 1; w.seq < q.batch; w.seq += 32) {
        const bool there = w.seq + lane < q.batch;
        w.s = Seq{0, 0, 0, 0};
        if (there) w.s = sequence(q, w.seq + lane);
        w.tiles = there ? t.tiles(w.s) : 0;
        some = __ballot_sync(0xffffffffu, w.tiles > 0);
        if (some) break;
      }
      if (!some) {  // not reached: steps are left
        w.left = 0;
        return;
      }
      const int l = __ffs(some) - 1;
      w.seq += l;
      w.s.q0 = __shfl_sync(0xffffffffu, w.s.q0, l), w.s.nq = __shfl_sync(0xffffffffu, w.s.nq, l);
      w.s.k0 = __shfl_sync(0xffffffffu, w.s.k0, l), w.s.nk = __shfl_sync(0xffffffffu, w.s.nk, l);
      w.tiles = __shfl_sync(0xffffffffu, w.tiles, l);
    }
  }
  t.range(w.s, w.tile, &w.lo, &w.hi);
  w.lo -= T::COST;
}

// Where a part of a divided tile goes: two slots a share, the first for the tile that it did not begin.
template <class T>
__device__ __forceinline__ int part_slot(const Walk& w) { return 2 * static_cast<int>(blockIdx.x) + (w.off <= T::COST ? 1 : 0); }
// The first of the shares that have a part of the tile that begins at step `begin`, and their number.
__device__ __forceinline__ int tile_shares(const Shares& p, int begin, int steps, int* first) {
  *first = share_of(p, begin);
  return share_of(p, begin + steps - 1) - *first + 1;
}
template <class T>
__device__ __forceinline__ int tile_begin(const Shares& p, const Walk& w) { return p.at + w.done - w.off + T::COST; }
__device__ __forceinline__ int tile_slot(int first, int i) { return i == 0 ? 2 * first + 1 : 2 * (first + i); }

// For the kernels that join: parts s up to `end`, eight, four or two at a time, so that their loads are in flight
// together and few are made for nothing: two or three parts of a long causal prompt's tile take one round, the ten or
// eleven of a short prompt over a long cache two, and so do the nine of a slice of a single token's.
template <int U>
struct Count {
  static constexpr int value = U;
};
template <class F>
__device__ __forceinline__ void some_parts(int s, int end, F f) {
#pragma unroll 1
  while (end - s > 4) f(Count<8>{}, s), s += 8;
  if (end - s > 2)
    f(Count<4>{}, s);
  else if (end > s)
    f(Count<2>{}, s);
}

// ------------------------------------------------------------------ waits

// A converged warp's bounded wait, in few instructions: the kernels' roles share the instruction cache, and a kernel
// that outgrows it runs at the speed of its misses (with 320 KB of code a tile's stores took 8000 cycles, with 130 KB
// 4000).  So what a wait does when it has lasted long is one function.
static __device__ __noinline__ bool waited_long(unsigned long long t0, unsigned long long limit_ns, uint32_t* err, uint32_t site) {
  const bool late = gtime() - t0 > limit_ns;
  const bool over = __any_sync(0xffffffffu, late || *reinterpret_cast<volatile uint32_t*>(err) != 0u);
  if (over && late && (threadIdx.x & 31) == 0) give_up(err, site);
  return over;
}
__device__ __forceinline__ bool wait_warp(const Watch& w, uint32_t bar, uint32_t parity, uint32_t site) {
  if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  const unsigned long long t0 = gtime();
#pragma unroll 1
  while (!__all_sync(0xffffffffu, mbar_test(bar, parity)))
    if (waited_long(t0, w.limit_ns, w.err, site)) return false;
  return true;
}

// A value that the compiler must take as new here: it makes no copies of a loop for each of its values.
__device__ __forceinline__ void anew(int& v) { asm volatile("" : "+r"(v)); }

// ------------------------------------------------------------------ items
//
// The loading warp walks over the share and hands its tiles to the other roles
// through a ring in shared memory.  It needs no wait for free entries: it loads at
// most two parts ahead of the products, which are at most two ahead of the stores.

struct Entry {
  Seq s;
  int head, tile, lo, hi;  // the share's steps of the tile; none: the end
  int from, shares;        // the shares that have parts of it (1: it is whole)
  int slot;                // where a part goes
  int begins;              // this share has the first of them
};
constexpr int RING = 8;
constexpr int64_t BEGUN_BYTES = (MAX_SHARES * 48ll + 255) / 256 * 256;  // an entry for each share in the workspace
static_assert(sizeof(Entry) == 48, "three 16-byte words");

// By the loading warp: entry n of the ring; `w` has no more: the end.  begun: a place in the workspace for each share.
template <class T>
__device__ __forceinline__ Entry put_item(const Shares& sh, const Walk& w, uint8_t* ring, uint32_t full, uint32_t n,
                                          Entry* begun, bool* open) {
  Entry e;
  e.s = w.s, e.head = w.head, e.tile = w.tile;
  e.lo = e.hi = 0, e.from = 0, e.shares = 1, e.slot = 0, e.begins = 0;
  if (walk_has(w)) {
    const Part p = walk_part<T>(w);
    e.lo = p.lo, e.hi = p.hi;
    if (!p.whole && p.hi > p.lo) {
      e.shares = tile_shares(sh, tile_begin<T>(sh, w), w.hi - w.lo - T::COST, &e.from);
      e.slot = part_slot<T>(w);
      e.begins = w.off <= T::COST;
    }
  }
  if ((threadIdx.x & 31) == 0) {
    int4* to = reinterpret_cast<int4*>(ring + n % RING * sizeof(Entry));
    const int4 x = make_int4(e.s.q0, e.s.nq, e.s.k0, e.s.nk), y = make_int4(e.head, e.tile, e.lo, e.hi),
               z = make_int4(e.from, e.shares, e.slot, e.begins);
    to[0] = x, to[1] = y, to[2] = z;
    mbar_arrive(full + 8 * (n % RING));
    // for the kernel that joins: the tile that this share begins and does not end, or at its end that there is none
    if (e.begins || (e.hi <= e.lo && !*open)) {
      to = reinterpret_cast<int4*>(begun + blockIdx.x);
      to[0] = x, to[1] = y, to[2] = z;
    }
  }
  *open |= e.begins != 0;
  __syncwarp();
  return e;
}
// By the others: false at the end, or if the wait ran out.
__device__ __forceinline__ bool get_item(const Watch& w, const uint8_t* ring, uint32_t full, uint32_t n, Entry* e) {
  if (!wait_warp(w, full + 8 * (n % RING), n / RING & 1u, S_FULL)) return false;
  const int4* from = reinterpret_cast<const int4*>(ring + n % RING * sizeof(Entry));
  const int4 a = from[0], b = from[1], c = from[2];
  e->s = {a.x, a.y, a.z, a.w};
  e->head = b.x, e->tile = b.y, e->lo = b.z, e->hi = b.w;
  e->from = c.x, e->shares = c.y, e->slot = c.z, e->begins = c.w;
  return e->hi > e->lo;
}

// ------------------------------------------------------------------ matrix instructions

// A tile of 128 rows by up to 128 elements lies in blocks of 64 elements, 128-byte swizzle, 16 KiB each.  As a K-major
// operand a block is one of smem_desc_sw128.
// As an MN-major operand (the 128 rows are the contraction): 64 elements further on the next block.
__device__ __forceinline__ uint64_t desc_rows(uint32_t addr) {
  uint64_t v = smem_desc_sw128(addr) & ~(static_cast<uint64_t>(0x3FFF) << 16);
  return v | (static_cast<uint64_t>(16384 >> 4) << 16);
}

// D[tensor memory] (+)= A . B^T over four times 16 contraction elements, bf16; a whole converged warp, in which one
// elected lane issues.  All four in one statement, as mma_kblock: one at a time, with the descriptors' arithmetic
// between them, an instruction took about 120 cycles to issue, and the tensor core needs 64 for it.
// A in tensor memory (8 columns each time), B MN-major (16 rows each time): 64 contraction elements.
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred E, A, T;\n\t.reg .b32 r;\n\tsetp.ne.b32 A, %4, 0;\n\tsetp.ne.b32 T, 1, 0;\n\t"
      "elect.sync r|E, 0xffffffff;\n\t"
      "@E tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, A;\n\t"
      "@E tcgen05.mma.cta_group::1.kind::f16 [%0], [%5], %6, %3, T;\n\t"
      "@E tcgen05.mma.cta_group::1.kind::f16 [%0], [%7], %8, %3, T;\n\t"
      "@E tcgen05.mma.cta_group::1.kind::f16 [%0], [%9], %10, %3, T;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(a + 8), "l"(b + 128), "r"(a + 16), "l"(b + 256), "r"(a + 24),
      "l"(b + 384));
}
// All of a head's elements: blocks of 64, whole (the loads fill what a head lacks with zeros).
template <int DP>
__device__ __forceinline__ void mma_head(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  mma_kblock<1, false>(d, a, b, idesc, 0u);
  if (DP == 128) mma_kblock<1, false>(d, a + (16384 >> 4), b + (16384 >> 4), idesc, 1u);
}

// 128 columns, loaded and waited for in one statement.
__device__ __forceinline__ void tmem_ld128_sync(uint32_t taddr, uint32_t (&x)[64], uint32_t (&y)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%128];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
      "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, "
      "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
      "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%129];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]),
        "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]),
        "=r"(x[16]), "=r"(x[17]), "=r"(x[18]), "=r"(x[19]), "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]),
        "=r"(x[24]), "=r"(x[25]), "=r"(x[26]), "=r"(x[27]), "=r"(x[28]), "=r"(x[29]), "=r"(x[30]), "=r"(x[31]),
        "=r"(x[32]), "=r"(x[33]), "=r"(x[34]), "=r"(x[35]), "=r"(x[36]), "=r"(x[37]), "=r"(x[38]), "=r"(x[39]),
        "=r"(x[40]), "=r"(x[41]), "=r"(x[42]), "=r"(x[43]), "=r"(x[44]), "=r"(x[45]), "=r"(x[46]), "=r"(x[47]),
        "=r"(x[48]), "=r"(x[49]), "=r"(x[50]), "=r"(x[51]), "=r"(x[52]), "=r"(x[53]), "=r"(x[54]), "=r"(x[55]),
        "=r"(x[56]), "=r"(x[57]), "=r"(x[58]), "=r"(x[59]), "=r"(x[60]), "=r"(x[61]), "=r"(x[62]), "=r"(x[63]),
        "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3]), "=r"(y[4]), "=r"(y[5]), "=r"(y[6]), "=r"(y[7]),
        "=r"(y[8]), "=r"(y[9]), "=r"(y[10]), "=r"(y[11]), "=r"(y[12]), "=r"(y[13]), "=r"(y[14]), "=r"(y[15]),
        "=r"(y[16]), "=r"(y[17]), "=r"(y[18]), "=r"(y[19]), "=r"(y[20]), "=r"(y[21]), "=r"(y[22]), "=r"(y[23]),
        "=r"(y[24]), "=r"(y[25]), "=r"(y[26]), "=r"(y[27]), "=r"(y[28]), "=r"(y[29]), "=r"(y[30]), "=r"(y[31]),
        "=r"(y[32]), "=r"(y[33]), "=r"(y[34]), "=r"(y[35]), "=r"(y[36]), "=r"(y[37]), "=r"(y[38]), "=r"(y[39]),
        "=r"(y[40]), "=r"(y[41]), "=r"(y[42]), "=r"(y[43]), "=r"(y[44]), "=r"(y[45]), "=r"(y[46]), "=r"(y[47]),
        "=r"(y[48]), "=r"(y[49]), "=r"(y[50]), "=r"(y[51]), "=r"(y[52]), "=r"(y[53]), "=r"(y[54]), "=r"(y[55]),
        "=r"(y[56]), "=r"(y[57]), "=r"(y[58]), "=r"(y[59]), "=r"(y[60]), "=r"(y[61]), "=r"(y[62]), "=r"(y[63])
      : "r"(taddr), "r"(taddr + 64)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16_sync(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ------------------------------------------------------------------ arithmetic

// 2^x by the special function unit, 2^-22 of the value: below the 2^-8 of a weight's rounding to bf16, and of either sign in
// the sums.  Results below 2^-126 become 0: of a row's weights the largest is 1 to 2^8.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// (a.x b.x + c.x, a.y b.y + c.y) and (a.x + b.x, a.y + b.y), two fp32 operations at a time.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// The largest of three; NaN only if all are.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// ------------------------------------------------------------------ results

// A warp stores 32 columns of its 32 rows as bf16 through 2 KB of shared memory at `stage`, row by row: lines of 64
// bytes.  (Each lane storing 16 bytes of its own row costs a cycle of the SM's memory pipe for each lane, 7000 for the 256
// rows of a tile.)  First each lane brings its own row, eight columns from 8 g on at a time; then `mine`, the lane's row
// in global memory (NULL: none), gets columns [col, col + 32), of which `cols` exist.
__device__ __forceinline__ uint32_t stage_at(int row, int g) { return row * 64 + ((g ^ ((row >> 1) & 3)) << 4); }
__device__ __forceinline__ void stage_row(uint8_t* stage, int g, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(stage + stage_at(threadIdx.x & 31, g)) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store_staged(const uint8_t* stage, const void* mine, int col, int cols) {
  const int lane = threadIdx.x & 31, part = lane % 4;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = lane / 4 + 8 * i;
    const uint64_t to = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine), row);
    const uint4 x = *reinterpret_cast<const uint4*>(stage + stage_at(row, part));
    if (to && part * 8 < cols) *reinterpret_cast<uint4*>(to + (col + part * 8) * 2) = x;
  }
  __syncwarp();  // before the next columns
}
// Parts of divided tiles lie as [dim / 4][rows][4] floats: a warp's 32 rows side by side.  Eight columns from col on.
__device__ __forceinline__ void store_part(float* part, int rows, int row, const float (&v)[8], int col, int dim) {
  if (col >= dim) return;
  float* p = part + (static_cast<int64_t>(col >> 2) * rows + row) * 4;
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + static_cast<int64_t>(rows) * 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// ------------------------------------------------------------------ host side

// [rows, heads, dim] by boxes of 64 elements, `box_heads` heads and `box_rows` rows (block_maps.cu).
bool encode_heads(CUtensorMap* map, const Heads& x, int64_t rows, int64_t heads, int64_t dim, int box_heads,
                  int box_rows);

}  // namespace tpo
