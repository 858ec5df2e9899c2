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
static_assert(MAX_SHARES <= ARRIVALS, "one arrival counter a block");
constexpr float kLog2e = 1.4426950408889634074f, kLn2 = 0.69314718055994530942f;

// ------------------------------------------------------------------ equal shares
//
// A launch's work is a list of tiles (outputs that one block can hold) by
// sequence, key head and position, each of some steps (what it contracts over,
// 128 at a time).  The lengths are known on the device only, and differ: so the
// list is cut by steps into as many equal shares as there are blocks, wherever
// the cuts fall.  A tile that a cut divides is computed in parts, in fp32, which
// the block that arrives last at the tile's counter joins in the shares' order:
// the same bits whoever comes last.  At most one tile begins and does not end
// in a share, and that share's number is the tile's counter.

// A share's place in the list, tile by tile.
struct Walk {
  // the share
  int64_t at, end;  // steps of the whole list
  // where it is
  int seq, head, tile, tiles;
  Seq s;
  int lo, hi;       // the tile's steps
  int64_t begin;    // of the tile, in the list
};

struct Part {
  int lo, hi;           // steps of this share
  bool whole;
  int64_t begin, end;   // of the tile, in the list
};

struct Shares {
  int64_t total;    // steps
  int count;        // shares
  int seq;          // where this block's share begins: sequence,
  int64_t before;   // and steps ahead of the sequence
};

__device__ __forceinline__ int64_t share_begin(const Shares& p, int64_t c) { return c * p.total / p.count; }
// The share that holds step x.
__device__ __forceinline__ int share_of(const Shares& p, int64_t x) {
  return static_cast<int>(((x + 1) * p.count - 1) / p.total);
}

// Steps of all tiles of a sequence (one key head), by a converged warp.
template <class T>
__device__ __forceinline__ int64_t steps_by_warp(const T& t, const Seq& s, int tiles) {
  int64_t sum = 0;
  for (int i = threadIdx.x & 31; i < tiles; i += 32) {
    int lo, hi;
    t.range(s, i, &lo, &hi);
    sum += hi - lo;
  }
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Steps of sequence i over all key heads; every thread of the block calls it,
// with its own i (at or past `batch`: none), and `tiles` gets the tiles' number.
template <class T>
__device__ int64_t cost_of(const T& t, const Sequences& q, int64_t i, int64_t* tiles) {
  Seq s{};
  int n = 0;
  int64_t sum = 0;
  if (i < q.batch) {
    s = sequence(q, i);
    n = t.tiles(s);
    if (n <= 4)
      for (int k = 0; k < n; ++k) {
        int lo, hi;
        t.range(s, k, &lo, &hi);
        sum += hi - lo;
      }
  }
  for (uint32_t many = __ballot_sync(0xffffffffu, n > 4); many; many &= many - 1) {
    const int l = __ffs(many) - 1;
    Seq o;
    o.q0 = 0, o.k0 = 0;
    o.nq = __shfl_sync(0xffffffffu, s.nq, l);
    o.nk = __shfl_sync(0xffffffffu, s.nk, l);
    const int64_t v = steps_by_warp(t, o, __shfl_sync(0xffffffffu, n, l));
    if ((threadIdx.x & 31) == l) sum = v;
  }
  *tiles = static_cast<int64_t>(n) * t.kv_heads;
  return sum * t.kv_heads;
}

struct PlanScratch {
  int64_t warp[32], warp2[32];
  Shares shares;
};

// Inclusive sum over the block's threads; *all gets the block's.
template <int THREADS>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* scratch, int64_t* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int o = 1; o < 32; o *= 2) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  int64_t before = 0, sum = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) before = sum;
    sum += scratch[w];
  }
  *all = sum;
  return v + before;
}

// Cuts the list; every thread of the block takes part.  At least MIN_STEPS a
// share, unless there are more tiles than such shares.
template <int THREADS, class T>
__device__ __noinline__ void plan_shares(const T& t, const Sequences& q, PlanScratch* sc) {
  constexpr int64_t MIN_STEPS = 2;
  int64_t total = 0, tiles = 0, mine = 0, scanned = 0;
  for (int64_t base = 0; base < q.batch; base += THREADS) {
    int64_t n, all;
    mine = cost_of(t, q, base + threadIdx.x, &n);
    scanned = block_scan<THREADS>(mine, sc->warp, &all) + total;
    total += all;
    block_scan<THREADS>(n, sc->warp2, &all);
    tiles += all;
  }
  Shares p;
  p.total = total;
  p.count = static_cast<int>(min(static_cast<int64_t>(gridDim.x), max(max(total / MIN_STEPS, tiles), int64_t(1))));
  p.count = static_cast<int>(min(static_cast<int64_t>(p.count), max(total, int64_t(1))));
  p.seq = p.before = 0;
  if (threadIdx.x == 0) sc->shares = p;
  __syncthreads();
  if (blockIdx.x >= p.count || total == 0) return;
  const int64_t at = share_begin(p, blockIdx.x);
  int64_t ahead = 0;
  for (int64_t base = 0; base < q.batch; base += THREADS) {
    int64_t n, all = total;
    if (q.batch > THREADS) {
      mine = cost_of(t, q, base + threadIdx.x, &n);
      scanned = block_scan<THREADS>(mine, sc->warp, &all) + ahead;
    }
    if (scanned - mine <= at && at < scanned) sc->shares.seq = static_cast<int>(base + threadIdx.x), sc->shares.before = scanned - mine;
    ahead += all;
  }
  __syncthreads();
}

// The first tile of this block's share, by a converged warp.
template <class T>
__device__ void walk_begin(const T& t, const Sequences& q, const Shares& p, Walk& w) {
  w.at = share_begin(p, blockIdx.x);
  w.end = share_begin(p, blockIdx.x + 1);
  if (blockIdx.x >= p.count || p.total == 0) w.at = w.end = 0;
  if (w.at >= w.end) return;
  w.seq = p.seq;
  w.s = sequence(q, w.seq);
  w.tiles = t.tiles(w.s);
  int64_t ahead = p.before;
  const int64_t a_head = w.tiles <= 1 ? 0 : steps_by_warp(t, w.s, w.tiles);
  if (w.tiles <= 1) {
    t.range(w.s, 0, &w.lo, &w.hi);
    w.head = static_cast<int>((w.at - ahead) / (w.hi - w.lo));
    w.tile = 0;
    w.begin = ahead + static_cast<int64_t>(w.head) * (w.hi - w.lo);
    return;
  }
  w.head = static_cast<int>((w.at - ahead) / a_head);
  ahead += a_head * w.head;
  const int lane = threadIdx.x & 31;
  for (int base = 0;; base += 32) {
    int lo = 0, hi = 0;
    if (base + lane < w.tiles) t.range(w.s, base + lane, &lo, &hi);
    int64_t v = hi - lo;
    for (int o = 1; o < 32; o *= 2) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, ahead + v > w.at);
    if (past) {
      const int l = __ffs(past) - 1;
      w.tile = base + l;
      w.lo = __shfl_sync(0xffffffffu, lo, l);
      w.hi = __shfl_sync(0xffffffffu, hi, l);
      w.begin = ahead + __shfl_sync(0xffffffffu, v, l) - (w.hi - w.lo);
      return;
    }
    if (base + 32 >= w.tiles) {  // not reached: the tile exists
      w.end = w.at;
      return;
    }
    ahead += __shfl_sync(0xffffffffu, v, 31);
  }
}
__device__ __forceinline__ bool walk_has(const Walk& w) { return w.at < w.end; }
__device__ __forceinline__ Part walk_part(const Walk& w) {
  Part r;
  r.begin = w.begin;
  r.end = w.begin + (w.hi - w.lo);
  const int64_t stop = w.end < r.end ? w.end : r.end;
  r.lo = w.lo + static_cast<int>(w.at - w.begin);
  r.hi = w.lo + static_cast<int>(stop - w.begin);
  r.whole = r.lo == w.lo && r.hi == w.hi;
  return r;
}
template <class T>
__device__ __forceinline__ void walk_next(const T& t, const Sequences& q, Walk& w) {
  w.begin += w.hi - w.lo;
  w.at = w.begin;
  if (w.at >= w.end) return;
  if (++w.tile == w.tiles) {
    w.tile = 0;
    if (++w.head == t.kv_heads) {
      w.head = 0;
      do {
        if (++w.seq >= q.batch) {  // not reached: steps are left
          w.at = w.end;
          return;
        }
        w.s = sequence(q, w.seq);
        w.tiles = t.tiles(w.s);
      } while (w.tiles == 0);
    }
  }
  t.range(w.s, w.tile, &w.lo, &w.hi);
}

// Where a part of a divided tile goes: two slots a share, the first for the tile that it did not begin.
__device__ __forceinline__ int part_slot(const Walk& w) {
  return 2 * static_cast<int>(blockIdx.x) + (w.at == w.begin ? 1 : 0);
}
__device__ __forceinline__ int tile_slot(int first, int i) { return i == 0 ? 2 * first + 1 : 2 * (first + i); }

// ------------------------------------------------------------------ matrix instructions

// A K-major tile of 128 rows by up to 128 elements: blocks of 64 elements, 128-byte swizzle, 16 KiB each.  Start of
// the 16 elements from 16 k on.
__device__ __forceinline__ uint64_t desc_k(uint64_t d, int k) {
  return d + static_cast<uint64_t>((k >> 2) * (16384 >> 4) + (k & 3) * 2);
}
// The same memory as an MN-major operand (its 128 rows are the contraction): 64 elements further on the next block.
__device__ __forceinline__ uint64_t desc_rows(uint32_t addr) {
  uint64_t v = smem_desc_sw128(addr) & ~(static_cast<uint64_t>(0x3FFF) << 16);
  return v | (static_cast<uint64_t>(16384 >> 4) << 16);
}

// D[tensor memory] (+)= A . B^T, 16 contraction elements, bf16, one elected lane of a converged warp; A in shared
// memory or in tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred E, A;\n\t.reg .b32 r;\n\tsetp.ne.b32 A, %4, 0;\n\telect.sync r|E, 0xffffffff;\n\t"
      "@E tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, A;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred E, A;\n\t.reg .b32 r;\n\tsetp.ne.b32 A, %4, 0;\n\telect.sync r|E, 0xffffffff;\n\t"
      "@E tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, A;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc));
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
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// ------------------------------------------------------------------ host side

// [rows, heads, dim] by boxes of 64 elements, `box_heads` heads and `box_rows` rows (block_maps.cu).
bool encode_heads(CUtensorMap* map, const Heads& x, int64_t rows, int64_t heads, int64_t dim, int box_heads,
                  int box_rows);

}  // namespace tpo
