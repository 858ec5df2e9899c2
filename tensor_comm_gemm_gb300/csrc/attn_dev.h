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

// ------------------------------------------------------------------ waits

// A converged warp's bounded wait.  The first tries (each of which the hardware may hold for a while) cost nothing
// but the instruction itself; the clock is read only when they have failed.
__device__ __forceinline__ bool wait_warp_long(const Watch& w, uint32_t bar, uint32_t parity, uint32_t site) {
  const unsigned long long t0 = gtime();
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
    if ((i & 15u) == 0u) {
      int stop = 0;
      if ((threadIdx.x & 31) == 0) {
        if (*reinterpret_cast<volatile uint32_t*>(w.err) != 0u) {
          stop = 1;
        } else if (gtime() - t0 > w.limit_ns) {
          give_up(w.err, site);
          stop = 1;
        }
      }
      if (__shfl_sync(0xffffffffu, stop, 0)) return false;
    }
  }
}
__device__ __forceinline__ bool wait_warp(const Watch& w, uint32_t bar, uint32_t parity, uint32_t site) {
#pragma unroll 1
  for (int i = 0; i < 8; ++i)
    if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  return wait_warp_long(w, bar, parity, site);
}

// ------------------------------------------------------------------ matrix instructions

// A tile of 128 rows by up to 128 elements lies in blocks of 64 elements, 128-byte swizzle, 16 KiB each.  As a K-major
// operand a block is one of smem_desc_sw128.
// As an MN-major operand (the 128 rows are the contraction): 64 elements further on the next block.
__device__ __forceinline__ uint64_t desc_rows(uint32_t addr) {
  uint64_t v = smem_desc_sw128(addr) & ~(static_cast<uint64_t>(0x3FFF) << 16);
  return v | (static_cast<uint64_t>(16384 >> 4) << 16);
}

// D[tensor memory] (+)= A . B^T over `count` (1 to 4) times 16 contraction elements, bf16; a whole converged warp, in
// which one elected lane issues.  All four in one statement: one at a time, with the descriptors' arithmetic between
// them, an instruction took about 120 cycles to issue, and the tensor core needs 64 for it.
// Both operands K-major in shared memory: a block of 64 elements.
__device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, int count) {
  asm volatile(
      "{\n\t.reg .pred E, A, T, P1, P2, P3;\n\t.reg .b32 r;\n\tsetp.ne.b32 A, %4, 0;\n\tsetp.ne.b32 T, 1, 0;\n\t"
      "elect.sync r|E, 0xffffffff;\n\tsetp.gt.and.s32 P1, %5, 1, E;\n\tsetp.gt.and.s32 P2, %5, 2, E;\n\t"
      "setp.gt.and.s32 P3, %5, 3, E;\n\t"
      "@E tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, A;\n\t"
      "@P1 tcgen05.mma.cta_group::1.kind::f16 [%0], %6, %7, %3, T;\n\t"
      "@P2 tcgen05.mma.cta_group::1.kind::f16 [%0], %8, %9, %3, T;\n\t"
      "@P3 tcgen05.mma.cta_group::1.kind::f16 [%0], %10, %11, %3, T;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(count), "l"(a + 2), "l"(b + 2), "l"(a + 4), "l"(b + 4), "l"(a + 6),
      "l"(b + 6));
}
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
// All of a head's elements: blocks of 64, `ksteps` times 16 of them.
template <int DP>
__device__ __forceinline__ void mma_head(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int ksteps) {
  mma4_ss(d, a, b, idesc, 0u, ksteps);
  if (DP == 128) mma4_ss(d, a + (16384 >> 4), b + (16384 >> 4), idesc, 1u, ksteps - 4);
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

// A warp stores 32 columns of its 32 rows (v: the lane's row) as bf16, through 2 KiB of shared memory at `stage`:
// row by row 64 bytes of a line at a time.  (Each lane storing 16 bytes of its own row costs a cycle of the SM's
// memory pipe for each lane, 7000 for the 256 rows of a tile.)  to[i], where rows (lane / 4 + 8 i) go, 0: nowhere;
// `cols` of the 32 exist.
struct RowsOut {
  uint64_t to[4];
};
__device__ __forceinline__ RowsOut rows_out(const void* mine) {  // mine: the lane's own row, NULL: none
  RowsOut r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.to[i] = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine), ((threadIdx.x & 31) >> 2) + 8 * i);
  return r;
}
__device__ __forceinline__ void store_rows(uint8_t* stage, const float (&v)[32], const RowsOut& r, int col, int cols) {
  const int lane = threadIdx.x & 31, part = lane & 3;
  __syncwarp();  // the chunk before has been read
#pragma unroll
  for (int g = 0; g < 4; ++g)
    *reinterpret_cast<uint4*>(stage + lane * 64 + ((g ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(pack_bf16(v[8 * g], v[8 * g + 1]), pack_bf16(v[8 * g + 2], v[8 * g + 3]),
                   pack_bf16(v[8 * g + 4], v[8 * g + 5]), pack_bf16(v[8 * g + 6], v[8 * g + 7]));
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = (lane >> 2) + 8 * i;
    const uint4 x = *reinterpret_cast<const uint4*>(stage + row * 64 + ((part ^ ((row >> 1) & 3)) << 4));
    if (r.to[i] && part * 8 < cols) *reinterpret_cast<uint4*>(r.to[i] + (col + part * 8) * 2) = x;
  }
}
// Parts of divided tiles lie as [dim / 4][rows][4] floats: a warp's 32 rows side by side.
__device__ __forceinline__ void store_part(float* part, int rows, int row, const float (&v)[32], int col, int dim) {
#pragma unroll
  for (int g = 0; g < 8; ++g)
    if (col + 4 * g < dim)
      *reinterpret_cast<float4*>(part + (static_cast<int64_t>((col >> 2) + g) * rows + row) * 4) =
          make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
}

// ------------------------------------------------------------------ host side

// [rows, heads, dim] by boxes of 64 elements, `box_heads` heads and `box_rows` rows (block_maps.cu).
bool encode_heads(CUtensorMap* map, const Heads& x, int64_t rows, int64_t heads, int64_t dim, int box_heads,
                  int box_rows);

}  // namespace tpo
