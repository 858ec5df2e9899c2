// Matrix products of the block operators on CTA pairs (sm_103a).
//
// A persistent kernel: each pair of CTAs computes tiles of 256 rows by up to
// 256 columns with the 2-SM tcgen05.mma (each CTA holds 128 rows of A and half
// of the B tile; fp32 accumulators in tensor memory, two of them, so that one
// tile's epilogue runs beside the next one's MMAs).  Warp 0 issues the TMA
// loads, warp 1 of the even CTA the MMAs, warps 2 to 9 the epilogue.
//
// One launch runs up to three products one tile list after another, so that
// the gradients of a layer (dx, and the weights' gradients) share one tail.
// Operands may be K-major (rows of contraction elements) or MN-major (the
// transposed matrix as it lies in memory), per product: both are loaded with
// the 128-byte swizzle, as [rows][64 contraction elements] or as blocks of
// [64 contraction rows][64 elements], and the MMA's descriptors say which.
//
// Bound by the tensor cores, and in a row of calls by the power limit, which
// lowers the clock.  4096^3 takes 86 us in a row of calls (1.60 PFLOP/s), with
// bias, GELU and z 92 there and 77 to 85 as a single launch under the profiler
// (tensor pipe 84 % busy); dx and dw of that layer in one launch 163 in a row
// (1.69) and 140 to 148 single (93 %); the gradients of gate and up of
// 3584 x 8192 from 8192 tokens 992 to 1043 single (1.85 to 1.94, 98 %; 1.7 in a
// row).  What is lost is the start (the first loads' latency, ~2 us), the last
// tile's epilogue (~4 us) and the last round's idle pairs, which plan_width
// trades against the higher cost per column of narrower tiles.  The loads are
// issued by a converged warp, one elected lane: from a thread of a diverged warp
// a TMA load cost 80 to 270 cycles and bounded every shape.
//
// Every wait is bounded by the device global timer (option wait_timeout_ms); on
// expiry the waiting thread records it in the handle's error word and the CTA
// winds down.

#include <algorithm>
#include <cstring>

#include "act.h"
#include "block.h"
#include "block_dev.h"
#include "ptx.h"

namespace tpo {

namespace {

constexpr int TM = 128;              // rows of one CTA; a pair's tile has 256
constexpr int TN = 256;              // most columns of a tile (accumulator width)
constexpr int A_BYTES = TM * KB;     // 16 KiB
constexpr int MAX_STAGES = 12;       // pipeline stages: an A block and half of the tile's B rows each
constexpr int EPI_WARPS_N = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS_N;
constexpr int CHUNK = 32;                   // columns of one epilogue step
constexpr int BOX = 32 * CHUNK * 2;         // bytes of one output box: 32 rows of 64 bytes
// The plain epilogue of products with few K blocks (weight gradients of few
// tokens), which the stores bound, takes 64 columns at a time, boxes of
// 128-byte rows, and gives a pipeline stage up for them: 4096x4096 from 16
// tokens 12.4 us, 12.7 with the narrow boxes; with 64 K blocks 91.4 and 90.0.
constexpr int STAGES_NARROW = 196608, STAGES_WIDE = 163840;  // bytes of pipeline stages
constexpr int OFF_BARS = STAGES_NARROW + EPI_WARPS_N * 2 * BOX;  // behind the staging boxes, two a warp
static_assert(OFF_BARS == STAGES_WIDE + EPI_WARPS_N * 2 * 2 * BOX, "one layout behind the stages and boxes");
constexpr int WIDE_KB = 16;  // K blocks of a product up to which its launch takes the wide boxes
constexpr int N_BARS = 2 * MAX_STAGES + 2 + 2 + 1;
constexpr int OFF_TMEM = OFF_BARS + 8 * N_BARS;
// Behind the tensor memory's address: whether a wait of the pair ran out, and
// (in the even CTA) the K blocks that it and its peer have loaded.
constexpr int OFF_FAILED = OFF_TMEM + 4, OFF_LOADED = OFF_TMEM + 8;
constexpr int SMEM = OFF_TMEM + 16 + 1024;  // and the slack to align the base
static_assert(SMEM <= 232448, "shared memory of one CTA");

// An output matrix: its maps for tensor stores (boxes of 32 and 64 columns), and its address for ragged edges.
struct OutMat {
  CUtensorMap map, wide;
  __nv_bfloat16* p;
  int64_t ld;
};
struct Prob {
  CUtensorMap a[2], b[2];
  OutMat y;
  int M, N;
  int tiles_m, tiles;   // row tiles, tiles in all
  int w;                // columns of a tile (EPI_GATED: of h; the accumulator has twice as many)
  int terms, kb_seg, kb;  // K blocks per term and in all
  int a_mn, b_mn;
};
struct Args {
  Prob q[3];
  OutMat y1, y2;
  int count, total;
  uint32_t stages, stage_bytes;
  int wide;             // 64-column boxes
  int act;
  const __nv_bfloat16 *bias, *residual;
  int64_t ldr;
  int bias_vec;         // the bias is 16-byte aligned
  int has1;             // y1 (and for EPI_GATED y2) are stored
  const float *sx, *sw0, *sw1;
  Watch watch;
};

struct TileAt {
  int q, row, col;
};
// Tile t of the launch: products in order; within one, groups of 8 row tiles
// are swept column by column, rows fastest, so that the tiles in flight share
// their B tiles and a group's A rows stay in L2 over the sweep.
__device__ __forceinline__ TileAt tile_at(const Args& p, int t) {
  TileAt o;
  o.q = 0;
  while (t >= p.q[o.q].tiles) t -= p.q[o.q++].tiles;
  const Prob& q = p.q[o.q];
  const int cols = q.tiles / q.tiles_m;
  const int grp = t / (8 * cols), first = grp * 8;
  const int rows = min(8, q.tiles_m - first);
  const int in = t - grp * 8 * cols;
  o.row = (first + in % rows) * (2 * TM);
  o.col = in / rows * q.w;
  return o;
}

struct Ring {  // the load warp's place in the pipeline
  uint32_t stage, phase, armed;
  uint32_t stages, bytes;  // stages of the ring, bytes of each
};

// Loads one tile's K blocks.  AMN: A is MN-major; BN_BOXES: MN-major boxes of
// this CTA's share of B (0: B is K-major).  A stage is one A block and one B
// block; the pair's bytes are expected on the even CTA's barrier.
template <bool FP8, bool AMN, int BN_BOXES>
__device__ __forceinline__ bool load_tile(const Args& p, Ring& g, uint32_t sbase, uint32_t full0, uint32_t full_lead,
                                          uint32_t empty0, uint32_t lead, uint32_t bytes, const CUtensorMap* ma,
                                          const CUtensorMap* mb, int terms, int kb_seg, int a0, int b0) {
  constexpr int KEL = FP8 ? KB : KB / 2;
  constexpr int NA = AMN ? 2 : 1, NB = BN_BOXES ? BN_BOXES : 1;
  for (int seg = 0; seg < terms; ++seg, ++ma, ++mb) {
    [[maybe_unused]] const uint64_t map_a = reinterpret_cast<uint64_t>(ma), map_b = reinterpret_cast<uint64_t>(mb);
    int kx = 0;
    for (int kk = 0; kk < kb_seg; ++kk, kx += KEL) {
      if (!wait_bar_warp(p.watch, empty0 + 8u * g.stage, g.phase ^ 1u, S_EMPTY)) return false;
      const uint32_t sa = sbase + g.stage * g.bytes, sb = sa + A_BYTES;
      Box x[NA + NB];
      if constexpr (AMN) {
        x[0] = {sa, map_a, a0, kx};
        x[1] = {sa + 8192u, map_a, a0 + 64, kx};
      } else {
        x[0] = {sa, map_a, kx, a0};
      }
      if constexpr (BN_BOXES > 0) {
        x[NA] = {sb, map_b, b0, kx};
        if constexpr (BN_BOXES > 1) x[NA + 1] = {sb + 8192u, map_b, b0 + 64, kx};
      } else {
        x[NA] = {sb, map_b, kx, b0};
      }
      stage_loads<2>(lead, full0 + 8u * g.stage, bytes, full_lead + 8u * g.stage, x);
      ++g.armed;
      if (++g.stage == g.stages) g.stage = 0, g.phase ^= 1u;
    }
  }
  return true;
}

// Bytes that one CTA loads for a K block.
template <int KIND>
__device__ __forceinline__ uint32_t kblock_bytes(const Prob& q) {
  if constexpr (KIND == EPI_GATED) return A_BYTES + q.w * KB;
  const int hb = q.w / 2;
  return A_BYTES + (q.b_mn ? (hb + 63) / 64 * 8192u : static_cast<uint32_t>(hb) * KB);
}

// Tells both CTAs of the pair that a wait ran out (one thread).
__device__ __forceinline__ void mark_failed(uint32_t sbase) {
  st_shared_cluster_u32(map_to_rank(sbase + OFF_FAILED, 0), 1u);
  st_shared_cluster_u32(map_to_rank(sbase + OFF_FAILED, 1), 1u);
}

// The load warp, converged (one elected lane issues each stage's loads).
template <int KIND, bool FP8>
__device__ void load_role(const Args& p, uint32_t sbase, uint32_t full0, uint32_t empty0, uint32_t rank, int pair,
                          int pairs) {
  const uint32_t full_lead = map_to_rank(full0, 0), lead = rank == 0 ? 1u : 0u;
  Ring g{0, 0, 0, p.stages, p.stage_bytes};
  bool ok = true;
  for (int t = pair; ok && t < p.total; t += pairs) {
    const TileAt T = tile_at(p, t);
    const Prob& q = p.q[T.q];
    const int a0 = T.row + TM * static_cast<int>(rank);
    if constexpr (KIND == EPI_GATED) {
      // the even CTA holds the tile's rows of wg, the odd one those of wu
      ok = load_tile<FP8, false, 0>(p, g, sbase, full0, full_lead, empty0, lead, 2u * kblock_bytes<KIND>(q), &q.a[0],
                                    &q.b[rank], 1, q.kb_seg, a0, T.col);
    } else {
      const int hb = q.w / 2, b0 = T.col + hb * static_cast<int>(rank), terms = q.terms, kbs = q.kb_seg;
      const int boxes = q.b_mn ? (hb + 63) / 64 : 0;
      const uint32_t bytes = 2u * kblock_bytes<KIND>(q);
      if constexpr (KIND == EPI_PLAIN) {
        if (q.a_mn)
          ok = boxes == 2 ? load_tile<FP8, true, 2>(p, g, sbase, full0, full_lead, empty0, lead, bytes, q.a, q.b,
                                                    terms, kbs, a0, b0)
                          : load_tile<FP8, true, 1>(p, g, sbase, full0, full_lead, empty0, lead, bytes, q.a, q.b,
                                                    terms, kbs, a0, b0);
        else
          ok = boxes == 2 ? load_tile<FP8, false, 2>(p, g, sbase, full0, full_lead, empty0, lead, bytes, q.a, q.b,
                                                     terms, kbs, a0, b0)
                          : load_tile<FP8, false, 1>(p, g, sbase, full0, full_lead, empty0, lead, bytes, q.a, q.b,
                                                     terms, kbs, a0, b0);
      } else {
        ok = load_tile<FP8, false, 0>(p, g, sbase, full0, full_lead, empty0, lead, bytes, q.a, q.b, terms, kbs, a0,
                                      b0);
      }
    }
  }
  if ((threadIdx.x & 31) == 0) {
    st_shared_cluster_u32(map_to_rank(sbase + OFF_LOADED + 4u * rank, 0), g.armed);
    if (!ok) mark_failed(sbase);
  }
  __syncwarp();
}

// After a wait of the pair ran out, in one thread of the even CTA, whose
// barriers all loads of the pair signal: waits until those in flight have
// landed, before either CTA gives up its shared memory.  Use j of the ring
// completes with its own arming and the bytes of both CTAs; where only one of
// them came to load K block j, the other's part is made up here.  (A K block is
// loaded once the MMAs have consumed the one that was in its stage, so only the
// latest `stages` can be in flight.)
template <int KIND>
__device__ __noinline__ void drain_loads(const Args& p, uint32_t sbase, uint32_t full0, int pair, int pairs) {
  const uint32_t own = ld_shared_u32(sbase + OFF_LOADED), peer = ld_shared_u32(sbase + OFF_LOADED + 4u);
  const uint32_t both = min(own, peer), end = max(own, peer), first = end > p.stages ? end - p.stages : 0u;
  uint32_t at = 0;  // the tile's first K block in the pair's sequence
  for (int t = pair; t < p.total && at < end; t += pairs) {
    const Prob& q = p.q[tile_at(p, t).q];
    const uint32_t next = at + static_cast<uint32_t>(q.kb), bytes = kblock_bytes<KIND>(q);
    for (uint32_t j = max(max(at, both), first); j < min(next, end); ++j) {
      const uint32_t bar = full0 + 8u * (j % p.stages);
      if (j < own)
        mbar_complete_tx(bar, bytes);  // armed for both, and the peer's will not come
      else
        mbar_expect_tx(bar, bytes);    // the peer's alone, not armed
    }
    at = next;
  }
  for (uint32_t j = first; j < end; ++j)
    wait_bar(p.watch, full0 + 8u * (j % p.stages), (j / p.stages) & 1u, S_DRAIN, false);
}

template <int KIND, bool FP8>
__device__ void mma_role(const Args& p, uint32_t sbase, uint32_t tmem, uint32_t full0, uint32_t empty0,
                         uint32_t tfull0, uint32_t tempty0, uint32_t drain, int pair, int pairs) {
  const uint32_t stages = p.stages, stage_bytes = p.stage_bytes;
  uint32_t stage = 0, phase = 0, ul = 0;
  bool ok = true;
  for (int t = pair; ok && t < p.total; t += pairs, ++ul) {
    const Prob& q = p.q[tile_at(p, t).q];
    const uint32_t acc = ul & 1u;
    const int a_mn = q.a_mn, b_mn = q.b_mn, kb = q.kb;
    const uint32_t idesc = idesc_n(make_idesc(FP8, 2 * TM), KIND == EPI_GATED ? 2 * q.w : q.w) |
                           (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
    const uint64_t da0 = a_mn ? desc_mn(sbase) : smem_desc_sw128(sbase);
    const uint64_t db0 = b_mn ? desc_mn(sbase + A_BYTES) : smem_desc_sw128(sbase + A_BYTES);
    const uint64_t step_a = a_mn ? 128u : 2u, step_b = b_mn ? 128u : 2u;
    if (!wait_bar_warp(p.watch, tempty0 + 8u * acc, ((ul >> 1) & 1u) ^ 1u, S_TEMPTY)) {
      ok = false;
      break;
    }
    tc_fence_after();
    const uint32_t d = tmem + acc * TN;
    for (int i = 0; i < kb; ++i) {
      if (!wait_bar_warp(p.watch, full0 + 8u * stage, phase, S_FULL)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint64_t off = static_cast<uint64_t>(stage_bytes >> 4) * stage;
      mma_kblock<2, FP8>(d, da0 + off, db0 + off, idesc, i > 0 ? 1u : 0u, step_a, step_b);
      mma_commit_cg<2>(empty0 + 8u * stage);
      if (++stage == stages) stage = 0, phase ^= 1u;
    }
    if (!ok) break;
    mma_commit_cg<2>(tfull0 + 8u * acc);
  }
  // Every MMA issued must complete before tensor memory is freed, also where
  // the epilogue has given up and nobody waits for the last tile.  (The arrival
  // in the odd CTA is the last of those from here.)
  mma_commit_cg<2>(drain);
  if ((threadIdx.x & 31) == 0) {
    wait_bar(p.watch, drain, 0u, S_DRAIN, false);
    if (!ok) mark_failed(sbase);
  }
  __syncwarp();
}

// 32 consecutive bf16 values as they lie in memory, and their addition.
struct Row32 {
  uint4 h[4];
};
__device__ __forceinline__ void load_row(const __nv_bfloat16* p, Row32& r) {
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) r.h[ch] = *reinterpret_cast<const uint4*>(p + 8 * ch);
}
__device__ __forceinline__ void add_row(const Row32& r, float (&v)[32]) {
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    const uint32_t w[4] = {r.h[ch].x, r.h[ch].y, r.h[ch].z, r.h[ch].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * ch + 2 * j] += __uint_as_float(w[j] << 16);
      v[8 * ch + 2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}
// The first `count` (fewer than 32, or of any alignment) one by one.
__device__ __forceinline__ void add_some(const __nv_bfloat16* p, int count, float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j < count) v[j] += __bfloat162float(p[j]);
}

template <int ACT, int KIND>
__device__ __forceinline__ void apply_act(float (&v)[32], const uint32_t (&u)[32], float su) {
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    v[j] = act_f<ACT>(v[j]);
    if constexpr (KIND == EPI_GATED) v[j] *= __uint_as_float(u[j]) * su;
  }
}

// The epilogue of one warp: its 32 rows (the tensor-memory lanes its number
// allows) of every other 32-column chunk of the tile.
template <int KIND, bool FP8>
__device__ void epilogue_role(const Args& p, uint32_t sbase, uint32_t tmem, uint32_t tfull0, uint32_t tempty0,
                              uint32_t rank, int pair, int pairs) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = warp & 3, half = (warp - 2) >> 2;
  const bool wide = KIND == EPI_PLAIN && p.wide;
  const uint32_t box_bytes = wide ? 2 * BOX : BOX;
  const uint32_t ebase = sbase + (wide ? STAGES_WIDE : STAGES_NARROW) + (warp - 2) * 2 * box_bytes;
  const float s0 = FP8 ? __ldg(p.sx) * __ldg(p.sw0) : 1.0f;
  const float s1 = FP8 && KIND == EPI_GATED ? __ldg(p.sx) * __ldg(p.sw1) : 1.0f;
  uint32_t ul = 0, nst = 0;
  // Rounds 32 values of row `lane` to bf16 into a staging box (64-byte swizzle)
  // and stores it.  A tensor store writes whole 16-byte groups, past the end of
  // rows that are no multiple of them: a chunk with such an edge is written
  // element by element.
  auto store = [&](const OutMat* out, const float(&v)[32], int ox, int oy, const Prob& q) {
    if (ox + CHUNK > q.N && (q.N & 7)) {
      if (oy + lane < q.M) {
        __nv_bfloat16* o = out->p + static_cast<int64_t>(oy + lane) * out->ld + ox;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (ox + j < q.N) o[j] = __float2bfloat16_rn(v[j]);
      }
      return;
    }
    const uint32_t buf = ebase + (nst & 1u) * box_bytes;
    ++nst;
    if (lane == 0) bulk_wait_read<1>();  // the store before last has read this buffer
    __syncwarp();
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
      uint32_t h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[8 * ch + 2 * j], v[8 * ch + 2 * j + 1]);
        h[j] = *reinterpret_cast<const uint32_t*>(&b2);
      }
      st_shared_v4(buf + lane * 64 + (static_cast<uint32_t>(ch ^ ((lane >> 1) & 3)) << 4), h[0], h[1], h[2], h[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(&out->map, buf, ox, oy);
      bulk_commit();
    }
  };
  for (int t = pair; t < p.total; t += pairs, ++ul) {
    const TileAt T = tile_at(p, t);
    const Prob& q = p.q[T.q];
    const uint32_t acc = ul & 1u;
    if (wide) {
      if (!wait_bar_warp(p.watch, tfull0 + 8u * acc, (ul >> 1) & 1u, S_TFULL)) break;
      tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * TN;
      const int oy = T.row + TM * static_cast<int>(rank) + quad * 32, nw = (q.w + 63) / 64;
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_to_rank(tempty0 + 8u * acc, 0));
      };
      if (half >= nw) release();
#pragma unroll 1
      for (int c = half; c < nw; c += 2) {
        uint32_t r[64];
        tmem_ld64_sync(taddr + c * 64, r);
        if (c + 2 >= nw) release();
        const int ox = T.col + c * 64, cols = min(64, q.w - c * 64);
        if (ox >= q.N || oy >= q.M) continue;  // wholly past the output's edge
        if (cols == 64 && (ox + 64 <= q.N || !(q.N & 7))) {
          const uint32_t buf = ebase + (nst & 1u) * box_bytes;
          ++nst;
          uint32_t h[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
            h[j] = *reinterpret_cast<const uint32_t*>(&b2);
          }
          if (lane == 0) bulk_wait_read<1>();  // the store before last has read this buffer
          __syncwarp();
#pragma unroll
          for (int ch = 0; ch < 8; ++ch)  // row `lane` of 128 bytes, 128-byte swizzle
            st_shared_v4(buf + lane * 128 + (static_cast<uint32_t>(ch ^ (lane & 7)) << 4), h[4 * ch], h[4 * ch + 1],
                         h[4 * ch + 2], h[4 * ch + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&q.y.wide, buf, ox, oy);
            bulk_commit();
          }
        } else {
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
          store(&q.y, v, ox, oy, q);
          if (cols > 32 && ox + 32 < q.N) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[32 + j]);
            store(&q.y, v, ox + 32, oy, q);
          }
        }
      }
      continue;
    }
    const int nch = (q.w + CHUNK - 1) / CHUNK;
    const int oy = T.row + TM * static_cast<int>(rank) + quad * 32;
    const int64_t row = static_cast<int64_t>(oy) + lane;
    // the residual of this warp's next chunk, in flight beside the MMAs and the chunk before it
    Row32 res;
    auto fetch_residual = [&](int c) {
      const int ox = T.col + c * CHUNK;
      if (KIND == EPI_LINEAR && p.residual && c < nch && row < q.M && ox + CHUNK <= q.N)
        load_row(p.residual + row * p.ldr + ox, res);
    };
    fetch_residual(half);
    if (!wait_bar_warp(p.watch, tfull0 + 8u * acc, (ul >> 1) & 1u, S_TFULL)) break;
    tc_fence_after();
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * TN;
    const int last = (nch - 1 - half) / 2 * 2 + half;  // this warp's last chunk (if it has any)
    auto release = [&] {  // the accumulator is read: hand it back to the MMA warp
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to_rank(tempty0 + 8u * acc, 0));
    };
    if (half >= nch) release();
#pragma unroll 1
    for (int c = half; c < nch; c += 2) {
      uint32_t r[32], u[32];
      tmem_ld32_sync(taddr + c * CHUNK, r);
      if constexpr (KIND == EPI_GATED) tmem_ld32_sync(taddr + q.w + c * CHUNK, u);
      if (c == last) release();
      const int ox = T.col + c * CHUNK;
      if (ox >= q.N || oy >= q.M) continue;  // wholly past the output's edge
      float v[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]) * s0;
      if constexpr (KIND == EPI_LINEAR) {
        if (p.bias) {
          if (p.bias_vec && ox + CHUNK <= q.N) {
            Row32 b;
            load_row(p.bias + ox, b);
            add_row(b, v);
          } else {
            add_some(p.bias + ox, q.N - ox, v);
          }
        }
        if (p.has1) store(&p.y1, v, ox, oy, q);
      }
      if constexpr (KIND == EPI_GATED) {
        if (p.has1) {
          store(&p.y1, v, ox, oy, q);
          float uf[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) uf[j] = __uint_as_float(u[j]) * s1;
          store(&p.y2, uf, ox, oy, q);
        }
      }
      if constexpr (KIND != EPI_PLAIN) {
        switch (p.act) {
          case TPO_ACT_RELU: apply_act<TPO_ACT_RELU, KIND>(v, u, s1); break;
          case TPO_ACT_GELU: apply_act<TPO_ACT_GELU, KIND>(v, u, s1); break;
          case TPO_ACT_GELU_TANH: apply_act<TPO_ACT_GELU_TANH, KIND>(v, u, s1); break;
          case TPO_ACT_SILU: apply_act<TPO_ACT_SILU, KIND>(v, u, s1); break;
          default: apply_act<TPO_ACT_NONE, KIND>(v, u, s1); break;
        }
      }
      if constexpr (KIND == EPI_LINEAR) {
        if (p.residual && row < q.M) {
          if (ox + CHUNK <= q.N)
            add_row(res, v);
          else
            add_some(p.residual + row * p.ldr + ox, q.N - ox, v);
        }
        fetch_residual(c + 2);
      }
      store(&q.y, v, ox, oy, q);
    }
  }
  if (lane == 0) bulk_wait_read<0>();  // the boxes are read; the stores themselves end with the kernel
  __syncwarp();
}

// Grid: two CTAs (a cluster) per pair, at most as many pairs as the device
// holds at once; pair p takes the tiles p, p + pairs, ... (claims from a
// counter kept late pairs busier but cost each tile a round trip: 4096^3 took
// 4 us longer with them).
template <int KIND, bool FP8>
__global__ void __launch_bounds__(THREADS, 1) products_kernel(const __grid_constant__ Args p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
  grid_dep_launch();
  const int warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_rank();
  const int pair = static_cast<int>(blockIdx.x) / 2, pairs = static_cast<int>(gridDim.x) / 2;
  const uint32_t full0 = sbase + OFF_BARS, empty0 = full0 + 8 * MAX_STAGES, tfull0 = empty0 + 8 * MAX_STAGES,
                 tempty0 = tfull0 + 16, drain = tempty0 + 16;
  if (threadIdx.x == 0) {
    for (int s = 0; s < MAX_STAGES; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8u * a, 1);
      mbar_init(tempty0 + 8u * a, 2 * EPI_WARPS_N);
    }
    mbar_init(drain, 1);
    st_shared_u32(sbase + OFF_FAILED, 0u);
    fence_barrier_init();
    for (int i = 0; i < p.count; ++i) {
      tma_prefetch_map(&p.q[i].a[0]);
      tma_prefetch_map(&p.q[i].b[0]);
    }
  }
  __syncwarp();
  cluster_sync();  // the peer's barriers exist before anyone signals them
  if (warp == 1) {
    tmem_alloc_cg<2>(sbase + OFF_TMEM, 2 * TN);
    tmem_relinquish_cg<2>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ld_shared_u32(sbase + OFF_TMEM);
  grid_dep_wait();  // from here on memory may depend on the launch before
  if (warp == 0) {
    load_role<KIND, FP8>(p, sbase, full0, empty0, rank, pair, pairs);
  } else if (warp == 1) {
    if (rank == 0) mma_role<KIND, FP8>(p, sbase, tmem, full0, empty0, tfull0, tempty0, drain, pair, pairs);
    __syncwarp();
  } else {
    epilogue_role<KIND, FP8>(p, sbase, tmem, tfull0, tempty0, rank, pair, pairs);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while its peer may still use it
  if (ld_shared_u32(sbase + OFF_FAILED)) {  // the same in both CTAs: written before the barrier only
    if (rank == 0 && threadIdx.x == 0) drain_loads<KIND>(p, sbase, full0, pair, pairs);
    __syncthreads();
    cluster_sync();
  }
  if (warp == 1) {
    if (rank == 1 && (threadIdx.x & 31) == 0) wait_bar(p.watch, drain, 0u, S_DRAIN, false);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_cg<2>(tmem, 2 * TN);
  }
}

// ------------------------------------------------------------------ host side

bool encode_out(OutMat* o, void* p, int64_t ld, int64_t M, int64_t N, bool wide) {
  o->p = static_cast<__nv_bfloat16*>(p);
  o->ld = ld;
  return encode(&o->map, p, false, N, M, ld, CHUNK, 32, CU_TENSOR_MAP_SWIZZLE_64B) &&
         (!wide || encode(&o->wide, p, false, N, M, ld, 2 * CHUNK, 32, CU_TENSOR_MAP_SWIZZLE_128B));
}

// Bytes of a CTA's share of a B block of a tile w columns wide (w of h for the
// gated form, whose accumulator has twice as many).
int b_bytes(int w, bool gated, bool b_mn) {
  const int rows = gated ? w : w / 2;
  return b_mn ? (rows + 63) / 64 * 8192 : rows * KB;
}

// Time in ns of one K block of a tile with `cols` accumulator columns: when all
// pairs work for long, and the power limit sets the clock (measured 355, 312,
// 280 and 212 at 256, 224, 192 and 128 columns), and in a round that leaves
// pairs idle or is short (two cycles a column at the full clock; below 128
// columns the loads' latency over the stages in flight, 175 to 190).
double kblock_full_ns(int cols) { return std::max(71.0 + 1.1 * cols, 165.0 + 0.31 * cols); }
double kblock_free_ns(int cols) { return std::max(1.05 * cols, 165.0 + 0.20 * cols); }
// Rows that do not begin on 128-byte lines touch two of them a box (measured
// 225 ns a K block at least, and 300 with a transposed B).
double kblock_least_ns(const Product& q, bool fp8) {
  const int lines = fp8 ? 128 : 64;
  double ns = 0;
  for (int t = 0; t < q.terms; ++t)
    if (q.a[t].ld % lines || q.b[t].ld % lines) ns = std::max(ns, q.b[t].mn_major && q.b[t].ld % lines ? 300.0 : 225.0);
  return ns;
}

}  // namespace

void plan_width(const Machine& mc, const Product* q, int count, bool fp8, bool gated, int* widths, double* us) {
  // the products' shapes: the first, and the others, which are alike
  const int most = gated ? TN / 2 : TN, kinds = count > 1 ? 2 : 1;
  double least[2] = {}, best_ns = 0;
  int64_t rows[2] = {}, kbs[2] = {};
  for (int i = 0; i < kinds; ++i) {
    least[i] = kblock_least_ns(q[i], fp8);
    rows[i] = static_cast<int64_t>(ceil_div(q[i].M, 2 * TM)) * (i == 0 ? 1 : count - 1);
    kbs[i] = static_cast<int64_t>(ceil_div(q[i].K, fp8 ? KB : KB / 2)) * q[i].terms;
  }
  int w[2] = {most, most}, best[2] = {0, 0};
  for (w[0] = most; w[0] >= CHUNK; w[0] -= CHUNK)
    for (w[1] = most; w[1] >= CHUNK; w[1] -= kinds > 1 ? 2 * CHUNK : most) {
      double ns = 0, full = 0, free = 0, longest = 0;  // full, free: a tile of the last product
      int64_t total = 0;
      for (int i = 0; i < kinds; ++i) {
        const int cols = gated ? 2 * w[i] : w[i];
        // a tile is as long as its K blocks, or the draining of its accumulator
        const double drain = 8.0 * cols + 300, k = static_cast<double>(kbs[i]);
        full = std::max(k * std::max(kblock_full_ns(cols), least[i]), drain);
        free = std::max(k * std::max(kblock_free_ns(cols), least[i]), drain);
        longest = std::max(longest, free + 12.0 * cols);
        const int64_t tiles = rows[i] * ceil_div(q[i].N, w[i]);
        ns += static_cast<double>(tiles) / mc.pairs * full;
        total += tiles;
      }
      const double tail = 12.0 * (gated ? 2 * w[kinds - 1] : w[kinds - 1]);  // the last tile's epilogue
      // the last round, only partly filled, takes a whole tile's time at the clock that it has
      const double part = static_cast<double>(total % mc.pairs) / mc.pairs;
      if (total <= mc.pairs)
        ns = longest;
      else
        ns = std::max(longest, ns + tail + (part > 0 ? std::max(0.0, free - part * full) : 0.0));
      if (!best[0] || ns < 0.97 * best_ns) best[0] = w[0], best[1] = w[1], best_ns = ns;
    }
  for (int i = 0; i < count; ++i) widths[i] = best[i == 0 ? 0 : 1];
  if (us) *us = 4.0 + best_ns * 1e-3;
}

namespace {

template <int KIND, bool FP8>
cudaError_t launch_pairs(const Args& p, int pairs, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, products_kernel<KIND, FP8>, p);
}

}  // namespace

cudaError_t configure_products(Machine* m) {
  if (!load_encode()) return cudaErrorNotSupported;
  const void* fns[] = {reinterpret_cast<const void*>(products_kernel<EPI_PLAIN, false>),
                       reinterpret_cast<const void*>(products_kernel<EPI_LINEAR, false>),
                       reinterpret_cast<const void*>(products_kernel<EPI_LINEAR, true>),
                       reinterpret_cast<const void*>(products_kernel<EPI_GATED, false>),
                       reinterpret_cast<const void*>(products_kernel<EPI_GATED, true>)};
  for (const void* f : fns) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
  }
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&m->sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(&m->pairs, products_kernel<EPI_PLAIN, false>, &cfg);
  if (e == cudaSuccess && m->pairs < 1) e = cudaErrorNotSupported;
  return e;
}

cudaError_t launch_products(const Machine& mc, const Product* q, int count, bool fp8, const Epi& e, const Watch& w,
                            cudaStream_t s) {
  // The forms of operands that the kernel has: with an epilogue, both K-major and one term; without, bf16 and B
  // MN-major.
  const bool plain = e.kind == EPI_PLAIN;
  if (count > 1 && !plain) return cudaErrorInvalidValue;
  for (int i = 0; i < count; ++i)
    for (int t = 0; t < (e.kind == EPI_GATED ? 2 : q[i].terms); ++t)
      if (q[i].b[t].mn_major != plain || (plain ? fp8 || q[i].a[t].mn_major != q[i].a[0].mn_major
                                                : q[i].a[0].mn_major || q[i].terms != 1))
        return cudaErrorInvalidValue;
  Args p;
  std::memset(&p, 0, sizeof(p));
  p.count = count;
  int widths[3];
  plan_width(mc, q, count, fp8, e.kind == EPI_GATED, widths, nullptr);
  int stage = 0;
  for (int i = 0; i < count; ++i)
    if (e.kind == EPI_PLAIN && ceil_div(q[i].K, KB / 2) * q[i].terms <= WIDE_KB) p.wide = 1;
  bool ok = true;
  for (int i = 0; i < count; ++i) {
    const Product& c = q[i];
    Prob& o = p.q[i];
    o.M = static_cast<int>(c.M), o.N = static_cast<int>(c.N);
    o.w = widths[i];
    const int hb = e.kind == EPI_GATED ? o.w : o.w / 2;
    stage = std::max(stage, A_BYTES + b_bytes(o.w, e.kind == EPI_GATED, c.b[0].mn_major));
    o.tiles_m = ceil_div(c.M, 2 * TM);
    o.tiles = o.tiles_m * ceil_div(c.N, o.w);
    o.kb_seg = ceil_div(c.K, fp8 ? KB : KB / 2);
    o.terms = c.terms;
    o.kb = o.kb_seg * c.terms;
    o.a_mn = c.a[0].mn_major, o.b_mn = c.b[0].mn_major;
    for (int t = 0; t < c.terms && ok; ++t)
      ok = encode_operand(&o.a[t], c.a[t], fp8, c.M, c.K, TM) && encode_operand(&o.b[t], c.b[t], fp8, c.N, c.K, hb);
    if (ok && e.kind == EPI_GATED) ok = encode_operand(&o.b[1], c.b[1], fp8, c.N, c.K, hb);
    ok = ok && encode_out(&o.y, c.out, c.ldo, c.M, c.N, p.wide);
    p.total += o.tiles;
  }
  if (e.out1) ok = ok && encode_out(&p.y1, e.out1, e.ld1, q[0].M, q[0].N, false);
  if (e.out2) ok = ok && encode_out(&p.y2, e.out2, e.ld2, q[0].M, q[0].N, false);
  if (!ok) return cudaErrorInvalidValue;
  p.stage_bytes = static_cast<uint32_t>(stage);
  p.stages = static_cast<uint32_t>(std::min(MAX_STAGES, (p.wide ? STAGES_WIDE : STAGES_NARROW) / stage));
  p.has1 = e.out1 != nullptr;
  p.act = e.act;
  p.bias = static_cast<const __nv_bfloat16*>(e.bias);
  p.bias_vec = reinterpret_cast<uintptr_t>(e.bias) % 16 == 0;
  p.residual = static_cast<const __nv_bfloat16*>(e.residual);
  p.ldr = e.ldr;
  p.sx = e.sx, p.sw0 = e.sw0, p.sw1 = e.sw1;
  p.watch = w;
  const int pairs = std::min(mc.pairs, p.total);
  switch (e.kind) {
    case EPI_LINEAR: return fp8 ? launch_pairs<EPI_LINEAR, true>(p, pairs, s) : launch_pairs<EPI_LINEAR, false>(p, pairs, s);
    case EPI_GATED: return fp8 ? launch_pairs<EPI_GATED, true>(p, pairs, s) : launch_pairs<EPI_GATED, false>(p, pairs, s);
    default: return launch_pairs<EPI_PLAIN, false>(p, pairs, s);
  }
}

}  // namespace tpo
