// What the two product kernels share: bounded waits, operand descriptors, and
// the tensor maps of their operands.
#pragma once

#include "block.h"
#include "ptx.h"

namespace tpo {

constexpr int KB = 128;  // bytes of contraction elements per K block

// Bound of the waits of a CTA that gave up, for what it has in flight.
constexpr unsigned long long DRAIN_NS = 2000000000ull;

enum Site : uint32_t { S_EMPTY = 1, S_FULL = 2, S_TEMPTY = 3, S_TFULL = 4, S_DRAIN = 5, S_STEPS = kSiteSteps };

__device__ inline void give_up(uint32_t* err, uint32_t site) {
  if (atomicCAS(err, 0u, 1u) == 0u) {
    err[1] = site;
    err[2] = blockIdx.x;
    __threadfence();
  }
}
// Bounded wait; with honor_abort a failure recorded by any CTA also ends it,
// without it (draining) the limit is DRAIN_NS.
__device__ inline bool wait_bar(const Watch& w, uint32_t bar, uint32_t parity, uint32_t site, bool honor_abort = true) {
  if (mbar_test(bar, parity)) return true;
  const unsigned long long limit = honor_abort ? w.limit_ns : DRAIN_NS;
  const unsigned long long t0 = gtime();
  for (uint32_t i = 1;; ++i) {
    if (mbar_test(bar, parity)) return true;
    if ((i & 15u) == 0u) {
      if (honor_abort && *reinterpret_cast<volatile uint32_t*>(w.err) != 0u) return false;
      if (gtime() - t0 > limit) {
        give_up(w.err, site);
        return false;
      }
    }
  }
}
// The same for a converged warp, with one result and every lane ordered after the phase.
__device__ __forceinline__ bool wait_bar_warp(const Watch& w, uint32_t bar, uint32_t parity, uint32_t site) {
  if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = wait_bar(w, bar, parity, site) ? 1 : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  if (ok) (void)mbar_test(bar, parity);
  return ok != 0;
}

// Descriptor of an MN-major tile: blocks of 64 elements by 64 contraction
// rows (128 bytes each, 128-byte swizzle), 8-row groups 1024 bytes apart,
// the next 64 elements 8192 bytes on.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  uint64_t v = smem_desc_sw128(addr) & ~(static_cast<uint64_t>(0x3FFF) << 16);
  return v | (static_cast<uint64_t>(8192 >> 4) << 16);
}

// Tensor loads of one pipeline stage, issued by a converged warp: inside the
// statement elect.sync picks the lane, which first arms `arm` with the stage's
// bytes (if arming is not 0) and then issues the loads, all completing on
// `bar`.  One thread of a diverged warp needs ~80 cycles for each load and the
// index arithmetic around it runs at the latency of every instruction; the
// whole warp keeps the operands in uniform registers and issues two loads in
// less than 50.  (Measured on all SMs: 120 bytes per cycle and SM from L2 with
// two 16 KiB boxes a stage, 88 from a single thread.)
struct Box {
  uint32_t dst;
  uint64_t map;
  int x, y;
};
#define TPO_LOAD(CG, D, M, X, Y)                                                                              \
  "@E cp.async.bulk.tensor.2d" CG ".shared::cluster.global.mbarrier::complete_tx::bytes [" D "], [" M ", {" X \
  ", " Y "}], [%3];\n\t"
#define TPO_ARM                                                                                               \
  "{\n\t.reg .pred E, F;\n\t.reg .b32 r;\n\telect.sync r|E, 0xffffffff;\n\tsetp.ne.and.b32 F, %0, 0, E;\n\t" \
  "@F mbarrier.arrive.expect_tx.shared::cta.b64 _, [%1], %2;\n\t"
#define TPO_BOX(b) "r"(b.dst), "l"(b.map), "r"(b.x), "r"(b.y)
#define TPO_STAGE_LOADS(CG)                                                                                   \
  if constexpr (N == 2)                                                                                       \
    asm volatile(TPO_ARM TPO_LOAD(CG, "%4", "%5", "%6", "%7") TPO_LOAD(CG, "%8", "%9", "%10", "%11") "}" ::"r"( \
                     arming), "r"(arm), "r"(bytes), "r"(bar), TPO_BOX(b[0]), TPO_BOX(b[1])                    \
                 : "memory");                                                                                 \
  else if constexpr (N == 3)                                                                                  \
    asm volatile(TPO_ARM TPO_LOAD(CG, "%4", "%5", "%6", "%7") TPO_LOAD(CG, "%8", "%9", "%10", "%11")          \
                     TPO_LOAD(CG, "%12", "%13", "%14", "%15") "}" ::"r"(arming),                              \
                 "r"(arm), "r"(bytes), "r"(bar), TPO_BOX(b[0]), TPO_BOX(b[1]), TPO_BOX(b[2])                  \
                 : "memory");                                                                                 \
  else                                                                                                        \
    asm volatile(TPO_ARM TPO_LOAD(CG, "%4", "%5", "%6", "%7") TPO_LOAD(CG, "%8", "%9", "%10", "%11")          \
                     TPO_LOAD(CG, "%12", "%13", "%14", "%15") TPO_LOAD(CG, "%16", "%17", "%18", "%19") "}" :: \
                         "r"(arming), "r"(arm), "r"(bytes), "r"(bar), TPO_BOX(b[0]), TPO_BOX(b[1]),           \
                 TPO_BOX(b[2]), TPO_BOX(b[3])                                                                 \
                 : "memory")
// CG 2: `bar` may be the pair's even CTA's (a shared::cluster address).
template <int CG, int N>
__device__ __forceinline__ void stage_loads(uint32_t arming, uint32_t arm, uint32_t bytes, uint32_t bar,
                                            const Box (&b)[N]) {
  if constexpr (CG == 2) {
    TPO_STAGE_LOADS(".cta_group::2");
  } else {
    TPO_STAGE_LOADS("");
  }
}
#undef TPO_LOAD
#undef TPO_ARM
#undef TPO_BOX
#undef TPO_STAGE_LOADS

// ------------------------------------------------------------------ host side (block_maps.cu)

bool load_encode();  // the driver's tensor-map encoder; false if there is none

// A [outer, inner] matrix with rows `ld` elements apart, of bf16 or e4m3.
bool encode(CUtensorMap* map, const void* base, bool fp8, int64_t inner, int64_t outer, int64_t ld, int box_inner,
            int box_outer, CUtensorMapSwizzle sw);
// An operand of `rows` rows: K-major boxes of `box_rows` rows by one K block,
// or MN-major boxes of 64 contraction rows by 64 elements.
bool encode_operand(CUtensorMap* map, const Operand& o, bool fp8, int64_t rows, int64_t K, int box_rows);

inline int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

}  // namespace tpo
