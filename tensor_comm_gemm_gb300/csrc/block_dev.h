// What the two product kernels share: bounded waits, operand descriptors, and
// the tensor maps of their operands.
#pragma once

#include "block.h"
#include "ptx.h"

namespace tpo {

constexpr int KB = 128;  // bytes of contraction elements per K block
constexpr unsigned long long WAIT_NS = 2000000000ull;  // bound of every wait

enum Site : uint32_t { S_EMPTY = 1, S_FULL = 2, S_TEMPTY = 3, S_TFULL = 4, S_DRAIN = 5 };

__device__ inline void give_up(uint32_t* err, uint32_t site) {
  if (atomicCAS(err, 0u, 1u) == 0u) {
    err[1] = site;
    err[2] = blockIdx.x;
    __threadfence();
  }
}
// Bounded wait; with honor_abort a failure recorded by any CTA also ends it.
__device__ inline bool wait_bar(uint32_t* err, uint32_t bar, uint32_t parity, uint32_t site, bool honor_abort = true) {
  if (mbar_test(bar, parity)) return true;
  const unsigned long long t0 = gtime();
  for (uint32_t i = 1;; ++i) {
    if (mbar_test(bar, parity)) return true;
    if ((i & 15u) == 0u) {
      if (honor_abort && *reinterpret_cast<volatile uint32_t*>(err) != 0u) return false;
      if (gtime() - t0 > WAIT_NS) {
        give_up(err, site);
        return false;
      }
    }
  }
}
// The same for a converged warp, with one result and every lane ordered after the phase.
__device__ __forceinline__ bool wait_bar_warp(uint32_t* err, uint32_t bar, uint32_t parity, uint32_t site) {
  if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = wait_bar(err, bar, parity, site) ? 1 : 0;
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
