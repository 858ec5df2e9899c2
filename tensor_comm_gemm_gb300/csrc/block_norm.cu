// Layer norm and its gradient (sm_103a).
//
// Both are bound by memory: each reads and writes every row once, so a row
// lives in the registers of the threads that share it.  `tpr` threads (a power
// of two; part of a warp, or whole warps of one block) hold a row as NV vectors
// of VEC elements each, thread l the vectors l, l + tpr, ...; rows whose
// address or pitch is no multiple of 16 bytes, or whose length is no multiple
// of the vector, take VEC = 1.  Rows too long for that are walked by one block
// in several passes.
//
// With many rows a block is persistent: its row groups take rows g, g + G, ...,
// and every thread keeps the vectors of its next rows in flight with
// asynchronous copies into its own part of shared memory, so no barrier is
// needed before they are read.
//
// Backward, a block also keeps the sums over its rows of dy xhat and dy for the
// columns its threads own in fp32 registers; they go to the workspace once,
// and a second kernel adds the blocks' sums in a fixed order.

#include <algorithm>
#include <cstring>
#include <initializer_list>

#include <cuda_bf16.h>

#include <type_traits>

#include "block.h"
#include "pdl.h"
#include "ptx.h"

namespace tpo {

namespace {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(bf16* p, float v) { *p = __float2bfloat16_rn(v); }

// VEC consecutive elements as they lie in memory (16 bytes of x's type, or one element).
template <class T, int VEC>
struct alignas(VEC * sizeof(T) > 16 ? 16 : VEC * sizeof(T)) Vec {
  T e[VEC];
};
template <class T, int VEC>
__device__ __forceinline__ Vec<T, VEC> load(const T* p) {
  return *reinterpret_cast<const Vec<T, VEC>*>(p);
}

// Sums over the `tpr` threads of a row, the same bits in each of them; `red`
// holds a value per warp and is free for the call after the next (the callers
// alternate between two).
__device__ __forceinline__ float lanes_sum(float a, int lanes) {
#pragma unroll
  for (int d = 16; d; d >>= 1)
    if (d < lanes) a += __shfl_xor_sync(0xffffffffu, a, d);
  return a;
}
// Barrier of the `tpr` threads of a row.  (A kernel with it holds all 16 of a
// block's barriers, so at most four such blocks run on an SM.)
__device__ __forceinline__ void group_barrier(int group, int tpr) {
  if (tpr > 32)
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpr) : "memory");
  else
    __syncwarp();
}
// The block's rows go together.
__device__ __forceinline__ float row_sum(float a, int tpr, float* red) {
  a = lanes_sum(a, tpr);
  if (tpr > 32) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = tpr >> 5;
    if (lane == 0) red[warp] = a;
    __syncthreads();
    a = lanes_sum(red[(warp & ~(per - 1)) + (lane & (per - 1))], per);
  }
  return a;
}
// The same where a row has whole warps, up to 16 of them, that keep their own
// pace; of two values at once.  (No step depends on tpr: lanes past the row's
// last warp add zeros.)  They also are a barrier of the row's threads.
__device__ __forceinline__ float group_sum(float a, int group, int tpr, float* red) {
  a = lanes_sum(a, 32);
  if (tpr > 32) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = tpr >> 5;
    if (lane == 0) red[warp] = a;
    group_barrier(group, tpr);
    const int w = lane & 15;
    a = w < per ? red[(warp & ~(per - 1)) + w] : 0.0f;
    a = lanes_sum(a, 16);
  } else {
    __syncwarp();
  }
  return a;
}
template <int LANES>
__device__ __forceinline__ void lanes_sums(float& a, float& b) {  // both chains at once
#pragma unroll
  for (int d = LANES / 2; d; d >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, d);
    b += __shfl_xor_sync(0xffffffffu, b, d);
  }
}
__device__ __forceinline__ float2 group_sums(float a, float b, int group, int tpr, float2* red) {
  lanes_sums<32>(a, b);
  if (tpr > 32) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = tpr >> 5;
    if (lane == 0) red[warp] = make_float2(a, b);
    group_barrier(group, tpr);
    const int w = lane & 15;
    const float2 v = w < per ? red[(warp & ~(per - 1)) + w] : make_float2(0.0f, 0.0f);
    a = v.x;
    b = v.y;
    lanes_sums<16>(a, b);
  } else {
    __syncwarp();
  }
  return make_float2(a, b);
}

// Two values at a time (the packed fp32 operations, which halve the
// instructions that otherwise bound these kernels).
struct Num {
  uint64_t v;
};
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ Num num(float a, float b) { return {pack2(a, b)}; }
__device__ __forceinline__ Num all(float x) { return num(x, x); }
__device__ __forceinline__ Num add(Num a, Num b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.v), "l"(b.v));
  return {r};
}
__device__ __forceinline__ Num mul(Num a, Num b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.v), "l"(b.v));
  return {r};
}
__device__ __forceinline__ Num fma(Num a, Num b, Num c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a.v), "l"(b.v), "l"(c.v));
  return {r};
}
__device__ __forceinline__ float total(Num a) {
  float x, y;
  unpack2(a.v, x, y);
  return x + y;
}

// A step of a thread's share of a row: a vector of VEC > 1 elements, or two
// single ones 32 apart.  Its values as fp32, and back (rounded).
constexpr int STRIDE1 = 32;
template <int VEC>
constexpr int NUMS = VEC > 1 ? VEC / 2 : 1;
template <class T, int VEC>
__device__ __forceinline__ void to_nums(const Vec<T, VEC>& v, Num (&o)[NUMS<VEC>]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) o[j] = num(v.e[2 * j], v.e[2 * j + 1]);
  } else {
    uint32_t w[VEC / 2];
    memcpy(w, &v, sizeof(w));
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) o[j] = num(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
  }
}
template <class T, int VEC>
__device__ __forceinline__ void read_nums(const T* p, Num (&o)[NUMS<VEC>]) {
  if constexpr (VEC > 1)
    to_nums<T, VEC>(load<T, VEC>(p), o);
  else
    o[0] = num(to_f(p[0]), to_f(p[STRIDE1]));
}
// left: how many of the row's elements there are from p on (VEC = 1: of which the step has the first and the 33rd).
template <class T, int VEC>
__device__ __forceinline__ void write_nums(T* p, const Num (&a)[NUMS<VEC>], int left) {
  if constexpr (VEC == 1) {
    float x, y;
    unpack2(a[0].v, x, y);
    if (left > 0) put(p, x);
    if (left > STRIDE1) put(p + STRIDE1, y);
  } else if (left > 0) {
    Vec<T, VEC> v;
    uint32_t w[VEC / 2];
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
      float x, y;
      unpack2(a[j].v, x, y);
      if constexpr (sizeof(T) == 4) {
        v.e[2 * j] = x;
        v.e[2 * j + 1] = y;
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        memcpy(&w[j], &h, 4);
      }
    }
    if constexpr (sizeof(T) == 2) memcpy(&v, w, sizeof(w));
    *reinterpret_cast<Vec<T, VEC>*>(p) = v;
  }
}
// The values of a step that exist; zeros for the others.
template <int VEC>
__device__ __forceinline__ void mask_nums(Num (&a)[NUMS<VEC>], int left) {
  if constexpr (VEC == 1) {
    float x, y;
    unpack2(a[0].v, x, y);
    a[0] = num(left > 0 ? x : 0.0f, left > STRIDE1 ? y : 0.0f);
  } else {
#pragma unroll
    for (int j = 0; j < NUMS<VEC>; ++j)
      if (left <= 0) a[j] = all(0.0f);
  }
}

// ------------------------------------------------------------ one row per group

// Few rows, short rows and long ones (bf16 vectors up to 32768 elements): one
// row per group of 2^lg threads, read once.  Latency bounds few rows: one of
// 4096 2.1 us in a row of calls, 256 3.5 us; instructions bound many short
// ones: 262144 x 128 35 us.  The variance is the mean square of the
// differences from the mean, of values that are already in registers.
template <class T, class W, int VEC, int NV>
__global__ void __launch_bounds__(512) norm_kernel(const NormArgs a, int lg) {
  __shared__ float red[2][32];
  constexpr int NN = NUMS<VEC>;
  grid_dep_launch();
  grid_dep_wait();
  const int tpr = 1 << lg, lane = threadIdx.x & (tpr - 1), k = static_cast<int>(a.k);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> lg) + (threadIdx.x >> lg);
  const bool live = row < a.n;
  const T* const x = static_cast<const T*>(a.x) + row * a.ldx;
  T* const y = static_cast<T*>(a.y) + row * a.ldy;
  const W *const gamma = static_cast<const W*>(a.gamma), *const beta = static_cast<const W*>(a.beta);
  const float inv_k = 1.0f / static_cast<float>(k);
  float mean, rstd;
  if constexpr (VEC > 1) {
    Vec<T, VEC> e[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * tpr) * VEC;
      e[i] = {};
      if (live && c < k) e[i] = load<T, VEC>(x + c);
    }
    Num v[NV][NN], s = all(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      to_nums<T, VEC>(e[i], v[i]);
#pragma unroll
      for (int j = 0; j < NN; ++j) s = add(s, v[i][j]);
    }
    mean = row_sum(total(s), tpr, red[0]) * inv_k;
    const Num minus = all(-mean);
    s = all(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < NN; ++j) v[i][j] = add(v[i][j], minus);
      mask_nums<VEC>(v[i], k - (lane + i * tpr) * VEC);
#pragma unroll
      for (int j = 0; j < NN; ++j) s = fma(v[i][j], v[i][j], s);
    }
    rstd = rsqrtf(row_sum(total(s), tpr, red[1]) * inv_k + a.eps);
    if (!live) return;
    const Num scale = all(rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * tpr) * VEC;
      if (c >= k) continue;
      Num g[NN], b[NN];
      if (gamma) read_nums<W, VEC>(gamma + c, g);
      if (beta) read_nums<W, VEC>(beta + c, b);
#pragma unroll
      for (int j = 0; j < NN; ++j) {
        v[i][j] = mul(v[i][j], scale);
        if (gamma) v[i][j] = mul(v[i][j], g[j]);
        if (beta) v[i][j] = add(v[i][j], b[j]);
      }
      write_nums<T, VEC>(y + c, v[i], k - c);
    }
  } else {
    float v[NV], s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = live && lane + i * tpr < k ? to_f(x[lane + i * tpr]) : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) s += v[i];
    mean = row_sum(s, tpr, red[0]) * inv_k;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = lane + i * tpr < k ? v[i] - mean : 0.0f;
      s += v[i] * v[i];
    }
    rstd = rsqrtf(row_sum(s, tpr, red[1]) * inv_k + a.eps);
    if (!live) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = lane + i * tpr;
      if (c < k) put(y + c, v[i] * rstd * (gamma ? to_f(gamma[c]) : 1.0f) + (beta ? to_f(beta[c]) : 0.0f));
    }
  }
  if (lane == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

// ------------------------------------------------------------------ many rows

// Asynchronous copy of 16 bytes to shared memory; zeros (and no access to src) if they do not exist.
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool exists) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(exists ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most AHEAD of this thread's latest copy groups are in flight.
template <int AHEAD>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD) : "memory");
}
// Rows in flight.  With VEC > 1 (16-byte rows) a thread copies the vectors that
// it will read itself, so it needs no barrier before them.  With VEC = 1 the
// group copies the aligned 16-byte units that hold the row, to the same offset
// modulo 16, and reads single elements after a barrier; the slot is free after
// the next one: that of the row's sum forward, where the registers hold the
// row then, and that before the next row backward.  Units at a row's ends
// bring a few bytes of what lies beside it, which nobody reads; where that
// might be outside the matrix (`edge`: the first and the last edge_rows(k)
// rows) only the row's own bytes are touched.
__device__ __forceinline__ int64_t edge_rows(int k) { return k >= 16 ? 1 : 16; }
__host__ __device__ inline uint32_t weight_bytes(int k, int elem) {
  return (static_cast<uint32_t>(k) * elem + 15u) & ~15u;
}
__host__ __device__ inline uint32_t row_bytes(int k, int elem) {
  return ((static_cast<uint32_t>(k) * elem + 15u) & ~15u) + 16u;
}
// A thread takes at most MOST of the units.
template <class T, int MOST>
__device__ __forceinline__ void copy_units(const T* src, int k, uint32_t dst, int lane, int tpr, bool edge) {
  const uint64_t p = reinterpret_cast<uint64_t>(src), lo = p & ~15ull;
  const int skip = static_cast<int>(p & 15), bytes = skip + k * static_cast<int>(sizeof(T));  // up to the row's end
  if (!edge) {
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      const int u = 16 * (lane + i * tpr);
      if (u < bytes)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + u), "l"(lo + u) : "memory");
    }
    return;
  }
#pragma unroll 1
  for (int u = 16 * lane; u < bytes; u += 16 * tpr) {
    if (u < skip) {  // the row's own elements of its first unit
      const int own = min(k, (16 - skip) / static_cast<int>(sizeof(T)));
      for (int c = 0; c < own; ++c) {
        const uint32_t to = dst + skip + c * static_cast<uint32_t>(sizeof(T));
        if constexpr (sizeof(T) == 4)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(to), "f"(src[c]) : "memory");
        else
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(__bfloat16_as_ushort(src[c])) : "memory");
      }
    } else {
      const int own = min(16, bytes - u);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + u), "l"(lo + u), "r"(own) : "memory");
    }
  }
}
// Where element 0 of row r of such a matrix is.
template <class T>
__device__ __forceinline__ const T* unit_row(const void* p, int64_t r, int64_t ld, const uint8_t* slot) {
  const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uint64_t>(p)) +
                      static_cast<uint32_t>(r) * static_cast<uint32_t>(ld) * static_cast<uint32_t>(sizeof(T));
  return reinterpret_cast<const T*>(slot + (at & 15u));
}

// A group is whole warps.  With VEC = 1, warp w of it holds the elements
// [w NV 32, (w + 1) NV 32), lane l every 32nd of them, two of them to a step:
// the offsets between a thread's elements are known to the compiler, and all
// warps but a row's last have nothing to mask.  Whole vectors are dealt out
// over the group instead (thread l has l, l + tpr, ...), which keeps the
// group's accesses of one step together: 16384 x 4096 backward took a ninth
// longer with vectors dealt out by warp.
constexpr int RING_THREADS = 512;
// Copies k weights to shared memory (VEC = 1: `none` where there are none) and
// adds zeros up to `all` (the block joins afterwards).
template <class W, int VEC>
__device__ __forceinline__ void keep_weights(W* to, const W* from, int k, int all, float none) {
  if (from || VEC == 1)
#pragma unroll 4
    for (int c = threadIdx.x * VEC; c < all; c += RING_THREADS * VEC) {
      Vec<W, VEC> v = {};
      if (c < k) {
        if (from)
          v = load<W, VEC>(from + c);
        else
          put(&v.e[0], none);
      }
      *reinterpret_cast<Vec<W, VEC>*>(to + c) = v;
    }
}
// A thread's first element, how far apart its steps are, and how many it has.
template <int VEC, int NV>
__device__ __forceinline__ int first_column(int tpr) {
  const int lane = static_cast<int>(threadIdx.x & (tpr - 1));
  return VEC > 1 ? lane * VEC : (lane >> 5) * NV * 32 + (lane & 31);
}
template <int VEC>
__device__ __forceinline__ int column_step(int tpr) {
  return VEC > 1 ? tpr * VEC : 2 * STRIDE1;
}
template <int VEC, int NV>
constexpr int STEPS = VEC > 1 ? NV : NV / 2;
// The most units of a row that a thread copies: up to NV elements a thread, and at most one unit more for the row.
template <class T, int NV>
constexpr int MOST_UNITS = NV * static_cast<int>(sizeof(T)) / 16 + 1;

// Rows of each group in flight or in use.  Two: with 32 KB and more a row set,
// that covers the memory's latency, and more only puts off the first rows and
// with them the first stores: 2048 x 4096 bf16 forward 9.9 us, 10.9 with three,
// 11.5 with four; level over many rows (16384 x 4096 backward with dres 83.7 us,
// 83.6 and 84.5).
constexpr int DEPTH = 2;

// Forward.  FULL: the group's vectors are exactly a row's.  8192 x 8192 bf16 in
// 45 us, 6.0 TB/s of 6.8, fp32 in 90; 2000 x 7777 (single elements) in 26 us, where the
// shared-memory accesses and the three barriers of a row, with 16 warps in
// step, bound it.
template <class T, class W, int VEC, int NV, bool FULL>
__global__ void __launch_bounds__(RING_THREADS, 1) norm_ring_kernel(const NormArgs a, int tpr) {
  extern __shared__ __align__(16) uint8_t smem[];  // gamma, beta, the rows in flight, slack to read past them
  __shared__ float red[4][RING_THREADS / 32];
  constexpr int NN = NUMS<VEC>, ST = STEPS<VEC, NV>;
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = RING_THREADS / tpr;
  const int c0 = first_column<VEC, NV>(tpr), step_c = column_step<VEC>(tpr);
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t row = static_cast<int64_t>(blockIdx.x) * groups + group;
  const int k = static_cast<int>(a.k);
  W* const gamma = reinterpret_cast<W*>(smem);
  W* const beta = reinterpret_cast<W*>(smem + weight_bytes(k, sizeof(W)));
  uint8_t* const ring = smem + 2 * weight_bytes(k, sizeof(W));
  // slot s of this thread's vectors, or of its group's row
  const uint32_t slot_bytes = VEC > 1 ? NV * RING_THREADS * 16 : groups * row_bytes(k, sizeof(T));
  uint8_t* const mine = ring + (VEC > 1 ? threadIdx.x * 16 : group * row_bytes(k, sizeof(T)));
  const int64_t edge = edge_rows(k);
  auto fetch = [&](int64_t r, int slot) {
    const bool live = r < a.n;
    const T* x = static_cast<const T*>(a.x) + (live ? r : 0) * a.ldx;
    const uint32_t to = smem_u32(mine) + slot * slot_bytes;
    if constexpr (VEC > 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (c0 + i * step_c);
        copy_async(to + i * (RING_THREADS * 16), x + (FULL || c < k ? c : 0), live && (FULL || c < k));
      }
    } else if (live) {
      copy_units<T, MOST_UNITS<T, NV>>(x, k, to, lane, tpr, r < edge || r >= a.n - edge);
    }
    copy_commit();
  };
  for (int d = 0; d < DEPTH; ++d) fetch(row + d * step, d);
  keep_weights<W, VEC>(gamma, static_cast<const W*>(a.gamma), k, k, 1.0f);
  keep_weights<W, VEC>(beta, static_cast<const W*>(a.beta), k, k, 0.0f);
  __syncthreads();
  const bool has_gamma = VEC == 1 || a.gamma != nullptr, has_beta = VEC == 1 || a.beta != nullptr;
  const float inv_k = 1.0f / static_cast<float>(k);
  int slot = 0, buf = 0;
  // WHOLE: all of this warp's elements exist.
  auto work = [&](auto whole, bool live) {
    constexpr bool WHOLE = decltype(whole)::value;
    const int own = WHOLE ? ST * step_c : live || VEC > 1 ? k - c0 : 0;  // elements from this thread's first on
    Num v[ST][NN], s = all(0.0f);
    if constexpr (VEC == 1) {
      const T* x = unit_row<T>(a.x, row, a.ldx, mine + slot * slot_bytes) + c0;
#pragma unroll
      for (int i = 0; i < ST; ++i) {
        read_nums<T, 1>(x + i * 64, v[i]);  // past the row's end: whatever lies there, in shared memory all the same
        if constexpr (!WHOLE) mask_nums<1>(v[i], own - i * 64);
      }
    } else {
#pragma unroll
      for (int i = 0; i < ST; ++i)
        read_nums<T, VEC>(reinterpret_cast<const T*>(mine + slot * slot_bytes + i * (RING_THREADS * 16)), v[i]);
      fetch(row + DEPTH * step, slot);  // the slot has been read (by this thread, its only reader)
    }
#pragma unroll
    for (int i = 0; i < ST; ++i)
#pragma unroll
      for (int j = 0; j < NN; ++j) s = add(s, v[i][j]);
    const float mean = group_sum(total(s), group, tpr, red[buf]) * inv_k;
    if constexpr (VEC == 1) fetch(row + DEPTH * step, slot);  // the slot has been read, by the whole group
    const Num minus = all(-mean);
    s = all(0.0f);
#pragma unroll
    for (int i = 0; i < ST; ++i) {
#pragma unroll
      for (int j = 0; j < NN; ++j) v[i][j] = add(v[i][j], minus);
      if constexpr (!WHOLE) mask_nums<VEC>(v[i], own - i * step_c);
#pragma unroll
      for (int j = 0; j < NN; ++j) s = fma(v[i][j], v[i][j], s);
    }
    const float rstd = rsqrtf(group_sum(total(s), group, tpr, red[buf + 1]) * inv_k + a.eps);
    const Num scale = all(rstd);
    T* const y = static_cast<T*>(a.y) + row * a.ldy + c0;
    if (live)
#pragma unroll
      for (int i = 0; i < ST; ++i) {
        const int c = i * step_c;
        if (!WHOLE && c >= own) continue;
        Num g[NN], b[NN];
        if (has_gamma) read_nums<W, VEC>(gamma + c0 + c, g);
        if (has_beta) read_nums<W, VEC>(beta + c0 + c, b);
#pragma unroll
        for (int j = 0; j < NN; ++j) {
          v[i][j] = mul(v[i][j], scale);
          if (has_gamma) v[i][j] = mul(v[i][j], g[j]);
          if (has_beta) v[i][j] = add(v[i][j], b[j]);
        }
        write_nums<T, VEC>(y + c, v[i], WHOLE ? 2 * STRIDE1 : own - c);
      }
    if (live && lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  };
  // every group of the block runs the same number of rounds
  const int64_t sets = (a.n + groups - 1) / groups;
  for (int64_t set = blockIdx.x; set < sets; set += gridDim.x, row += step) {
    const bool live = row < a.n;
    if constexpr (VEC > 1) {
      copy_wait<DEPTH - 1>();
      work(std::bool_constant<FULL>(), live);
    } else {
      copy_wait<DEPTH - 1>();
      group_barrier(group, tpr);  // the row is there
      if (live && (c0 & ~31) + NV * 32 <= k)  // one answer per warp
        work(std::true_type(), true);
      else
        work(std::false_type(), live);
    }
    if (++slot == DEPTH) slot = 0;
    buf ^= 2;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Adds the sums of a block's row groups in their order and stores them:
// part[blockIdx.x][2][k].  `sums`: [groups][2][k] floats of shared memory,
// which a lone group of single elements does without.
template <int VEC, int NV>
__device__ __forceinline__ void store_sums(const Num (&dg)[STEPS<VEC, NV>][NUMS<VEC>],
                                           const Num (&db)[STEPS<VEC, NV>][NUMS<VEC>], int k, int tpr, float* sums,
                                           float* part) {
  const int c0 = first_column<VEC, NV>(tpr), step_c = column_step<VEC>(tpr);
  const int group = threadIdx.x / tpr, groups = RING_THREADS / tpr;
  float* const out = part + static_cast<int64_t>(blockIdx.x) * 2 * k;
  auto put_all = [&](float* to) {
#pragma unroll
    for (int i = 0; i < STEPS<VEC, NV>; ++i) {
      const int c = c0 + i * step_c;
      if constexpr (VEC == 1) {
        write_nums<float, 1>(to + c, dg[i], k - c);
        write_nums<float, 1>(to + k + c, db[i], k - c);
      } else if (c < k) {
#pragma unroll
        for (int j = 0; j < NUMS<VEC>; ++j) {  // k is even where values come in pairs
          memcpy(to + c + j * 2, &dg[i][j], sizeof(Num));
          memcpy(to + k + c + j * 2, &db[i][j], sizeof(Num));
        }
      }
    }
  };
  if (VEC == 1 && groups == 1) {
    put_all(out);
    return;
  }
  put_all(sums + group * 2 * k);
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * k; c += 4 * RING_THREADS) {
    float v[4] = {};
#pragma unroll 1
    for (int q = 0; q < groups; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j * RING_THREADS < 2 * k) v[j] += sums[q * 2 * k + c + j * RING_THREADS];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j * RING_THREADS < 2 * k) out[c + j * RING_THREADS] = v[j];
  }
}

// Backward, rows in flight as forward: x, dy and (if given) dres of a row.
// With xhat = (x - mean) rstd and w = dy gamma:
// dx = rstd (w - mean(w) - xhat mean(w xhat)) + dres.  16384 x 4096 bf16 with
// dres in 84 us with the column sums behind it (537 MB, 6.4 TB/s in all);
// 777 x 5003 f32 in 20 us with them: 5.1 rows per SM in two groups are three
// rounds, and the start, the last round and the sums do not overlap.
template <class T, class W, int VEC, int NV>
__global__ void __launch_bounds__(RING_THREADS, 1) norm_bwd_ring_kernel(const NormArgs a, int tpr,
                                                                        float* part) {
  extern __shared__ __align__(16) uint8_t smem[];  // gamma, the rows in flight, slack to read past them
  __shared__ float2 red[2][RING_THREADS / 32];
  constexpr int NN = NUMS<VEC>, ST = STEPS<VEC, NV>;
  constexpr bool KEEP = NV * VEC <= 20;  // xhat and dy gamma stay in registers from the sums to dx
  static_assert(KEEP || VEC > 1, "single elements are read once");
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = RING_THREADS / tpr;
  const int c0 = first_column<VEC, NV>(tpr), step_c = column_step<VEC>(tpr);
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t row = static_cast<int64_t>(blockIdx.x) * groups + group;
  const int k = static_cast<int>(a.k);
  const int arrays = a.dres && a.y ? 3 : 2;
  // bf16 gamma of few vectors stays in registers, other gammas in shared memory
  constexpr bool GREG = KEEP && VEC > 1 && sizeof(W) == 2;
  W* const gamma = reinterpret_cast<W*>(smem);
  uint8_t* const ring = smem + (GREG ? 0u : weight_bytes(tpr * NV * VEC, sizeof(W)));
  const bool has_gamma = VEC == 1 || a.gamma != nullptr;
  // slot s, matrix w: this thread's vectors, or its group's row
  const uint32_t part_bytes = VEC > 1 ? NV * RING_THREADS * 16 : groups * row_bytes(k, sizeof(T));
  uint8_t* const mine = ring + (VEC > 1 ? threadIdx.x * 16 : group * row_bytes(k, sizeof(T)));
  auto at = [&](int slot, int which) { return mine + (slot * arrays + which) * part_bytes; };
  // a vector past the row's end, or of a row past the last, is zeros: it adds nothing to any sum
  const int64_t edge = edge_rows(k);
  auto fetch = [&](int64_t r, int slot) {
    const bool live = r < a.n;
    const int64_t q = live ? r : 0;
    const T *x = static_cast<const T*>(a.x) + q * a.ldx, *dy = static_cast<const T*>(a.dy) + q * a.lddy;
    const T* dres = static_cast<const T*>(a.dres) + q * a.lddres;
    const uint32_t tx = smem_u32(at(slot, 0)), td = smem_u32(at(slot, 1)), tr = smem_u32(at(slot, 2));
    if constexpr (VEC > 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (c0 + i * step_c);
        const bool in = live && c < k;
        const int o = in ? c : 0;
        copy_async(tx + i * (RING_THREADS * 16), x + o, in);
        copy_async(td + i * (RING_THREADS * 16), dy + o, in);
        if (arrays == 3) copy_async(tr + i * (RING_THREADS * 16), dres + o, in);
      }
    } else if (live) {
      const bool at_edge = r < edge || r >= a.n - edge;
      copy_units<T, MOST_UNITS<T, NV>>(x, k, tx, lane, tpr, at_edge);
      copy_units<T, MOST_UNITS<T, NV>>(dy, k, td, lane, tpr, at_edge);
      if (arrays == 3) copy_units<T, MOST_UNITS<T, NV>>(dres, k, tr, lane, tpr, at_edge);
    }
    copy_commit();
  };
  for (int d = 0; d < DEPTH; ++d) fetch(row + d * step, d);
  Vec<W, VEC> gk[GREG ? NV : 1];
  if constexpr (GREG) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * step_c;
      gk[i] = {};
      if (has_gamma && c < k) gk[i] = load<W, VEC>(static_cast<const W*>(a.gamma) + c);
    }
  } else {
    // zeros past the row's end
    keep_weights<W, VEC>(gamma, static_cast<const W*>(a.gamma), k, tpr * NV * VEC, 1.0f);
    __syncthreads();
  }
  Num dg[ST][NN], db[ST][NN];
#pragma unroll
  for (int i = 0; i < ST; ++i)
#pragma unroll
    for (int j = 0; j < NN; ++j) dg[i][j] = db[i][j] = all(0.0f);
  const float inv_k = 1.0f / static_cast<float>(k);
  int slot = 0, buf = 0;
  float mean = row < a.n ? a.mean[row] : 0.0f, rstd = row < a.n ? a.rstd[row] : 0.0f;
  // WHOLE (VEC = 1): all of this warp's elements exist.
  auto work = [&](auto whole, bool live) {
    constexpr bool WHOLE = decltype(whole)::value;
    const T *ux = nullptr, *ud = nullptr;  // VEC = 1: this thread's first element of each row
    if constexpr (VEC == 1) {
      ux = unit_row<T>(a.x, row, a.ldx, at(slot, 0)) + c0;
      ud = unit_row<T>(a.dy, row, a.lddy, at(slot, 1)) + c0;
    }
    const int own = live ? k - c0 : 0;  // elements from this thread's first on
    const Num minus = all(-mean), scale = all(rstd);
    Num s1 = all(0.0f), s2 = s1;
    // xhat and w = dy gamma of step i
    auto values = [&](int i, Num(&h)[NN], Num(&w)[NN], bool first) {
      Num g[NN];
      if constexpr (VEC > 1) {
        read_nums<T, VEC>(reinterpret_cast<const T*>(at(slot, 0) + i * (RING_THREADS * 16)), h);
        read_nums<T, VEC>(reinterpret_cast<const T*>(at(slot, 1) + i * (RING_THREADS * 16)), w);
      } else {
        // past the row's end: whatever lies there, in shared memory all the same
        read_nums<T, 1>(ux + i * 64, h);
        read_nums<T, 1>(ud + i * 64, w);
        if constexpr (!WHOLE) {
          mask_nums<1>(h, own - i * 64);
          mask_nums<1>(w, own - i * 64);
        }
      }
      if (has_gamma) {
        if constexpr (GREG)
          to_nums<W, VEC>(gk[i], g);
        else
          read_nums<W, VEC>(gamma + c0 + i * step_c, g);
      }
#pragma unroll
      for (int j = 0; j < NN; ++j) {
        h[j] = mul(add(h[j], minus), scale);
        if (first) {
          dg[i][j] = fma(w[j], h[j], dg[i][j]);
          db[i][j] = add(db[i][j], w[j]);
        }
        if (has_gamma) w[j] = mul(w[j], g[j]);
      }
    };
    Num hk[KEEP ? ST : 1][NN], wk[KEEP ? ST : 1][NN];
#pragma unroll
    for (int i = 0; i < ST; ++i) {
      Num(&h)[NN] = hk[KEEP ? i : 0];
      Num(&w)[NN] = wk[KEEP ? i : 0];
      values(i, h, w, true);
#pragma unroll
      for (int j = 0; j < NN; ++j) {
        s1 = add(s1, w[j]);
        s2 = fma(w[j], h[j], s2);
      }
    }
    if (!a.y) return;
    const float2 t = group_sums(total(s1), total(s2), group, tpr, red[buf]);
    const Num m1 = all(-t.x * inv_k), m2 = all(-t.y * inv_k);
    T* const dx = static_cast<T*>(a.y) + row * a.ldy + c0;
    const T* ur = unit_row<T>(a.dres, row, a.lddres, at(slot, 2)) + c0;
    auto finish = [&](auto with) {
      constexpr bool DRES = decltype(with)::value;
#pragma unroll
      for (int i = 0; i < ST; ++i) {
        Num(&h)[NN] = hk[KEEP ? i : 0];
        Num(&w)[NN] = wk[KEEP ? i : 0];
        if constexpr (!KEEP) values(i, h, w, false);
        Num r[NN];
        if constexpr (DRES && VEC > 1)
          read_nums<T, VEC>(reinterpret_cast<const T*>(at(slot, 2) + i * (RING_THREADS * 16)), r);
        else if constexpr (DRES)
          read_nums<T, VEC>(ur + i * 64, r);
#pragma unroll
        for (int j = 0; j < NN; ++j) {
          const Num q = fma(h[j], m2, add(w[j], m1));
          r[j] = DRES ? fma(q, scale, r[j]) : mul(q, scale);
        }
        write_nums<T, VEC>(dx + i * step_c, r, WHOLE ? 2 * STRIDE1 : own - i * step_c);
      }
    };
    if (arrays == 3)
      finish(std::true_type());
    else
      finish(std::false_type());
  };
  const int64_t sets = (a.n + groups - 1) / groups;
  for (int64_t set = blockIdx.x; set < sets; set += gridDim.x, row += step) {
    const bool live = row < a.n;
    const float mean_n = row + step < a.n ? a.mean[row + step] : 0.0f;
    const float rstd_n = row + step < a.n ? a.rstd[row + step] : 0.0f;
    if constexpr (VEC > 1) {
      copy_wait<DEPTH - 1>();
      work(std::false_type(), live);
      fetch(row + DEPTH * step, slot);  // the slot has been read (by this thread, its only reader)
    } else {
      const bool later = set != blockIdx.x;
      if (later)
        copy_wait<DEPTH - 2>();
      else
        copy_wait<DEPTH - 1>();
      group_barrier(group, tpr);  // the row is there, and every thread is done with the one before
      if (later) fetch(row + (DEPTH - 1) * step, slot == 0 ? DEPTH - 1 : slot - 1);
      if (live && (c0 & ~31) + NV * 32 <= k)  // one answer per warp
        work(std::true_type(), true);
      else
        work(std::false_type(), live);
    }
    if (++slot == DEPTH) slot = 0;
    buf ^= 1;
    mean = mean_n;
    rstd = rstd_n;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (!part) return;
  __syncthreads();  // the ring is free: it holds the columns' sums now
  store_sums<VEC, NV>(dg, db, k, tpr, reinterpret_cast<float*>(ring), part);
}

// ----------------------------------------------------------------- short rows

// Backward for many rows of up to 128 elements: `tpr` lanes a row, a vector
// each, several rows a warp where they are shorter, and U rows at a time whose
// loads are all in flight before the first is used.  No barriers; the
// weights of a lane's columns and their gradients' sums stay in registers.
// 262144 x 128 bf16 54 us, 95 in the kernel above, whose groups are whole warps;
// 262144 x 64 30 and 95; fp32 262144 x 128 87 and 125.  (Forward the same
// arrangement was no faster than one row per group: 38 and 35 us.)  What is
// left over the memory's 30 and 15 us are the sums over the lanes, two for each
// row.
template <class T, int VEC>
__device__ __forceinline__ void read_or_zeros(const T* p, bool exists, Num (&v)[NUMS<VEC>]) {
  Vec<T, VEC> e = {};
  if (exists) e = load<T, VEC>(p);
  to_nums<T, VEC>(e, v);
}
constexpr int SHORT_THREADS = 640;  // one block per SM: a part of the columns' sums each
template <class T, class W, int VEC>
__global__ void __launch_bounds__(SHORT_THREADS, 1) norm_short_bwd_kernel(const NormArgs a, int tpr, float* part) {
  extern __shared__ __align__(16) uint8_t smem[];  // [groups][2][k] floats
  constexpr int NN = NUMS<VEC>, U = 2;
  grid_dep_launch();
  grid_dep_wait();
  const int per_warp = 32 / tpr, k = static_cast<int>(a.k), c = (threadIdx.x & (tpr - 1)) * VEC;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (SHORT_THREADS / 32) + (threadIdx.x >> 5);
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (SHORT_THREADS / 32) * per_warp;
  const bool has_dres = a.dres && a.y;
  Num g[NN], dg[NN], db[NN];
  if (a.gamma) read_or_zeros<W, VEC>(static_cast<const W*>(a.gamma) + c, c < k, g);
#pragma unroll
  for (int j = 0; j < NN; ++j) dg[j] = db[j] = all(0.0f);
  const float inv_k = 1.0f / static_cast<float>(k);
  for (int64_t base = warp * per_warp; base < a.n; base += U * groups) {  // the same rounds for all of the warp
    const int64_t row = base + (threadIdx.x & 31) / tpr;
    Num h[U][NN], w[U][NN];
    float mean[U], rstd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = row + u * groups;
      const bool live = r < a.n;
      read_or_zeros<T, VEC>(static_cast<const T*>(a.x) + r * a.ldx + c, live && c < k, h[u]);
      read_or_zeros<T, VEC>(static_cast<const T*>(a.dy) + r * a.lddy + c, live && c < k, w[u]);
      mean[u] = live ? a.mean[r] : 0.0f;
      rstd[u] = live ? a.rstd[r] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = row + u * groups;
      const Num minus = all(-mean[u]), scale = all(rstd[u]);
      Num s1 = all(0.0f), s2 = s1, q[NN];
      if (has_dres) read_or_zeros<T, VEC>(static_cast<const T*>(a.dres) + r * a.lddres + c, r < a.n && c < k, q);
#pragma unroll
      for (int j = 0; j < NN; ++j) {  // where there is no element dy is 0, and xhat adds nothing
        Num &hv = h[u][j], &wv = w[u][j];
        hv = mul(add(hv, minus), scale);
        dg[j] = fma(wv, hv, dg[j]);
        db[j] = add(db[j], wv);
        if (a.gamma) wv = mul(wv, g[j]);
        s1 = add(s1, wv);
        s2 = fma(wv, hv, s2);
      }
      if (!a.y) continue;
      const Num m1 = all(-lanes_sum(total(s1), tpr) * inv_k), m2 = all(-lanes_sum(total(s2), tpr) * inv_k);
      if (r >= a.n) continue;
#pragma unroll
      for (int j = 0; j < NN; ++j) {
        const Num d = fma(h[u][j], m2, add(w[u][j], m1));
        q[j] = has_dres ? fma(d, scale, q[j]) : mul(d, scale);
      }
      write_nums<T, VEC>(static_cast<T*>(a.y) + r * a.ldy + c, q, k - c);
    }
  }
  if (!part) return;
  float* const sums = reinterpret_cast<float*>(smem);
  float* const mine = sums + static_cast<int>(threadIdx.x / tpr) * 2 * k + c;
  if (c < k)
#pragma unroll
    for (int j = 0; j < NN; ++j) {
      memcpy(mine + 2 * j, &dg[j], sizeof(Num));
      memcpy(mine + k + 2 * j, &db[j], sizeof(Num));
    }
  __syncthreads();
  // 2 k columns, up to 256 of them; each the groups' sums in their order
  for (int o = threadIdx.x; o < 2 * k; o += SHORT_THREADS) {
    float v = 0.0f;
    for (int q = 0; q < SHORT_THREADS / tpr; ++q) v += sums[q * 2 * k + o];
    part[static_cast<int64_t>(blockIdx.x) * 2 * k + o] = v;
  }
}

// ------------------------------------------------------------------ long rows

__device__ float block_sum(float v, float* part) {
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < 32; ++w) s += part[w];
  return s;
}

// Rows too long for a group's registers: one block per row, three passes (the
// later two mostly from L2).
template <class T, class W>
__global__ void __launch_bounds__(1024) norm_long_kernel(const NormArgs a) {
  __shared__ float red[32];
  grid_dep_launch();
  grid_dep_wait();
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  T* y = static_cast<T*>(a.y) + row * a.ldy;
  const W *gamma = static_cast<const W*>(a.gamma), *beta = static_cast<const W*>(a.beta);
  float s = 0.0f;
  for (int64_t j = threadIdx.x; j < a.k; j += 1024) s += to_f(x[j]);
  const float mean = block_sum(s, red) / a.k;
  s = 0.0f;
  for (int64_t j = threadIdx.x; j < a.k; j += 1024) {
    const float d = to_f(x[j]) - mean;
    s += d * d;
  }
  const float rstd = 1.0f / sqrtf(block_sum(s, red) / a.k + a.eps);
  for (int64_t j = threadIdx.x; j < a.k; j += 1024)
    put(&y[j], (to_f(x[j]) - mean) * rstd * (gamma ? to_f(gamma[j]) : 1.0f) + (beta ? to_f(beta[j]) : 0.0f));
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

template <class T, class W>
__global__ void __launch_bounds__(1024) norm_long_dx_kernel(const NormArgs a) {
  __shared__ float red[32];
  grid_dep_launch();
  grid_dep_wait();
  const int64_t row = blockIdx.x;
  const T *x = static_cast<const T*>(a.x) + row * a.ldx, *dy = static_cast<const T*>(a.dy) + row * a.lddy;
  const T* dres = a.dres ? static_cast<const T*>(a.dres) + row * a.lddres : nullptr;
  T* dx = static_cast<T*>(a.y) + row * a.ldy;
  const W* gamma = static_cast<const W*>(a.gamma);
  const float mean = a.mean[row], rstd = a.rstd[row];
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t j = threadIdx.x; j < a.k; j += 1024) {
    const float v = to_f(dy[j]) * (gamma ? to_f(gamma[j]) : 1.0f);
    s1 += v;
    s2 += v * ((to_f(x[j]) - mean) * rstd);
  }
  s1 = block_sum(s1, red) / a.k;
  s2 = block_sum(s2, red) / a.k;
  for (int64_t j = threadIdx.x; j < a.k; j += 1024) {
    const float v = to_f(dy[j]) * (gamma ? to_f(gamma[j]) : 1.0f);
    const float xhat = (to_f(x[j]) - mean) * rstd;
    put(&dx[j], rstd * (v - s1 - xhat * s2) + (dres ? to_f(dres[j]) : 0.0f));
  }
}

// Sums over the rows g, g + gridDim.y, ... of dy xhat and dy, one thread per column.
template <class T>
__global__ void __launch_bounds__(256) norm_long_dw_kernel(const NormArgs a, float* part) {
  grid_dep_launch();
  grid_dep_wait();
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (j >= a.k) return;
  float dg = 0.0f, db = 0.0f;
#pragma unroll 4
  for (int64_t i = blockIdx.y; i < a.n; i += gridDim.y) {
    const float d = to_f(static_cast<const T*>(a.dy)[i * a.lddy + j]);
    dg += d * ((to_f(static_cast<const T*>(a.x)[i * a.ldx + j]) - a.mean[i]) * a.rstd[i]);
    db += d;
  }
  part[static_cast<int64_t>(blockIdx.y) * 2 * a.k + j] = dg;
  part[static_cast<int64_t>(blockIdx.y) * 2 * a.k + a.k + j] = db;
}

// ------------------------------------------------------------------ host side

template <class F>
cudaError_t with_types(int dtype, int wdtype, F f) {
  if (dtype == TPO_F32) return wdtype == TPO_F32 ? f(float(), float()) : f(float(), bf16());
  return wdtype == TPO_F32 ? f(bf16(), float()) : f(bf16(), bf16());
}
template <class F>
cudaError_t with_nv(int nv, F f) {
  switch (nv) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    default: return f(std::integral_constant<int, 8>());
  }
}

bool vec_ok(const void* p, int64_t ld, int64_t rows, int elem) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld * elem % 16 == 0);
}

// How a row is shared: vectors per thread and threads per row; tpr = 0 when it is too long.
struct Share {
  int nv, tpr;
};
Share share(int64_t vecs, int nv, int most_nv, int most_tpr, int least_tpr = 1) {
  Share s{nv, least_tpr};
  while (static_cast<int64_t>(s.tpr) * s.nv < vecs) {
    if (s.tpr < most_tpr)
      s.tpr *= 2;
    else if (s.nv < most_nv)
      s.nv *= 2;
    else
      return {0, 0};
  }
  return s;
}

// The shared memory of a block with DEPTH rows per group and `fixed` bytes of
// weights; 0: too much.
constexpr size_t RING_SMEM = 226 * 1024;
size_t ring_smem(bool vec, const Share& h, int arrays, int64_t k, int elem, size_t fixed) {
  if (!h.tpr) return 0;
  const size_t slot = arrays * (vec ? static_cast<size_t>(RING_THREADS) * h.nv * 16
                                    : static_cast<size_t>(RING_THREADS / h.tpr) * row_bytes(static_cast<int>(k), elem));
  // single elements are also read past the row's end
  const size_t all = fixed + (vec ? 0 : static_cast<size_t>(h.tpr) * h.nv * elem) + DEPTH * slot;
  return all <= RING_SMEM ? all : 0;
}

// Of some numbers of vectors a thread, the one that leaves the fewest of a
// group's places without a vector (the first of equals); f: whether it will do.
template <class F>
Share share_best(int64_t vecs, std::initializer_list<int> nvs, F f) {
  Share best{0, 0};
  for (int nv : nvs) {
    const Share s = share(vecs, nv, nv, RING_THREADS, 32);
    if (s.tpr && f(s) && (!best.tpr || s.tpr * nv < best.tpr * best.nv)) best = s;
  }
  return best;
}
// Single elements.  Up to 20 a thread, so that longer rows still fit (bf16 1000 x 9001 backward 28 us, 45 in the plain
// kernels); where fewer hold the row, the number makes no difference (f32 777 x 5003 19.8 us with 20, 19.5 with 12).
Share share_single(int64_t k, int arrays, int elem, int welem, int weights) {
  return share_best(k, {20, 16, 12, 8}, [&](const Share& s) {
    return ring_smem(false, s, arrays, k, elem, weights * weight_bytes(s.tpr * s.nv, welem)) > 0;
  });
}

template <class K>
cudaError_t allow_smem(K* kernel) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_SMEM);
}

}  // namespace

cudaError_t launch_norm(const Machine& mc, const NormArgs& a, int dtype, int wdtype, cudaStream_t s) {
  return with_types(dtype, wdtype, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    constexpr int V = 16 / sizeof(T);
    const bool vec = a.k % V == 0 && vec_ok(a.x, a.ldx, a.n, sizeof(T)) && vec_ok(a.y, a.ldy, a.n, sizeof(T)) &&
                     vec_ok(a.gamma, 0, 1, 4) && vec_ok(a.beta, 0, 1, 4);
    const int64_t vecs = vec ? a.k / V : a.k;
    // Rows for most of the SMs' persistent blocks (one of 512 threads per SM):
    // keep rows in flight.  Fewer rows: one row per group, as many threads as it
    // has vectors (latency).  1024 rows of 4096 7.0 us and 8.3, 400 4.7 and 3.8;
    // 1024 of 8192 10.7 and 13.1, 152 4.8 and 3.8; single elements, 400 of 5003
    // 7.9 and 11.3.  8192 rows of 8192, 46 us: two blocks per SM, with 64
    // registers a thread, were a sixth slower than one.
    const Share m = vec ? share_best(vecs, {4, 3, 5}, [](const Share&) { return true; })
                        : share_single(a.k, 1, sizeof(T), sizeof(W), 2);
    const int64_t sets = m.tpr ? (a.n + RING_THREADS / m.tpr - 1) / (RING_THREADS / m.tpr) : 0;
    // (16384 rows of 256, a third of whose group's places would hold a vector: 6.4 us, 8.4 in flight; of 512, two
    // thirds: 11.3 and 10.0)
    if (3 * sets >= 2 * static_cast<int64_t>(mc.sms) && (!vec || 2 * vecs >= m.tpr * m.nv)) {
      const size_t smem = ring_smem(vec, m, 1, a.k, sizeof(T), 2 * weight_bytes(static_cast<int>(a.k), sizeof(W)));
      const dim3 grid(static_cast<unsigned>(std::min<int64_t>(sets, mc.sms)));
      auto run = [&](auto kernel) {
        const cudaError_t e = allow_smem(kernel);
        return e != cudaSuccess ? e : launch_pdl(kernel, grid, dim3(RING_THREADS), smem, s, a, m.tpr);
      };
      auto run_vec = [&](auto nv) {
        constexpr int NV = decltype(nv)::value;
        return static_cast<int64_t>(m.tpr) * NV == vecs ? run(norm_ring_kernel<T, W, V, NV, true>)
                                                        : run(norm_ring_kernel<T, W, V, NV, false>);
      };
      if (smem) {
        if (vec && m.nv == 3) return run_vec(std::integral_constant<int, 3>());
        if (vec && m.nv == 4) return run_vec(std::integral_constant<int, 4>());
        if (vec) return run_vec(std::integral_constant<int, 5>());
        if (m.nv == 8) return run(norm_ring_kernel<T, W, 1, 8, false>);
        if (m.nv == 12) return run(norm_ring_kernel<T, W, 1, 12, false>);
        return m.nv == 16 ? run(norm_ring_kernel<T, W, 1, 16, false>) : run(norm_ring_kernel<T, W, 1, 20, false>);
      }
    }
    const Share h = share(vecs, 1, 8, 512);
    if (!h.tpr) return launch_pdl(norm_long_kernel<T, W>, dim3(static_cast<unsigned>(a.n)), dim3(1024), 0, s, a);
    const int threads = std::max(h.tpr, 128), rows = threads / h.tpr;
    int lg = 0;
    while (1 << lg < h.tpr) ++lg;
    const dim3 grid(static_cast<unsigned>((a.n + rows - 1) / rows));
    return with_nv(h.nv, [&](auto nv) {
      constexpr int NV = decltype(nv)::value;
      if (vec) return launch_pdl(norm_kernel<T, W, V, NV>, grid, dim3(threads), 0, s, a, lg);
      return launch_pdl(norm_kernel<T, W, 1, NV>, grid, dim3(threads), 0, s, a, lg);
    });
  });
}

cudaError_t launch_norm_bwd(const Machine& mc, const NormArgs& a, int dtype, int wdtype, float* part, cudaStream_t s) {
  return with_types(dtype, wdtype, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    constexpr int V = 16 / sizeof(T);
    const bool wants = a.dgamma || a.dbeta;
    const bool vec = a.k % V == 0 && vec_ok(a.x, a.ldx, a.n, sizeof(T)) && vec_ok(a.dy, a.lddy, a.n, sizeof(T)) &&
                     vec_ok(a.dres, a.lddres, a.n, sizeof(T)) && vec_ok(a.y, a.ldy, a.n, sizeof(T)) &&
                     vec_ok(a.gamma, 0, 1, 4);
    const int64_t vecs = vec ? a.k / V : a.k;
    if (!wants) part = nullptr;
    int parts = 0;
    cudaError_t e = cudaSuccess;
    // Whole vectors: 16 elements a thread, whose xhat and dy gamma then stay in
    // registers; 24 or (bf16: fp32 rows in flight would not fit) 32 where rows
    // are too long for that, and 24 where that leaves a quarter fewer places,
    // in bf16 rows long enough for it to pay: 8192 x 5120 59 us, 67 with 16;
    // 2560 33.7 and 36.1; but 1536 22.6 and 21.8; fp32 4096 x 6144 57.5 and 55.2.
    constexpr int NV = 16 / V;
    const int arrays = a.dres && a.y ? 3 : 2;
    auto kept = [&](const Share& s) -> size_t {  // gamma in shared memory
      return vec && s.nv == NV && sizeof(W) == 2 ? 0 : weight_bytes(s.tpr * s.nv * (vec ? V : 1), sizeof(W));
    };
    Share h{0, 0};
    if (vec) {
      h = share(vecs, NV, NV, RING_THREADS, 32);
      auto fits = [&](const Share& s) { return ring_smem(true, s, arrays, a.k, sizeof(T), kept(s)) > 0; };
      const Share more =
          sizeof(T) == 2 ? share_best(vecs, {2 * NV, 3 * NV / 2}, fits) : share_best(vecs, {3 * NV / 2}, fits);
      if (!h.tpr || (sizeof(T) == 2 && a.k > 2048 && more.tpr && 4 * more.tpr * more.nv <= 3 * h.tpr * h.nv)) h = more;
    } else {
      h = share_single(a.k, arrays, sizeof(T), sizeof(W), 1);
    }
    const size_t ring = ring_smem(vec, h, arrays, a.k, sizeof(T), kept(h));
    // Rows that would have a vector in at most a quarter of a warp's places, where every block's warps have some
    const Share few = vec && vecs <= 8 * NV ? share(vecs, 1, 1, 32) : Share{0, 0};
    if (few.tpr && a.n / (32 / few.tpr) >= static_cast<int64_t>(mc.sms) * (SHORT_THREADS / 32)) {
      parts = std::min(mc.sms, NORM_PARTS);
      const size_t smem = static_cast<size_t>(SHORT_THREADS / few.tpr) * 8 * a.k;
      e = allow_smem(norm_short_bwd_kernel<T, W, V>);
      if (e == cudaSuccess)
        e = launch_pdl(norm_short_bwd_kernel<T, W, V>, dim3(parts), dim3(SHORT_THREADS), smem, s, a, few.tpr, part);
    } else if (ring && a.n > 0) {
      const int64_t sets = (a.n + RING_THREADS / h.tpr - 1) / (RING_THREADS / h.tpr);
      parts = static_cast<int>(std::min<int64_t>({sets, mc.sms, NORM_PARTS}));
      // the slots later hold every group's fp32 sums
      const size_t smem = std::max(ring, kept(h) + static_cast<size_t>(RING_THREADS / h.tpr) * 8 * a.k);
      auto run = [&](auto kernel) {
        const cudaError_t c = allow_smem(kernel);
        return c != cudaSuccess ? c : launch_pdl(kernel, dim3(parts), dim3(RING_THREADS), smem, s, a, h.tpr, part);
      };
      if (vec && h.nv == NV)
        e = run(norm_bwd_ring_kernel<T, W, V, NV>);
      else if (vec && h.nv == 3 * NV / 2)
        e = run(norm_bwd_ring_kernel<T, W, V, 3 * NV / 2>);
      else if (vec)
        e = run(norm_bwd_ring_kernel<T, W, V, sizeof(T) == 2 ? 2 * NV : NV>);
      else if (h.nv == 8)
        e = run(norm_bwd_ring_kernel<T, W, 1, 8>);
      else if (h.nv == 12)
        e = run(norm_bwd_ring_kernel<T, W, 1, 12>);
      else if (h.nv == 16)
        e = run(norm_bwd_ring_kernel<T, W, 1, 16>);
      else
        e = run(norm_bwd_ring_kernel<T, W, 1, 20>);
    } else if (a.n > 0) {
      // the weights' gradients first: dx may overwrite dy
      parts = static_cast<int>(std::min<int64_t>(a.n, 32));
      if (wants)
        e = launch_pdl(norm_long_dw_kernel<T>, dim3(static_cast<unsigned>((a.k + 255) / 256), parts), dim3(256), 0, s,
                       a, part);
      if (e == cudaSuccess && a.y)
        e = launch_pdl(norm_long_dx_kernel<T, W>, dim3(static_cast<unsigned>(a.n)), dim3(1024), 0, s, a);
    }
    if (e == cudaSuccess && wants)
      e = launch_column_sums(part, parts, 2, a.k, a.dgamma, a.dbeta, wdtype, s);
    return e;
  });
}

}  // namespace tpo
