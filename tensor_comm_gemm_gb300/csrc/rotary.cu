// Rotary positions (sm_103a): pairs of elements of each head turn by an angle
// that grows with the token's position.
//
// The angle is position x frequency, and a position may be in the millions: the
// product is taken in turns, as a 64-bit fraction of one turn that wraps around
// (an entry of the table is 2^64 times the frequency's turns per position), so
// that it is exact for every position and its top 32 bits give the angle to
// 2^-26 turns.  A block computes its tokens' sines and cosines once, in shared
// memory, and all heads of the token use them.
//
// Bound by memory: every element is read and written once.  Measured with a flushed
// L2: a prompt's queries and keys in bf16 (302 MB moved) 50.5 us, 5.98 TB/s or 90 %
// of the measured copy bandwidth; 29 MB in fp32 12.2 us and one token 7.0 us, of
// which about 6 are a launch on a cold cache.

#include <cuda_bf16.h>

#include <algorithm>

#include "attn.h"
#include "pdl.h"
#include "ptx.h"

namespace tpo {

namespace {

using bf16 = __nv_bfloat16;
constexpr int THREADS = 256;
constexpr int MAX_TOKENS = 32;  // of a block

struct Shape {
  int heads, rot, turning, still;  // of a head: items that turn, items behind them that are copied
  int tokens;                      // of a block
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void narrow(float v, float& o) { o = v; }
__device__ __forceinline__ void narrow(float v, bf16& o) { o = __float2bfloat16_rn(v); }

// V consecutive elements, moved as one access.
template <class T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

// One item turns V pairs (halves), or V / 2 (pairs; a single one where V is 1),
// or copies V elements.
template <class T, int V, bool PAIRS>
__global__ void __launch_bounds__(THREADS) rotary_kernel(RotaryArgs a, Shape d) {
  extern __shared__ float turn[];  // [tokens][rot / 2] cosines, then sines
  using Item = Vec<T, V>;
  grid_dep_launch();
  grid_dep_wait();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * d.tokens;
  const int count = static_cast<int>(min(static_cast<int64_t>(d.tokens), a.n - t0)), half = d.rot / 2;
  float *cosine = turn, *sine = turn + d.tokens * half;
  for (int i = threadIdx.x; i < count * half; i += THREADS) {
    const int tok = i / half;
    const int64_t pos = a.pos ? a.pos[t0 + tok] : t0 + tok;
    const uint64_t part = static_cast<uint64_t>(pos) * a.table[i - tok * half];
    float s, c;
    // rounded to 24 bits of half a turn, 2^-26 turns at most: fp32 results are off by 3.0e-8 of their size, of which their own
    // rounding is 2.6e-8
    sincospif(static_cast<float>(static_cast<int32_t>(part >> 32)) * 0x1p-31f, &s, &c);
    cosine[i] = c * a.magnitude;
    sine[i] = (a.inverse ? -s : s) * a.magnitude;
  }
  __syncthreads();
  const int per_head = d.turning + d.still, total = count * d.heads * per_head;
  for (int i = threadIdx.x; i < total; i += THREADS) {
    const int th = i / per_head, j = i - th * per_head, tok = th / d.heads, h = th - tok * d.heads;
    int64_t row = t0 + tok;
    const T* x = static_cast<const T*>(a.x.p) + row * a.x.ld + h * a.x.hs;
    if (a.rows) {
      row = a.rows[row];
      if (row < 0 || row >= a.ny) continue;
    }
    T* y = const_cast<T*>(static_cast<const T*>(a.y.p)) + row * a.y.ld + h * a.y.hs;
    if (j >= d.turning) {
      const int e = d.rot + (j - d.turning) * V;
      *reinterpret_cast<Item*>(y + e) = *reinterpret_cast<const Item*>(x + e);
      continue;
    }
    if constexpr (PAIRS && V > 1) {
      Item v = *reinterpret_cast<const Item*>(x + j * V);
#pragma unroll
      for (int p = 0; p < V / 2; ++p) {
        const float c = cosine[tok * half + j * (V / 2) + p], s = sine[tok * half + j * (V / 2) + p];
        const float l = widen(v.e[2 * p]), r = widen(v.e[2 * p + 1]);
        narrow(l * c - r * s, v.e[2 * p]);
        narrow(l * s + r * c, v.e[2 * p + 1]);
      }
      *reinterpret_cast<Item*>(y + j * V) = v;
    } else {
      const int ea = PAIRS ? 2 * j : j * V, eb = PAIRS ? 2 * j + 1 : half + j * V;
      Item l = *reinterpret_cast<const Item*>(x + ea), r = *reinterpret_cast<const Item*>(x + eb);
#pragma unroll
      for (int p = 0; p < V; ++p) {
        const float c = cosine[tok * half + j * V + p], s = sine[tok * half + j * V + p];
        const float u = widen(l.e[p]), w = widen(r.e[p]);
        narrow(u * c - w * s, l.e[p]);
        narrow(u * s + w * c, r.e[p]);
      }
      *reinterpret_cast<Item*>(y + ea) = l;
      *reinterpret_cast<Item*>(y + eb) = r;
    }
  }
}

template <class T, int V>
cudaError_t launch_as(const Machine& mc, const RotaryArgs& a, cudaStream_t s) {
  const bool pairs = a.layout == TPO_ROTARY_PAIRS;
  const bool in_place = a.x.p == a.y.p && !a.rows;
  Shape d;
  d.heads = static_cast<int>(a.heads), d.rot = static_cast<int>(a.rot);
  d.turning = d.rot / (pairs && V > 1 ? V : 2 * V);
  d.still = in_place ? 0 : static_cast<int>(a.dim - a.rot) / V;
  // about eight items a thread, where that leaves no SM without a block
  const int64_t items = a.heads * (d.turning + d.still);
  if (items == 0) return cudaSuccess;
  int64_t tokens = std::min<int64_t>(8 * THREADS / items + 1, a.n / (2 * mc.sms) + 1);
  tokens = std::min<int64_t>(tokens, MAX_TOKENS);
  while (tokens > 1 && tokens * a.rot * 4 > 32768) --tokens;
  d.tokens = static_cast<int>(tokens);
  const dim3 grid(static_cast<unsigned>((a.n + tokens - 1) / tokens));
  const size_t smem = static_cast<size_t>(tokens) * a.rot * 4;
  return pairs ? launch_pdl(rotary_kernel<T, V, true>, grid, dim3(THREADS), smem, s, a, d)
               : launch_pdl(rotary_kernel<T, V, false>, grid, dim3(THREADS), smem, s, a, d);
}

}  // namespace

cudaError_t launch_rotary(const Machine& mc, const RotaryArgs& a, int dtype, cudaStream_t s) {
  const int elem = dtype == TPO_F32 ? 4 : 2, v = 16 / elem;
  // 16-byte accesses where every address and the halves or pairs allow them
  const int64_t unit = a.layout == TPO_ROTARY_PAIRS ? a.rot : a.rot / 2;
  const int64_t strides = a.x.ld | a.x.hs | a.y.ld | a.y.hs | a.dim | unit;
  const bool wide = strides % v == 0 && reinterpret_cast<uintptr_t>(a.x.p) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(a.y.p) % 16 == 0;
  if (dtype == TPO_F32) return wide ? launch_as<float, 4>(mc, a, s) : launch_as<float, 1>(mc, a, s);
  return wide ? launch_as<bf16, 8>(mc, a, s) : launch_as<bf16, 1>(mc, a, s);
}

}  // namespace tpo
