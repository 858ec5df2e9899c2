// Shared by the host side (attention.cu) and the kernels of the attention
// sublayer's operators.  Private to libtpoverlap; include/tpoverlap.h has the
// contract.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "block.h"

namespace tpo {

// [rows, heads, dim] with unit stride in dim: element (i, h, j) at p + i * ld + h * hs + j.
struct Heads {
  const void* p;
  int64_t ld, hs;
};

// Where the sequences lie: rows [q_start[i], q_start[i + 1]) of the queries, and
// of the keys k_len[i] rows from k_start[i] on (k_len NULL: up to k_start[i + 1]).
// Both NULL: one sequence of all rows.
struct Sequences {
  int64_t batch, n, nk;
  const int32_t *q_start, *k_start, *k_len;
};
struct Seq {
  int q0, nq, k0, nk;  // rows of a tensor: at most 2^30
};
// Sequence i, held inside the tensors whatever the arrays say.
__device__ __forceinline__ Seq sequence(const Sequences& s, int64_t i) {
  // all loads before the first use of one
  const int32_t* ke = s.k_len ? s.k_len + i : s.k_start ? s.k_start + i + 1 : nullptr;
  const int64_t q0 = s.q_start ? s.q_start[i] : 0, q1 = s.q_start ? s.q_start[i + 1] : s.n;
  const int64_t k0 = s.k_start ? s.k_start[i] : 0, k1 = ke ? *ke : s.nk;
  auto in = [](int64_t v, int64_t lo, int64_t hi) { return static_cast<int>(v < lo ? lo : v > hi ? hi : v); };
  Seq r;
  r.q0 = in(q0, 0, s.n);
  r.nq = in(q1, r.q0, s.n) - r.q0;
  r.k0 = in(k0, 0, s.nk);
  r.nk = s.k_len ? in(k1, 0, s.nk - r.k0) : in(k1, r.k0, s.nk) - r.k0;
  return r;
}

// Keys that query t of a sequence sees.
__device__ __forceinline__ int keys_seen(const Seq& s, int t, int causal) {
  return causal ? max(0, t - s.nq + 1 + s.nk) : s.nk;
}

struct AttnArgs {
  Sequences seq;
  int64_t heads, kv_heads, dim;
  int causal;
  float scale;
  Heads q, k, v, out;
  float* lse;  // [n, heads]
  Heads dout, dq, dk, dv;
};

// Steps that a tile costs beside its own, where the work is cut into shares: what it takes to fill the pipeline again
// (attention over 8192 tokens took 446, 424, 405 and 406 us with 1 to 4, packed sequences 61, 56, 55 and 53; its
// gradient 786, 785, 789 and 791, of odd sequences 82, 80, 82 and 84).
constexpr int FWD_TILE_COST = 4, BWD_TILE_COST = 2;
// Steps and costs that a launch can count in 32 bits (one more than these says that there are too many).
constexpr int64_t MAX_STEPS = 2147483646;

// Set the kernels' attributes.
cudaError_t configure_attention();
cudaError_t launch_attention(const Machine& mc, const AttnArgs& a, const Watch& w, void* ws, cudaStream_t s);
int64_t need_attention(int64_t n, int64_t nk, int64_t heads, int64_t kv_heads, int64_t dim);
cudaError_t configure_attention_bwd();
cudaError_t launch_attention_bwd(const Machine& mc, const AttnArgs& a, const Watch& w, void* ws, cudaStream_t s);
int64_t need_attention_bwd(int64_t n, int64_t nk, int64_t heads, int64_t kv_heads, int64_t dim);

struct RotaryArgs {
  int64_t n, heads, dim, rot;
  Heads x, y;
  const int32_t *pos, *rows;
  int64_t ny;
  const uint64_t* table;
  float magnitude;
  int layout, inverse;
};
cudaError_t launch_rotary(const Machine& mc, const RotaryArgs& a, int dtype, cudaStream_t s);

}  // namespace tpo
