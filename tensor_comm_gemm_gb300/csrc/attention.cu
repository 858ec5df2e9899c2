// Host side of the attention sublayer's operators: argument checks and the
// launches of each call.  See include/tpoverlap.h for the contract.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn.h"
#include "block_host.h"

using namespace tpo;

namespace {

constexpr int64_t kMaxHeads = 65535, kMaxHeadDim = 128, kMaxGroup = 128, kMaxRotaryDim = 8192;

// An argument [rows, heads, dim] of `elem`-byte elements at pitches ld and hs.
struct HeadsArg {
  const char* name;
  const void* p;
  int64_t rows, heads, dim, ld, hs;
  int elem;
  Heads get() const { return {p, ld, hs}; }
};

// Checks its address and pitches (multiples of `unit` bytes) and replaces the
// pitches that a single row or head does not have.
tpo_status check_heads(HeadsArg& a, int unit) {
  if (a.rows == 0) {
    a.ld = a.hs = round_up(a.dim, 16);
    return TPO_OK;
  }
  if (!a.p || reinterpret_cast<uintptr_t>(a.p) % static_cast<uintptr_t>(unit))
    return fail(TPO_ERR_INVALID_ARG, "%s must be non-NULL and %d-byte aligned", a.name, unit);
  if (a.heads == 1) a.hs = round_up(a.dim, 16);
  if (a.rows == 1) a.ld = round_up(a.dim, 16);
  if (a.ld < a.dim || a.ld > (1ll << 34) || a.hs < a.dim || a.hs > (1ll << 34))
    return fail(TPO_ERR_INVALID_ARG, "%s: pitches %lld of rows and %lld of heads are outside [%lld, 2^34]", a.name,
                (long long)a.ld, (long long)a.hs, (long long)a.dim);
  if (a.ld * a.elem % unit || a.hs * a.elem % unit)
    return fail(TPO_ERR_UNSUPPORTED, "%s: pitches %lld and %lld must be multiples of %d bytes", a.name,
                (long long)a.ld, (long long)a.hs, unit);
  return TPO_OK;
}

tpo_status check_shape(int64_t batch, int64_t n, int64_t nk, int64_t heads, int64_t kv_heads, int64_t dim) {
  if (batch < 1 || batch > kMaxSize || n < 0 || n > kMaxSize || nk < 0 || nk > kMaxSize)
    return fail(TPO_ERR_INVALID_ARG, "sizes out of range: batch=%lld in [1, 2^30], n=%lld and nk=%lld in [0, 2^30]",
                (long long)batch, (long long)n, (long long)nk);
  if (kv_heads < 1 || heads < 1 || heads > kMaxHeads || heads % kv_heads)
    return fail(TPO_ERR_INVALID_ARG, "heads=%lld must be a multiple of kv_heads=%lld, at most %lld", (long long)heads,
                (long long)kv_heads, (long long)kMaxHeads);
  if (heads / kv_heads > kMaxGroup)
    return fail(TPO_ERR_UNSUPPORTED, "%lld heads share one of the keys, at most %lld are supported",
                (long long)(heads / kv_heads), (long long)kMaxGroup);
  if (dim < 1) return fail(TPO_ERR_INVALID_ARG, "dim=%lld must be positive", (long long)dim);
  if (dim % 8 || dim > kMaxHeadDim)
    return fail(TPO_ERR_UNSUPPORTED, "dim=%lld must be a multiple of 8 up to %lld", (long long)dim,
                (long long)kMaxHeadDim);
  return TPO_OK;
}

// The sum over i < count of (a i + b) / m, rounded down; none is negative.  m steps on, a term has grown by a.
int64_t sum_of_quotients(int64_t count, int64_t a, int64_t b, int64_t m) {
  int64_t sum = 0;
  for (int64_t r = 0; r < std::min(count, m); ++r) {
    const int64_t terms = (count - 1 - r) / m + 1;
    sum += terms * ((a * r + b) / m) + a * (terms * (terms - 1) / 2);
  }
  return sum;
}

// Steps and costs of one key head's tiles, as Tiles::range gives them on the device, for a sequence of all rows: of
// queries, `tok` tokens a tile, and (a gradient's) of keys, 128 a tile.
int64_t steps_of_queries(int64_t n, int64_t nk, int64_t tok, bool causal, int64_t cost) {
  if (n == 0) return 0;
  const int64_t tiles = (n + tok - 1) / tok, last = std::max<int64_t>(0, nk - 1) / 128;
  if (!causal) return tiles * (cost + 1 + last);
  // tile i's last token sees nk - n + (i + 1) tok keys, the last tile's all; a key more than 128 j are j steps more
  const int64_t first = n - nk < tok ? 0 : (n - nk) / tok;
  const int64_t before_last = std::max<int64_t>(0, tiles - 1 - first);
  return tiles * (cost + 1) + last + sum_of_quotients(before_last, tok, nk - n + (first + 1) * tok - 1, 128);
}
int64_t steps_of_keys(int64_t n, int64_t nk, int64_t tok, bool causal, int64_t cost) {
  const int64_t tiles = (nk + 127) / 128, queries = std::max<int64_t>(1, (n + tok - 1) / tok);
  if (!causal || n == 0) return tiles * (cost + queries);
  // the queries of the first (128 i - nk + n) / tok tiles do not see tile i's keys
  const int64_t first = nk > n ? (nk - n + 127) / 128 : 0;
  return tiles * (cost + queries) - sum_of_quotients(std::max<int64_t>(0, tiles - first), 128, 128 * first - nk + n, tok);
}

// The device counts a launch's steps in 32 bits.  It checks that itself where it has the lengths.
tpo_status check_steps(const AttnArgs& a, bool gradient) {
  if (a.seq.batch > 1 || a.seq.q_start || a.seq.k_start || a.seq.k_len) return TPO_OK;
  const int64_t n = a.seq.n, nk = a.seq.nk, tok = 128 / (a.heads / a.kv_heads);
  const int64_t most = gradient ? std::max(steps_of_queries(n, nk, tok, a.causal, BWD_TILE_COST),
                                           steps_of_keys(n, nk, tok, a.causal, BWD_TILE_COST))
                                : steps_of_queries(n, nk, 2 * tok, a.causal, FWD_TILE_COST);
  if (most > MAX_STEPS / a.kv_heads)
    return fail(TPO_ERR_UNSUPPORTED, "%lld queries of %lld heads with %lld keys have more than 2^31 - 2 steps",
                (long long)n, (long long)a.heads, (long long)nk);
  return TPO_OK;
}

// Also lets keys that have no arrays of their own lie as the queries do.
tpo_status check_sequences(Sequences& s, float scale) {
  if (!(scale > 0.0f) || scale > 1e38f) return fail(TPO_ERR_INVALID_ARG, "scale must be positive, at most 1e38");
  if (tpo_status st = check_vec("q_start", s.q_start, 4)) return st;
  if (tpo_status st = check_vec("k_start", s.k_start, 4)) return st;
  if (tpo_status st = check_vec("k_len", s.k_len, 4)) return st;
  if (s.batch > 1 && !s.q_start) return fail(TPO_ERR_INVALID_ARG, "q_start is needed with more than one sequence");
  if (!s.k_start && !s.k_len) s.k_start = s.q_start;
  if (s.batch > 1 && !s.k_start) return fail(TPO_ERR_INVALID_ARG, "k_start is needed with k_len and more than one sequence");
  return TPO_OK;
}

}  // namespace

extern "C" {

tpo_status tpo_rotary_table(int64_t rot, double base, int scaling, double factor, double low, double high,
                            int64_t original, uint64_t* table) {
  if (rot < 0 || rot % 2 || rot > kMaxRotaryDim)
    return fail(TPO_ERR_INVALID_ARG, "rot=%lld must be even, in [0, %lld]", (long long)rot, (long long)kMaxRotaryDim);
  if (!(base > 0.0) || std::isinf(base)) return fail(TPO_ERR_INVALID_ARG, "base must be positive and finite");
  if (scaling < TPO_ROTARY_UNSCALED || scaling > TPO_ROTARY_BY_PARTS)
    return fail(TPO_ERR_INVALID_ARG, "scaling=%d is not a tpo_rotary_scaling", scaling);
  if (scaling != TPO_ROTARY_UNSCALED && (!(factor > 0.0) || std::isinf(factor)))
    return fail(TPO_ERR_INVALID_ARG, "factor must be positive and finite");
  if (scaling == TPO_ROTARY_BY_PARTS && (!(low < high) || std::isinf(low) || std::isinf(high) || original < 1))
    return fail(TPO_ERR_INVALID_ARG, "low must be less than high, and original at least 1");
  if (!table && rot > 0) return fail(TPO_ERR_INVALID_ARG, "table must be non-NULL");
  constexpr double kTurn = 6.283185307179586476925;
  auto turns_of = [&](int64_t i) {  // pair i's, a position
    double f = std::pow(base, -2.0 * static_cast<double>(i) / static_cast<double>(rot));
    if (scaling == TPO_ROTARY_LINEAR) f /= factor;
    if (scaling == TPO_ROTARY_BY_PARTS) {
      const double turns = static_cast<double>(original) * f / kTurn;
      const double keep = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
      f *= keep + (1.0 - keep) / factor;
    }
    return f / kTurn;
  };
  for (int64_t i = 0; i < rot / 2; ++i)
    if (!std::isfinite(turns_of(i)))
      return fail(TPO_ERR_INVALID_ARG, "the frequency of pair %lld is not finite: base=%g, factor=%g", (long long)i, base,
                  factor);
  for (int64_t i = 0; i < rot / 2; ++i) {
    const double turns = turns_of(i);
    table[i] = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 64));  // below 2^64: 53 bits
  }
  return TPO_OK;
}

tpo_status tpo_rotary(tpo_block* b, int64_t n, int64_t heads, int64_t dim, int64_t rot, int dtype, int layout,
                      int inverse, float magnitude, const int32_t* pos, const uint64_t* table, const void* x,
                      int64_t ldx, int64_t hx, const int32_t* rows, int64_t ny, void* y, int64_t ldy, int64_t hy,
                      void* stream) {
  if (n < 0 || n > kMaxSize || heads < 1 || heads > kMaxHeads || dim < 1 || dim > kMaxRotaryDim || ny < 0 ||
      ny > (1ll << 31))
    return fail(TPO_ERR_INVALID_ARG,
                "sizes out of range: n=%lld in [0, 2^30], heads=%lld in [1, %lld], dim=%lld in [1, %lld], ny=%lld in "
                "[0, 2^31]", (long long)n, (long long)heads, (long long)kMaxHeads, (long long)dim,
                (long long)kMaxRotaryDim, (long long)ny);
  if (rot < 0 || rot > dim || rot % 2)
    return fail(TPO_ERR_INVALID_ARG, "rot=%lld must be even, in [0, dim=%lld]", (long long)rot, (long long)dim);
  if (dtype != TPO_BF16 && dtype != TPO_F32)
    return fail(TPO_ERR_INVALID_ARG, "rotary types are TPO_BF16 (0) or TPO_F32 (2): dtype=%d", dtype);
  if (layout != TPO_ROTARY_HALVES && layout != TPO_ROTARY_PAIRS)
    return fail(TPO_ERR_INVALID_ARG, "layout=%d is not a tpo_rotary_layout", layout);
  if (!std::isfinite(magnitude)) return fail(TPO_ERR_INVALID_ARG, "magnitude must be finite");
  if (!rows && ny != n) return fail(TPO_ERR_INVALID_ARG, "without rows, ny=%lld must be n=%lld", (long long)ny, (long long)n);
  const int elem = dtype == TPO_F32 ? 4 : 2;
  HeadsArg ax{"x", x, n, heads, dim, ldx, hx, elem}, ay{"y", y, ny, heads, dim, ldy, hy, elem};
  if (tpo_status st = check_heads(ax, elem)) return st;
  if (tpo_status st = check_heads(ay, elem)) return st;
  if (tpo_status st = check_vec("pos", pos, 4)) return st;
  if (tpo_status st = check_vec("rows", rows, 4)) return st;
  if (n > 0 && rot > 0 && (!table || reinterpret_cast<uintptr_t>(table) % 8))
    return fail(TPO_ERR_INVALID_ARG, "table must be non-NULL and 8-byte aligned");
  if (n > 0 && x == y && (rows || ax.ld != ay.ld || ax.hs != ay.hs))
    return fail(TPO_ERR_INVALID_ARG, "y may be x only with the same pitches and without rows");
  if (tpo_status st = check_block(b, 0)) return st;
  if (n == 0 || ny == 0) return TPO_OK;
  RotaryArgs a{};
  a.n = n, a.heads = heads, a.dim = dim, a.rot = rot, a.x = ax.get(), a.y = ay.get(), a.pos = pos, a.rows = rows;
  a.ny = ny, a.table = table, a.magnitude = magnitude, a.layout = layout, a.inverse = inverse != 0;
  return launched(launch_rotary(b->machine, a, dtype, static_cast<cudaStream_t>(stream)));
}

int64_t tpo_attention_workspace(int64_t n, int64_t nk, int64_t heads, int64_t kv_heads, int64_t dim) {
  if (check_shape(1, n, nk, heads, kv_heads, dim) != TPO_OK) return -1;
  return need_attention(n, nk, heads, kv_heads, dim);
}

int64_t tpo_attention_bwd_workspace(int64_t n, int64_t nk, int64_t heads, int64_t kv_heads, int64_t dim) {
  if (check_shape(1, n, nk, heads, kv_heads, dim) != TPO_OK) return -1;
  return need_attention_bwd(n, nk, heads, kv_heads, dim);
}

tpo_status tpo_attention(tpo_block* b, int64_t batch, int64_t n, int64_t nk, int64_t heads, int64_t kv_heads,
                         int64_t dim, const int32_t* q_start, const int32_t* k_start, const int32_t* k_len, int causal,
                         float scale, const void* q, int64_t ldq, int64_t hq, const void* k, int64_t ldk, int64_t hk,
                         const void* v, int64_t ldv, int64_t hv, void* out, int64_t ldo, int64_t ho, float* lse,
                         void* stream) {
  if (tpo_status st = check_shape(batch, n, nk, heads, kv_heads, dim)) return st;
  AttnArgs a{};
  a.seq = {batch, n, nk, q_start, k_start, k_len};
  if (tpo_status st = check_sequences(a.seq, scale)) return st;
  a.heads = heads, a.kv_heads = kv_heads, a.dim = dim, a.causal = causal != 0, a.scale = scale;
  if (tpo_status st = check_steps(a, false)) return st;
  HeadsArg aq{"q", q, n, heads, dim, ldq, hq, 2}, ak{"k", k, nk, kv_heads, dim, ldk, hk, 2},
      av{"v", v, nk, kv_heads, dim, ldv, hv, 2}, ao{"out", out, n, heads, dim, ldo, ho, 2};
  HeadsArg* need[] = {&aq, &ak, &av, &ao};
  for (HeadsArg* h : need)
    if (tpo_status st = check_heads(*h, 16)) return st;
  if (tpo_status st = check_vec("lse", lse, 4)) return st;
  if (tpo_status st = check_block(b, need_attention(n, nk, heads, kv_heads, dim))) return st;
  if (n == 0) return TPO_OK;
  a.q = aq.get(), a.k = ak.get(), a.v = av.get(), a.out = ao.get(), a.lse = lse;
  return launched(launch_attention(b->machine, a, b->watch(), b->ws(), static_cast<cudaStream_t>(stream)));
}

tpo_status tpo_attention_bwd(tpo_block* b, int64_t batch, int64_t n, int64_t nk, int64_t heads, int64_t kv_heads,
                             int64_t dim, const int32_t* q_start, const int32_t* k_start, const int32_t* k_len,
                             int causal, float scale, const void* dout, int64_t lddo, int64_t hdo, const void* q,
                             int64_t ldq, int64_t hq, const void* k, int64_t ldk, int64_t hk, const void* v,
                             int64_t ldv, int64_t hv, const void* out, int64_t ldo, int64_t ho, const float* lse,
                             void* dq, int64_t lddq, int64_t hdq, void* dk, int64_t lddk, int64_t hdk, void* dv,
                             int64_t lddv, int64_t hdv, void* stream) {
  if (tpo_status st = check_shape(batch, n, nk, heads, kv_heads, dim)) return st;
  AttnArgs a{};
  a.seq = {batch, n, nk, q_start, k_start, k_len};
  if (tpo_status st = check_sequences(a.seq, scale)) return st;
  a.heads = heads, a.kv_heads = kv_heads, a.dim = dim, a.causal = causal != 0, a.scale = scale;
  if (tpo_status st = check_steps(a, true)) return st;
  HeadsArg ado{"dout", dout, n, heads, dim, lddo, hdo, 2}, aq{"q", q, n, heads, dim, ldq, hq, 2},
      ak{"k", k, nk, kv_heads, dim, ldk, hk, 2}, av{"v", v, nk, kv_heads, dim, ldv, hv, 2},
      ao{"out", out, n, heads, dim, ldo, ho, 2}, adq{"dq", dq, n, heads, dim, lddq, hdq, 2},
      adk{"dk", dk, nk, kv_heads, dim, lddk, hdk, 2}, adv{"dv", dv, nk, kv_heads, dim, lddv, hdv, 2};
  HeadsArg* need[] = {&ado, &aq, &ak, &av, &ao, &adq, &adk, &adv};
  for (HeadsArg* h : need)
    if (tpo_status st = check_heads(*h, 16)) return st;
  if (n > 0 && !lse) return fail(TPO_ERR_INVALID_ARG, "lse of the forward call is needed");
  if (tpo_status st = check_vec("lse", lse, 4)) return st;
  if (tpo_status st = check_block(b, need_attention_bwd(n, nk, heads, kv_heads, dim))) return st;
  if (n == 0 && nk == 0) return TPO_OK;
  a.q = aq.get(), a.k = ak.get(), a.v = av.get(), a.out = ao.get(), a.lse = const_cast<float*>(lse);
  a.dout = ado.get(), a.dq = adq.get(), a.dk = adk.get(), a.dv = adv.get();
  return launched(
      launch_attention_bwd(b->machine, a, b->watch(), b->ws(), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
