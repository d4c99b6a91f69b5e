// Log probabilities of given tokens with entropy and best alternatives, and
// their gradient (sm_103a).
//
// With z = scale * logits, m = max z, S = sum e^(z - m), Q = sum e^(z - m)(z - m):
//   lse = m + log S,   logp = (z_id - m) - log S,   entropy = log S - Q / S.
// One pass over the logits: every thread keeps a running (m, S, Q); when the
// maximum grows by t = m_old - m_new <= 0, S <- S e^t and Q <- e^t (Q + t S).
// Pairs of partial results are joined by the same rule.  Everything is taken
// from differences to the maximum, so an offset common to the row does not
// cancel digits; lse, which holds the offset, comes with the remainder of its
// rounding, so that the gradient can form p = e^((z - lse) - rest) without it
// (a row of nothing but the type's lowest value has lse = that value: without
// the remainder every p would be 1).
//
// A row is read by a cluster of 1 to 8 CTAs (few long rows need many SMs);
// partial results are joined through shared memory and then distributed
// shared memory.  A thread loads 32 values at a time, so one look at their
// maximum serves all of them; an exponential, a clamp and five additions and
// products are left per value (two values an instruction where the hardware
// has it), which a bf16 row just hides under its loads.
//
// Best alternatives are found from maxima.  A key is 64 bits, the
// order-preserving image of the logit above the complement of the column, so
// equal logits rank by column and no two keys are equal.  Each thread keeps
// the maximum of every 32 values it has read.  If k threads have seen a value
// of at least b, the k best are at least b; such a bound is taken from the
// threads' maxima, few values reach it, and these are read once more, where a
// maximum says so, and ranked by counting.  If more values reach the bound
// than the list holds (many equal logits), the row is read again and each
// warp keeps a sorted list of its 32 best keys, into which it inserts one at a
// time.
//
// Measured, 8192 x 32000 bf16: 97 us (80% of the copy rate), with 20 alternatives
// 137; gradient 152 (the copy rate) with the entropy's term and without; 1024 x
// 128257 fp32 with 20 alternatives 92 (84%).
#include <cooperative_groups.h>
#include <math_constants.h>

#include "okls_internal.h"
#include "okls_lm.cuh"

namespace cg = cooperative_groups;

namespace okls {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFar = -200.0f;  // e^-200 is 0 in fp32: bounds a difference to the maximum

struct Stat {
  float m, s, q;
};

__device__ __forceinline__ Stat stat_join(const Stat& a, const Stat& b) {
  Stat r;
  r.m = fmaxf(a.m, b.m);
  // a side without a possible value (m = -inf, s = 0) has weight 0
  const float ta = fmaxf(a.m - r.m, kFar), tb = fmaxf(b.m - r.m, kFar);
  const float ea = a.m == -CUDART_INF_F ? 0.0f : exp2f(ta * kLog2e);
  const float eb = b.m == -CUDART_INF_F ? 0.0f : exp2f(tb * kLog2e);
  r.s = a.s * ea + b.s * eb;
  r.q = (ea > 0.0f ? ea * fmaf(ta, a.s, a.q) : a.q * 0.0f) + (eb > 0.0f ? eb * fmaf(tb, b.s, b.q) : b.q * 0.0f);
  return r;
}

__device__ __forceinline__ Stat stat_shfl_xor(const Stat& a, int o) {
  return {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o),
          __shfl_xor_sync(0xffffffffu, a.q, o)};
}

// ------------------------------------------------------------ alternatives
typedef unsigned long long Key;

// fp32 order as unsigned order; -0 counts as 0 and NaN as -inf
__device__ __forceinline__ uint32_t ord_bits(float v) {
  if (v != v) v = -CUDART_INF_F;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float ord_value(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u ^ 0x80000000u) : ~u);
}
__device__ __forceinline__ Key make_key(float v, uint32_t col) {
  return (static_cast<Key>(ord_bits(v)) << 32) | static_cast<Key>(~col);
}

// Insert one key (the same in all lanes) into the warp's list, which is
// sorted downwards across the lanes.
__device__ __forceinline__ void list_insert(Key& mine, Key cand, int lane) {
  const int at = __popc(__ballot_sync(0xffffffffu, mine > cand));
  const Key up = __shfl_up_sync(0xffffffffu, mine, 1);
  if (lane > at) mine = up;
  if (lane == at) mine = cand;
}

// The 32 best of two sorted lists, sorted: the larger of a[i] and b[31 - i]
// form a bitonic list of them, which five compare-exchange steps sort.
template <class V>
__device__ __forceinline__ V list_merge(V a, V b, int lane) {
  const V rb = __shfl_sync(0xffffffffu, b, 31 - lane);
  V v = a > rb ? a : rb;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const V w = __shfl_xor_sync(0xffffffffu, v, o);
    const bool keep_max = (lane & o) == 0;
    v = keep_max ? (v > w ? v : w) : (v > w ? w : v);
  }
  return v;
}

// 128 threads: a row's fixed costs are a CTA's, so small CTAs hide them under
// other rows' loads (8192 x 32000 bf16: 512 threads 144 us, 256 110, 128 96).
constexpr int kScoreThreads = 128;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kVecs = 4;  // vectors of 8 values a thread loads at a time
// A row goes to one warp when it is short, or when there are rows for 16
// warps on every SM (bf16, a CTA a row against a warp: 8192 x 4000 22 and 13 us,
// 8192 x 16000 56 and 48); longer rows leave the SMs unevenly filled.
constexpr int kWarpRow = 16384, kWarpRowFew = 4096;

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Two fp32 values in one instruction.
typedef unsigned long long Pair;
__device__ __forceinline__ Pair pair_of(float lo, float hi) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(Pair p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

struct Best {
  Key list;
  Key bound;  // keys at or below it cannot be among the k best
  float bound_v;
};

// The lanes' values in descending order (bitonic).
template <class V>
__device__ __forceinline__ V sort_lanes(V v, int lane) {
#pragma unroll
  for (int w = 2; w <= 32; w <<= 1)
#pragma unroll
    for (int o = w >> 1; o > 0; o >>= 1) {
      const V x = __shfl_xor_sync(0xffffffffu, v, o);
      // descending in even blocks of w lanes, ascending in odd ones
      const bool keep_max = ((lane & o) == 0) == ((lane & w) == 0);
      v = keep_max ? (v > x ? v : x) : (v > x ? x : v);
    }
  return v;
}

// Offers the warp's values to its list: lane values z[j], j < count, whose
// columns are col + (j / W) * stride + j % W of the row at `row`; vm is the
// lane's maximum.
template <class T, int N, int W>
__device__ __forceinline__ void offer(Best& B, const float (&z)[N], float vm, int count, const T* row, uint32_t col,
                                      uint32_t stride, int lane, int k, Key* cta_bound) {
  // one lane reads it for the warp: other warps raise it at any time, and the
  // steps below need every lane to hold the same bound
  Key shared = 0;
  if (lane == 0) shared = *reinterpret_cast<volatile Key*>(cta_bound);
  shared = __shfl_sync(0xffffffffu, shared, 0);
  if (shared > B.bound) {
    B.bound = shared;
    B.bound_v = ord_value(static_cast<uint32_t>(shared >> 32));
  }
  if (!__any_sync(0xffffffffu, count > 0 && !(vm < B.bound_v))) return;
  if (N > 1 && B.bound == 0) {
    // the k-th best of 32 of the warp's values, one a lane
    const uint32_t kth = __shfl_sync(0xffffffffu, sort_lanes(count > 0 ? ord_bits(vm) : 0u, lane), k - 1);
    if (kth > 0) B.bound = (static_cast<Key>(kth) << 32) - 1;
    B.bound_v = kth > 0 ? ord_value(kth - 1) : -CUDART_INF_F;
  }
  uint32_t mask = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) mask |= !(z[j] < B.bound_v) ? 1u << j : 0u;
  if (count < 32) mask &= (1u << count) - 1u;
  while (__any_sync(0xffffffffu, mask != 0)) {
    Key cand = 0;
    if (mask) {
      const int j = __ffs(mask) - 1;
      mask &= mask - 1;
      const uint32_t c = col + static_cast<uint32_t>(j / W) * stride + static_cast<uint32_t>(j % W);
      cand = make_key(to_f32(row[c]), c);
    }
    unsigned todo = __ballot_sync(0xffffffffu, cand > B.bound);
    while (todo) {
      const int src = __ffs(todo) - 1;
      todo &= todo - 1;
      const Key c = __shfl_sync(0xffffffffu, cand, src);
      if (c > B.bound) {
        list_insert(B.list, c, lane);
        const Key kth = __shfl_sync(0xffffffffu, B.list, k - 1);
        if (kth > B.bound) B.bound = kth;
      }
    }
  }
  if (B.bound) B.bound_v = ord_value(static_cast<uint32_t>(B.bound >> 32));
  if (lane == 0 && B.bound) atomicMax(cta_bound, B.bound);
}

// Adds N values of this lane to its running sums (values that are not there
// are -inf); returns their maximum.
template <int N, bool SCALED>
__device__ __forceinline__ float take(Stat& L, const float (&z)[N], float scale) {
  float vm = z[0];
#pragma unroll
  for (int j = 1; j < N; ++j) vm = max_nan(vm, z[j]);
  // products are rounded before the differences, as m was: a fused difference
  // would leave the rounding error of a huge masked logit
  const float top = SCALED ? __fmul_rn(vm, scale) : vm;
  if (top != top) {
    L.s = top;  // the row's sums are NaN from here on; the others still rank
#pragma unroll
    for (int j = 0; j < N; ++j) vm = fmaxf(vm, z[j]);
    return vm;
  }
  if (top > L.m) {
    if (L.m == -CUDART_INF_F) {
      // no possible value so far: s and q are 0 (or NaN, which stays)
      L.m = top;
    } else {
      const float t = fmaxf(L.m - top, kFar);
      const float f = ex2(t * kLog2e);
      L.q = f * fmaf(t, L.s, L.q);
      L.s *= f;
      L.m = top;
    }
  }
  if (L.m == -CUDART_INF_F) return vm;  // impossible values only
  Pair s = pair_of(0.0f, 0.0f), q = s;
  const Pair minus_m = pair_of(-L.m, -L.m), l2e = pair_of(kLog2e, kLog2e), sc = pair_of(scale, scale);
#pragma unroll
  for (int j = 0; j + 1 < N; j += 2) {
    Pair v = pair_of(z[j], z[j + 1]);
    if (SCALED) v = mul2(v, sc);
    float d0, d1, x0, x1;
    unpair(add2(v, minus_m), d0, d1);
    const Pair d = pair_of(fmaxf(d0, kFar), fmaxf(d1, kFar));
    unpair(mul2(d, l2e), x0, x1);
    const Pair e = pair_of(ex2(x0), ex2(x1));
    s = add2(s, e);
    q = fma2(e, d, q);
  }
  float s0, s1, q0, q1;
  unpair(s, s0, s1);
  unpair(q, q0, q1);
  if (N & 1) {
    const float d = fmaxf((SCALED ? __fmul_rn(z[N - 1], scale) : z[N - 1]) - L.m, kFar);
    const float e = ex2(d * kLog2e);
    s0 += e;
    q0 = fmaf(e, d, q0);
  }
  L.s += s0 + s1;
  L.q += q0 + q1;
  return vm;
}

// Results of a row from the sums L (the same in all lanes) and the list.
template <class T, bool TOP>
__device__ __forceinline__ void write_row(const ScoreArgs& A, int64_t row, const T* z, const Stat& L, Key best, int lane,
                                          int k) {
  const bool none = L.m == -CUDART_INF_F && L.s == 0.0f;  // no possible token
  // a sum that is NaN (a NaN logit) makes everything NaN, and so does an
  // infinite maximum, whose sum is 0
  const float logs = logf(L.s);
  const float lse = none ? -CUDART_INF_F : (L.s != L.s ? L.s : __fadd_rn(L.m, logs));
  // a log probability is -inf where no token is possible
  auto logp_of = [&](float v) { return none ? -CUDART_INF_F : __fsub_rn(__fsub_rn(__fmul_rn(v, A.scale), L.m), logs); };
  if (lane == 0) {
    if (A.lse) A.lse[row] = lse;
    if (A.lse_rest) {
      // m + log S - lse exactly: the error of a rounded sum of two, whichever is larger
      const float t = __fsub_rn(lse, L.m);
      const float rest = __fadd_rn(__fsub_rn(L.m, __fsub_rn(lse, t)), __fsub_rn(logs, t));
      A.lse_rest[row] = none ? 0.0f : rest;
    }
    if (A.entropy) A.entropy[row] = none ? 0.0f : logs - L.q / L.s;
    if (A.logp) {
      const int64_t id = token_at(A.ids, A.ids_i64, row);
      if (id >= A.vocab) atomicOr(A.status, kStBadToken);
      float lp = 0.0f;
      if (id >= 0 && id < A.vocab) lp = logp_of(to_f32(z[id]));
      A.logp[row] = lp;
    }
  }
  if (TOP && lane < k) {
    const uint32_t col = ~static_cast<uint32_t>(best);
    A.top_ids[row * k + lane] = static_cast<int32_t>(col);
    A.top_logp[row * k + lane] = logp_of(ord_value(static_cast<uint32_t>(best >> 32)));
  }
}

// How a row lies in memory: a 16-byte aligned body of vectors of 8 columns,
// and fewer than 16 columns before and after it, taken one by one.
struct Layout {
  int64_t head, nvec, tail0, edge;
};
template <class T>
__device__ __forceinline__ Layout layout_of(const T* z, int64_t vocab) {
  Layout Y;
  const int64_t mis = (reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T);
  Y.head = min(vocab, mis ? static_cast<int64_t>(16 / sizeof(T)) - mis : int64_t(0));
  Y.nvec = (vocab - Y.head) / 8;
  Y.tail0 = Y.head + Y.nvec * 8;
  Y.edge = Y.head + (vocab - Y.tail0);
  return Y;
}

// Values of kVecs vectors i, i + step, ... of this lane (-inf where there are
// none); returns how many there are.
template <class T>
__device__ __forceinline__ int load_block(const T* z, const Layout& Y, int64_t i, int64_t step, float (&v)[kVecs * 8]) {
  int count = 0;
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    float t[8];
    if (i + u * step < Y.nvec) {
      load8(z + Y.head + (i + u * step) * 8, t);
      count += 8;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = -CUDART_INF_F;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[u * 8 + j] = t[j];
  }
  return count;
}

// Sums of a warp's share of a row: vectors first + lane, + step, ... and, for
// the first share, the columns outside the body.  With TOP, block b's maximum
// goes to maxima[b * stride], and `most` is the thread's maximum (order bits,
// 0 where it has read nothing).
template <class T, bool TOP, bool SCALED>
__device__ __forceinline__ void read_row(const ScoreArgs& A, const T* z, const Layout& Y, int64_t first, int64_t step,
                                         Stat& L, int lane, float* maxima, int stride, uint32_t& most, float& edge_v) {
  int b = 0;
  most = 0;
  for (int64_t v0 = first; v0 < Y.nvec; v0 += step * kVecs, ++b) {
    float v[kVecs * 8];
    const int count = load_block(z, Y, v0 + lane, step, v);
    const float vm = take<kVecs * 8, SCALED>(L, v, A.scale);
    if (TOP) {
      maxima[b * stride] = vm;
      if (count > 0) most = max(most, ord_bits(vm));
    }
  }
  edge_v = 0.0f;
  if (first == 0 && Y.edge > 0) {
    const int64_t col = lane < Y.head ? lane : Y.tail0 + (lane - Y.head);
    edge_v = lane < Y.edge ? to_f32(z[col]) : -CUDART_INF_F;
    float v[1] = {edge_v};
    take<1, SCALED>(L, v, A.scale);
    if (TOP && lane < Y.edge) most = max(most, ord_bits(edge_v));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L = stat_join(L, stat_shfl_xor(L, o));
}

constexpr uint32_t kOrdNegInf = 0x007FFFFFu;  // ord_bits(-inf)

// Appends a key to list[0 .. cap); the count goes on past cap.
__device__ __forceinline__ void push_key(float v, uint32_t col, Key* list, int cap, int* count) {
  const int at = atomicAdd(count, 1);
  if (at < cap) list[at] = make_key(v, col);
}

// The least possible value that `bound` (order bits) lets through.
__device__ __forceinline__ float least_value(uint32_t bound) {
  return ord_value(bound > kOrdNegInf ? bound : kOrdNegInf + 1);
}

// When fewer than k threads have seen a possible value, impossible ones are
// among the best; their first k columns are enough of them.
template <class T>
__device__ __forceinline__ void collect_impossible(const T* z, int64_t vocab, int t, int k, Key* list, int cap, int* count) {
  if (t >= k || t >= vocab) return;
  const float v = to_f32(z[t]);
  if (ord_bits(v) == kOrdNegInf) push_key(v, static_cast<uint32_t>(t), list, cap, count);
}

// Rank of thread t's key among list[0 .. n).
__device__ __forceinline__ int rank_of(Key mine, const Key* list, int n) {
  int r = 0;
#pragma unroll 8
  for (int j = 0; j < n; ++j) r += list[j] > mine ? 1 : 0;
  return r;
}

// The list by insertion, for any row.
template <class T>
__device__ __forceinline__ Key insert_row(const T* z, const Layout& Y, int64_t first, int64_t step, int lane, int k,
                                          Key* bound) {
  Best B = {0, 0, -CUDART_INF_F};
  for (int64_t v0 = first; v0 < Y.nvec; v0 += step * kVecs) {
    float v[kVecs * 8];
    const int count = load_block(z, Y, v0 + lane, step, v);
    float vm = v[0];
#pragma unroll
    for (int j = 1; j < kVecs * 8; ++j) vm = fmaxf(vm, v[j]);
    offer<T, kVecs * 8, 8>(B, v, vm, count, z, static_cast<uint32_t>(Y.head + (v0 + lane) * 8),
                           static_cast<uint32_t>(step * 8), lane, k, bound);
  }
  if (first == 0 && Y.edge > 0) {
    const int64_t col = lane < Y.head ? lane : Y.tail0 + (lane - Y.head);
    float v[1] = {lane < Y.edge ? to_f32(z[col]) : -CUDART_INF_F};
    offer<T, 1, 1>(B, v, v[0], lane < Y.edge ? 1 : 0, z, static_cast<uint32_t>(col), 0u, lane, k, bound);
  }
  return B.list;
}

// Short rows: a warp each.
constexpr int kWarpList = 256;  // keys; a row whose bound is 0 has fewer columns
constexpr int kWarpBlocks = static_cast<int>((kWarpRow + 32 * 8 * kVecs - 1) / (32 * 8 * kVecs));
template <class T, bool TOP, bool SCALED>
__global__ void __launch_bounds__(kScoreThreads) k_token_logprobs_warp(const ScoreArgs A) {
  __shared__ Key lists[TOP ? kScoreWarps : 1][TOP ? kWarpList : 1];
  __shared__ float maxima[TOP ? kScoreWarps : 1][TOP ? kWarpBlocks : 1][32];
  __shared__ Key bounds[kScoreWarps];
  __shared__ int counts[kScoreWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k = TOP ? A.top_k : 1;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kScoreWarps + warp;
  if (row >= A.rows) return;
  const T* z = static_cast<const T*>(A.logits) + row * A.ldl;
  const Layout Y = layout_of(z, A.vocab);
  Stat L = {-CUDART_INF_F, 0.0f, 0.0f};
  uint32_t most;
  float edge_v;
  float* mine = TOP ? &maxima[warp][0][lane] : nullptr;
  read_row<T, TOP, SCALED>(A, z, Y, 0, 32, L, lane, mine, 32, most, edge_v);
  Key best = 0;
  if (TOP) {
    Key* list = lists[warp];
    if (lane == 0) counts[warp] = 0, bounds[warp] = 0;
    // the k-th largest of the lanes' maxima
    const uint32_t bound = __shfl_sync(0xffffffffu, sort_lanes(most, lane), k - 1);
    const float least = least_value(bound);
    __syncwarp();
    int b = 0;
    for (int64_t v0 = 0; v0 < Y.nvec; v0 += 32 * kVecs, ++b) {
      if (!(mine[b * 32] >= least)) continue;
      float v[kVecs * 8];
      load_block(z, Y, v0 + lane, 32, v);
      const uint32_t col = static_cast<uint32_t>(Y.head + (v0 + lane) * 8);
#pragma unroll
      for (int j = 0; j < kVecs * 8; ++j)
        if (v[j] >= least) push_key(v[j], col + (j / 8) * 256 + j % 8, list, kWarpList, &counts[warp]);
    }
    if (lane < Y.edge && edge_v >= least)
      push_key(edge_v, static_cast<uint32_t>(lane < Y.head ? lane : Y.tail0 + (lane - Y.head)), list, kWarpList, &counts[warp]);
    if (bound <= kOrdNegInf) collect_impossible(z, A.vocab, lane, k, list, kWarpList, &counts[warp]);
    __syncwarp();
    const int n = counts[warp];
    if (n <= kWarpList) {
      // every lane ranks up to 8 keys before any is moved
      Key key[kWarpList / 32];
      int at[kWarpList / 32];
#pragma unroll
      for (int i = 0; i < kWarpList / 32; ++i) {
        at[i] = 32;
        if (i * 32 < n && i * 32 + lane < n) {
          key[i] = list[i * 32 + lane];
          at[i] = rank_of(key[i], list, n);
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kWarpList / 32; ++i)
        if (at[i] < 32) list[at[i]] = key[i];
      __syncwarp();
      best = list[lane];
    } else {
      best = insert_row(z, Y, 0, 32, lane, k, &bounds[warp]);
    }
  }
  write_row<T, TOP>(A, row, z, L, best, lane, k);
}

// Longer rows: a cluster of CTAs each.
constexpr int kCtaBlocks = 32;  // maxima a thread keeps: 131072 columns a CTA
constexpr int kCtaList = 256;   // keys
constexpr int kHits = 512;
template <class T, bool TOP, bool SCALED>
__global__ void __launch_bounds__(kScoreThreads) k_token_logprobs(const ScoreArgs A, int keep_maxima) {
  __shared__ Stat stats[kScoreWarps];
  __shared__ Stat cta_stat;
  __shared__ Key list[TOP ? kCtaList : 1];  // candidates, or the warps' lists
  __shared__ Key sorted[32];                        // the CTA's best
  __shared__ uint16_t hits[TOP ? kHits : 1];        // (thread, block) whose maximum reaches the bound
  __shared__ uint32_t tops[kScoreWarps];
  __shared__ float maxima[TOP ? kCtaBlocks : 1][kScoreThreads];
  __shared__ Key cta_bound;
  __shared__ int count, nhits;
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank(), nct = cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int k = TOP ? A.top_k : 1;
  const int64_t row = blockIdx.x / nct;
  const T* z = static_cast<const T*>(A.logits) + row * A.ldl;
  const Layout Y = layout_of(z, A.vocab);
  const int64_t first = int64_t(rank) * kScoreThreads + warp * 32, step = int64_t(nct) * kScoreThreads;
  Stat L = {-CUDART_INF_F, 0.0f, 0.0f};
  uint32_t most;
  float edge_v;
  // a row too long for the maxima overwrites one and is read again
  const int stride = TOP && keep_maxima ? kScoreThreads : 0;
  read_row<T, TOP, SCALED>(A, z, Y, first, step, L, lane, &maxima[0][tid], stride, most, edge_v);

  // join: warps, CTAs
  if (lane == 0) stats[warp] = L;
  if (TOP) {
    // the m-th largest maximum of each warp, m = ceil(k / warps): the least
    // of these is reached by k threads
    uint32_t left = most, mth = 0;
    for (int i = 0; i < (k + kScoreWarps - 1) / kScoreWarps; ++i) {
      mth = __reduce_max_sync(0xffffffffu, left);
      const unsigned who = __ballot_sync(0xffffffffu, left == mth);
      if (lane == __ffs(who) - 1) left = 0;
    }
    if (lane == 0) tops[warp] = mth;
    if (tid == 0) count = 0, nhits = 0, cta_bound = 0;
    if (tid < 32) sorted[tid] = 0;
  }
  __syncthreads();
  if (warp == 0) {
    L = stats[lane & (kScoreWarps - 1)];  // every kScoreWarps lanes form the same sum
#pragma unroll
    for (int o = kScoreWarps / 2; o > 0; o >>= 1) L = stat_join(L, stat_shfl_xor(L, o));
    if (lane == 0) cta_stat = L;
  }
  if (TOP) {
    uint32_t bound = 0xFFFFFFFFu;
#pragma unroll
    for (int w = 0; w < kScoreWarps; ++w) bound = min(bound, tops[w]);
    const float least = least_value(bound);
    if (keep_maxima) {
      const int blocks = static_cast<int>((Y.nvec - first + step * kVecs - 1) / (step * kVecs));
      for (int b = 0; b < blocks; ++b)
        if (maxima[b][tid] >= least) {
          const int at = atomicAdd(&nhits, 1);
          if (at < kHits) hits[at] = static_cast<uint16_t>(b * kScoreThreads + tid);
        }
      if (first == 0 && lane < Y.edge && edge_v >= least)
        push_key(edge_v, static_cast<uint32_t>(lane < Y.head ? lane : Y.tail0 + (lane - Y.head)), list, kCtaList, &count);
      if (rank == 0 && bound <= kOrdNegInf) collect_impossible(z, A.vocab, tid, k, list, kCtaList, &count);
      __syncthreads();
      // a warp reads the 32 values of a hit, one a lane
      const int nh = nhits <= kHits ? nhits : 0;
#pragma unroll 4
      for (int h = warp; h < nh; h += kScoreWarps) {
        const int64_t i = int64_t(rank) * kScoreThreads + hits[h] % kScoreThreads +
                          ((hits[h] / kScoreThreads) * kVecs + lane / 8) * step;
        const int64_t col = Y.head + i * 8 + lane % 8;
        const float v = i < Y.nvec ? to_f32(z[col]) : -CUDART_INF_F;
        if (v >= least) push_key(v, static_cast<uint32_t>(col), list, kCtaList, &count);
      }
      if (tid == 0 && nhits > kHits) count = kCtaList + 1;
    } else if (tid == 0) {
      count = kCtaList + 1;
    }
    __syncthreads();
    const int n = count;
    if (n <= kCtaList) {
      for (int i = tid; i < n; i += kScoreThreads) {
        const Key mine = list[i];
        const int at = rank_of(mine, list, n);
        if (at < 32) sorted[at] = mine;
      }
      __syncthreads();
    } else {
      const Key mine = insert_row(z, Y, first, step, lane, k, &cta_bound);
      __syncthreads();
      list[warp * 32 + lane] = mine;
      __syncthreads();
      if (warp == 0) {
        Key best = mine;
        for (int w = 1; w < kScoreWarps; ++w) best = list_merge(best, list[w * 32 + lane], lane);
        sorted[lane] = best;
      }
    }
  }
  if (nct > 1)
    cluster.sync();
  else
    __syncwarp();
  if (rank == 0 && warp == 0) {
    Key best = TOP ? sorted[lane] : 0;
    for (uint32_t r = 1; r < nct; ++r) {
      L = stat_join(L, *cluster.map_shared_rank(&cta_stat, r));
      if (TOP) best = list_merge(best, cluster.map_shared_rank(sorted, r)[lane], lane);
    }
    write_row<T, TOP>(A, row, z, L, best, lane, k);
  }
  // the other CTAs stay until rank 0 has read their shared memory
  if (nct > 1) cluster.sync();
}

// --------------------------------------------------------------- gradient
// dlogits = scale (g ([j = id] - p) - h p (log p + H)): one read, one write,
// bound by memory.  A CTA is short (16 KB of bf16 in and out), so its logits are
// on their way while the row's statistics are looked up (statistics first, 8192
// x 32000 bf16 took 197 us instead of 152).
// Each CTA takes kGradCols columns of a row, each thread 4 vectors of 8.
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;
constexpr int kGradCols = kGradThreads * 8 * kGradVecs;

struct RowGrad {
  float scale, lse, h;
  float rest2;  // -rest log2(e)
  float c;      // -g - h (entropy - rest)
};

template <bool ENT>
__device__ __forceinline__ float grad_of(const RowGrad& R, float z) {
  // log p = (z - lse) - rest; -inf logits have p = 0 and no gradient
  const float d = __fsub_rn(__fmul_rn(z, R.scale), R.lse);
  const float p = ex2(fmaf(d, kLog2e, R.rest2)) * R.scale;
  return p * (ENT ? fmaf(-R.h, fmaxf(d, kFar), R.c) : R.c);
}

template <class T, bool ENT>
__global__ void __launch_bounds__(kGradThreads) k_token_logprobs_grad(const ScoreGradArgs A, int parts) {
  const int64_t row = blockIdx.x / parts;
  const int64_t c0 = (blockIdx.x - row * parts) * int64_t(kGradCols);
  const int64_t c1 = min(A.vocab, c0 + kGradCols);
  const T* z = static_cast<const T*>(A.logits) + row * A.ldl;
  T* o = static_cast<T*>(A.dlogits) + row * A.ldd;
  const int64_t mz = (reinterpret_cast<uintptr_t>(z + c0) & 15) / sizeof(T);
  const int64_t mo = (reinterpret_cast<uintptr_t>(o + c0) & 15) / sizeof(T);
  const int64_t head = min(c1 - c0, mz ? static_cast<int64_t>(16 / sizeof(T)) - mz : int64_t(0));
  const int64_t b0 = c0 + head;
  const int nvec = mz == mo ? static_cast<int>((c1 - b0) / 8) : 0;
  // the logits are on their way before the row's statistics are looked up
  Pack<T> v[kGradVecs];
#pragma unroll
  for (int u = 0; u < kGradVecs; ++u) {
    const int i = threadIdx.x + u * kGradThreads;
    if (i < nvec) v[u].load(z + b0 + i * 8);
  }
  RowGrad R;
  R.scale = A.scale;
  R.lse = A.lse[row];
  int64_t id = token_at(A.ids, A.ids_i64, row);
  if (id < 0 || id >= A.vocab) id = -1;
  const float g = id >= 0 ? A.dlogp[row] : 0.0f;
  R.h = ENT ? A.dentropy[row] : 0.0f;
  const float rest = A.lse_rest ? A.lse_rest[row] : 0.0f;
  R.rest2 = -rest * kLog2e;
  R.c = ENT ? -g - R.h * (A.entropy[row] - rest) : -g;
  float own = g * A.scale;  // the given token's own term
  if (R.lse == -CUDART_INF_F) {
    // no possible token: z - lse would be NaN
    R.lse = R.rest2 = R.h = R.c = own = 0.0f;
  }
  auto one = [&](int64_t c) {
    const float d = grad_of<ENT>(R, to_f32(z[c]));
    o[c] = from_f32<T>(c == id ? d + own : d);
  };
  if (mz != mo) {
    // the two rows are aligned differently: element by element
#pragma unroll 4
    for (int64_t c = c0 + threadIdx.x; c < c1; c += kGradThreads) one(c);
    return;
  }
  const int64_t t0 = b0 + nvec * 8;
  if (threadIdx.x < head) one(c0 + threadIdx.x);
  if (threadIdx.x < c1 - t0) one(t0 + threadIdx.x);
#pragma unroll
  for (int u = 0; u < kGradVecs; ++u) {
    const int i = threadIdx.x + u * kGradThreads;
    if (i >= nvec) break;
    const int64_t c = b0 + i * 8;
    float d[8];
    v[u].unpack(d);
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] = grad_of<ENT>(R, d[j]);
    if (id >= c && id < c + 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j == id) d[j] += own;
    }
    store8(o + c, d);
  }
}

template <class T, bool TOP, bool SCALED>
cudaError_t run_score(const ScoreArgs& A, int num_sms, cudaStream_t st) {
  if (A.vocab <= kWarpRowFew || (A.vocab <= kWarpRow && A.rows >= 16 * num_sms)) {
    k_token_logprobs_warp<T, TOP, SCALED>
        <<<static_cast<unsigned>(lm_div_up(A.rows, kScoreWarps)), kScoreThreads, 0, st>>>(A);
    return cudaGetLastError();
  }
  // CTAs per row: enough to fill the SMs four times while each still has a
  // few vectors per thread
  int nct = 1;
  while (nct < 8 && A.rows * nct < 4 * num_sms && A.vocab / (nct * 2) >= kScoreThreads * 8) nct *= 2;
  // and enough to keep the maxima of a long row
  constexpr int64_t kept = int64_t(kCtaBlocks) * kScoreThreads * 8 * kVecs;
  while (TOP && nct < 8 && A.vocab > kept * nct) nct *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(A.rows * nct));
  cfg.blockDim = dim3(kScoreThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nct;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_token_logprobs<T, TOP, SCALED>, A, static_cast<int>(A.vocab <= kept * nct));
}

template <class T>
cudaError_t score_of(const ScoreArgs& A, int num_sms, cudaStream_t st) {
  const bool scaled = A.scale != 1.0f;
  if (A.top_k > 0) return scaled ? run_score<T, true, true>(A, num_sms, st) : run_score<T, true, false>(A, num_sms, st);
  return scaled ? run_score<T, false, true>(A, num_sms, st) : run_score<T, false, false>(A, num_sms, st);
}

template <class T>
cudaError_t grad_of_rows(const ScoreGradArgs& A, cudaStream_t st) {
  const int parts = static_cast<int>(lm_div_up(A.vocab, kGradCols));
  const unsigned grid = static_cast<unsigned>(A.rows * parts);
  if (A.dentropy)
    k_token_logprobs_grad<T, true><<<grid, kGradThreads, 0, st>>>(A, parts);
  else
    k_token_logprobs_grad<T, false><<<grid, kGradThreads, 0, st>>>(A, parts);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_token_logprobs(const ScoreArgs& A, int dtype, int num_sms, cudaStream_t st) {
  if (A.rows <= 0) return cudaSuccess;
  return dtype == kDtBf16 ? score_of<__nv_bfloat16>(A, num_sms, st) : score_of<float>(A, num_sms, st);
}

cudaError_t launch_token_logprobs_grad(const ScoreGradArgs& A, int dtype, cudaStream_t st) {
  if (A.rows <= 0) return cudaSuccess;
  return dtype == kDtBf16 ? grad_of_rows<__nv_bfloat16>(A, st) : grad_of_rows<float>(A, st);
}

}  // namespace okls
