// Log probabilities of given tokens with entropy and best alternatives, and
// their gradient (sm_103a).
//
// With z = scale * logits, m = max z, S = sum e^(z - m), Q = sum e^(z - m)(z - m):
//   lse = m + log S,   logp = z_id - lse,   entropy = log S - Q / S.
// One pass over the logits: every thread keeps a running (m, S, Q); when the
// maximum grows by t = m_old - m_new <= 0, S <- S e^t and Q <- e^t (Q + t S).
// Pairs of partial results are joined by the same rule.  The entropy is taken
// from differences to the maximum, so an offset common to the row does not
// cancel digits.
//
// A row is read by a cluster of 1 to 8 CTAs (few long rows need many SMs);
// partial results are joined through shared memory and then distributed
// shared memory.  A thread loads 32 values at a time, so one look at their
// maximum serves all of them; an exponential, a clamp and five additions and
// products are left per value (two values an instruction where the hardware
// has it), which a bf16 row just hides under its loads.
//
// Best alternatives ride along: each warp keeps the 32 best (logit, column)
// keys sorted across its lanes.  A key is 64 bits, the order-preserving image
// of the logit above the complement of the column, so equal logits rank by
// column and no two keys are equal.  A warp's first 1024 values give a first
// bound, the k-th largest of its lanes' maxima; a CTA-wide bound (the best of
// its warps' k-th keys) then rejects almost every group of 32 values with the
// maximum that the sums need anyway, and about k ln(vocab / k) insertions a
// row are left.
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
__device__ __forceinline__ Key list_merge(Key a, Key b, int lane) {
  const Key rb = __shfl_sync(0xffffffffu, b, 31 - lane);
  Key v = a > rb ? a : rb;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Key w = __shfl_xor_sync(0xffffffffu, v, o);
    const bool keep_max = (lane & o) == 0;
    v = keep_max ? (v > w ? v : w) : (v > w ? w : v);
  }
  return v;
}

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kVecs = 4;  // vectors of 8 values a thread loads at a time

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

// k-th largest of the lanes' values.
__device__ __forceinline__ uint32_t kth_of_lanes(uint32_t v, int k, int lane) {
#pragma unroll
  for (int w = 2; w <= 32; w <<= 1)
#pragma unroll
    for (int o = w >> 1; o > 0; o >>= 1) {
      const uint32_t x = __shfl_xor_sync(0xffffffffu, v, o);
      // descending in even blocks of w lanes, ascending in odd ones
      const bool keep_max = ((lane & o) == 0) == ((lane & w) == 0);
      v = keep_max ? max(v, x) : min(v, x);
    }
  return __shfl_sync(0xffffffffu, v, k - 1);
}

// Offers the warp's values to its list: lane values z[j], j < count, whose
// columns are col + (j / W) * stride + j % W of the row at `row`; vm is the
// lane's maximum.
template <class T, int N, int W>
__device__ __forceinline__ void offer(Best& B, const float (&z)[N], float vm, int count, const T* row, uint32_t col,
                                      uint32_t stride, int lane, int k, Key* cta_bound) {
  const Key shared = *reinterpret_cast<volatile Key*>(cta_bound);
  if (shared > B.bound) {
    B.bound = shared;
    B.bound_v = ord_value(static_cast<uint32_t>(shared >> 32));
  }
  if (!__any_sync(0xffffffffu, count > 0 && !(vm < B.bound_v))) return;
  if (N > 1 && B.bound == 0) {
    // the k-th best of 32 of the warp's values, one a lane
    const uint32_t kth = kth_of_lanes(count > 0 ? ord_bits(vm) : 0u, k, lane);
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
    L.s = top;  // the row's sums are NaN from here on
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

template <class T, bool TOP, bool SCALED>
__global__ void __launch_bounds__(kScoreThreads) k_token_logprobs(const ScoreArgs A) {
  __shared__ Stat stats[kScoreWarps];
  __shared__ Stat cta_stat;
  __shared__ Key lists[TOP ? kScoreWarps : 1][32];
  __shared__ Key cta_bound;
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank(), nct = cluster.num_blocks();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k = TOP ? A.top_k : 1;
  const int64_t vocab = A.vocab;
  const int64_t row = blockIdx.x / nct;
  if (TOP) {
    if (threadIdx.x == 0) cta_bound = 0;
    __syncthreads();
  }
  const T* z = static_cast<const T*>(A.logits) + row * A.ldl;
  Stat L = {-CUDART_INF_F, 0.0f, 0.0f};
  Best B = {0, 0, -CUDART_INF_F};
  // 16-byte aligned body; the columns before and after it one by one
  const int64_t mis = (reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T);
  const int64_t head = min(vocab, mis ? static_cast<int64_t>(16 / sizeof(T)) - mis : int64_t(0));
  const int64_t nvec = (vocab - head) / 8;
  const int64_t tail0 = head + nvec * 8;
  const int64_t step = int64_t(nct) * kScoreThreads;  // vectors between a thread's vectors
  for (int64_t v0 = int64_t(rank) * kScoreThreads + warp * 32; v0 < nvec; v0 += step * kVecs) {
    const int64_t i = v0 + lane;
    float v[kVecs * 8];
    int count = 0;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      float t[8];
      if (i + u * step < nvec) {
        load8(z + head + (i + u * step) * 8, t);
        count += 8;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = -CUDART_INF_F;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u * 8 + j] = t[j];
    }
    const float vm = take<kVecs * 8, SCALED>(L, v, A.scale);
    if (TOP)
      offer<T, kVecs * 8, 8>(B, v, vm, count, z, static_cast<uint32_t>(head + i * 8), static_cast<uint32_t>(step * 8),
                             lane, k, &cta_bound);
  }
  if (rank == 0 && warp == 0) {
    const int64_t edge = head + (vocab - tail0);  // < 16 columns
    const int64_t col = lane < head ? lane : tail0 + (lane - head);
    float v[1] = {lane < edge ? to_f32(z[col]) : -CUDART_INF_F};
    const float vm = take<1, SCALED>(L, v, A.scale);
    if (TOP)
      offer<T, 1, 1>(B, v, vm, lane < edge ? 1 : 0, z, static_cast<uint32_t>(col), 0u, lane, k, &cta_bound);
  }

  // join: lanes, warps, CTAs
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L = stat_join(L, stat_shfl_xor(L, o));
  if (lane == 0) stats[warp] = L;
  if (TOP) lists[warp][lane] = B.list;
  __syncthreads();
  if (warp == 0) {
    L = stats[lane & (kScoreWarps - 1)];  // every 8 lanes form the same sum
#pragma unroll
    for (int o = kScoreWarps / 2; o > 0; o >>= 1) L = stat_join(L, stat_shfl_xor(L, o));
    if (lane == 0) cta_stat = L;
  }
  if (TOP) {
#pragma unroll 1
    for (int o = kScoreWarps / 2; o > 0; o >>= 1) {
      if (warp < o) lists[warp][lane] = list_merge(lists[warp][lane], lists[warp + o][lane], lane);
      __syncthreads();
    }
  }
  if (nct > 1) cluster.sync();
  if (rank == 0 && warp == 0) {
    Key best = TOP ? lists[0][lane] : 0;
    for (uint32_t r = 1; r < nct; ++r) {
      L = stat_join(L, *cluster.map_shared_rank(&cta_stat, r));
      if (TOP) best = list_merge(best, cluster.map_shared_rank(&lists[0][0], r)[lane], lane);
    }
    const bool none = L.m == -CUDART_INF_F && L.s == 0.0f;  // no possible token
    // a sum that is NaN (a NaN logit) makes everything NaN, and so does an
    // infinite maximum, whose sum is 0
    const float logs = logf(L.s);
    const float lse = none ? -CUDART_INF_F : (L.s != L.s ? L.s : L.m + logs);
    if (lane == 0) {
      if (A.lse) A.lse[row] = lse;
      if (A.entropy) A.entropy[row] = none ? 0.0f : logs - L.q / L.s;
      if (A.logp) {
        const int64_t id = token_at(A.ids, A.ids_i64, row);
        if (id >= vocab) atomicOr(A.status, kStBadToken);
        float lp = 0.0f;
        if (id >= 0 && id < vocab) lp = none ? -CUDART_INF_F : __fsub_rn(__fmul_rn(to_f32(z[id]), A.scale), lse);
        A.logp[row] = lp;
      }
    }
    if (TOP && lane < k) {
      const uint32_t col = ~static_cast<uint32_t>(best);
      A.top_ids[row * k + lane] = static_cast<int32_t>(col);
      A.top_logp[row * k + lane] =
          none ? -CUDART_INF_F : __fsub_rn(__fmul_rn(ord_value(static_cast<uint32_t>(best >> 32)), A.scale), lse);
    }
  }
  // the other CTAs stay until rank 0 has read their shared memory
  if (nct > 1) cluster.sync();
}

// --------------------------------------------------------------- gradient
// dlogits = scale (g ([j = id] - p) - h p (log p + H)): one read, one write.
// Each CTA takes kGradCols columns of a row, each thread 4 vectors of 8.
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;
constexpr int kGradCols = kGradThreads * 8 * kGradVecs;

struct RowGrad {
  float scale, lse, h, c;  // c = -g - h entropy
};

template <bool ENT>
__device__ __forceinline__ float grad_of(const RowGrad& R, float z) {
  // log p = z - lse; -inf logits have p = 0 and no gradient
  const float lp = __fsub_rn(__fmul_rn(z, R.scale), R.lse);
  const float p = ex2(lp * kLog2e) * R.scale;
  return p * (ENT ? fmaf(-R.h, fmaxf(lp, kFar), R.c) : R.c);
}

template <class T, bool ENT>
__global__ void __launch_bounds__(kGradThreads) k_token_logprobs_grad(const ScoreGradArgs A, int parts) {
  const int64_t row = blockIdx.x / parts;
  const int64_t c0 = (blockIdx.x - row * parts) * int64_t(kGradCols);
  const int64_t c1 = min(A.vocab, c0 + kGradCols);
  const T* z = static_cast<const T*>(A.logits) + row * A.ldl;
  T* o = static_cast<T*>(A.dlogits) + row * A.ldd;
  RowGrad R;
  R.scale = A.scale;
  R.lse = A.lse[row];
  int64_t id = token_at(A.ids, A.ids_i64, row);
  if (id < 0 || id >= A.vocab) id = -1;
  const float g = id >= 0 ? A.dlogp[row] : 0.0f;
  R.h = ENT ? A.dentropy[row] : 0.0f;
  R.c = ENT ? -g - R.h * A.entropy[row] : -g;
  float own = g * A.scale;  // the given token's own term
  if (R.lse == -CUDART_INF_F) {
    // no possible token: z - lse would be NaN
    R.lse = R.h = R.c = own = 0.0f;
  }
  auto one = [&](int64_t c) {
    const float d = grad_of<ENT>(R, to_f32(z[c]));
    o[c] = from_f32<T>(c == id ? d + own : d);
  };
  const int64_t mz = (reinterpret_cast<uintptr_t>(z + c0) & 15) / sizeof(T);
  const int64_t mo = (reinterpret_cast<uintptr_t>(o + c0) & 15) / sizeof(T);
  if (mz != mo) {
    // the two rows are aligned differently: element by element
#pragma unroll 4
    for (int64_t c = c0 + threadIdx.x; c < c1; c += kGradThreads) one(c);
    return;
  }
  const int64_t head = min(c1 - c0, mz ? static_cast<int64_t>(16 / sizeof(T)) - mz : int64_t(0));
  const int64_t b0 = c0 + head;
  const int nvec = static_cast<int>((c1 - b0) / 8);
  const int64_t t0 = b0 + nvec * 8;
  if (threadIdx.x < head) one(c0 + threadIdx.x);
  if (threadIdx.x < c1 - t0) one(t0 + threadIdx.x);
  float v[kGradVecs][8];
#pragma unroll
  for (int u = 0; u < kGradVecs; ++u) {
    const int i = threadIdx.x + u * kGradThreads;
    if (i < nvec) load8(z + b0 + i * 8, v[u]);
  }
#pragma unroll
  for (int u = 0; u < kGradVecs; ++u) {
    const int i = threadIdx.x + u * kGradThreads;
    if (i >= nvec) break;
    const int64_t c = b0 + i * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[u][j] = grad_of<ENT>(R, v[u][j]);
    if (id >= c && id < c + 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j == id) v[u][j] += own;
    }
    store8(o + c, v[u]);
  }
}

template <class T, bool TOP, bool SCALED>
cudaError_t run_score(const ScoreArgs& A, int num_sms, cudaStream_t st) {
  // CTAs per row: enough to fill the SMs four times while each still has a
  // few vectors per thread
  int nct = 1;
  while (nct < 8 && A.rows * nct < 4 * num_sms && A.vocab / (nct * 2) >= kScoreThreads * 8) nct *= 2;
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
  return cudaLaunchKernelEx(&cfg, k_token_logprobs<T, TOP, SCALED>, A);
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

cudaError_t launch_token_logprobs_grad(const ScoreGradArgs& A, int dtype, int num_sms, cudaStream_t st) {
  (void)num_sms;
  if (A.rows <= 0) return cudaSuccess;
  return dtype == kDtBf16 ? grad_of_rows<__nv_bfloat16>(A, st) : grad_of_rows<float>(A, st);
}

}  // namespace okls
