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
// shared memory.
//
// Best alternatives ride along: each warp keeps the 32 best (logit, column)
// keys sorted across its lanes.  A key is 64 bits, the order-preserving image
// of the logit above the complement of the column, so equal logits rank by
// column and no two keys are equal.  A CTA-wide bound (the best of its warps'
// k-th keys) rejects almost every value with the comparison that the running
// maximum needs anyway; k ln(vocab / k) insertions are expected per row.
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

constexpr int kScoreThreads = 512;
constexpr int kScoreWarps = kScoreThreads / 32;

template <bool TOP>
struct Lane {
  Stat st;
  Key list;
  Key bound;    // keys at or below it cannot be among the k best
  float bound_v;
};

// One vector of N consecutive columns starting at col (N = 8) or one column
// (N = 1); every lane of the warp calls with its own vector or with `valid`
// false.
template <bool TOP, int N>
__device__ __forceinline__ void take(Lane<TOP>& L, const float (&z)[N], uint32_t col, bool valid, float scale,
                                     int lane, int k, Key* cta_bound) {
  float vm = z[0];
#pragma unroll
  for (int j = 1; j < N; ++j) vm = fmaxf(vm, z[j]);
  if (valid) {
    const float top = __fmul_rn(vm, scale);
    if (top > L.st.m) {
      if (L.st.m == -CUDART_INF_F) {
        // no possible value so far: s and q are 0 (or NaN, which stays)
        L.st.m = top;
      } else {
        const float t = fmaxf(L.st.m - top, kFar);
        const float f = exp2f(t * kLog2e);
        L.st.q = f * fmaf(t, L.st.s, L.st.q);
        L.st.s *= f;
        L.st.m = top;
      }
    }
    if (L.st.m != -CUDART_INF_F) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        // the product is rounded before the difference, as m was: a fused
        // difference would leave the rounding error of a huge masked logit
        const float d = __fsub_rn(__fmul_rn(z[j], scale), L.st.m);
        const float e = exp2f(d * kLog2e);
        L.st.s += e;
        L.st.q = fmaf(e, fmaxf(d, kFar), L.st.q);
      }
    } else {
      // only impossible values or NaN
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (z[j] != z[j]) L.st.s = z[j];
    }
  }
  if (TOP) {
    if (__any_sync(0xffffffffu, valid && !(vm < L.bound_v))) {
#pragma unroll 1
      for (int j = 0; j < N; ++j) {
        float zj = z[0];
#pragma unroll
        for (int i = 1; i < N; ++i) zj = i == j ? z[i] : zj;
        const Key cand = valid ? make_key(zj, col + j) : 0;
        unsigned todo = __ballot_sync(0xffffffffu, cand > L.bound);
        while (todo) {
          const int src = __ffs(todo) - 1;
          todo &= todo - 1;
          const Key c = __shfl_sync(0xffffffffu, cand, src);
          if (c > L.bound) {
            list_insert(L.list, c, lane);
            const Key kth = __shfl_sync(0xffffffffu, L.list, k - 1);
            if (kth > L.bound) L.bound = kth;
          }
        }
      }
      if (lane == 0) atomicMax(cta_bound, L.bound);
    }
    const Key b = *reinterpret_cast<volatile Key*>(cta_bound);
    if (b > L.bound) L.bound = b;
    L.bound_v = L.bound ? ord_value(static_cast<uint32_t>(L.bound >> 32)) : -CUDART_INF_F;
  }
}

template <class T, bool TOP>
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

  for (int64_t row = blockIdx.x / nct; row < A.rows; row += gridDim.x / nct) {
    if (TOP && threadIdx.x == 0) cta_bound = 0;
    if (TOP) __syncthreads();
    const T* z = static_cast<const T*>(A.logits) + row * A.ldl;
    Lane<TOP> L;
    L.st = {-CUDART_INF_F, 0.0f, 0.0f};
    L.list = 0;
    L.bound = 0;
    L.bound_v = -CUDART_INF_F;
    // 16-byte aligned body; the columns before and after it one by one
    const int64_t mis = (reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T);
    const int64_t head = min(vocab, mis ? static_cast<int64_t>(16 / sizeof(T)) - mis : int64_t(0));
    const int64_t nvec = (vocab - head) / 8;
    const int64_t tail0 = head + nvec * 8;
    if (rank == 0 && warp == 0) {
      const int64_t edge = head + (vocab - tail0);  // < 16 columns
      const int64_t col = lane < head ? lane : tail0 + (lane - head);
      float v[1] = {lane < edge ? to_f32(z[col]) : 0.0f};
      take<TOP, 1>(L, v, static_cast<uint32_t>(col), lane < edge, A.scale, lane, k, &cta_bound);
    }
    const int64_t step = int64_t(nct) * kScoreThreads;
    for (int64_t v0 = int64_t(rank) * kScoreThreads + warp * 32; v0 < nvec; v0 += step) {
      const int64_t i = v0 + lane;
      float v[8] = {};
      const int64_t col = head + i * 8;
      if (i < nvec) load8(z + col, v);
      take<TOP, 8>(L, v, static_cast<uint32_t>(col), i < nvec, A.scale, lane, k, &cta_bound);
    }

    // join: lanes, warps, CTAs
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L.st = stat_join(L.st, stat_shfl_xor(L.st, o));
    if (lane == 0) stats[warp] = L.st;
    if (TOP) lists[warp][lane] = L.list;
    __syncthreads();
    if (warp == 0) {
      Stat s = lane < kScoreWarps ? stats[lane] : Stat{-CUDART_INF_F, 0.0f, 0.0f};
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s = stat_join(s, stat_shfl_xor(s, o));
      if (lane == 0) cta_stat = s;
      L.st = s;
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
        L.st = stat_join(L.st, *cluster.map_shared_rank(&cta_stat, r));
        if (TOP) best = list_merge(best, cluster.map_shared_rank(&lists[0][0], r)[lane], lane);
      }
      const Stat s = L.st;
      const bool none = s.m == -CUDART_INF_F && s.s == 0.0f;  // no possible token
      // a sum that is NaN (a NaN or +inf logit) makes everything NaN
      const float logs = logf(s.s);
      const float lse = none ? -CUDART_INF_F : (s.s != s.s ? s.s : s.m + logs);
      if (lane == 0) {
        if (A.lse) A.lse[row] = lse;
        if (A.entropy) A.entropy[row] = none ? 0.0f : logs - s.q / s.s;
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
    // the next row's lists and sums overwrite what rank 0 reads
    if (nct > 1)
      cluster.sync();
    else
      __syncthreads();
  }
}

// --------------------------------------------------------------- gradient
// dlogits = scale (g ([j = id] - p) - h p (log p + H)): one read, one write.
// Each CTA takes kGradCols columns of a row.
constexpr int kGradThreads = 256;
constexpr int kGradCols = kGradThreads * 8 * 4;

struct RowGrad {
  float scale, lse, neg_g, h, ent;  // neg_g = -g
};

__device__ __forceinline__ float grad_of(const RowGrad& R, float z) {
  // log p = z - lse; -inf logits have p = 0 and no gradient
  const float lp = __fsub_rn(__fmul_rn(z, R.scale), R.lse);
  const float p = exp2f(lp * kLog2e);
  return R.scale * p * fmaf(-R.h, fmaxf(lp, kFar) + R.ent, R.neg_g);
}

template <class T>
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
  R.neg_g = -g;
  R.h = A.dentropy ? A.dentropy[row] : 0.0f;
  R.ent = A.dentropy ? A.entropy[row] : 0.0f;
  const bool none = R.lse == -CUDART_INF_F;
  const float add = none ? 0.0f : g * A.scale;  // the given token's own term
  auto one = [&](int64_t c) {
    const float d = none ? 0.0f : grad_of(R, to_f32(z[c]));
    o[c] = from_f32<T>(c == id ? d + add : d);
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
  const int64_t nvec = (c1 - b0) / 8;
  const int64_t t0 = b0 + nvec * 8;
  if (threadIdx.x < head) one(c0 + threadIdx.x);
  if (threadIdx.x < c1 - t0) one(t0 + threadIdx.x);
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < nvec; i += kGradThreads) {
    const int64_t c = b0 + i * 8;
    float v[8];
    load8(z + c, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = none ? 0.0f : grad_of(R, v[j]);
      v[j] = c + j == id ? d + add : d;
    }
    store8(o + c, v);
  }
}

template <class T, bool TOP>
cudaError_t run_score(const ScoreArgs& A, int num_sms, cudaStream_t st) {
  // CTAs per row: enough to fill the SMs twice while each still has a few
  // vectors per thread
  int nct = 1;
  while (nct < 8 && A.rows * nct < 2 * num_sms && A.vocab / (nct * 2) >= kScoreThreads * 8) nct *= 2;
  const int64_t rows_at_once = 4 * num_sms / nct;
  const int64_t grid = (A.rows < rows_at_once ? A.rows : rows_at_once) * nct;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kScoreThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nct;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_token_logprobs<T, TOP>, A);
}

}  // namespace

cudaError_t launch_token_logprobs(const ScoreArgs& A, int dtype, int num_sms, cudaStream_t st) {
  if (A.rows <= 0) return cudaSuccess;
  if (dtype == kDtBf16)
    return A.top_k > 0 ? run_score<__nv_bfloat16, true>(A, num_sms, st) : run_score<__nv_bfloat16, false>(A, num_sms, st);
  return A.top_k > 0 ? run_score<float, true>(A, num_sms, st) : run_score<float, false>(A, num_sms, st);
}

cudaError_t launch_token_logprobs_grad(const ScoreGradArgs& A, int dtype, int num_sms, cudaStream_t st) {
  (void)num_sms;
  if (A.rows <= 0) return cudaSuccess;
  const int parts = static_cast<int>(lm_div_up(A.vocab, kGradCols));
  const unsigned grid = static_cast<unsigned>(A.rows * parts);
  if (dtype == kDtBf16)
    k_token_logprobs_grad<__nv_bfloat16><<<grid, kGradThreads, 0, st>>>(A, parts);
  else
    k_token_logprobs_grad<float><<<grid, kGradThreads, 0, st>>>(A, parts);
  return cudaGetLastError();
}

}  // namespace okls
