// Token embedding with scaling, and its gradient by sorted tokens (sm_103a).
//
//   out[t] = scale W[id_t];     dW[v] = base[v] + scale sum_{t: id_t = v} dy[t].
//
// Both are bound by memory.  The gradient is a sum by key: the token
// positions are sorted by id in one cluster (radix passes whose counters the
// CTAs exchange through distributed shared memory), then the sorted list is
// cut into chunks of kRun positions, one CTA per chunk and column slice.  A
// CTA writes the rows that begin and end inside its chunk; a row that spans
// chunks leaves one partial sum per chunk, which a last launch joins in
// order.  So a frequent token is spread over many CTAs, no sum depends on
// the order in which CTAs run, and no row needs an atomic.
#include <cooperative_groups.h>

#include "okls_internal.h"
#include "okls_lm.cuh"

namespace cg = cooperative_groups;

namespace okls {
namespace {

// ---------------------------------------------------------------- forward
constexpr int kSeg = 1024;  // columns of a row that one warp copies

template <class T, class O, bool VEC>
__global__ void __launch_bounds__(256) k_embedding(const EmbedArgs A, int segs, int64_t items) {
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (item >= items) return;
  const int64_t t = item / segs;
  const int64_t e0 = (item - t * segs) * kSeg;
  const int64_t id = token_at(A.ids, A.ids_i64, t);
  if (id >= A.vocab && lane == 0) atomicOr(A.status, kStBadToken);
  const bool keep = id >= 0 && id < A.vocab;
  const T* w = static_cast<const T*>(A.weight) + (keep ? id : 0) * A.ldw;
  O* o = static_cast<O*>(A.out) + t * A.ldo;
  if (VEC) {
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t e = e0 + i * 256 + lane * 8;
      if (keep && e + 8 <= A.dim) load8(w + e, v[i]);
      if (!keep) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t e = e0 + i * 256 + lane * 8;
      if (e + 8 <= A.dim) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= A.scale;
        store8(o + e, v[i]);
      } else {
        for (int64_t c = e; c < A.dim; ++c) o[c] = from_f32<O>(keep ? to_f32(w[c]) * A.scale : 0.0f);
      }
    }
  } else {
#pragma unroll 8
    for (int i = 0; i < kSeg / 32; ++i) {
      const int64_t e = e0 + i * 32 + lane;
      if (e < A.dim) o[e] = from_f32<O>(keep ? to_f32(w[e]) * A.scale : 0.0f);
    }
  }
}

template <class T, class O>
cudaError_t run_embedding(const EmbedArgs& A, cudaStream_t st) {
  const int segs = static_cast<int>(lm_div_up(A.dim, kSeg));
  const int64_t items = A.tokens * segs;
  const int64_t grid = lm_div_up(items, 8);
  const bool vec = lm_aligned(A.weight, A.ldw, A.vocab, sizeof(T), 16) &&
                   lm_aligned(A.out, A.ldo, A.tokens, sizeof(O), 16);
  if (vec)
    k_embedding<T, O, true><<<static_cast<unsigned>(grid), 256, 0, st>>>(A, segs, items);
  else
    k_embedding<T, O, false><<<static_cast<unsigned>(grid), 256, 0, st>>>(A, segs, items);
  return cudaGetLastError();
}

// ------------------------------------------------------------------- sort
// Stable radix sort of (id, position) by id in one cluster of up to 8 CTAs.
// Padding gets the key `vocab` and sorts to the end.  Each warp owns a
// contiguous span of the list and a row of digit counters; a pass counts
// digits per warp, turns the counts into offsets (prefix over warps within
// the CTA, over CTAs through distributed shared memory, then over digits),
// and moves the pairs, 32 at a time in order, with __match_any_sync ranks.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxBins = 1 << kMaxDigitBits;
constexpr int kSortSmem = (kSortWarps * kMaxBins + 2 * kMaxBins + 32) * 4;

struct SortArgs {
  const void* ids;
  int32_t ids_i64;
  int64_t tokens;
  uint32_t vocab;
  int32_t digit_bits, passes;
  uint32_t *key[2], *pos[2];
  uint8_t* present;  // [vocab]: 1 where a row has a token
  uint32_t* status;
};

__global__ void __launch_bounds__(kSortThreads) k_embed_sort(const SortArgs A) {
  extern __shared__ uint32_t sm[];
  uint32_t* wcnt = sm;                             // [warp][bin]
  uint32_t* hist = sm + kSortWarps * kMaxBins;     // [bin], read by the other CTAs
  uint32_t* offs = hist + kMaxBins;                // [bin]
  uint32_t* wsum = offs + kMaxBins;                // [warp]
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank(), nct = cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bins = 1 << A.digit_bits;
  const uint32_t dmask = bins - 1;

  for (int64_t v = rank * kSortThreads + tid; v < A.vocab; v += int64_t(nct) * kSortThreads) A.present[v] = 0;

  const int64_t nwarps = int64_t(nct) * kSortWarps;
  const int64_t span = lm_div_up(lm_div_up(A.tokens, nwarps), 32) * 32;
  const int64_t lo = (int64_t(rank) * kSortWarps + warp) * span;
  const int64_t hi = min(A.tokens, lo + span);

  for (int p = 0; p < A.passes; ++p) {
    const uint32_t* sk = A.key[(p + 1) & 1];
    const uint32_t* sp = A.pos[(p + 1) & 1];
    uint32_t* dk = A.key[p & 1];
    uint32_t* dp = A.pos[p & 1];
    const int shift = p * A.digit_bits;
    uint32_t* mine = wcnt + warp * kMaxBins;
    for (int b = lane; b < bins; b += 32) mine[b] = 0;
    __syncwarp();
    for (int64_t i = lo + lane; i < hi; i += 32) {
      uint32_t k;
      if (p == 0) {
        const int64_t id = token_at(A.ids, A.ids_i64, i);
        if (id >= A.vocab) atomicOr(A.status, kStBadToken);
        k = id >= 0 && id < A.vocab ? static_cast<uint32_t>(id) : A.vocab;
      } else {
        k = sk[i];
      }
      atomicAdd(&mine[(k >> shift) & dmask], 1u);
    }
    __syncthreads();
    for (int b = tid; b < bins; b += kSortThreads) {
      uint32_t run = 0;
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = wcnt[w * kMaxBins + b];
        wcnt[w * kMaxBins + b] = run;
        run += c;
      }
      hist[b] = run;
    }
    cluster.sync();
    // bins <= 512 < threads: one bin a thread
    uint32_t total = 0, before = 0;
    if (tid < bins)
      for (uint32_t r = 0; r < nct; ++r) {
        const uint32_t c = cluster.map_shared_rank(hist, r)[tid];
        before += r < rank ? c : 0u;
        total += c;
      }
    uint32_t inc = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    uint32_t basew = 0;
    for (int w = 0; w < warp; ++w) basew += wsum[w];
    if (tid < bins) offs[tid] = basew + inc - total + before;
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      const int64_t i = i0 + lane;
      const bool in = i < hi;
      uint32_t k = 0, q = 0;
      if (in) {
        if (p == 0) {
          const int64_t id = token_at(A.ids, A.ids_i64, i);
          k = id >= 0 && id < A.vocab ? static_cast<uint32_t>(id) : A.vocab;
          q = static_cast<uint32_t>(i);
          if (k < A.vocab) A.present[k] = 1;
        } else {
          k = sk[i];
          q = sp[i];
        }
      }
      const uint32_t d = in ? (k >> shift) & dmask : 0xFFFFFFFFu;
      const uint32_t peers = __match_any_sync(0xffffffffu, d);
      const uint32_t below = __popc(peers & ((1u << lane) - 1u));
      uint32_t at = 0;
      if (in) at = offs[d] + mine[d] + below;
      __syncwarp();
      if (in && below == 0) mine[d] += __popc(peers);
      __syncwarp();
      if (in) {
        dk[at] = k;
        dp[at] = q;
      }
    }
    // the pairs reach the cluster's other CTAs; hist may be rewritten
    cluster.sync();
  }
}

// ------------------------------------------------------------- sum by key
constexpr int kRun = 32;      // sorted positions of one chunk
constexpr int kSlice = 2048;  // columns of one CTA: 256 threads x 8

struct ReduceArgs {
  const void* dy;
  int64_t lddy;
  const uint32_t *key, *pos;  // sorted
  const uint8_t* present;
  int64_t tokens, vocab, dim;
  float scale;
  const void* base;
  int64_t ldbase;
  void* out;
  int64_t ldo;
  float* part;  // [chunk][head, tail][dim]: sums of rows that span chunks
  int64_t chunks;
  int32_t slices;
};

template <class O, bool VEC>
__device__ __forceinline__ void write_row(const ReduceArgs& A, int64_t v, int64_t e0, const float (&acc)[8]) {
  O* o = static_cast<O*>(A.out) + v * A.ldo;
  const O* b = A.base ? static_cast<const O*>(A.base) + v * A.ldbase : nullptr;
  if (VEC && e0 + 8 <= A.dim) {
    float r[8];
    if (b) {
      load8(b + e0, r);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = fmaf(acc[j], A.scale, r[j]);
    store8(o + e0, r);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e0 + j < A.dim) o[e0 + j] = from_f32<O>(fmaf(acc[j], A.scale, b ? to_f32(b[e0 + j]) : 0.0f));
  }
}

template <class T, bool VEC>
__device__ __forceinline__ void load_row8(const T* row, int64_t e0, int64_t dim, float (&v)[8]) {
  if (VEC && e0 + 8 <= dim) {
    load8(row + e0, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e0 + j < dim ? to_f32(row[e0 + j]) : 0.0f;
  }
}

template <class T, class O, bool VEC>
__global__ void __launch_bounds__(256) k_embed_reduce(const ReduceArgs A) {
  __shared__ uint32_t sk[kRun], sp[kRun];
  const int64_t b = blockIdx.x;
  const int64_t chunk = b / A.slices;
  const int64_t e0 = (b - chunk * A.slices) * kSlice + threadIdx.x * 8;
  const int64_t i0 = chunk * kRun;
  const int n = static_cast<int>(min(static_cast<int64_t>(kRun), A.tokens - i0));
  if (threadIdx.x < n) {
    sk[threadIdx.x] = A.key[i0 + threadIdx.x];
    sp[threadIdx.x] = A.pos[i0 + threadIdx.x];
  }
  const uint32_t prev = i0 > 0 ? A.key[i0 - 1] : 0xFFFFFFFFu;
  const uint32_t next = i0 + n < A.tokens ? A.key[i0 + n] : 0xFFFFFFFFu;
  __syncthreads();
  if (e0 >= A.dim) return;
  const uint32_t vocab = static_cast<uint32_t>(A.vocab);
  const T* dy = static_cast<const T*>(A.dy);
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
  bool from_before = sk[0] == prev;
  constexpr int U = 4;  // rows in flight
  for (int i = 0; i < n; i += U) {
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u < n && sk[i + u] < vocab) load_row8<T, VEC>(dy + int64_t(sp[i + u]) * A.lddy, e0, A.dim, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= n) break;
      const uint32_t k = sk[i + u];
      if (k >= vocab) return;  // padding fills the rest of the list
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += v[u][j];
      const bool last = i + u + 1 == n;
      if (last ? k != next : k != sk[i + u + 1]) {
        if (from_before) {
          float* p = A.part + (chunk * 2) * A.dim;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (e0 + j < A.dim) p[e0 + j] = acc[j];
        } else {
          write_row<O, VEC>(A, k, e0, acc);
        }
        from_before = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
      } else if (last) {
        // the row goes on in the next chunk: a head slot when it also came
        // from the previous one, this chunk's tail slot otherwise
        float* p = A.part + (chunk * 2 + (from_before ? 0 : 1)) * A.dim;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (e0 + j < A.dim) p[e0 + j] = acc[j];
      }
    }
  }
}

// Rows without a token: base, or zeros.
template <class O, bool VEC>
__global__ void __launch_bounds__(256) k_embed_fill(const ReduceArgs A) {
  const int64_t b = blockIdx.x;
  const int64_t v = b / A.slices;
  const int64_t e0 = (b - v * A.slices) * kSlice + threadIdx.x * 8;
  if (e0 >= A.dim || A.present[v]) return;
  const float zero[8] = {};
  write_row<O, VEC>(A, v, e0, zero);
}

// Rows that span chunks.  The owner is the chunk in which the row begins; it
// adds its tail and the head slots of the chunks that follow: 4 groups of
// threads take every fourth slot, then the groups' sums are added in order.
constexpr int kJoinCols = 512;
template <class O>
__global__ void __launch_bounds__(512) k_embed_join(const ReduceArgs A) {
  __shared__ float sum[4][kJoinCols];
  const int64_t chunk = blockIdx.x;
  const int64_t i0 = chunk * kRun, end = i0 + kRun;
  if (end >= A.tokens) return;  // the last chunk has no successor
  const uint32_t k = A.key[end - 1];
  if (k >= A.vocab || A.key[end] != k) return;               // nothing spans the boundary
  if (A.key[i0] == k && i0 > 0 && A.key[i0 - 1] == k) return;  // began in an earlier chunk
  // end of the run: first position past `end` with another key
  int64_t lo = end, hi = A.tokens;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (A.key[mid] == k)
      lo = mid + 1;
    else
      hi = mid;
  }
  const int64_t last = (lo - 1) / kRun;  // last chunk of the row
  const int grp = threadIdx.x >> 7, t = threadIdx.x & 127;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * kJoinCols + t * 4;
  float acc[4] = {};
  for (int64_t c = chunk + grp; c <= last; c += 4) {
    const float* p = A.part + (c * 2 + (c == chunk ? 1 : 0)) * A.dim;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c0 + j < A.dim) acc[j] += p[c0 + j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) sum[grp][t * 4 + j] = acc[j];
  __syncthreads();
  const int64_t col = static_cast<int64_t>(blockIdx.y) * kJoinCols + threadIdx.x;
  if (col >= A.dim) return;
  const float s = (sum[0][threadIdx.x] + sum[1][threadIdx.x]) + (sum[2][threadIdx.x] + sum[3][threadIdx.x]);
  const float b0 = A.base ? to_f32(static_cast<const O*>(A.base)[k * A.ldbase + col]) : 0.0f;
  static_cast<O*>(A.out)[k * A.ldo + col] = from_f32<O>(fmaf(s, A.scale, b0));
}

struct GradPlan {
  size_t key[2], pos[2], present, part, total;
  int64_t chunks;
};

GradPlan plan_grad(int64_t tokens, int64_t vocab, int64_t dim) {
  GradPlan g;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  g.chunks = lm_div_up(tokens, kRun);
  for (int i = 0; i < 2; ++i) {
    g.key[i] = take(static_cast<size_t>(tokens) * 4);
    g.pos[i] = take(static_cast<size_t>(tokens) * 4);
  }
  g.present = take(static_cast<size_t>(vocab));
  g.part = take(static_cast<size_t>(g.chunks) * 2 * dim * 4);
  g.total = at;
  return g;
}

template <class T, class O>
cudaError_t run_reduce(const ReduceArgs& R, bool in_place, bool vec, cudaStream_t st) {
  if (!in_place && R.vocab > 0) {
    const unsigned grid = static_cast<unsigned>(R.vocab * R.slices);
    vec ? k_embed_fill<O, true><<<grid, 256, 0, st>>>(R) : k_embed_fill<O, false><<<grid, 256, 0, st>>>(R);
  }
  if (R.tokens > 0) {
    const unsigned grid = static_cast<unsigned>(R.chunks * R.slices);
    vec ? k_embed_reduce<T, O, true><<<grid, 256, 0, st>>>(R) : k_embed_reduce<T, O, false><<<grid, 256, 0, st>>>(R);
    if (R.chunks > 1)
      k_embed_join<O><<<dim3(static_cast<unsigned>(R.chunks), static_cast<unsigned>(lm_div_up(R.dim, kJoinCols))),
                        512, 0, st>>>(R);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_embedding(const EmbedArgs& A, int weight_dtype, cudaStream_t st) {
  if (A.tokens <= 0) return cudaSuccess;
  if (weight_dtype == kDtBf16)
    return A.out_dtype == kDtBf16 ? run_embedding<__nv_bfloat16, __nv_bfloat16>(A, st)
                                  : run_embedding<__nv_bfloat16, float>(A, st);
  return A.out_dtype == kDtBf16 ? run_embedding<float, __nv_bfloat16>(A, st) : run_embedding<float, float>(A, st);
}

size_t embedding_grad_workspace(int64_t tokens, int64_t vocab, int64_t dim) {
  return plan_grad(tokens, vocab, dim).total;
}

cudaError_t launch_embedding_grad(const EmbedGradArgs& A, int dy_dtype, int out_dtype, void* workspace, int num_sms,
                                  cudaStream_t st) {
  (void)num_sms;
  const GradPlan g = plan_grad(A.tokens, A.vocab, A.dim);
  char* ws = static_cast<char*>(workspace);
  ReduceArgs R = {};
  R.dy = A.dy, R.lddy = A.lddy;
  R.tokens = A.tokens, R.vocab = A.vocab, R.dim = A.dim, R.scale = A.scale;
  R.base = A.base, R.ldbase = A.ldbase, R.out = A.out, R.ldo = A.ldo;
  R.present = reinterpret_cast<const uint8_t*>(ws + g.present);
  R.part = reinterpret_cast<float*>(ws + g.part);
  R.chunks = g.chunks;
  R.slices = static_cast<int32_t>(lm_div_up(A.dim, kSlice));
  if (A.tokens > 0) {
    SortArgs S = {};
    S.ids = A.ids, S.ids_i64 = A.ids_i64, S.tokens = A.tokens;
    S.vocab = static_cast<uint32_t>(A.vocab);
    int bits = 1;
    while ((int64_t(1) << bits) <= A.vocab) ++bits;  // keys 0 .. vocab
    S.passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
    S.digit_bits = (bits + S.passes - 1) / S.passes;
    for (int i = 0; i < 2; ++i) {
      S.key[i] = reinterpret_cast<uint32_t*>(ws + g.key[i]);
      S.pos[i] = reinterpret_cast<uint32_t*>(ws + g.pos[i]);
    }
    S.present = reinterpret_cast<uint8_t*>(ws + g.present);
    S.status = A.status;
    const int out_buf = (S.passes - 1) & 1;
    R.key = S.key[out_buf], R.pos = S.pos[out_buf];
    static PerDevice pd;
    cudaError_t e = once_per_device(pd, [](int) {
      return cudaFuncSetAttribute(k_embed_sort, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const int nct = A.tokens <= 4096 ? 1 : A.tokens <= 8192 ? 2 : A.tokens <= 16384 ? 4 : 8;
    cfg.gridDim = dim3(nct);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = kSortSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = nct;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_embed_sort, S);
    if (e != cudaSuccess) return e;
  } else {
    const cudaError_t e = cudaMemsetAsync(ws + g.present, 0, static_cast<size_t>(A.vocab), st);
    if (e != cudaSuccess) return e;
  }
  const bool in_place = A.base == A.out;
  const int eb = out_dtype == kDtBf16 ? 2 : 4;
  const bool vec = lm_aligned(A.dy, A.lddy, A.tokens, dy_dtype == kDtBf16 ? 2 : 4, 16) &&
                   lm_aligned(A.out, A.ldo, A.vocab, eb, 16) &&
                   (!A.base || lm_aligned(A.base, A.ldbase, A.vocab, eb, 16));
  if (dy_dtype == kDtBf16)
    return out_dtype == kDtBf16 ? run_reduce<__nv_bfloat16, __nv_bfloat16>(R, in_place, vec, st)
                                : run_reduce<__nv_bfloat16, float>(R, in_place, vec, st);
  return out_dtype == kDtBf16 ? run_reduce<float, __nv_bfloat16>(R, in_place, vec, st)
                              : run_reduce<float, float>(R, in_place, vec, st);
}

}  // namespace okls
