// Token embedding with scaling, and its gradient by sorted tokens (sm_103a).
//
//   out[t] = scale W[id_t];     dW[v] = base[v] + scale sum_{t: id_t = v} dy[t].
//
// Both are bound by memory.  The gradient is a sum by key: the token
// positions are sorted by id in one cluster (radix passes whose counters the
// CTAs exchange through distributed shared memory), then the sorted list is
// cut into chunks of 16 to 64 positions, one CTA per chunk and column slice.  A
// CTA writes the rows that begin and end inside its chunk; a row that spans
// chunks leaves one partial sum per chunk, which a last launch joins in
// order.  So a frequent token is spread over many CTAs, no sum depends on
// the order in which CTAs run, and no row needs an atomic.  The rest of the
// launch that sums writes the rows without a token.
//
// Measured, bf16 in: rows of 16363 tokens x 2048 21 us (95% of the copy rate);
// gradient of them into 32000 x 2048 fp32 77 us against 48 of its bytes (sort
// 15, sums and zero rows 53, join 9); 32768 tokens into 131072 x 2048 195 us
// against 178, added to a base 361 against 336.
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
// It is bound by latency (a handful of dependent trips to L2 and to the other
// CTAs a pass), so a span is loaded kHeld steps of 32 at once.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxBins = 1 << kMaxDigitBits;
constexpr int kSortSmem = (kSortWarps * kMaxBins + 2 * kMaxBins + 32) * 4;
constexpr int kMaxSortCtas = 8;
constexpr int kHeld = 8;

struct SortArgs {
  const void* ids;
  int32_t ids_i64;
  int64_t tokens;
  uint32_t vocab;
  int32_t digit_bits, passes;
  uint32_t *key[2], *pos[2];
  uint8_t* present;  // [vocab, rounded up to 16]: 1 where a row has a token
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

  for (int64_t v = rank * kSortThreads + tid; v < (int64_t(A.vocab) + 15) / 16; v += int64_t(nct) * kSortThreads)
    reinterpret_cast<uint4*>(A.present)[v] = make_uint4(0, 0, 0, 0);

  const int64_t nwarps = int64_t(nct) * kSortWarps;
  const int64_t span = lm_div_up(lm_div_up(A.tokens, nwarps), 32) * 32;
  const int64_t lo = (int64_t(rank) * kSortWarps + warp) * span;
  const int64_t hi = min(A.tokens, lo + span);
  uint32_t* mine = wcnt + warp * kMaxBins;

  for (int p = 0; p < A.passes; ++p) {
    const uint32_t* sk = A.key[(p + 1) & 1];
    const uint32_t* sp = A.pos[(p + 1) & 1];
    uint32_t* dk = A.key[p & 1];
    uint32_t* dp = A.pos[p & 1];
    const int shift = p * A.digit_bits;
    uint32_t key[kHeld], pos[kHeld];
    // the pairs of steps i0, i0 + 32, ... (key 0xFFFFFFFF past the end)
    auto load = [&](int64_t i0) {
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        const int64_t i = i0 + u * 32 + lane;
        key[u] = 0xFFFFFFFFu;
        pos[u] = static_cast<uint32_t>(i);
        if (i < hi) {
          if (p == 0) {
            const int64_t id = token_at(A.ids, A.ids_i64, i);
            if (id >= A.vocab) atomicOr(A.status, kStBadToken);
            key[u] = id >= 0 && id < A.vocab ? static_cast<uint32_t>(id) : A.vocab;
          } else {
            key[u] = sk[i];
            pos[u] = sp[i];
          }
        }
      }
    };
    for (int b = lane; b < bins; b += 32) mine[b] = 0;
    __syncwarp();
    for (int64_t i0 = lo; i0 < hi; i0 += kHeld * 32) {
      load(i0);
#pragma unroll
      for (int u = 0; u < kHeld; ++u)
        if (key[u] != 0xFFFFFFFFu) atomicAdd(&mine[(key[u] >> shift) & dmask], 1u);
    }
    __syncthreads();
    for (int b = tid; b < bins; b += kSortThreads) {
      uint32_t run = 0;
#pragma unroll 16
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
    if (tid < bins) {
#pragma unroll
      for (uint32_t r = 0; r < kMaxSortCtas; ++r)
        if (r < nct) {
          const uint32_t c = cluster.map_shared_rank(hist, r)[tid];
          before += r < rank ? c : 0u;
          total += c;
        }
    }
    uint32_t inc = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    const uint32_t ws = lane < warp ? wsum[lane] : 0u;
    const uint32_t basew = __reduce_add_sync(0xffffffffu, ws);
    if (tid < bins) offs[tid] = basew + inc - total + before;
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += kHeld * 32) {
      // a span of one load is still in the registers
      if (span > kHeld * 32) load(i0);
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        if (i0 + u * 32 >= hi) break;
        const bool in = key[u] != 0xFFFFFFFFu;
        if (p == 0 && in && key[u] < A.vocab) A.present[key[u]] = 1;
        const uint32_t d = in ? (key[u] >> shift) & dmask : 0xFFFFFFFFu;
        const uint32_t peers = __match_any_sync(0xffffffffu, d);
        const uint32_t below = __popc(peers & ((1u << lane) - 1u));
        uint32_t at = 0;
        if (in) at = offs[d] + mine[d] + below;
        __syncwarp();
        if (in && below == 0) mine[d] += __popc(peers);
        __syncwarp();
        if (in) {
          dk[at] = key[u];
          dp[at] = pos[u];
        }
      }
    }
    // the pairs reach the cluster's other CTAs; hist may be rewritten
    cluster.sync();
  }
}

// ------------------------------------------------------------- sum by key
constexpr int kMaxRun = 64;   // sorted positions of one chunk: see run_of
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
  int32_t run;  // positions of one chunk
  int32_t slices;
  int32_t sum_ctas;  // chunks * slices; the launch's other CTAs fill
};

// Column of element j of thread t: 8 consecutive columns a thread for rows
// that start on 16-byte boundaries, else N threads' consecutive columns an
// access (8 a thread there would put neighbouring lanes 32 bytes apart in every
// access: 79 tokens into 37178 x 3435 fp32 534 us instead of 104, 100 tokens
// added to 65536 x 2049 607 instead of 190).
template <bool VEC, int N>
__device__ __forceinline__ int64_t col_of(int64_t c0, int t, int j) {
  return VEC ? c0 + t * 8 + j : c0 + j * N + t;
}

// What lies past the end is zero, or with ANY the last column again: it is not
// stored, and loads without branches all start together.
template <bool VEC, int N, bool ANY, class T>
__device__ __forceinline__ void load_cols(const T* row, int64_t c0, int t, int64_t dim, Pack<T>& p) {
  if (VEC && c0 + t * 8 + 8 <= dim) {
    p.load(row + c0 + t * 8);
  } else {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t c = col_of<VEC, N>(c0, t, j);
      v[j] = ANY ? to_f32(row[min(c, dim - 1)]) : c < dim ? to_f32(row[c]) : 0.0f;
    }
    p.pack(v);
  }
}
template <bool VEC, int N, class T>
__device__ __forceinline__ void store_cols(T* row, int64_t c0, int t, int64_t dim, const Pack<T>& p) {
  if (VEC && c0 + t * 8 + 8 <= dim) {
    p.store(row + c0 + t * 8);
  } else {
    float v[8];
    p.unpack(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t c = col_of<VEC, N>(c0, t, j);
      if (c < dim) row[c] = from_f32<T>(v[j]);
    }
  }
}

constexpr int kSumThreads = kSlice / 8;

template <class O, bool VEC>
__device__ __forceinline__ void write_row(const ReduceArgs& A, int64_t v, int64_t c0, const float (&acc)[8]) {
  Pack<O> p;
  float r[8];
  if (A.base) {
    load_cols<VEC, kSumThreads, false>(static_cast<const O*>(A.base) + v * A.ldbase, c0, threadIdx.x, A.dim, p);
    p.unpack(r);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = 0.0f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = fmaf(acc[j], A.scale, r[j]);
  p.pack(r);
  store_cols<VEC, kSumThreads>(static_cast<O*>(A.out) + v * A.ldo, c0, threadIdx.x, A.dim, p);
}

// CTA b < sum_ctas: the sums of one chunk in one slice of columns.
template <class T, class O, bool VEC>
__device__ __forceinline__ void sum_chunk(const ReduceArgs& A, int64_t b) {
  __shared__ uint32_t sk[kMaxRun], sp[kMaxRun];
  const int64_t chunk = b / A.slices;
  const int64_t c0 = (b - chunk * A.slices) * kSlice;  // first column of the slice
  const int64_t i0 = chunk * A.run;
  const int n = static_cast<int>(min(static_cast<int64_t>(A.run), A.tokens - i0));
  if (threadIdx.x < n) {
    sk[threadIdx.x] = A.key[i0 + threadIdx.x];
    sp[threadIdx.x] = A.pos[i0 + threadIdx.x];
  }
  const uint32_t prev = i0 > 0 ? A.key[i0 - 1] : 0xFFFFFFFFu;
  const uint32_t next = i0 + n < A.tokens ? A.key[i0 + n] : 0xFFFFFFFFu;
  __syncthreads();
  if (col_of<VEC, kSumThreads>(c0, threadIdx.x, 0) >= A.dim) return;
  const uint32_t vocab = static_cast<uint32_t>(A.vocab);
  const T* dy = static_cast<const T*>(A.dy);
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
  bool from_before = sk[0] == prev;
  constexpr int U = sizeof(T) == 2 ? 8 : 4;  // rows in flight
  for (int i = 0; i < n; i += U) {
    if (sk[i] >= vocab) return;  // padding fills the rest of the list
    Pack<T> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // past the end the first row again (see ANY)
      const int at = i + u < n && sk[i + u] < vocab ? i + u : i;
      load_cols<VEC, kSumThreads, true>(dy + int64_t(sp[at]) * A.lddy, c0, threadIdx.x, A.dim, v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= n) break;
      const uint32_t k = sk[i + u];
      if (k >= vocab) return;
      float x[8];
      v[u].unpack(x);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += x[j];
      const bool last = i + u + 1 == n;
      const bool ends = last ? k != next : k != sk[i + u + 1];
      if (ends && !from_before) {
        write_row<O, VEC>(A, k, c0, acc);
      } else if (ends || last) {
        // a row of several chunks: the sum goes to this chunk's head slot when
        // the row came from the chunk before, to its tail slot otherwise
        float* p = A.part + (chunk * 2 + (from_before ? 0 : 1)) * A.dim;
        if (VEC && c0 + threadIdx.x * 8 + 8 <= A.dim && A.dim % 4 == 0) {
          store8(p + c0 + threadIdx.x * 8, acc);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int64_t c = col_of<VEC, kSumThreads>(c0, threadIdx.x, j);
            if (c < A.dim) p[c] = acc[j];
          }
        }
      }
      if (ends) {
        from_before = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
      }
    }
  }
}

// The other CTAs: rows without a token become base, or zeros.  A CTA takes 32
// consecutive rows, so that which of them are absent is one look; its warps
// take pieces of 256 columns of them in turn, 4 at a time (a row at a time by
// the whole CTA: 19 tokens added to 122738 x 153 191 us instead of 54).  It
// reads and writes base and out alone, so their alignment decides (VEC),
// whatever dy's.
constexpr int kFillRows = 32;
constexpr int kFillHeld = 4;
template <class O, bool VEC>
__device__ __forceinline__ void fill_rows(const ReduceArgs& A, int64_t b) {
  const int lane = threadIdx.x & 31;
  const int64_t v0 = b * kFillRows, v = v0 + lane;
  const unsigned absent = __ballot_sync(0xffffffffu, v < A.vocab && !A.present[v]);
  const float zero[8] = {};
  constexpr unsigned kWarps = kSumThreads / 32;
  const unsigned pieces = static_cast<unsigned>((A.dim + 255) / 256);  // of a row
  for (unsigned i = threadIdx.x >> 5; i < kFillRows * pieces; i += kWarps * kFillHeld) {
    Pack<O> p[kFillHeld];
    unsigned row[kFillHeld];
    int64_t c0[kFillHeld];
    bool on[kFillHeld];
#pragma unroll
    for (int u = 0; u < kFillHeld; ++u) {
      const unsigned at = i + u * kWarps;
      row[u] = at / pieces;
      c0[u] = static_cast<int64_t>(at - row[u] * pieces) * 256;
      on[u] = row[u] < kFillRows && (absent >> (row[u] & 31) & 1u);
      p[u].pack(zero);
      if (A.base && on[u])
        load_cols<VEC, 32, false>(static_cast<const O*>(A.base) + (v0 + row[u]) * A.ldbase, c0[u], lane, A.dim, p[u]);
    }
#pragma unroll
    for (int u = 0; u < kFillHeld; ++u)
      if (on[u]) store_cols<VEC, 32>(static_cast<O*>(A.out) + (v0 + row[u]) * A.ldo, c0[u], lane, A.dim, p[u]);
  }
}

// VEC: every tensor's rows are 16-byte aligned; VECO: out's and base's are.
template <class T, class O, bool VEC, bool VECO>
__global__ void __launch_bounds__(kSumThreads, 3) k_embed_rows(const ReduceArgs A) {
  if (blockIdx.x < A.sum_ctas)
    sum_chunk<T, O, VEC>(A, blockIdx.x);
  else
    fill_rows<O, VECO>(A, blockIdx.x - A.sum_ctas);
}

// Rows that span chunks.  The owner is the chunk in which the row begins; it
// adds its tail and the head slots of the chunks that follow.  A warp takes
// one chunk and 128 columns; the rows of more than kLongRow chunks are left to
// the whole CTA, whose warps add an eighth of the slots each.
constexpr int kJoinCols = 128;
constexpr int kJoinWarps = 8;
constexpr int kLongRow = 64;

// Sum of the row's slots of chunks c0 .. c1 - 1 (c0 its first chunk or
// later), 8 loads at a time.
__device__ __forceinline__ void sum_slots(const ReduceArgs& A, int64_t owner, int64_t c0, int64_t c1, int64_t col,
                                          float (&acc)[4]) {
  constexpr int U = 8;
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = 0.0f;
  if (A.dim % 4 == 0) {
    if (col >= A.dim) return;
    for (int64_t c = c0; c < c1; c += U) {
      float4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = c + u < c1 ? *reinterpret_cast<const float4*>(A.part + ((c + u) * 2 + (c + u == owner ? 1 : 0)) * A.dim + col)
                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int u = 0; u < U; ++u) acc[0] += v[u].x, acc[1] += v[u].y, acc[2] += v[u].z, acc[3] += v[u].w;
    }
  } else {
    for (int64_t c = c0; c < c1; c += U) {
      float v[U][4];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[u][j] = c + u < c1 && col + j < A.dim ? A.part[((c + u) * 2 + (c + u == owner ? 1 : 0)) * A.dim + col + j] : 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += v[u][j];
    }
  }
}

template <class O>
__device__ __forceinline__ void write_sum(const ReduceArgs& A, uint32_t k, int64_t col, const float (&acc)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (col + j >= A.dim) continue;
    const float b0 = A.base ? to_f32(static_cast<const O*>(A.base)[k * A.ldbase + col + j]) : 0.0f;
    static_cast<O*>(A.out)[k * A.ldo + col + j] = from_f32<O>(fmaf(acc[j], A.scale, b0));
  }
}

template <class O>
__global__ void __launch_bounds__(kJoinWarps * 32) k_embed_join(const ReduceArgs A) {
  __shared__ int64_t long_last[kJoinWarps];
  __shared__ float part[kJoinWarps][kJoinCols];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t chunk = static_cast<int64_t>(blockIdx.x) * kJoinWarps + warp;
  const int64_t i0 = chunk * A.run, end = i0 + A.run;
  const int64_t col = static_cast<int64_t>(blockIdx.y) * kJoinCols + lane * 4;
  if (lane == 0) long_last[warp] = 0;
  if (end < A.tokens) {  // the last chunk has no successor
    const uint32_t k = A.key[end - 1], after = A.key[end], at0 = A.key[i0], before = i0 > 0 ? A.key[i0 - 1] : 0xFFFFFFFFu;
    // something spans the boundary, and it did not begin in an earlier chunk
    if (k < A.vocab && after == k && !(at0 == k && before == k)) {
      // the row's last chunk: the last one that begins with its key (the keys
      // are sorted), looked for 32 chunks at a time
      int64_t last = chunk + 1;
      for (;;) {
        const int64_t c = last + 1 + lane;
        const unsigned same = __ballot_sync(0xffffffffu, c * A.run < A.tokens && A.key[c * A.run] == k);
        last += __popc(same);
        if (same != 0xffffffffu) break;
      }
      if (last - chunk < kLongRow) {
        float acc[4];
        sum_slots(A, chunk, chunk, last + 1, col, acc);
        write_sum<O>(A, k, col, acc);
      } else if (lane == 0) {
        long_last[warp] = last;
      }
    }
  }
  __syncthreads();
  for (int w = 0; w < kJoinWarps; ++w) {
    const int64_t last = long_last[w];
    if (last == 0) continue;
    const int64_t owner = static_cast<int64_t>(blockIdx.x) * kJoinWarps + w;
    const int64_t share = lm_div_up(last + 1 - owner, kJoinWarps);
    const int64_t c0 = owner + warp * share, c1 = min(last + 1, c0 + share);
    float acc[4];
    sum_slots(A, owner, c0, c1, col, acc);
#pragma unroll
    for (int j = 0; j < 4; ++j) part[warp][lane * 4 + j] = acc[j];
    __syncthreads();
    if (warp == 0) {
      for (int u = 1; u < kJoinWarps; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += part[u][lane * 4 + j];
      write_sum<O>(A, A.key[(owner + 1) * A.run - 1], col, acc);
    }
    __syncthreads();
  }
}

// Positions of a chunk: short chunks for short lists, to have CTAs for every
// SM; long ones leave fewer partial sums to write and join.
int run_of(int64_t tokens) { return tokens <= 8192 ? 16 : tokens <= 24576 ? 32 : kMaxRun; }

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
  g.chunks = lm_div_up(tokens, run_of(tokens));
  for (int i = 0; i < 2; ++i) {
    g.key[i] = take(static_cast<size_t>(tokens) * 4);
    g.pos[i] = take(static_cast<size_t>(tokens) * 4);
  }
  g.present = take(static_cast<size_t>(vocab) + 16);
  g.part = take(static_cast<size_t>(g.chunks) * 2 * dim * 4);
  g.total = at;
  return g;
}

template <class T, class O>
cudaError_t run_reduce(ReduceArgs R, bool in_place, bool vec, bool vec_out, cudaStream_t st) {
  R.sum_ctas = static_cast<int32_t>(R.chunks * R.slices);
  const int64_t fill = in_place ? 0 : lm_div_up(R.vocab, kFillRows);
  const unsigned grid = static_cast<unsigned>(R.sum_ctas + fill);
  if (grid > 0) {
    if (vec)
      k_embed_rows<T, O, true, true><<<grid, kSumThreads, 0, st>>>(R);
    else if (vec_out)
      k_embed_rows<T, O, false, true><<<grid, kSumThreads, 0, st>>>(R);
    else
      k_embed_rows<T, O, false, false><<<grid, kSumThreads, 0, st>>>(R);
  }
  if (R.chunks > 1)
    k_embed_join<O><<<dim3(static_cast<unsigned>(lm_div_up(R.chunks, kJoinWarps)),
                           static_cast<unsigned>(lm_div_up(R.dim, kJoinCols))),
                      kJoinWarps * 32, 0, st>>>(R);
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

cudaError_t launch_embedding_grad(const EmbedGradArgs& A, int dy_dtype, int out_dtype, void* workspace,
                                  cudaStream_t st) {
  const GradPlan g = plan_grad(A.tokens, A.vocab, A.dim);
  char* ws = static_cast<char*>(workspace);
  ReduceArgs R = {};
  R.dy = A.dy, R.lddy = A.lddy;
  R.tokens = A.tokens, R.vocab = A.vocab, R.dim = A.dim, R.scale = A.scale;
  R.base = A.base, R.ldbase = A.ldbase, R.out = A.out, R.ldo = A.ldo;
  R.present = reinterpret_cast<const uint8_t*>(ws + g.present);
  R.part = reinterpret_cast<float*>(ws + g.part);
  R.chunks = g.chunks, R.run = run_of(A.tokens);
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
    // two steps of 32 a warp, up to 8 CTAs
    int nct = 1;
    while (nct < kMaxSortCtas && A.tokens > int64_t(nct) * kSortThreads * 2) nct *= 2;
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
  const bool vec_out = lm_aligned(A.out, A.ldo, A.vocab, eb, 16) && (!A.base || lm_aligned(A.base, A.ldbase, A.vocab, eb, 16));
  const bool vec = vec_out && lm_aligned(A.dy, A.lddy, A.tokens, dy_dtype == kDtBf16 ? 2 : 4, 16);
  if (dy_dtype == kDtBf16)
    return out_dtype == kDtBf16 ? run_reduce<__nv_bfloat16, __nv_bfloat16>(R, in_place, vec, vec_out, st)
                                : run_reduce<__nv_bfloat16, float>(R, in_place, vec, vec_out, st);
  return out_dtype == kDtBf16 ? run_reduce<float, __nv_bfloat16>(R, in_place, vec, vec_out, st)
                              : run_reduce<float, float>(R, in_place, vec, vec_out, st);
}

}  // namespace okls
