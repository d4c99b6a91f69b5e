// 4-bit weights with a scale (and a zero point) for each group of a row:
// quantisation, and the product with a few rows of activations (sm_103a).
//
//   y[r, j] = sum over groups g of scale[j, g] sum over p in g of (c[j, p] - zero[j, g]) x[r, p]
//
// A generation step reads every weight once for a few tokens, so the codes'
// bytes bound it.  What has to keep up with them is the way from nibbles to
// products: small whole numbers and x are exact in bf16 and their products exact in
// fp32, so the tensor core takes them (16 weights' rows x 16 of the sum x 8 tokens an
// instruction); tokens that are not there are zero columns.  fp32 activations
// go in as three bf16 terms, whose sum is the value, with three instructions
// instead of one.  A group's partial sum is scaled in fp32 and added to the
// running sum there.  What the numbers are off by (the zero point, and the 16 or 8
// of their form) is a factor of the group's sum of x, from a product with ones.
//
// The order of a sum's terms is free, so each lane takes the codes where they
// lie: 8 codes of a word are four pairs (c0, c4), (c1, c5), ..., which a shift, a
// mask and an or turn into bf16 pairs, and the activations are paired alike.
//
// Two kernels: k_int4_stream for generated tokens (one wave of CTAs, x in shared
// memory), k_int4_matmul for more rows or longer ones than that holds.  Measured
// (bf16, L2 flushed): 1 row, 131072 x 2048 with zero points in 36.9 us (4.1 TB/s; 2.6 of
// four instructions a clock from 14 warps an SM, which wait for results of their own and for the
// tensor pipe's turn, hardly for memory), 5504 x 2048 in 4.6 us without its call; 16 rows,
// 11008 x 4096 in 18 us (1.6 a clock: x's staging and its barrier, then the same waits and
// x's reads from shared memory).
#include <cuda_bf16.h>
#include <math_constants.h>

#include "okls_internal.h"
#include "okls_lm.cuh"

namespace okls {
namespace {

constexpr int kMmThreads = 256;
constexpr int kMmWarps = kMmThreads / 32;
constexpr int kMmRows = 16;    // weights' rows of a CTA; its warps share the sum
constexpr int kMmChunk = 128;  // codes of a row that a warp takes at a time

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same with nothing to add to.
__device__ __forceinline__ void mma16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// Codes 0..15 in bits 0-3 and 16-19 as bf16 values of c - 8: 0x4300 | c is
// 128 + c, and 136 is taken away (both exact).
__device__ __forceinline__ uint32_t codes_bf16(uint32_t q) {
  const uint32_t v = (q & 0x000F000Fu) | 0x43004300u, off = 0x43084308u;
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&off));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Eight values of x as they lie in memory.
template <class X>
struct Raw {
  uint4 u[sizeof(X) / 2];
  __device__ __forceinline__ void load(const X* x) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(X) / 2); ++i) u[i] = reinterpret_cast<const uint4*>(x)[i];
  }
  // the first `count`, zeros behind them
  __device__ __forceinline__ void load_some(const X* x, int count) {
    uint32_t w[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (sizeof(X) == 4)
        w[i] = i < count ? reinterpret_cast<const uint32_t*>(x)[i] : 0u;
      else if (i < count)
        w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const unsigned short*>(x)[i]) << (16 * (i & 1));
    }
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(X) / 2); ++i) u[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  __device__ __forceinline__ void none() {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(X) / 2); ++i) u[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    if constexpr (sizeof(X) == 4) {
      const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
      unpack8(u[0], v);
    }
  }
};

// Eight values of x as the four pairs (0, 4), (1, 5), (2, 6), (3, 7) of each
// of their bf16 terms.
template <class X>
struct Terms;
template <>
struct Terms<__nv_bfloat16> {
  static constexpr int kCount = 1;
  uint32_t p[1][4];
  __device__ __forceinline__ void pair(const uint4& u) {
    p[0][0] = __byte_perm(u.x, u.z, 0x5410), p[0][1] = __byte_perm(u.x, u.z, 0x7632);
    p[0][2] = __byte_perm(u.y, u.w, 0x5410), p[0][3] = __byte_perm(u.y, u.w, 0x7632);
  }
  __device__ __forceinline__ void take(const Raw<__nv_bfloat16>& r) { pair(r.u[0]); }
  __device__ __forceinline__ void none() { p[0][0] = p[0][1] = p[0][2] = p[0][3] = 0; }
};
template <>
struct Terms<float> {
  static constexpr int kCount = 3;
  uint32_t p[3][4];
  // v = t0 + t1 + t2: each term is the upper half of what is left, cut off, so
  // that three times 8 bits are fp32's 24 and none overflows.  (An infinity is
  // its own first term; a NaN reaches the second.)
  __device__ __forceinline__ void split(const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo = v[i], hi = v[i + 4];
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        p[t][i] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
        if (t == 2) break;
        const float tl = __uint_as_float(p[t][i] << 16), th = __uint_as_float(p[t][i] & 0xFFFF0000u);
        lo = mag_bits(lo) == 0x7F800000u ? 0.0f : lo - tl;
        hi = mag_bits(hi) == 0x7F800000u ? 0.0f : hi - th;
      }
    }
  }
  __device__ __forceinline__ void take(const Raw<float>& r) {
    float v[8];
    r.values(v);
    split(v);
  }
  __device__ __forceinline__ void none() {
#pragma unroll
    for (int t = 0; t < 3; ++t) p[t][0] = p[t][1] = p[t][2] = p[t][3] = 0;
  }
};

// Group of a column: pieces of 32 and 64 columns are groups, longer groups are multiples of 128.
template <int GW>
__device__ __forceinline__ int group_of(int col, int64_t group) {
  return GW < 4 ? col / (32 * GW) : group == 128 ? col >> 7 : static_cast<int>((static_cast<uint32_t>(col) >> 7) / static_cast<uint32_t>(group >> 7));
}

__device__ __forceinline__ uint32_t half_at(const void* p, int64_t i) {
  return __ldg(static_cast<const unsigned short*>(p) + i);
}

// A lane's part of a chunk: two rows, 4 words of 8 codes each, in kLoads
// pieces that belong to one group each.
template <int GW>
struct Codes {
  static constexpr int kLoads = 4 / GW;
  uint32_t q[2][4];
  uint32_t sz[2][kLoads];  // bf16 scale, zero point above it

  __device__ __forceinline__ float scale(int h, int l) const { return __uint_as_float(sz[h][l] << 16); }
  __device__ __forceinline__ float zero(int h, int l) const { return __uint_as_float(sz[h][l] & 0xFFFF0000u); }

  template <bool ZERO>
  __device__ __forceinline__ void load(const Int4Args& A, const int64_t (&row)[2], int64_t k0, int t) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool there = row[h] < A.n;
      const uint8_t* base = A.codes + row[h] * A.ldq;
      const int64_t bytes = (A.k + 1) >> 1;
#pragma unroll
      for (int l = 0; l < kLoads; ++l) {
        const int64_t at = k0 / 2 + l * 16 * GW + t * 4 * GW;
        uint32_t w[GW];
#pragma unroll
        for (int i = 0; i < GW; ++i) w[i] = 0;
        if (there) {
          if (at + 4 * GW <= bytes) {
            if constexpr (GW == 4)
              asm("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(base + at));
            else if constexpr (GW == 2)
              asm("ld.global.nc.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(base + at));
            else
              asm("ld.global.nc.b32 %0, [%1];" : "=r"(w[0]) : "l"(base + at));
          } else {
            for (int b = 0; b < 4 * GW; ++b)
              if (at + b < bytes) w[b / 4] |= static_cast<uint32_t>(base[at + b]) << (8 * (b & 3));
          }
        }
#pragma unroll
        for (int i = 0; i < GW; ++i) q[h][l * GW + i] = w[i];
        const int64_t first = k0 + l * 32 * GW;
        sz[h][l] = 0;
        if (there && first < A.k) {
          const int64_t g = group_of<GW>(static_cast<int>(first), A.group);
          sz[h][l] = half_at(A.scale, row[h] * A.lds_row + g * A.lds_group);
          if (ZERO) sz[h][l] |= half_at(A.zero, row[h] * A.ldz_row + g * A.ldz_group) << 16;
        }
      }
    }
  }
};

// Eight warps share the chunks of 16 weights' rows; NT tiles of 8 tokens.
template <class X, int NT, int GW, bool ZERO>
__global__ void __launch_bounds__(kMmThreads) k_int4_matmul(const Int4Args A) {
  __shared__ float red[kMmWarps][NT * 8][kMmRows + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kMmRows;
  const int64_t row[2] = {row0 + g, row0 + g + 8};
  const int64_t col0 = static_cast<int64_t>(blockIdx.y) * (NT * 8);
  const int64_t chunks = (A.k + kMmChunk - 1) / kMmChunk;
  float y[NT][4] = {};
  Codes<GW> now, next;
  if (warp < chunks) now.template load<ZERO>(A, row, static_cast<int64_t>(warp) * kMmChunk, t);
  for (int64_t c = warp; c < chunks; c += kMmWarps) {
    const int64_t k0 = c * kMmChunk;
    if (c + kMmWarps < chunks) next.template load<ZERO>(A, row, k0 + kMmWarps * kMmChunk, t);
#pragma unroll
    for (int l = 0; l < Codes<GW>::kLoads; ++l) {
      float acc[NT][4] = {}, ones[NT][4] = {};
#pragma unroll
      for (int w = l * GW; w < (l + 1) * GW; ++w) {
        uint32_t a[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t q0 = now.q[0][w] >> (8 * i), q1 = now.q[1][w] >> (8 * i);
          a[i][0] = codes_bf16(q0), a[i][1] = codes_bf16(q1);
          a[i][2] = codes_bf16(q0 >> 4), a[i][3] = codes_bf16(q1 >> 4);
        }
        const int64_t at = k0 + l * 32 * GW + t * 8 * GW + (w % GW) * 8;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int64_t col = col0 + nt * 8 + g;
          Terms<X> x;
          x.none();
          if (col < A.rows && at < A.k) {
            const X* src = static_cast<const X*>(A.x) + col * A.ldx + at;
            Raw<X> r;
            if (A.x_vec && at + 8 <= A.k)
              r.load(src);
            else
              r.load_some(src, static_cast<int>(min(A.k - at, int64_t(8))));
            x.take(r);
          }
#pragma unroll
          for (int f = 0; f < Terms<X>::kCount; ++f) {
            mma16816(acc[nt], a[0], x.p[f][0], x.p[f][1]);
            mma16816(acc[nt], a[1], x.p[f][2], x.p[f][3]);
            if (ZERO) {
              const uint32_t one[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
              mma16816(ones[nt], one, x.p[f][0], x.p[f][1]);
              mma16816(ones[nt], one, x.p[f][2], x.p[f][3]);
            }
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = ZERO ? fmaf(8.0f - now.zero(i >> 1, l), ones[nt][i], acc[nt][i]) : acc[nt][i];
          y[nt][i] = fmaf(now.scale(i >> 1, l), v, y[nt][i]);
        }
      }
    }
    now = next;
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[warp][nt * 8 + 2 * t + (i & 1)][g + 8 * (i >> 1)] = y[nt][i];
  __syncthreads();
  for (int i = threadIdx.x; i < NT * 8 * kMmRows; i += kMmThreads) {
    const int r = i % kMmRows, c = i / kMmRows;
    if (row0 + r >= A.n || col0 + c >= A.rows) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kMmWarps; ++w) v += red[w][c][r];
    const int64_t at = (col0 + c) * A.ldy + row0 + r;
    if (A.out_dtype == kDtF32) {
      float* o = static_cast<float*>(A.out) + at;
      *o = A.accumulate ? *o + v : v;
    } else {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(A.out) + at;
      *o = __float2bfloat16_rn(A.accumulate ? __bfloat162float(*o) + v : v);
    }
  }
}

// ------------------------------------------------------------------ stream
// The form for tokens that are generated.  Persistent CTAs stage x in shared
// memory once, in the order in which lanes take it (16 bytes a lane for each
// word of codes, already paired), with its sums over each piece of a group.  A
// CTA has a run of tiles of 16 weights' rows, whose chunks (16 rows x 256 codes) go to its
// warps in turn: at any time they read neighbouring memory (warps with runs of
// chunks of their own, 1 or 2 KB of a row apart, waited for memory half of the
// time).  Every warp fills a ring of its own with asynchronous copies of its chunks
// and their scales, and leaves its part of a tile's sums in shared memory; every few
// tiles the CTA adds the parts up, in the warps' order.
//
// Instructions cost more than bytes here, so the codes' way is two of them a
// pair: a shift brings a nibble to the fraction's upper bits, a mask and an or
// make it bf16 16 + c.  The 16 + zero too many are taken away with the sum of x.
// (That costs a sum two bits, which fp32 activations are given back: there 24 is
// taken away from the pair.)
constexpr int kStreamSmem = 226 * 1024;
constexpr int kStreamChunk = 256;  // codes of a row that a warp takes at a time

// W warps; NT tiles of 8 tokens; GW words of a lane's piece of a group.
template <class X, int NT, int GW, bool ZERO>
struct Stream {
  static constexpr int kWarps = NT == 1 ? 8 : 16;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kCtas = NT == 1 ? 2 : 1;  // on an SM
  static constexpr int kAhead = NT == 1 ? 3 : 2;
  static constexpr int kTerms = Terms<X>::kCount;
  static constexpr int kLoads = 8 / GW;  // pieces of a chunk that belong to one group each
  static constexpr int kScales = kLoads * (ZERO ? 2 : 1);
  static constexpr int kStage = 2048 + 32 * kScales;
  static constexpr int kRings = kWarps * kAhead * kStage;
  static constexpr int kSums = kLoads * NT * 8;  // sums of x in a chunk
  // 16-byte unit of x of (chunk, word, term, token, lane of four)
  __device__ static __forceinline__ int unit(int chunk, int word, int term, int tokens, int token, int t) {
    return (((chunk * 8 + word) * kTerms + term) * tokens + token) * 4 + t;
  }
  static constexpr int kBuffers = NT == 1 ? 2 : 1;  // of parts of sums
  // tiles whose parts a buffer holds, in some 8 KB (16 for 16 tokens)
  __host__ __device__ static constexpr int batch(int tokens) { return tokens * NT >= 16 ? 1 : 16 / (tokens * NT); }
  __host__ __device__ static constexpr int part_floats(int tokens) { return kBuffers * batch(tokens) * kWarps * kMmRows * tokens; }
  // x, its sums, parts of sums, the rings
  static int64_t bytes(int64_t chunks, int tokens) {
    return chunks * (512 * kTerms * tokens + 4 * kSums) + 4 * part_floats(tokens) + kRings;
  }
};

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// The first `bytes` <= 16 of them, zeros behind.
__device__ __forceinline__ void copy_some(uint32_t to, const void* from, const void* valid, int bytes) {
  bytes = max(0, min(16, bytes));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(bytes > 0 ? from : valid), "r"(bytes) : "memory");
}

// The same where `on` is not zero.
__device__ __forceinline__ void copy16_if(int on, uint32_t to, const void* from) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t@p cp.async.cg.shared.global [%1], [%2], 16;\n\t}" ::"r"(on), "r"(to), "l"(from)
               : "memory");
}
__device__ __forceinline__ uint32_t shared32(uint32_t at) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ uint2 shared64(uint32_t at) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ uint4 shared128(uint32_t at) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at) : "memory");
  return r;
}

// bf16 16 + c (EXACT: c - 8) of the nibbles that the shift brought to bits 3-6
// and 19-22.  (mask and ones come in registers: with two constants it is two instructions)
template <bool EXACT>
struct Unpack {
  uint32_t mask, ones;
  __device__ __forceinline__ Unpack() { asm volatile("mov.b32 %0, 0x00780078;\n\tmov.b32 %1, 0x41804180;" : "=r"(mask), "=r"(ones)); }
  __device__ __forceinline__ uint32_t operator()(uint32_t q) const {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(q), "r"(mask), "r"(ones));  // (q & mask) | ones
    if (!EXACT) return r;
    const uint32_t off = 0x41C041C0u;  // 24
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&r), *reinterpret_cast<const __nv_bfloat162*>(&off));
    return *reinterpret_cast<const uint32_t*>(&d);
  }
};

template <class X, int NT, int GW, bool ZERO>
__global__ void __launch_bounds__(Stream<X, NT, GW, ZERO>::kThreads, Stream<X, NT, GW, ZERO>::kCtas)
    k_int4_stream(const Int4Args A, int tokens_all, int tidy, int cta_tiles, int cta_more) {
  typedef Stream<X, NT, GW, ZERO> G;
  constexpr bool kExact = sizeof(X) == 4;
  extern __shared__ uint4 xs[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int col0 = blockIdx.y * tokens_all, tokens = min(tokens_all, static_cast<int>(A.rows) - col0);
  const int chunks = static_cast<int>((A.k + kStreamChunk - 1) / kStreamChunk);
  float* sums = reinterpret_cast<float*>(xs + static_cast<size_t>(chunks) * 32 * G::kTerms * tokens);
  float* parts = sums + static_cast<size_t>(chunks) * G::kSums;
  unsigned char* ring = reinterpret_cast<unsigned char*>(parts + G::part_floats(tokens_all)) + warp * G::kAhead * G::kStage;

  // this CTA's tiles; their chunks, counted on from one tile to the next, go to the warps in turn
  const int block = blockIdx.x, cta_tile = block * cta_tiles + min(block, cta_more), end_tile = cta_tile + cta_tiles + (block < cta_more);
  const int tile0 = cta_tile + warp / chunks, begin = warp % chunks;

  // A row of a chunk is 8 pieces of 16 bytes; a lane copies pieces t and t + 4 of
  // rows 2 g and 2 g + 1 (the product's rows g and g + 8, so that the scales of a
  // lane's two rows are neighbours).  They lie at piece ^ turn, so that a warp's reads of the words of
  // one group (16 bytes of 8 rows, 32 of 4 or 64 of 2 at a time) meet no bank twice.
  const int turn = GW == 4 ? (g & 1) * 4 : GW == 2 ? (g & 3) * 2 : g;
  const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring)), ring_end = ring_at + G::kAhead * G::kStage;
  const uint32_t put0 = g * 256 + (t ^ turn) * 16, put1 = g * 256 + ((t + 4) ^ turn) * 16;
  int load_tile = tile0, load_chunk = begin;
  uint32_t load_at = ring_at;
  const uint8_t *src0 = nullptr, *src1 = nullptr;
  // scales: 8 rows of one piece's group a lane, the lanes of zero points behind those of scales
  const bool s_zero = ZERO && lane >= 2 * G::kLoads;
  const int s_load = (lane >> 1) % G::kLoads;
  const int64_t s_pitch = 2 * (s_zero ? A.ldz_group : A.lds_group);
  const char* s_src = nullptr;
  // scales that lie in another way come one by one: loaded with a chunk, put beside it with the next
  constexpr int kSingles = G::kScales / 2;
  uint32_t single[kSingles];
  uint32_t single_at = 0;
  const auto put_singles = [&]() {
    if (single_at == 0) return;
#pragma unroll
    for (int i = 0; i < kSingles; ++i)
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(single_at + (i * 32 + lane) * 2), "h"(static_cast<unsigned short>(single[i])) : "memory");
    single_at = 0;
  };
  const auto load_singles = [&](uint32_t to, int first, int row) {
    single_at = to;
#pragma unroll
    for (int i = 0; i < kSingles; ++i) {
      const int piece = (i * 32 + lane) / 16, r = row + (lane & 15);
      const int col = first + (piece % G::kLoads) * 32 * GW;
      const bool of_zero = ZERO && piece >= G::kLoads;
      single[i] = 0;
      if (r < A.n && col < A.k)
        single[i] = half_at(of_zero ? A.zero : A.scale, r * (of_zero ? A.ldz_row : A.lds_row) +
                                                            group_of<GW>(col, A.group) * (of_zero ? A.ldz_group : A.lds_group));
    }
  };
  {
    const int64_t row = static_cast<int64_t>(load_tile) * kMmRows;
    src0 = A.codes + (row + 2 * g) * A.ldq + t * 16 + load_chunk * (kStreamChunk / 2), src1 = src0 + A.ldq;
    s_src = static_cast<const char*>(s_zero ? A.zero : A.scale) + 2 * (row + (lane & 1) * 8) + (load_chunk * G::kLoads + s_load) * s_pitch;
  }
  // from one of the warp's chunks to the next, and what a step over a tile's end adds
  const int64_t s_turn = G::kWarps * G::kLoads * s_pitch, s_wrap = 2 * kMmRows - chunks * G::kLoads * s_pitch;
  const int64_t src_wrap = kMmRows * A.ldq - chunks * (kStreamChunk / 2);
  // chunks that need no look at the matrix's end, nor at groups that are longer than a piece
  const int whole_chunks = static_cast<int>(A.k / kStreamChunk);
  const int whole_tiles = GW < 4 || A.group == 128 ? static_cast<int>(A.n / kMmRows) : 0;
  const auto fetch = [&]() {
    put_singles();
    if (load_tile < end_tile) {
      if (load_chunk < whole_chunks && load_tile < whole_tiles) {
        copy16(load_at + put0, src0), copy16(load_at + put1, src0 + 64);
        copy16(load_at + put0 + 128, src1), copy16(load_at + put1 + 128, src1 + 64);
        if (tidy)
          copy16_if(lane < 2 * G::kScales, load_at + 2048 + lane * 16, s_src);
        else
          load_singles(load_at + 2048, load_chunk * kStreamChunk, load_tile * kMmRows);
      } else {
        const int first = load_chunk * kStreamChunk, row = load_tile * kMmRows;
        const int bytes = static_cast<int>((A.k + 1) >> 1) - first / 2 - t * 16;
        const int b0 = row + 2 * g < A.n ? bytes : 0, b1 = row + 2 * g + 1 < A.n ? bytes : 0;
        copy_some(load_at + put0, src0, A.codes, b0), copy_some(load_at + put1, src0 + 64, A.codes, b0 - 64);
        copy_some(load_at + put0 + 128, src1, A.codes, b1), copy_some(load_at + put1 + 128, src1 + 64, A.codes, b1 - 64);
        if (!tidy) {
          load_singles(load_at + 2048, first, row);
        } else if (lane < 2 * G::kScales) {
          const int col = first + s_load * 32 * GW;
          const int srow = row + (lane & 1) * 8;
          const void* base = s_zero ? A.zero : A.scale;
          copy_some(load_at + 2048 + lane * 16, static_cast<const char*>(base) + 2 * static_cast<int64_t>(srow) + group_of<GW>(col, A.group) * s_pitch,
                    base, col < A.k ? 2 * min(static_cast<int>(A.n) - srow, 8) : 0);
        }
      }
      src0 += G::kWarps * kStreamChunk / 2, src1 += G::kWarps * kStreamChunk / 2, s_src += s_turn;
      load_chunk += G::kWarps;
#pragma unroll 1
      while (load_chunk >= chunks) load_chunk -= chunks, ++load_tile, src0 += src_wrap, src1 += src_wrap, s_src += s_wrap;
    }
    load_at = load_at + G::kStage == ring_end ? ring_at : load_at + G::kStage;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < G::kAhead - 1; ++i) fetch();

  // stage x: 8 values a thread, of some tokens at a time, neighbouring threads along a row
  {
    constexpr int kTurns = 16 / sizeof(X);  // loads on their way together
    for (int k8 = threadIdx.x; k8 < chunks * 32; k8 += G::kThreads) {
      const int c = k8 >> 5, j = k8 & 31, l = j / (4 * GW), lane_t = (j / GW) & 3, w = l * GW + j % GW;
      const int64_t at = static_cast<int64_t>(k8) * 8;
      const int count = static_cast<int>(max(int64_t(0), min(A.k - at, int64_t(8))));
      const X* from = static_cast<const X*>(A.x) + col0 * A.ldx + at;
      uint4* to = xs + G::unit(c, w, 0, tokens, 0, lane_t);
#pragma unroll 1
      for (int col = 0; col < tokens; col += kTurns) {
        Raw<X> raw[kTurns];
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
          if (col + i >= tokens) break;
          if (A.x_vec && count == 8)
            raw[i].load(from + (col + i) * A.ldx);
          else
            raw[i].load_some(from + (col + i) * A.ldx, count);
        }
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
          if (col + i >= tokens) break;
          Terms<X> x;
          x.take(raw[i]);
#pragma unroll
          for (int f = 0; f < G::kTerms; ++f) to[(f * tokens + col + i) * 4] = make_uint4(x.p[f][0], x.p[f][1], x.p[f][2], x.p[f][3]);
        }
      }
    }
  }
  __syncthreads();

  // where the lane's units of x are, in bytes, from a word and a term to the
  // next (a token that is not there repeats the last one: its columns are not stored)
  const uint32_t x_term = tokens * 64, x_word = x_term * G::kTerms;
  uint32_t x_at[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    x_at[nt] = static_cast<uint32_t>(__cvta_generic_to_shared(xs + min(nt * 8 + g, tokens - 1) * 4 + t));
  const uint32_t sums_at = static_cast<uint32_t>(__cvta_generic_to_shared(sums)) + 8 * t;
  if (!kExact || ZERO) {
    // the pieces' sums of x: products with ones
    const uint32_t one[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    for (int c = warp; c < chunks; c += G::kWarps) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int l = 0; l < G::kLoads; ++l) {
          float acc[4] = {};
#pragma unroll
          for (int w = l * GW; w < (l + 1) * GW; ++w)
#pragma unroll
            for (int f = 0; f < G::kTerms; ++f) {
              const uint4 x = shared128(x_at[nt] + (c * 8 + w) * x_word + f * x_term);
              mma16816(acc, one, x.x, x.y);
              mma16816(acc, one, x.z, x.w);
            }
          if (g == 0) *reinterpret_cast<float2*>(sums + c * G::kSums + (l * NT + nt) * 8 + 2 * t) = make_float2(acc[0], acc[1]);
        }
      }
    }
    __syncthreads();
  }

  float y[NT][4] = {};
  const auto store = [&](int64_t row, int col, float v) {
    if (row >= A.n || col >= tokens) return;
    const int64_t at = (col0 + col) * A.ldy + row;
    if (A.out_dtype == kDtF32) {
      float* o = static_cast<float*>(A.out) + at;
      *o = A.accumulate ? *o + v : v;
    } else {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(A.out) + at;
      *o = __float2bfloat16_rn(A.accumulate ? __bfloat162float(*o) + v : v);
    }
  };
  const Unpack<kExact> unpack;
  const int batch = G::batch(tokens_all), buffer = batch * G::kWarps * kMmRows * tokens;
  uint32_t stage = ring_at;
  int tile = tile0, chunk = begin;
  for (int base = cta_tile, turns = 0; base < end_tile; base += batch, ++turns) {
    const int stop = min(base + batch, end_tile);
    float* mine = parts + (G::kBuffers == 2 ? (turns & 1) * buffer : 0);
#pragma unroll 1
    while (tile < stop) {
      uint32_t xw[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) xw[nt] = x_at[nt] + chunk * 8 * x_word;
      const uint32_t sum_at = sums_at + chunk * G::kSums * 4;
      fetch();
      asm volatile("cp.async.wait_group %0;" ::"n"(G::kAhead - 1) : "memory");
      __syncwarp();
#pragma unroll
      for (int l = 0; l < G::kLoads; ++l) {
        uint32_t q[2][GW];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t r = stage + g * 256 + h * 128;
          if constexpr (GW == 4) {
            const uint4 v = shared128(r + ((l * 4 + t) ^ turn) * 16);
            q[h][0] = v.x, q[h][1] = v.y, q[h][2] = v.z, q[h][3] = v.w;
          } else if constexpr (GW == 2) {
            const uint2 v = shared64(r + ((l * 2 + (t >> 1)) ^ turn) * 16 + (t & 1) * 8);
            q[h][0] = v.x, q[h][1] = v.y;
          } else {
            q[h][0] = shared32(r + (l ^ turn) * 16 + t * 4);
          }
        }
        float acc[NT][4];
#pragma unroll
        for (int w = 0; w < GW; ++w) {
          const uint32_t u0 = q[0][w], u1 = q[1][w];
          const uint32_t a0[4] = {unpack(u0 << 3), unpack(u1 << 3), unpack(u0 >> 1), unpack(u1 >> 1)};
          const uint32_t a1[4] = {unpack(u0 >> 5), unpack(u1 >> 5), unpack(u0 >> 9), unpack(u1 >> 9)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int f = 0; f < G::kTerms; ++f) {
              const uint4 x = shared128(xw[nt] + (l * GW + w) * x_word + f * x_term);
              if (w == 0 && f == 0)
                mma16816_first(acc[nt], a0, x.x, x.y);
              else
                mma16816(acc[nt], a0, x.x, x.y);
              mma16816(acc[nt], a1, x.z, x.w);
            }
          }
        }
        // scales, and what is too much in the codes, of rows 2 g and 2 g + 1
        const uint32_t sv = shared32(stage + 2048 + l * 32 + g * 4);
        const float s[2] = {__uint_as_float(sv << 16), __uint_as_float(sv & 0xFFFF0000u)};
        float z[2] = {kExact ? 0.0f : 24.0f, kExact ? 0.0f : 24.0f};
        if (ZERO) {
          const uint32_t zv = shared32(stage + 2048 + (G::kLoads + l) * 32 + g * 4);
          z[0] = (kExact ? -8.0f : 16.0f) + __uint_as_float(zv << 16), z[1] = (kExact ? -8.0f : 16.0f) + __uint_as_float(zv & 0xFFFF0000u);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (!kExact || ZERO) {
            const uint2 v = shared64(sum_at + (l * NT + nt) * 32);
            const float x0 = __uint_as_float(v.x), x1 = __uint_as_float(v.y);
            acc[nt][0] = fmaf(-z[0], x0, acc[nt][0]), acc[nt][1] = fmaf(-z[0], x1, acc[nt][1]);
            acc[nt][2] = fmaf(-z[1], x0, acc[nt][2]), acc[nt][3] = fmaf(-z[1], x1, acc[nt][3]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) y[nt][i] = fmaf(s[i >> 1], acc[nt][i], y[nt][i]);
        }
      }
      stage = stage + G::kStage == ring_end ? ring_at : stage + G::kStage;
      __syncwarp();
      chunk += G::kWarps;
      if (chunk >= chunks) {
        // leave this tile's part
        float* to = mine + ((tile - base) * G::kWarps + warp) * kMmRows * tokens;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int col = nt * 8 + 2 * t + i;
            if (col < tokens) *reinterpret_cast<float2*>(to + col * kMmRows + 2 * g) = make_float2(y[nt][i], y[nt][2 + i]);
            y[nt][i] = y[nt][2 + i] = 0.0f;
          }
        }
        do
          chunk -= chunks, ++tile;
        while (chunk >= chunks);
      }
    }
    __syncthreads();
    // (a warp has a part of a tile if one of the tile's chunks is its turn)
    for (int j = threadIdx.x / kMmRows; j < (stop - base) * tokens; j += G::kThreads / kMmRows) {
      const int r = threadIdx.x % kMmRows, b = j / tokens, c = j - b * tokens, first = (base + b - cta_tile) * chunks;
      const float* from = mine + (b * G::kWarps * tokens + c) * kMmRows + r;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < G::kWarps; ++w)
        if (((w - first) & (G::kWarps - 1)) < chunks) v += from[w * kMmRows * tokens];
      store(static_cast<int64_t>(base + b) * kMmRows + r, c, v);
    }
    if (G::kBuffers == 1) __syncthreads();
  }
}

// ---------------------------------------------------------------- quantise
// 16 lanes take a group, two neighbouring values (a byte of codes) each at a
// time.  Without zero points scale = bf16(amax / 7) and c = round(x / scale) + 8
// in 1..15; with them the group's range, 0 included, is spread over 0..15:
// scale = bf16((hi - lo) / 15), zero = bf16(-lo / scale), c = round(x / scale +
// zero).  The codes are made with the rounded scale and zero.
template <class X>
__global__ void __launch_bounds__(256) k_int4_quantize(const Int4QuantArgs A) {
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 4;
  const int64_t groups = (A.cols + A.group - 1) / A.group;
  const int lane = threadIdx.x & 15;
  const bool there = unit < A.rows * groups;
  const int64_t row = there ? unit / groups : 0, g = there ? unit % groups : 0;
  const int64_t begin = g * A.group, end = there ? min(begin + A.group, A.cols) : begin;
  const X* x = static_cast<const X*>(A.x) + row * A.ldx;
  float lo = 0.0f, hi = 0.0f;
  uint32_t mag = 0;
  for (int64_t i = begin + 2 * lane; i < end; i += 32) {
    const float a = to_f32(x[i]), b = i + 1 < end ? to_f32(x[i + 1]) : 0.0f;
    lo = fminf(lo, fminf(a, b)), hi = fmaxf(hi, fmaxf(a, b));
    mag = max(mag, max(mag_bits(a), mag_bits(b)));
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, o));
  }
  if (!there) return;
  const bool sym = A.zero == nullptr;
  // (halves: the range of a group may pass fp32's)
  float s = sym ? __fdiv_rn(fmaxf(-lo, hi), 7.0f) : 2.0f * __fdiv_rn(0.5f * hi - 0.5f * lo, 15.0f);
  __nv_bfloat16 sb = __float2bfloat16_rn(fmaxf(s, kFp8AmaxFloor));
  if (mag >= 0x7F800000u) sb = __float2bfloat16_rn(CUDART_NAN_F);
  s = __bfloat162float(sb);
  const __nv_bfloat16 zb = __float2bfloat16_rn(sym ? 8.0f : __fdiv_rn(-lo, s));
  const float z = __bfloat162float(zb), least = sym ? 1.0f : 0.0f;
  for (int64_t i = begin + 2 * lane; i < end; i += 32) {
    uint32_t byte = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (i + h >= end) break;
      const float v = __fadd_rn(__fdiv_rn(to_f32(x[i + h]), s), z);
      byte |= static_cast<uint32_t>(fminf(fmaxf(rintf(v), least), 15.0f)) << (4 * h);
    }
    A.codes[row * A.ldq + i / 2] = static_cast<uint8_t>(byte);
  }
  if (lane == 0) {
    static_cast<__nv_bfloat16*>(A.scale)[row * A.lds_row + g * A.lds_group] = sb;
    if (!sym) static_cast<__nv_bfloat16*>(A.zero)[row * A.ldz_row + g * A.ldz_group] = zb;
  }
}

template <class X, int NT, int GW, bool ZERO>
cudaError_t launch_stream(const Int4Args& A, int tokens, bool tidy, int num_sms, cudaStream_t st) {
  typedef Stream<X, NT, GW, ZERO> G;
  static PerDevice pd;
  const cudaError_t e = once_per_device(pd, [](int) {
    return cudaFuncSetAttribute(k_int4_stream<X, NT, GW, ZERO>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem);
  });
  if (e != cudaSuccess) return e;
  const int64_t chunks = lm_div_up(A.k, kStreamChunk), tiles = lm_div_up(A.n, kMmRows);
  const int64_t smem = G::bytes(chunks, tokens), fit = 227 * 1024 / (smem + 1024);
  const int64_t ctas = num_sms * (fit < 1 ? 1 : fit > G::kCtas ? G::kCtas : fit);
  const dim3 grid(static_cast<unsigned>(tiles < ctas ? tiles : ctas), static_cast<unsigned>(lm_div_up(A.rows, tokens)));
  k_int4_stream<X, NT, GW, ZERO><<<grid, G::kThreads, static_cast<size_t>(smem), st>>>(A, tokens, tidy, static_cast<int>(tiles / grid.x), static_cast<int>(tiles % grid.x));
  return cudaGetLastError();
}

// Tokens, up to `most`, that a pass of the kernel's form holds in shared memory.
template <class G>
int64_t stream_fit(int64_t chunks, int64_t most) {
  int64_t fit = 0;
  while (fit < most && G::bytes(chunks, static_cast<int>(fit) + 1) <= kStreamSmem) ++fit;
  return fit;
}

template <class X, int GW, bool ZERO>
cudaError_t launch_form(const Int4Args& A, int num_sms, cudaStream_t st) {
  // scales of neighbouring rows side by side, groups on 16-byte boundaries
  const auto ordered = [](const void* p, int64_t row, int64_t group) {
    return row == 1 && group % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  };
  const bool tidy = ordered(A.scale, A.lds_row, A.lds_group) && (!ZERO || ordered(A.zero, A.ldz_row, A.ldz_group));
  if (A.n <= (1 << 30)) {
    // One pass or two of up to 8 tokens, or of up to 16.  Up to four of at least 8 where the weights
    // are large: 48 rows, 2^24 codes in 4096 x 4096, take 31 us instead of the other kernel's 38, in 65536 x 2048
    // 143 instead of 380; 4096 x 1024 19 instead of 15; four passes of 4 (16 rows, 4096 x 16384) 68 instead of 58.
    constexpr int64_t kLarge = 1 << 23;
    const int64_t chunks = lm_div_up(A.k, kStreamChunk), rows = A.rows;
    const int64_t few = stream_fit<Stream<X, 1, GW, ZERO>>(chunks, 8), more = stream_fit<Stream<X, 2, GW, ZERO>>(chunks, 16);
    if (rows <= 8 && 2 * few >= rows)
      return launch_stream<X, 1, GW, ZERO>(A, static_cast<int>(few < rows ? lm_div_up(rows, 2) : rows), tidy, num_sms, st);
    const int64_t passes = more > 0 ? lm_div_up(rows, more) : 5;
    if (passes <= (more >= 8 && A.n * A.k >= kLarge ? 4 : 2))
      return launch_stream<X, 2, GW, ZERO>(A, static_cast<int>(lm_div_up(rows, passes)), tidy, num_sms, st);
  }
  const dim3 grid(static_cast<unsigned>(lm_div_up(A.n, kMmRows)), static_cast<unsigned>(lm_div_up(A.rows, 32)));
  k_int4_matmul<X, 4, GW, ZERO><<<grid, kMmThreads, 0, st>>>(A);
  return cudaGetLastError();
}

template <class X, int GW>
cudaError_t launch_zero(const Int4Args& A, int num_sms, cudaStream_t st) {
  return A.zero ? launch_form<X, GW, true>(A, num_sms, st) : launch_form<X, GW, false>(A, num_sms, st);
}

template <class X>
cudaError_t launch_typed(const Int4Args& A, int num_sms, cudaStream_t st) {
  if (A.group == 32) return launch_zero<X, 1>(A, num_sms, st);
  if (A.group == 64) return launch_zero<X, 2>(A, num_sms, st);
  return launch_zero<X, 4>(A, num_sms, st);
}

}  // namespace

cudaError_t launch_int4_matmul(const Int4Args& A, int x_dtype, int num_sms, cudaStream_t st) {
  return x_dtype == kDtF32 ? launch_typed<float>(A, num_sms, st) : launch_typed<__nv_bfloat16>(A, num_sms, st);
}

cudaError_t launch_int4_quantize(const Int4QuantArgs& A, int dtype, cudaStream_t st) {
  const int64_t units = A.rows * lm_div_up(A.cols, A.group);
  if (units == 0) return cudaSuccess;
  const unsigned grid = static_cast<unsigned>(lm_div_up(units * 16, 256));
  if (dtype == kDtF32)
    k_int4_quantize<float><<<grid, 256, 0, st>>>(A);
  else
    k_int4_quantize<__nv_bfloat16><<<grid, 256, 0, st>>>(A);
  return cudaGetLastError();
}

}  // namespace okls
