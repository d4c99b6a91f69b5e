// 4-bit weights with a scale (and a zero point) for each group of a row:
// quantisation, and the product with a few rows of activations (sm_103a).
//
//   y[r, j] = sum over groups g of scale[j, g] sum over p in g of (c[j, p] - zero[j, g]) x[r, p]
//
// A generation step reads every weight once for a few tokens, so the codes'
// bytes bound it.  What has to keep up with them is the way from nibbles to
// products: c - 8 and x are exact in bf16 and their products exact in fp32, so
// the tensor core takes them (16 weights' rows x 16 of the sum x 8 tokens an
// instruction); tokens that are not there are zero columns.  fp32 activations
// go in as three bf16 terms, whose sum is the value, with three instructions
// instead of one.  A group's partial sum is scaled in fp32 and added to the
// running sum there.  With zero points, one more instruction with a factor of
// ones gives the group's sum of x, which (zero - 8) scale takes away.
//
// The order of a sum's terms is free, so each lane takes the codes where they
// lie: 8 codes of a word are four pairs (c0, c4), (c1, c5), ..., which a mask
// and an or turn into bf16 128 + c, and the activations are paired alike.
#include <cuda_bf16.h>
#include <math_constants.h>

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

// Codes 0..15 in bits 0-3 and 16-19 as bf16 values of c - 8: 0x4300 | c is
// 128 + c, and 136 is taken away (both exact).
__device__ __forceinline__ uint32_t codes_bf16(uint32_t q) {
  const uint32_t v = (q & 0x000F000Fu) | 0x43004300u, off = 0x43084308u;
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&off));
  return *reinterpret_cast<const uint32_t*>(&r);
}

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
  __device__ __forceinline__ void load(const __nv_bfloat16* x) { pair(*reinterpret_cast<const uint4*>(x)); }
  __device__ __forceinline__ void load_some(const __nv_bfloat16* x, int count) {
    uint32_t w[4] = {};
    const unsigned short* s = reinterpret_cast<const unsigned short*>(x);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < count) w[i / 2] |= static_cast<uint32_t>(s[i]) << (16 * (i & 1));
    pair(make_uint4(w[0], w[1], w[2], w[3]));
  }
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
  __device__ __forceinline__ void load(const float* x) {
    float v[8];
    load8(x, v);
    split(v);
  }
  __device__ __forceinline__ void load_some(const float* x, int count) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < count ? x[i] : 0.0f;
    split(v);
  }
  __device__ __forceinline__ void none() {
#pragma unroll
    for (int t = 0; t < 3; ++t) p[t][0] = p[t][1] = p[t][2] = p[t][3] = 0;
  }
};

__device__ __forceinline__ float bf16_at(const void* p, int64_t i) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const unsigned short*>(p) + i)) << 16);
}

// A lane's part of a chunk: two rows, 4 words of 8 codes each, in kLoads
// pieces that belong to one group each.
template <int GW>
struct Codes {
  static constexpr int kLoads = 4 / GW;
  uint32_t q[2][4];
  float s[2][kLoads], z[2][kLoads];

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
        s[h][l] = 0.0f, z[h][l] = 8.0f;
        if (there && first < A.k) {
          const int64_t g = first / A.group;
          s[h][l] = bf16_at(A.scale, row[h] * A.lds_row + g * A.lds_group);
          if (ZERO) z[h][l] = bf16_at(A.zero, row[h] * A.ldz_row + g * A.ldz_group);
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
            if (A.x_vec && at + 8 <= A.k)
              x.load(src);
            else
              x.load_some(src, static_cast<int>(min(A.k - at, int64_t(8))));
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
          const float v = ZERO ? fmaf(8.0f - now.z[i >> 1][l], ones[nt][i], acc[nt][i]) : acc[nt][i];
          y[nt][i] = fmaf(now.s[i >> 1][l], v, y[nt][i]);
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

template <class X, int NT, int GW>
cudaError_t launch_zero(const Int4Args& A, dim3 grid, cudaStream_t st) {
  if (A.zero)
    k_int4_matmul<X, NT, GW, true><<<grid, kMmThreads, 0, st>>>(A);
  else
    k_int4_matmul<X, NT, GW, false><<<grid, kMmThreads, 0, st>>>(A);
  return cudaGetLastError();
}

template <class X, int NT>
cudaError_t launch_group(const Int4Args& A, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(lm_div_up(A.n, kMmRows)), static_cast<unsigned>(lm_div_up(A.rows, NT * 8)));
  if (A.group == 32) return launch_zero<X, NT, 1>(A, grid, st);
  if (A.group == 64) return launch_zero<X, NT, 2>(A, grid, st);
  return launch_zero<X, NT, 4>(A, grid, st);
}

template <class X>
cudaError_t launch_typed(const Int4Args& A, cudaStream_t st) {
  if (A.rows <= 8) return launch_group<X, 1>(A, st);
  if (A.rows <= 16) return launch_group<X, 2>(A, st);
  return launch_group<X, 4>(A, st);
}

}  // namespace

cudaError_t launch_int4_matmul(const Int4Args& A, int x_dtype, cudaStream_t st) {
  return x_dtype == kDtF32 ? launch_typed<float>(A, st) : launch_typed<__nv_bfloat16>(A, st);
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
