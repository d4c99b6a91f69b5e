// RMS norm with the residual's addition, output in 32, 16 or 8 bits, and its
// gradient (sm_103a).
//
//   s = x + residual (rounded to the stream's type),  rstd = (mean s^2 + eps)^-1/2,
//   y = s rstd w;   with xhat = s rstd, g = dy w:
//   ds = rstd (g - xhat mean(g xhat)) + dres,   dw = sum_rows dy xhat.
//
// Both are bound by memory: a row is read once into registers, reduced by
// one CTA, and written from the same registers.  A warp covers 256 columns
// with 8 elements a lane, so a row of D columns takes ceil(D / 256) warp
// chunks, NV of them per warp.  A group of 128 columns with one 8-bit scale
// lies inside a warp chunk: its largest magnitude is a shuffle maximum, and
// the codes leave from the registers that hold y.
#include "okls_internal.h"
#include "okls_lm.cuh"

namespace okls {
namespace {

constexpr int kChunk = 256;  // columns of one warp chunk: 32 lanes x 8

// Column of element j of warp chunk c for this lane: 8 consecutive columns a
// lane for 16-byte accesses, or 32 consecutive columns an access otherwise.
template <bool VEC>
__device__ __forceinline__ int col_of(int c, int lane, int j) {
  return VEC ? c * kChunk + lane * 8 + j : c * kChunk + j * 32 + lane;
}

template <class T, bool VEC>
__device__ __forceinline__ void load_chunk(const T* row, int c, int lane, int dim, float (&v)[8]) {
  if (VEC && c * kChunk + lane * 8 + 8 <= dim) {
    load8(row + c * kChunk + lane * 8, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = col_of<VEC>(c, lane, j);
      v[j] = e < dim ? to_f32(row[e]) : 0.0f;
    }
  }
}

template <class T, bool VEC>
__device__ __forceinline__ void store_chunk(T* row, int c, int lane, int dim, const float (&v)[8]) {
  if (VEC && c * kChunk + lane * 8 + 8 <= dim) {
    store8(row + c * kChunk + lane * 8, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = col_of<VEC>(c, lane, j);
      if (e < dim) row[e] = from_f32<T>(v[j]);
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void load_chunk_dt(const void* base, int dt, int64_t off, int c, int lane, int dim,
                                              float (&v)[8]) {
  if (dt == kDtBf16)
    load_chunk<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(base) + off, c, lane, dim, v);
  else
    load_chunk<float, VEC>(static_cast<const float*>(base) + off, c, lane, dim, v);
}

// Sum over the CTA's warps; `slots` holds 2 x 32 floats, used in turn so that
// one barrier per sum is enough.
__device__ __forceinline__ float cta_sum(float v, float* slots, int& turn) {
  v = warp_sum(v);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  float* s = slots + turn * 32;
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < nw ? s[lane] : 0.0f);
}

// Codes and scales of one warp chunk (two groups of 128 columns).
template <bool VEC>
__device__ __forceinline__ void store_chunk_fp8(const NormArgs& A, int64_t row, int c, int lane, const float (&y)[8]) {
  uint8_t* q = static_cast<uint8_t*>(A.out) + row * A.ldo;
  float* sc = A.out_scale + row * A.lds_row;
  if (VEC) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, mag_bits(y[j]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    float mul, scale;
    fp8_scales(m, &mul, &scale);
    const int e0 = c * kChunk + lane * 8;
    const uint2 code = e4m3x8(y, mul);
    if (e0 + 8 <= A.dim) {
      *reinterpret_cast<uint2*>(q + e0) = code;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (e0 + j < A.dim) q[e0 + j] = static_cast<uint8_t>((j < 4 ? code.x : code.y) >> (8 * (j & 3)));
    }
    const int g = c * 2 + (lane >> 4);
    if ((lane & 15) == 0 && g * kFp8Group < A.dim) sc[g * A.lds_group] = scale;
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) m = max(m, mag_bits(y[4 * h + j]));
      m = __reduce_max_sync(0xffffffffu, m);
      float mul, scale;
      fp8_scales(m, &mul, &scale);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = col_of<false>(c, lane, 4 * h + j);
        if (e < A.dim) q[e] = static_cast<uint8_t>(e4m3x2(y[4 * h + j] * mul, 0.0f));
      }
      const int g = c * 2 + h;
      if (lane == 0 && g * kFp8Group < A.dim) sc[g * A.lds_group] = scale;
    }
  }
}

template <class T, int NV, bool VEC>
__global__ void __launch_bounds__(512) k_rms_norm(const NormArgs A) {
  __shared__ float slots[64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  int turn = 0;
  float w[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) load_chunk_dt<VEC>(A.weight, A.weight_dtype, 0, warp + i * nw, lane, A.dim, w[i]);
  const float inv_dim = 1.0f / static_cast<float>(A.dim);
  for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x) {
    float s[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
      load_chunk<T, VEC>(static_cast<const T*>(A.x) + row * A.ldx, warp + i * nw, lane, A.dim, s[i]);
    if (A.residual) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float r[8];
        load_chunk<T, VEC>(static_cast<const T*>(A.residual) + row * A.ldr, warp + i * nw, lane, A.dim, r);
        // the stream is held in its own type: what is normed is what is kept
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] = to_f32(from_f32<T>(s[i][j] + r[j]));
        store_chunk<T, VEC>(static_cast<T*>(A.res_out) + row * A.ldro, warp + i * nw, lane, A.dim, s[i]);
      }
    }
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) q = fmaf(s[i][j], s[i][j], q);
    const float rstd = rsqrtf(cta_sum(q, slots, turn) * inv_dim + A.eps);
    if (A.rstd && threadIdx.x == 0) A.rstd[row] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = warp + i * nw;
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = s[i][j] * rstd * w[i][j];
      if (A.out_dtype == kDtE4m3)
        store_chunk_fp8<VEC>(A, row, c, lane, y);
      else if (A.out_dtype == kDtBf16)
        store_chunk<__nv_bfloat16, VEC>(static_cast<__nv_bfloat16*>(A.out) + row * A.ldo, c, lane, A.dim, y);
      else
        store_chunk<float, VEC>(static_cast<float*>(A.out) + row * A.ldo, c, lane, A.dim, y);
    }
  }
}

template <class T, int NV, bool VEC>
__global__ void __launch_bounds__(512) k_rms_norm_grad(const NormGradArgs A) {
  __shared__ float slots[64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  int turn = 0;
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_chunk_dt<VEC>(A.weight, A.weight_dtype, 0, warp + i * nw, lane, A.dim, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  const float inv_dim = 1.0f / static_cast<float>(A.dim);
  for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x) {
    float xh[NV][8], g[NV][8];
    const float rstd = A.rstd[row];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_chunk<T, VEC>(static_cast<const T*>(A.s) + row * A.lds, warp + i * nw, lane, A.dim, xh[i]);
      load_chunk_dt<VEC>(A.dy, A.dy_dtype, row * A.lddy, warp + i * nw, lane, A.dim, g[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] *= rstd;
        dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
        g[i][j] *= w[i][j];
        dot = fmaf(g[i][j], xh[i][j], dot);
      }
    const float mean = cta_sum(dot, slots, turn) * inv_dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = warp + i * nw;
      float d[8];
      if (A.dres)
        load_chunk<T, VEC>(static_cast<const T*>(A.dres) + row * A.lddres, c, lane, A.dim, d);
      else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = fmaf(rstd, g[i][j] - xh[i][j] * mean, d[j]);
      store_chunk<T, VEC>(static_cast<T*>(A.ds) + row * A.ldds, c, lane, A.dim, d);
    }
  }
  if (A.part) {
    // dim columns of partial sums per CTA, in this lane's column order
    float* p = A.part + static_cast<int64_t>(blockIdx.x) * A.dim;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = col_of<VEC>(warp + i * nw, lane, j);
        if (e < A.dim) p[e] = dw[i][j];
      }
  }
}

// dweight[d] = sum over CTAs of their partial sums, in a fixed order: 32
// columns a block, 32 partial rows at a time.
__global__ void __launch_bounds__(1024) k_rms_norm_dweight(const float* part, int nparts, int dim, float* dweight) {
  __shared__ float t[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  float v = 0.0f;
  if (col < dim)
    for (int p = threadIdx.y; p < nparts; p += 32) v += part[static_cast<int64_t>(p) * dim + col];
  t[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = warp_sum(t[threadIdx.x][threadIdx.y]);
  const int out = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && out < dim) dweight[out] = v;
}

struct Shape {
  int nv, warps;
};

// Two chunks a warp; one when there are too few rows to fill the SMs (a row
// then takes the most threads it can); four or eight past 16 warps.
Shape norm_shape(int64_t rows, int dim, int num_sms) {
  const int chunks = static_cast<int>(lm_div_up(dim, kChunk));
  int nv = (rows < num_sms || chunks == 1) ? 1 : 2;
  while (lm_div_up(chunks, nv) > 16) nv *= 2;
  return {nv, static_cast<int>(lm_div_up(chunks, nv))};
}

int norm_grid(int64_t rows, int warps, int num_sms) {
  const int per_sm = 48 / warps > 16 ? 16 : (48 / warps < 1 ? 1 : 48 / warps);
  return static_cast<int>(rows < int64_t(num_sms) * per_sm ? rows : int64_t(num_sms) * per_sm);
}

int grad_grid(int64_t rows, int warps, int num_sms) {
  const int per_sm = 24 / warps > 8 ? 8 : (24 / warps < 1 ? 1 : 24 / warps);
  return static_cast<int>(rows < int64_t(num_sms) * per_sm ? rows : int64_t(num_sms) * per_sm);
}

template <class T, bool VEC>
void run_norm(const NormArgs& A, Shape sh, int grid, cudaStream_t st) {
  const int threads = sh.warps * 32;
  switch (sh.nv) {
    case 1: k_rms_norm<T, 1, VEC><<<grid, threads, 0, st>>>(A); break;
    case 2: k_rms_norm<T, 2, VEC><<<grid, threads, 0, st>>>(A); break;
    case 4: k_rms_norm<T, 4, VEC><<<grid, threads, 0, st>>>(A); break;
    default: k_rms_norm<T, 8, VEC><<<grid, threads, 0, st>>>(A); break;
  }
}

template <class T, bool VEC>
void run_grad(const NormGradArgs& A, Shape sh, int grid, cudaStream_t st) {
  const int threads = sh.warps * 32;
  switch (sh.nv) {
    case 1: k_rms_norm_grad<T, 1, VEC><<<grid, threads, 0, st>>>(A); break;
    case 2: k_rms_norm_grad<T, 2, VEC><<<grid, threads, 0, st>>>(A); break;
    case 4: k_rms_norm_grad<T, 4, VEC><<<grid, threads, 0, st>>>(A); break;
    default: k_rms_norm_grad<T, 8, VEC><<<grid, threads, 0, st>>>(A); break;
  }
}

int elem_bytes(int dt) { return dt == kDtF32 ? 4 : dt == kDtBf16 ? 2 : 1; }

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& A, int dtype, int num_sms, cudaStream_t st) {
  if (A.rows <= 0) return cudaSuccess;
  const Shape sh = norm_shape(A.rows, A.dim, num_sms);
  const int grid = norm_grid(A.rows, sh.warps, num_sms), eb = elem_bytes(dtype);
  const bool vec = lm_aligned(A.x, A.ldx, A.rows, eb, 16) &&
                   (!A.residual || (lm_aligned(A.residual, A.ldr, A.rows, eb, 16) &&
                                    lm_aligned(A.res_out, A.ldro, A.rows, eb, 16))) &&
                   lm_aligned(A.weight, 0, 1, 1, 16) &&
                   lm_aligned(A.out, A.ldo, A.rows, elem_bytes(A.out_dtype), A.out_dtype == kDtE4m3 ? 8 : 16);
  if (dtype == kDtBf16)
    vec ? run_norm<__nv_bfloat16, true>(A, sh, grid, st) : run_norm<__nv_bfloat16, false>(A, sh, grid, st);
  else
    vec ? run_norm<float, true>(A, sh, grid, st) : run_norm<float, false>(A, sh, grid, st);
  return cudaGetLastError();
}

size_t rms_norm_grad_workspace(int64_t rows, int64_t dim, int num_sms) {
  const Shape sh = norm_shape(rows, static_cast<int>(dim), num_sms);
  return static_cast<size_t>(grad_grid(rows, sh.warps, num_sms)) * static_cast<size_t>(dim) * sizeof(float);
}

cudaError_t launch_rms_norm_grad(const NormGradArgs& A, int s_dtype, float* dweight, int num_sms, cudaStream_t st) {
  if (A.rows <= 0) return dweight ? cudaMemsetAsync(dweight, 0, sizeof(float) * A.dim, st) : cudaSuccess;
  const Shape sh = norm_shape(A.rows, A.dim, num_sms);
  const int grid = grad_grid(A.rows, sh.warps, num_sms), eb = elem_bytes(s_dtype);
  const bool vec = lm_aligned(A.s, A.lds, A.rows, eb, 16) && lm_aligned(A.ds, A.ldds, A.rows, eb, 16) &&
                   (!A.dres || lm_aligned(A.dres, A.lddres, A.rows, eb, 16)) &&
                   lm_aligned(A.dy, A.lddy, A.rows, elem_bytes(A.dy_dtype), 16) &&
                   lm_aligned(A.weight, 0, 1, 1, 16);
  if (s_dtype == kDtBf16)
    vec ? run_grad<__nv_bfloat16, true>(A, sh, grid, st) : run_grad<__nv_bfloat16, false>(A, sh, grid, st);
  else
    vec ? run_grad<float, true>(A, sh, grid, st) : run_grad<float, false>(A, sh, grid, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !dweight) return e;
  k_rms_norm_dweight<<<static_cast<int>(lm_div_up(A.dim, 32)), dim3(32, 32), 0, st>>>(A.part, grid, A.dim, dweight);
  return cudaGetLastError();
}

}  // namespace okls
