// Quantisation to e4m3 with a scale for each group of 128, in either
// orientation or both from one read (sm_103a).
//
//   a = max(amax, 2^-100),  q = e4m3(x (448 / a)),  scale = a / 448.
//
// Bound by memory: 2 or 4 bytes in and 1 (or 2) out per element.  A CTA takes
// one 128 x 128 tile, which holds whole groups of every kind: rows of the
// tile, columns of the tile (the transposed matrix's row groups), and the
// square block.  Each of 256 threads keeps an 8 x 8 patch in registers, so
// row maxima are shuffles over the 16 lanes of a tile row, column maxima a
// shuffle and one exchange over the 8 warps, and the transposed codes leave
// through a shared-memory tile in runs of 8 bytes.
#include "okls_internal.h"
#include "okls_lm.cuh"

namespace okls {
namespace {

constexpr int kTile = 128;
constexpr int kPitchT = kTile + 8;  // bytes; keeps 8-byte runs of neighbouring columns in distinct banks

template <class T, bool VEC, bool SQUARE>
__global__ void __launch_bounds__(256) k_fp8_quantize(const QuantArgs A) {
  __shared__ __align__(16) uint8_t tq[kTile * kPitchT];
  __shared__ uint32_t cmax[8][kTile];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cx = (tid & 15) * 8, ry = (tid >> 4) * 8;  // this thread's patch
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kTile, c0 = static_cast<int64_t>(blockIdx.x) * kTile;

  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + ry + i, c = c0 + cx;
    const T* p = static_cast<const T*>(A.x) + r * A.ldx + c;
    if (VEC && r < A.rows && c + 8 <= A.cols) {
      load8(p, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = r < A.rows && c + j < A.cols ? to_f32(p[j]) : 0.0f;
    }
  }

  // group maxima: per tile row (16 lanes), per tile column (all threads of a
  // column), or of the whole tile
  uint32_t rm[8], cm[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) cm[j] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    rm[i] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = mag_bits(v[i][j]);
      rm[i] = max(rm[i], b);
      cm[j] = max(cm[j], b);
    }
  }
  if (SQUARE) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, rm[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) cmax[0][warp] = m;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, lane < 8 ? cmax[0][lane] : 0u);
#pragma unroll
    for (int i = 0; i < 8; ++i) rm[i] = cm[i] = m;
  } else {
    if (A.q) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) rm[i] = max(rm[i], __shfl_xor_sync(0xffffffffu, rm[i], o));
    }
    if (A.qt) {
#pragma unroll
      for (int j = 0; j < 8; ++j) cm[j] = max(cm[j], __shfl_xor_sync(0xffffffffu, cm[j], 16));
      if (lane < 16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) cmax[warp][cx + j] = cm[j];
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 8; ++w)
#pragma unroll
        for (int j = 0; j < 8; ++j) cm[j] = max(cm[j], cmax[w][cx + j]);
    }
  }

  if (A.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + ry + i, c = c0 + cx;
      float mul, scale;
      fp8_scales(rm[i], &mul, &scale);
      if (r < A.rows && c < A.cols) {
        const uint2 code = e4m3x8(v[i], mul);
        uint8_t* q = A.q + r * A.ldq + c;
        if (c + 8 <= A.cols && (reinterpret_cast<uintptr_t>(q) & 7) == 0) {
          *reinterpret_cast<uint2*>(q) = code;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c + j < A.cols) q[j] = static_cast<uint8_t>((j < 4 ? code.x : code.y) >> (8 * (j & 3)));
        }
      }
      if (!SQUARE && (tid & 15) == 0 && r < A.rows)
        A.scale[r * A.lds_row + static_cast<int64_t>(blockIdx.x) * A.lds_group] = scale;
    }
    if (SQUARE && tid == 0) {
      float mul, scale;
      fp8_scales(rm[0], &mul, &scale);
      A.scale[static_cast<int64_t>(blockIdx.y) * A.lds_row + static_cast<int64_t>(blockIdx.x) * A.lds_group] = scale;
    }
  }

  if (A.qt) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float mul, scale;
      fp8_scales(cm[j], &mul, &scale);
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = v[i][j];
      *reinterpret_cast<uint2*>(tq + (cx + j) * kPitchT + ry) = e4m3x8(t, mul);
      if (!SQUARE && tid < 16 && c0 + cx + j < A.cols)
        A.scale_t[(c0 + cx + j) * A.ldst_row + static_cast<int64_t>(blockIdx.y) * A.ldst_group] = scale;
    }
    if (SQUARE && tid == 0) {
      float mul, scale;
      fp8_scales(cm[0], &mul, &scale);
      A.scale_t[static_cast<int64_t>(blockIdx.x) * A.ldst_row + static_cast<int64_t>(blockIdx.y) * A.ldst_group] = scale;
    }
    __syncthreads();
    // 128 transposed rows of 16 runs of 8 codes
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int u = tid + i * 256, c = u >> 4, r = (u & 15) * 8;
      if (c0 + c >= A.cols || r0 + r >= A.rows) continue;
      const uint2 code = *reinterpret_cast<const uint2*>(tq + c * kPitchT + r);
      uint8_t* q = A.qt + (c0 + c) * A.ldqt + r0 + r;
      if (r0 + r + 8 <= A.rows && (reinterpret_cast<uintptr_t>(q) & 7) == 0) {
        *reinterpret_cast<uint2*>(q) = code;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (r0 + r + j < A.rows) q[j] = static_cast<uint8_t>((j < 4 ? code.x : code.y) >> (8 * (j & 3)));
      }
    }
  }
}

template <class T>
void run_quant(const QuantArgs& A, int square, bool vec, dim3 grid, cudaStream_t st) {
  if (square)
    vec ? k_fp8_quantize<T, true, true><<<grid, 256, 0, st>>>(A) : k_fp8_quantize<T, false, true><<<grid, 256, 0, st>>>(A);
  else
    vec ? k_fp8_quantize<T, true, false><<<grid, 256, 0, st>>>(A) : k_fp8_quantize<T, false, false><<<grid, 256, 0, st>>>(A);
}

}  // namespace

cudaError_t launch_fp8_quantize(const QuantArgs& A, int dtype, int square, cudaStream_t st) {
  if (A.rows <= 0 || A.cols <= 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>(lm_div_up(A.cols, kTile)), static_cast<unsigned>(lm_div_up(A.rows, kTile)));
  const bool vec = lm_aligned(A.x, A.ldx, A.rows, dtype == kDtBf16 ? 2 : 4, 16);
  if (dtype == kDtBf16)
    run_quant<__nv_bfloat16>(A, square, vec, grid, st);
  else
    run_quant<float>(A, square, vec, grid, st);
  return cudaGetLastError();
}

}  // namespace okls
