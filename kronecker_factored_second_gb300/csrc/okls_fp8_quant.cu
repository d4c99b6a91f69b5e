// Quantisation to e4m3 with a scale for each group of 128, in either
// orientation or both from one read (sm_103a).
//
//   a = max(amax, 2^-100),  q = e4m3(x (448 / a)),  scale = a / 448.
//
// Bound by memory: 2 or 4 bytes in and 1 (or 2) out per element.  A CTA takes
// one 128 x 128 tile, which holds whole groups of every kind: rows of the
// tile, columns of the tile (the transposed matrix's row groups), and the
// square block.  Each of 256 threads keeps an 8 x 8 patch in its own type
// (bf16 packed: 32 registers), so four tiles are in flight on an SM.  Maxima
// are taken on magnitude bits, two bf16 values an instruction; row maxima are
// gathered over the 16 lanes of a tile row by exchanging halves (8 shuffles
// for 8 rows), column maxima through shared memory.  The quotients are formed
// once per group, one a thread, and read back; the transposed codes leave
// through a shared-memory tile in runs of 8 bytes.
//
// Measured, 8192 x 11008 bf16: rows 47 us (85% of the copy rate), both
// orientations 73 (73%), square blocks in both 67 (79%); with fp32 patches and a
// quotient per thread and group 138, 190 and 156.
#include "okls_internal.h"
#include "okls_lm.cuh"

namespace okls {
namespace {

constexpr int kTile = 128;
constexpr int kPitchT = kTile + 8;  // bytes; keeps 8-byte runs of neighbouring columns in distinct banks

// 8 elements of one row in their own type, with magnitude maxima as the bits
// of fp32 values.
template <class T>
struct Row8;
template <>
struct Row8<float> {
  float v[8];
  __device__ __forceinline__ void load(const float* p) { load8(p, v); }
  __device__ __forceinline__ void put(int j, float x) { v[j] = x; }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  }
  __device__ __forceinline__ void unpack(float (&o)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = v[j];
  }
};
template <>
struct Row8<__nv_bfloat16> {
  uint32_t u[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    u[0] = a.x, u[1] = a.y, u[2] = a.z, u[3] = a.w;
  }
  __device__ __forceinline__ void put(int j, __nv_bfloat16 x) {
    const uint32_t b = __bfloat16_as_ushort(x);
    u[j >> 1] = j & 1 ? (u[j >> 1] & 0xFFFFu) | (b << 16) : (u[j >> 1] & 0xFFFF0000u) | b;
  }
  __device__ __forceinline__ void clear() { u[0] = u[1] = u[2] = u[3] = 0; }
  __device__ __forceinline__ void unpack(float (&o)[8]) const { unpack8(make_uint4(u[0], u[1], u[2], u[3]), o); }
};

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Magnitude maxima of an 8 x 8 patch by row and by column.
__device__ __forceinline__ void patch_max(const Row8<float> (&v)[8], uint32_t (&rm)[8], uint32_t (&cm)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) cm[j] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    rm[i] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = mag_bits(v[i].v[j]);
      rm[i] = max(rm[i], b);
      cm[j] = max(cm[j], b);
    }
  }
}
__device__ __forceinline__ void patch_max(const Row8<__nv_bfloat16> (&v)[8], uint32_t (&rm)[8], uint32_t (&cm)[8]) {
  uint32_t c2[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t r2 = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t b = v[i].u[p] & 0x7FFF7FFFu;
      r2 = max_u16x2(r2, b);
      c2[p] = max_u16x2(c2[p], b);
    }
    rm[i] = max(r2 << 16, r2 & 0xFFFF0000u);
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    cm[2 * p] = c2[p] << 16;
    cm[2 * p + 1] = c2[p] & 0xFFFF0000u;
  }
}

// One step of a maximum over lanes that differ in bit `o`: both send the half
// that the other keeps.
template <int N>
__device__ __forceinline__ void exchange_max(uint32_t (&m)[8], int o, int lane) {
  const bool upper = lane & o;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? m[i] : m[i + N / 2], o);
    m[i] = max(upper ? m[i + N / 2] : m[i], got);
  }
}

template <class T, bool VEC, bool SQUARE>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2) k_fp8_quantize(const QuantArgs A) {
  __shared__ __align__(16) uint8_t tq[kTile * kPitchT];
  __shared__ uint32_t rmax[kTile], cmax[8][kTile];
  __shared__ __align__(16) float rmul[kTile], cmul[kTile];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cx = (tid & 15) * 8, ry = (tid >> 4) * 8;  // this thread's patch
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kTile, c0 = static_cast<int64_t>(blockIdx.x) * kTile;

  Row8<T> v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + ry + i, c = c0 + cx;
    const T* p = static_cast<const T*>(A.x) + r * A.ldx + c;
    if (VEC && r < A.rows && c + 8 <= A.cols) {
      v[i].load(p);
    } else {
      v[i].clear();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (r < A.rows && c + j < A.cols) v[i].put(j, p[j]);
    }
  }
  uint32_t rm[8], cm[8];
  patch_max(v, rm, cm);

  if (SQUARE) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, rm[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) rmax[warp] = m;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int w = 1; w < 8; ++w) m = max(m, rmax[w]);
      float mul, scale;
      fp8_scales(m, &mul, &scale);
      rmul[0] = mul;
      if (A.q) A.scale[static_cast<int64_t>(blockIdx.y) * A.lds_row + static_cast<int64_t>(blockIdx.x) * A.lds_group] = scale;
      if (A.qt)
        A.scale_t[static_cast<int64_t>(blockIdx.x) * A.ldst_row + static_cast<int64_t>(blockIdx.y) * A.ldst_group] = scale;
    }
    __syncthreads();
  } else {
    if (A.q) {
      // lane bits 3, 2, 1 pick the row that a lane ends with
      exchange_max<8>(rm, 8, lane);
      exchange_max<4>(rm, 4, lane);
      exchange_max<2>(rm, 2, lane);
      rm[0] = max(rm[0], __shfl_xor_sync(0xffffffffu, rm[0], 1));
      if ((lane & 1) == 0) rmax[ry + ((lane >> 3) & 1) * 4 + ((lane >> 2) & 1) * 2 + ((lane >> 1) & 1)] = rm[0];
    }
    if (A.qt) {
      exchange_max<8>(cm, 16, lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) cmax[warp][cx + (lane >> 4) * 4 + j] = cm[j];
    }
    __syncthreads();
    if (tid < kTile) {
      if (A.q) {
        float mul, scale;
        fp8_scales(rmax[tid], &mul, &scale);
        rmul[tid] = mul;
        if (r0 + tid < A.rows)
          A.scale[(r0 + tid) * A.lds_row + static_cast<int64_t>(blockIdx.x) * A.lds_group] = scale;
      }
    } else if (A.qt) {
      const int c = tid - kTile;
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < 8; ++w) m = max(m, cmax[w][c]);
      float mul, scale;
      fp8_scales(m, &mul, &scale);
      cmul[c] = mul;
      if (c0 + c < A.cols)
        A.scale_t[(c0 + c) * A.ldst_row + static_cast<int64_t>(blockIdx.y) * A.ldst_group] = scale;
    }
    __syncthreads();
  }

  if (A.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + ry + i, c = c0 + cx;
      if (r >= A.rows || c >= A.cols) continue;
      float t[8];
      v[i].unpack(t);
      const uint2 code = e4m3x8(t, SQUARE ? rmul[0] : rmul[ry + i]);
      uint8_t* q = A.q + r * A.ldq + c;
      if (c + 8 <= A.cols && (reinterpret_cast<uintptr_t>(q) & 7) == 0) {
        *reinterpret_cast<uint2*>(q) = code;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < A.cols) q[j] = static_cast<uint8_t>((j < 4 ? code.x : code.y) >> (8 * (j & 3)));
      }
    }
  }

  if (A.qt) {
    // codes by rows, packed by columns: byte i of a column's run is row i
    uint32_t lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float t[8], u[8];
      v[i].unpack(t);
      v[i + 1].unpack(u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float mul = SQUARE ? rmul[0] : cmul[cx + j];
        const uint32_t two = e4m3x2(t[j] * mul, u[j] * mul);
        if (i == 0) lo[j] = two;
        if (i == 2) lo[j] |= two << 16;
        if (i == 4) hi[j] = two;
        if (i == 6) hi[j] |= two << 16;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) *reinterpret_cast<uint2*>(tq + (cx + j) * kPitchT + ry) = make_uint2(lo[j], hi[j]);
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
