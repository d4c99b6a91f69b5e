// RMS norm with the residual's addition, output in 32, 16 or 8 bits, and its
// gradient (sm_103a).
//
//   s = x + residual (rounded to the stream's type),  rstd = (mean s^2 + eps)^-1/2,
//   y = s rstd w;   with xhat = s rstd, g = dy w:
//   ds = rstd (g - xhat mean(g xhat)) + dres,   dw = sum_rows dy xhat.
//
// Both are bound by memory: a row is read once into registers, reduced by one
// CTA, and written from the same registers.  A warp chunk is 256 columns, 8
// elements a lane; a warp takes NV chunks and a row as many warps as it needs.
// Rows are held in their own type (packed), so that a CTA is small (2 warps
// for 2048 bf16 columns) and many rows are in flight on an SM.  The gradient
// keeps the weight's sums of its columns in registers over all rows of a CTA,
// and loads rows ahead through a ring in shared memory: each thread copies
// and later reads its own elements, so the ring needs no barrier.
//
// Measured, 16384 x 5504 bf16 with a residual: bf16 output 108 us (98% of the
// copy rate), 8-bit output 113 (82%), gradient 114 (93%; 7 us of it the weight's
// partial sums and their launch).  Eight chunks a warp were slower (128 and
// 172 us: fewer rows in flight), rows ahead in registers too (gradient 239).
//
// A group of 128 columns with one 8-bit scale lies inside a warp chunk: its
// largest magnitude is two warp reductions, each lane divides for one group
// of the warp's, and the codes leave from the registers that hold y.
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

template <bool VEC, class T>
__device__ __forceinline__ void load_chunk(const T* row, int c, int lane, int dim, Pack<T>& p) {
  if (VEC && c * kChunk + lane * 8 + 8 <= dim) {
    p.load(row + c * kChunk + lane * 8);
  } else {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = col_of<VEC>(c, lane, j);
      v[j] = e < dim ? to_f32(row[e]) : 0.0f;
    }
    p.pack(v);
  }
}

template <bool VEC, class T>
__device__ __forceinline__ void store_chunk(T* row, int c, int lane, int dim, const Pack<T>& p) {
  if (VEC && c * kChunk + lane * 8 + 8 <= dim) {
    p.store(row + c * kChunk + lane * 8);
  } else {
    float v[8];
    p.unpack(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = col_of<VEC>(c, lane, j);
      if (e < dim) row[e] = from_f32<T>(v[j]);
    }
  }
}

// The same for a tensor whose type is known at run time only.
template <bool VEC>
__device__ __forceinline__ void load_any(const void* base, int dt, int64_t off, int c, int lane, int dim,
                                         float (&v)[8]) {
  if (dt == kDtBf16) {
    Pack<__nv_bfloat16> p;
    load_chunk<VEC>(static_cast<const __nv_bfloat16*>(base) + off, c, lane, dim, p);
    p.unpack(v);
  } else {
    Pack<float> p;
    load_chunk<VEC>(static_cast<const float*>(base) + off, c, lane, dim, p);
    p.unpack(v);
  }
}
template <bool VEC>
__device__ __forceinline__ void store_any(void* base, int dt, int64_t off, int c, int lane, int dim,
                                          const float (&v)[8]) {
  if (dt == kDtBf16) {
    Pack<__nv_bfloat16> p;
    p.pack(v);
    store_chunk<VEC>(static_cast<__nv_bfloat16*>(base) + off, c, lane, dim, p);
  } else {
    Pack<float> p;
    p.pack(v);
    store_chunk<VEC>(static_cast<float*>(base) + off, c, lane, dim, p);
  }
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

template <class T, int NV, bool VEC>
__global__ void __launch_bounds__(512) k_rms_norm(const NormArgs A) {
  __shared__ float slots[64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  int turn = 0;
  const int64_t row = blockIdx.x;
  Pack<T> s[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) load_chunk<VEC>(static_cast<const T*>(A.x) + row * A.ldx, warp + i * nw, lane, A.dim, s[i]);
  if (A.residual) {
    Pack<T> r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
      load_chunk<VEC>(static_cast<const T*>(A.residual) + row * A.ldr, warp + i * nw, lane, A.dim, r[i]);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a[8], b[8];
      s[i].unpack(a);
      r[i].unpack(b);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] += b[j];
      // the stream is held in its own type: what is normed is what is kept
      s[i].pack(a);
      store_chunk<VEC>(static_cast<T*>(A.res_out) + row * A.ldro, warp + i * nw, lane, A.dim, s[i]);
    }
  }
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float a[8];
    s[i].unpack(a);
#pragma unroll
    for (int j = 0; j < 8; ++j) q = fmaf(a[j], a[j], q);
  }
  const float rstd = rsqrtf(cta_sum(q, slots, turn) * (1.0f / static_cast<float>(A.dim)) + A.eps);
  if (A.rstd && threadIdx.x == 0) A.rstd[row] = rstd;

  auto y_of = [&](int i, float(&y)[8]) {
    float w[8];
    load_any<VEC>(A.weight, A.weight_dtype, 0, warp + i * nw, lane, A.dim, w);
    s[i].unpack(y);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = y[j] * rstd * w[j];
  };
  if (A.out_dtype != kDtE4m3) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float y[8];
      y_of(i, y);
      store_any<VEC>(A.out, A.out_dtype, row * A.ldo, warp + i * nw, lane, A.dim, y);
    }
    return;
  }
  // 8 bits: lane 2 i + h divides for group h of the warp's chunk i
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float y[8];
    y_of(i, y);
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t m = mag_bits(y[j]);
      if (VEC ? lane < 16 : j < 4)
        lo = max(lo, m);
      else
        hi = max(hi, m);
    }
    lo = __reduce_max_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if ((lane >> 1) == i) amax = lane & 1 ? hi : lo;
  }
  float mul, scale;
  fp8_scales(amax, &mul, &scale);
  if (lane < 2 * NV) {
    const int g = (warp + (lane >> 1) * nw) * 2 + (lane & 1);
    if (g * kFp8Group < A.dim) A.out_scale[row * A.lds_row + g * A.lds_group] = scale;
  }
  uint8_t* o = static_cast<uint8_t*>(A.out) + row * A.ldo;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = warp + i * nw;
    float y[8];
    y_of(i, y);
    if (VEC) {
      const float m = __shfl_sync(0xffffffffu, mul, 2 * i + (lane >> 4));
      const uint2 code = e4m3x8(y, m);
      const int e0 = c * kChunk + lane * 8;
      if (e0 + 8 <= A.dim) {
        *reinterpret_cast<uint2*>(o + e0) = code;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (e0 + j < A.dim) o[e0 + j] = static_cast<uint8_t>((j < 4 ? code.x : code.y) >> (8 * (j & 3)));
      }
    } else {
      const float m0 = __shfl_sync(0xffffffffu, mul, 2 * i), m1 = __shfl_sync(0xffffffffu, mul, 2 * i + 1);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = col_of<false>(c, lane, j);
        if (e < A.dim) o[e] = static_cast<uint8_t>(e4m3x2(y[j] * (j < 4 ? m0 : m1), 0.0f));
      }
    }
  }
}

// 16 bytes into shared memory without registers; the first `bytes` of them
// from global memory, zeros after that.
__device__ __forceinline__ void copy16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the latest `pending` groups of this thread have landed.
__device__ __forceinline__ void copy_wait(int pending) {
  switch (pending) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
  }
}
constexpr int kMaxAhead = 4;

// Copies one lane's 8 elements of chunk c into its slot.
template <class T>
__device__ __forceinline__ void copy_chunk(Pack<T>* dst, const T* row, int c, int lane, int dim) {
  const int e0 = c * kChunk + lane * 8;
  constexpr int per = 16 / sizeof(T);
#pragma unroll
  for (int h = 0; h < static_cast<int>(sizeof(Pack<T>) / 16); ++h) {
    const int e = e0 + h * per;
    const int n = e >= dim ? 0 : e + per <= dim ? per : dim - e;
    copy16(reinterpret_cast<char*>(dst) + h * 16, row + (n ? e : 0), n * static_cast<int>(sizeof(T)));
  }
}

// Rows ahead in a ring of `ring` rows (shared memory: per row and thread NV
// packs of s, dy and dres).  Needs 16-byte aligned rows.
template <class T, class D, int NV>
__global__ void __launch_bounds__(512) k_rms_norm_grad_ring(const NormGradArgs A, int ring) {
  extern __shared__ __align__(16) char ring_mem[];
  __shared__ float slots[64];
  __shared__ float rstds[16][kMaxAhead];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = blockDim.x >> 5, nt = blockDim.x;
  // [stage][tensor][chunk][thread]
  const int s_bytes = nt * NV * static_cast<int>(sizeof(Pack<T>)), d_bytes = nt * NV * static_cast<int>(sizeof(Pack<D>));
  const int stage_bytes = s_bytes * 2 + d_bytes;
  auto s_at = [&](int st, int i) { return reinterpret_cast<Pack<T>*>(ring_mem + st * stage_bytes) + i * nt + tid; };
  auto e_at = [&](int st, int i) { return reinterpret_cast<Pack<T>*>(ring_mem + st * stage_bytes + s_bytes) + i * nt + tid; };
  auto d_at = [&](int st, int i) {
    return reinterpret_cast<Pack<D>*>(ring_mem + st * stage_bytes + 2 * s_bytes) + i * nt + tid;
  };
  auto fetch = [&](int64_t row, int st) {
    if (row < A.rows) {
      if (lane == 0)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                         static_cast<uint32_t>(__cvta_generic_to_shared(&rstds[warp][st]))),
                     "l"(A.rstd + row)
                     : "memory");
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        copy_chunk(s_at(st, i), static_cast<const T*>(A.s) + row * A.lds, warp + i * nw, lane, A.dim);
        copy_chunk(d_at(st, i), static_cast<const D*>(A.dy) + row * A.lddy, warp + i * nw, lane, A.dim);
        if (A.dres) copy_chunk(e_at(st, i), static_cast<const T*>(A.dres) + row * A.lddres, warp + i * nw, lane, A.dim);
      }
    }
    copy_commit();
  };
  for (int st = 0; st < ring; ++st) fetch(blockIdx.x + static_cast<int64_t>(st) * gridDim.x, st);

  int turn = 0, st = 0;
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    load_any<true>(A.weight, A.weight_dtype, 0, warp + i * nw, lane, A.dim, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  const float inv_dim = 1.0f / static_cast<float>(A.dim);
  for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x) {
    copy_wait(ring - 1);
    __syncwarp();  // lane 0's copy of rstd
    const float r = rstds[warp][st];
    Pack<T> s[NV], e[NV];
    Pack<D> dy[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = *s_at(st, i);
      dy[i] = *d_at(st, i);
      if (A.dres) e[i] = *e_at(st, i);
    }
    __syncwarp();
    fetch(row + static_cast<int64_t>(ring) * gridDim.x, st);
    if (++st == ring) st = 0;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a[8], g[8];
      s[i].unpack(a);
      dy[i].unpack(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float p = g[j] * (a[j] * r);
        dw[i][j] += p;
        dot = fmaf(p, w[i][j], dot);
      }
    }
    const float mean = cta_sum(dot, slots, turn) * inv_dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a[8], g[8], d[8];
      s[i].unpack(a);
      dy[i].unpack(g);
      if (A.dres) {
        e[i].unpack(d);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = fmaf(r, g[j] * w[i][j] - a[j] * r * mean, d[j]);
      Pack<T> o;
      o.pack(d);
      store_chunk<true>(static_cast<T*>(A.ds) + row * A.ldds, warp + i * nw, lane, A.dim, o);
    }
  }
  copy_wait(0);
  if (A.part) {
    float* p = A.part + static_cast<int64_t>(blockIdx.x) * A.dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Pack<float> o;
      o.pack(dw[i]);
      if (A.dim % 4 == 0) {
        store_chunk<true>(p, warp + i * nw, lane, A.dim, o);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int col = col_of<true>(warp + i * nw, lane, j);
          if (col < A.dim) p[col] = dw[i][j];
        }
      }
    }
  }
}

// The same with the rows loaded straight into registers: for rows that are
// not 16-byte aligned, or too long for the ring.
template <class T, class D, int NV, bool VEC>
__global__ void __launch_bounds__(512) k_rms_norm_grad(const NormGradArgs A) {
  __shared__ float slots[64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  int turn = 0;
  float dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  const float inv_dim = 1.0f / static_cast<float>(A.dim);
  for (int64_t row = blockIdx.x; row < A.rows; row += gridDim.x) {
    const float r = A.rstd[row];
    Pack<T> s[NV];
    Pack<D> dy[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      load_chunk<VEC>(static_cast<const T*>(A.s) + row * A.lds, warp + i * nw, lane, A.dim, s[i]);
      load_chunk<VEC>(static_cast<const D*>(A.dy) + row * A.lddy, warp + i * nw, lane, A.dim, dy[i]);
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float w[8], a[8], g[8];
      load_any<VEC>(A.weight, A.weight_dtype, 0, warp + i * nw, lane, A.dim, w);
      s[i].unpack(a);
      dy[i].unpack(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float p = g[j] * (a[j] * r);
        dw[i][j] += p;
        dot = fmaf(p, w[j], dot);
      }
    }
    const float mean = cta_sum(dot, slots, turn) * inv_dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = warp + i * nw;
      float w[8], a[8], g[8], d[8];
      load_any<VEC>(A.weight, A.weight_dtype, 0, c, lane, A.dim, w);
      s[i].unpack(a);
      dy[i].unpack(g);
      Pack<T> o;
      if (A.dres) {
        load_chunk<VEC>(static_cast<const T*>(A.dres) + row * A.lddres, c, lane, A.dim, o);
        o.unpack(d);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = fmaf(r, g[j] * w[j] - a[j] * r * mean, d[j]);
      o.pack(d);
      store_chunk<VEC>(static_cast<T*>(A.ds) + row * A.ldds, c, lane, A.dim, o);
    }
  }
  if (A.part) {
    // dim columns of partial sums per CTA, in this lane's column order
    float* p = A.part + static_cast<int64_t>(blockIdx.x) * A.dim;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = col_of<VEC>(warp + i * nw, lane, j);
        if (col < A.dim) p[col] = dw[i][j];
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
#pragma unroll 8
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

// Chunks per warp: as many as `most` (small CTAs, many rows in flight) when
// there are rows for every SM, else as few as leave at most 16 warps (the
// shortest time for one row).
Shape norm_shape(int64_t rows, int dim, int num_sms, int most) {
  const int chunks = static_cast<int>(lm_div_up(dim, kChunk));
  int nv = 1;
  if (rows >= 2 * num_sms)
    while (nv < most && nv < chunks) nv *= 2;
  while (lm_div_up(chunks, nv) > 16) nv *= 2;
  return {nv, static_cast<int>(lm_div_up(chunks, nv))};
}

Shape grad_shape(int64_t rows, int dim, int num_sms) { return norm_shape(rows, dim, num_sms, 2); }

// CTAs of the gradient: about 20 warps an SM
int grad_grid(int64_t rows, Shape sh, int num_sms) {
  const int per_sm = (20 + sh.warps / 2) / sh.warps;
  const int64_t most = int64_t(num_sms) * (per_sm < 1 ? 1 : per_sm > 10 ? 10 : per_sm);
  return static_cast<int>(rows < most ? rows : most);
}

template <class T, bool VEC>
void run_norm(const NormArgs& A, Shape sh, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(A.rows), threads = sh.warps * 32;
  switch (sh.nv) {
    case 1: k_rms_norm<T, 1, VEC><<<grid, threads, 0, st>>>(A); break;
    case 2: k_rms_norm<T, 2, VEC><<<grid, threads, 0, st>>>(A); break;
    case 4: k_rms_norm<T, 4, VEC><<<grid, threads, 0, st>>>(A); break;
    default: k_rms_norm<T, 8, VEC><<<grid, threads, 0, st>>>(A); break;
  }
}

template <class T, class D, int NV>
cudaError_t run_grad_nv(const NormGradArgs& A, Shape sh, int grid, int num_sms, bool vec, cudaStream_t st) {
  const int threads = sh.warps * 32;
  const int row_bytes = threads * NV * static_cast<int>(2 * sizeof(Pack<T>) + sizeof(Pack<D>));
  const int per_sm = static_cast<int>(lm_div_up(grid, num_sms));
  constexpr int kSmemPerSm = 216 * 1024;
  int ring = kSmemPerSm / (per_sm * (row_bytes + 2048));
  if (ring > kMaxAhead) ring = kMaxAhead;
  if (vec && ring >= 1) {
    static PerDevice pd;
    const cudaError_t e = once_per_device(pd, [](int) {
      return cudaFuncSetAttribute(k_rms_norm_grad_ring<T, D, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerSm);
    });
    if (e != cudaSuccess) return e;
    k_rms_norm_grad_ring<T, D, NV><<<grid, threads, ring * row_bytes, st>>>(A, ring);
  } else if (vec) {
    k_rms_norm_grad<T, D, NV, true><<<grid, threads, 0, st>>>(A);
  } else {
    k_rms_norm_grad<T, D, NV, false><<<grid, threads, 0, st>>>(A);
  }
  return cudaGetLastError();
}

template <class T, class D>
cudaError_t run_grad(const NormGradArgs& A, Shape sh, int grid, int num_sms, bool vec, cudaStream_t st) {
  switch (sh.nv) {
    case 1: return run_grad_nv<T, D, 1>(A, sh, grid, num_sms, vec, st);
    case 2: return run_grad_nv<T, D, 2>(A, sh, grid, num_sms, vec, st);
    case 4: return run_grad_nv<T, D, 4>(A, sh, grid, num_sms, vec, st);
    default: return run_grad_nv<T, D, 8>(A, sh, grid, num_sms, vec, st);
  }
}

int elem_bytes(int dt) { return dt == kDtF32 ? 4 : dt == kDtBf16 ? 2 : 1; }

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& A, int dtype, int num_sms, cudaStream_t st) {
  if (A.rows <= 0) return cudaSuccess;
  const int eb = elem_bytes(dtype);
  const Shape sh = norm_shape(A.rows, A.dim, num_sms, 4);
  const bool vec = lm_aligned(A.x, A.ldx, A.rows, eb, 16) &&
                   (!A.residual || (lm_aligned(A.residual, A.ldr, A.rows, eb, 16) &&
                                    lm_aligned(A.res_out, A.ldro, A.rows, eb, 16))) &&
                   lm_aligned(A.weight, 0, 1, 1, 16) &&
                   lm_aligned(A.out, A.ldo, A.rows, elem_bytes(A.out_dtype), A.out_dtype == kDtE4m3 ? 8 : 16);
  if (dtype == kDtBf16)
    vec ? run_norm<__nv_bfloat16, true>(A, sh, st) : run_norm<__nv_bfloat16, false>(A, sh, st);
  else
    vec ? run_norm<float, true>(A, sh, st) : run_norm<float, false>(A, sh, st);
  return cudaGetLastError();
}

size_t rms_norm_grad_workspace(int64_t rows, int64_t dim, int num_sms) {
  const Shape sh = grad_shape(rows, static_cast<int>(dim), num_sms);
  return static_cast<size_t>(grad_grid(rows, sh, num_sms)) * static_cast<size_t>(dim) * sizeof(float);
}

cudaError_t launch_rms_norm_grad(const NormGradArgs& A, int s_dtype, float* dweight, int num_sms, cudaStream_t st) {
  if (A.rows <= 0) return dweight ? cudaMemsetAsync(dweight, 0, sizeof(float) * A.dim, st) : cudaSuccess;
  const Shape sh = grad_shape(A.rows, A.dim, num_sms);
  const int grid = grad_grid(A.rows, sh, num_sms), eb = elem_bytes(s_dtype);
  const bool vec = lm_aligned(A.s, A.lds, A.rows, eb, 16) && lm_aligned(A.ds, A.ldds, A.rows, eb, 16) &&
                   (!A.dres || lm_aligned(A.dres, A.lddres, A.rows, eb, 16)) &&
                   lm_aligned(A.dy, A.lddy, A.rows, elem_bytes(A.dy_dtype), 16) &&
                   lm_aligned(A.weight, 0, 1, 1, 16);
  typedef __nv_bfloat16 B;
  const bool b = A.dy_dtype == kDtBf16;
  const cudaError_t e = s_dtype == kDtBf16
                            ? (b ? run_grad<B, B>(A, sh, grid, num_sms, vec, st) : run_grad<B, float>(A, sh, grid, num_sms, vec, st))
                            : (b ? run_grad<float, B>(A, sh, grid, num_sms, vec, st)
                                 : run_grad<float, float>(A, sh, grid, num_sms, vec, st));
  if (e != cudaSuccess || !dweight) return e;
  k_rms_norm_dweight<<<static_cast<int>(lm_div_up(A.dim, 32)), dim3(32, 32), 0, st>>>(A.part, grid, A.dim, dweight);
  return cudaGetLastError();
}

}  // namespace okls
