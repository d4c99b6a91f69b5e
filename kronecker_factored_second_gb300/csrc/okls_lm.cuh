// Device helpers of the language-model operators: typed loads and stores of
// 8 consecutive elements, warp sums, e4m3 codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "okls_lm.h"

namespace okls {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// 8 consecutive elements from a 16-byte aligned address.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
// A bf16 value is the upper half of an fp32 value.
__device__ __forceinline__ void unpack8(const uint4& a, float (&v)[8]) {
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(p), v);
}
// 32 bytes to a 32-byte aligned address: a whole memory sector.  Two 16-byte
// stores with neighbouring lanes 32 bytes apart write half sectors, which
// halves the rate of a kernel that mostly writes (262 MB: 80 against 40 us).
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    const uint32_t w[8] = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]),
                           __float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
    store32(p, w);
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// 8 consecutive elements in their own type.
template <class T>
struct Pack;
template <>
struct Pack<float> {
  float v[8];
  __device__ __forceinline__ void unpack(float (&o)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = v[j];
  }
  __device__ __forceinline__ void pack(const float (&o)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = o[j];
  }
  __device__ __forceinline__ void load(const float* p) { load8(p, v); }
  __device__ __forceinline__ void store(float* p) const { store8(p, v); }
};
template <>
struct Pack<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void unpack(float (&o)[8]) const { unpack8(u, o); }
  __device__ __forceinline__ void pack(const float (&o)[8]) {
    u = make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Magnitude bits: ordered like the magnitudes, with infinities and NaNs
// above every finite value, so an integer maximum carries a NaN along.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Multiplier and scale of a group from its largest magnitude bits: fp32
// quotients rounded to nearest.
__device__ __forceinline__ void fp8_scales(uint32_t amax_bits, float* mul, float* scale) {
  const float a = amax_bits < __float_as_uint(kFp8AmaxFloor) ? kFp8AmaxFloor : __uint_as_float(amax_bits);
  *mul = __fdiv_rn(kFp8Max, a);
  *scale = __fdiv_rn(a, kFp8Max);
}

// e4m3 codes of two values (the first in the low byte), round to nearest
// even; NaN gives a NaN code.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float mul) {
  uint2 r;
  r.x = e4m3x2(v[0] * mul, v[1] * mul) | (e4m3x2(v[2] * mul, v[3] * mul) << 16);
  r.y = e4m3x2(v[4] * mul, v[5] * mul) | (e4m3x2(v[6] * mul, v[7] * mul) << 16);
  return r;
}

// Token id t of an int32 or int64 array.
__device__ __forceinline__ int64_t token_at(const void* ids, int ids_i64, int64_t t) {
  return ids_i64 ? static_cast<const int64_t*>(ids)[t] : static_cast<const int32_t*>(ids)[t];
}

inline bool lm_aligned(const void* p, int64_t ld, int64_t rows, int elem_bytes, int to) {
  return reinterpret_cast<uintptr_t>(p) % to == 0 && (rows <= 1 || (ld * elem_bytes) % to == 0);
}

}  // namespace okls
