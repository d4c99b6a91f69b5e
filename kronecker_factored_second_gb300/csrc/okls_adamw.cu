// AdamW step over many tensors in one launch, with moments in 32 bits or in
// 8 (sm_103a).
//
//   m <- b1 m + (1 - b1) g,   v <- b2 v + (1 - b2) g^2
//   p <- p - lr wd p - (lr / (1 - b1^t)) m / (sqrt(v / (1 - b2^t)) + eps)
//
// The tensors' addresses and lengths are a table in the kernel's parameters
// (up to 28 KB of them): no copy of a table to the device, nothing to keep
// alive, and a captured launch carries its own.  A CTA takes one chunk of one
// tensor, which it finds by a binary search over the chunks' first numbers.
//
// 8 bits: m, and r = sqrt(v), are e4m3 codes with an fp32 scale for each 128
// elements (a = max(amax, 2^-100), scale = a / 448, as in the 8-bit products).
// The root is kept because it has half the range of v: the smallest code is
// 2^-17.8 of the group's largest value, 2^-35.6 of the largest v.  The update
// uses the moments before their rounding.  Rounding to nearest would lose
// every change below half a code (with b2 = 0.999, v would move only where g^2
// is some hundred times v); so a value between two codes takes one of them by
// chance, such that its mean is kept.  A root that is not zero does not become
// zero: the next update is divided by it.  The chances are 16-bit numbers from
// Philox-2x32 (Salmon, Moraes, Dror, Shaw 2011) with five rounds, a function of
// the seed, the step, the tensor's number and the element, so a step is
// reproducible and does not depend on the launch's shape.
//
// Measured (L2 flushed): 131M fp32 elements with 32-bit moments in 529 us (6.9
// TB/s: memory), bf16 ones with 8-bit moments in 339 us (3.9 TB/s: some 75
// instructions an element take three of four issue slots, and most ready warps wait for
// their turn; with one tile instead of four for a CTA 380; 64 registers a thread, past
// which 64 to 80 bytes are spilled); 49 tensors of 2048 in 10.3 us (8.6 of them the
// call's work on the host).
#include <math_constants.h>

#include "okls_lm.cuh"

namespace okls {
namespace {

constexpr int kAdamThreads = 256;
constexpr int kTableFew = 56;  // 4 KB of parameters
constexpr float kCodeSmall = 0.015625f;    // 2^-6, the smallest normal e4m3 value
constexpr float kCodeTiny = 0.001953125f;  // 2^-9, the smallest e4m3 value

// The tensors of a launch, by value.
template <int N>
struct AdamwTable {
  AdamwEntry t[N];
  int32_t first[N];  // number of the tensor's first chunk
  int32_t num;
  AdamwScalars s;
  const AdamwScalars* s_dev;  // where the step number lives on the device
};

template <int N>
__device__ __forceinline__ int find_tensor(const AdamwTable<N>& T, int chunk) {
  int lo = 0, hi = T.num - 1;  // the last tensor whose first chunk is at most `chunk`
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (T.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ bool all_aligned(const AdamwEntry& e, uintptr_t to) {
  return ((reinterpret_cast<uintptr_t>(e.p) | reinterpret_cast<uintptr_t>(e.g) | reinterpret_cast<uintptr_t>(e.m) |
           reinterpret_cast<uintptr_t>(e.v)) & (to - 1)) == 0;
}

// One element with 32-bit moments.
__device__ __forceinline__ void adamw32(const AdamwScalars& s, float& p, float g, float& m, float& v) {
  m = fmaf(s.beta1, m, s.rest1 * g);
  v = fmaf(s.beta2, v, s.rest2 * g * g);
  const float den = fmaf(__fsqrt_rn(v), s.root, s.eps);
  p = fmaf(-s.rate, __fdiv_rn(m, den), fmaf(-s.decay, p, p));
}

// 32-bit moments: elementwise, 8 elements a thread and pass.
constexpr int kChunk32 = 8192;
template <class P, class G, int N>
__global__ void __launch_bounds__(kAdamThreads) k_adamw32(const __grid_constant__ AdamwTable<N> T) {
  const int chunk = blockIdx.x, which = find_tensor(T, chunk);
  const AdamwEntry& e = T.t[which];
  const int64_t begin = static_cast<int64_t>(chunk - T.first[which]) * kChunk32;
  const int64_t end = min(begin + kChunk32, e.count);
  const AdamwScalars s = T.s_dev ? *T.s_dev : T.s;
  P* p = static_cast<P*>(e.p);
  const G* g = static_cast<const G*>(e.g);
  float *m = static_cast<float*>(e.m), *v = static_cast<float*>(e.v);
  int64_t from = begin;
  if (all_aligned(e, 16)) {
    from = begin + ((end - begin) & ~int64_t(7));
#pragma unroll 2
    for (int64_t i = begin + threadIdx.x * 8; i < from; i += kAdamThreads * 8) {
      Pack<P> pp;
      Pack<G> pg;
      float a[8], b[8], c[8], d[8];
      pp.load(p + i);
      pg.load(g + i);
      load8(m + i, c);
      load8(v + i, d);
      pp.unpack(a);
      pg.unpack(b);
#pragma unroll
      for (int j = 0; j < 8; ++j) adamw32(s, a[j], b[j], c[j], d[j]);
      pp.pack(a);
      pp.store(p + i);
      store8(m + i, c);
      store8(v + i, d);
    }
  }
  for (int64_t i = from + threadIdx.x; i < end; i += kAdamThreads) {
    float a = to_f32(p[i]), c = m[i], d = v[i];
    adamw32(s, a, to_f32(g[i]), c, d);
    p[i] = from_f32<P>(a), m[i] = c, v[i] = d;
  }
}

// ------------------------------------------------------------------ 8 bits
// Two random words for a pair of elements.
__device__ __forceinline__ uint2 philox(uint32_t x, uint32_t y, uint32_t key) {
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const uint64_t w = static_cast<uint64_t>(x) * 0xD256D193u;
    x = static_cast<uint32_t>(w >> 32) ^ (key + i * 0x9E3779B9u) ^ y;
    y = static_cast<uint32_t>(w);
  }
  return make_uint2(x, y);
}

// A magnitude x of a group, rounded to a code's value: y = x 448 / a goes up
// with the probability that keeps the mean.  The 20 bits below a normal
// value's three fraction bits are cut off after a random number of 16 bits
// (and a half) was added to them; adding 2^-6 to a value below it puts the
// fixed steps of 2^-9 there at the same place.  y is taken in two words
// (448 / a = mul + rest), so that the border which the random number sets is met
// exactly.
__device__ __forceinline__ float round_exact(float x, float mul, float rest, uint32_t random, bool root) {
  const float p = x * mul, off = p < kCodeSmall ? kCodeSmall : 0.0f;
  const float t = p + off;
  const float low = fmaf(x, rest, fmaf(x, mul, -p)) + (p - (t - off));
  const float y = t + low, under = low - (y - t);  // y + under, with under at most half of y's last bit
  uint32_t b = __float_as_uint(y) + (random << 4) + 8u;
  if ((b & 0xFFFFFu) == 0 && under < 0.0f) --b;
  const float q = __uint_as_float(b & 0xFFF00000u) - off;
  return root && x > 0.0f ? fmaxf(q, kCodeTiny) : q;
}

// The same from one word with its sign, which is off by two of its last bits
// at most.  A sum that ends within 4 bits of a border (12 instead of 8 bits
// are added, so that those are the last 8), and a y below the normal values
// that is not 0, leave it to round_exact: `near` keeps the least distance, `small`
// the least y.  A y past 448 by its own error stays below the next code.
struct Doubt {
  uint32_t near = ~0u, small = ~0u;
  __device__ __forceinline__ bool any() const { return near < 8u || small < 2u * __float_as_uint(kCodeSmall) - 1u; }
};
// random20: the random number 4 bits up.
__device__ __forceinline__ float round_code(float y, uint32_t random20, Doubt& d) {
  const uint32_t u = __float_as_uint(y), b = u + random20 + 12u;
  d.near = min(d.near, b & 0xFFFFFu);
  d.small = min(d.small, u + u - 1u);
  return __uint_as_float(b & 0xFFF00000u);
}

// fp32's root of a normal v, to its last bit but for one in some thousands; 0 for 0: a Newton
// step on the hardware's estimate of the reciprocal root.
__device__ __forceinline__ float root_of(float v) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaxf(v, 1.1754944e-38f)));
  const float r = v * y;
  return fmaf(fmaf(-r, r, v), 0.5f * y, r);
}
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// The larger magnitude, or NaN.
__device__ __forceinline__ float max_mag(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

__device__ __forceinline__ void codes_to_f32(uint32_t w, float* v) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * h)), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
    v[2 * h] = f.x, v[2 * h + 1] = f.y;
  }
}

// What the multiplier 448 / a lost to its rounding.
__device__ __forceinline__ float mul_rest(uint32_t amax_bits, float mul) {
  const float a = fmaxf(__uint_as_float(amax_bits), kFp8AmaxFloor);
  return __fdiv_rn(fmaf(-a, mul, kFp8Max), a);
}

// Scale and multiplier of a group; a group that holds a NaN or an infinity
// stands for NaN.
__device__ __forceinline__ void state_scales(uint32_t amax_bits, float* mul, float* scale) {
  fp8_scales(amax_bits, mul, scale);
  if (amax_bits >= 0x7F800000u) *scale = CUDART_NAN_F;
}

// The moments of one element after the step, each product and sum rounded (what a code is must
// not hang on how a compiler joins them).
__device__ __forceinline__ float second8(const AdamwScalars& s, float r, float g) {
  return __fadd_rn(__fmul_rn(s.beta2, __fmul_rn(r, r)), __fmul_rn(__fmul_rn(s.rest2, g), g));
}
__device__ __forceinline__ float first8(const AdamwScalars& s, float m, float g) {
  return __fadd_rn(__fmul_rn(s.beta1, m), __fmul_rn(s.rest1, g));
}
__device__ __forceinline__ float update8(const AdamwScalars& s, float p, float m, float r) {
  return fmaf(-s.rate * m, reciprocal(fmaf(r, s.root, s.eps)), fmaf(-s.decay, p, p));
}

// Squares leave fp32's range long before the moments do (at beta2 = 0.999 those of gradients below
// 2^-58 or past 2^69).  A warp that meets one goes through its 32 x 16 elements here, one by one and
// twice instead of holding them, which the common way is spared.  Where v is no normal number, the
// root of beta2 r^2 + rest2 g^2 is formed of r and g that a power of two brings into fp32's middle.
constexpr float kNormal = 0x1p-126f;
constexpr float kFarRoot = 0x1p-62f;
constexpr uint32_t kWideRoots = 0x6C800000u;  // 2^90: kFarRoot times 448 / 2^90 is a number, past it it may be 0
__device__ __forceinline__ bool root_far(const AdamwScalars& s, float r, float g, float& root) {
  const float v = second8(s, r, g);
  root = root_of(v);
  if ((v >= kNormal && v < CUDART_INF_F) || (r == 0.0f && g == 0.0f)) return false;
  const bool large = v > 1.0f;
  const float up = large ? 0x1p-65f : 0x1p120f, down = large ? 0x1p65f : 0x1p-120f;
  r *= up, g *= up;
  root = __fsqrt_rn(s.beta2 * r * r + s.rest2 * g * g) * down;
  return true;
}
template <class P, class G>
__device__ __forceinline__ void adamw8_far(const AdamwEntry& e, const AdamwScalars& s, int64_t i, uint32_t low) {
  const int count = static_cast<int>(max(int64_t(0), min(e.count - i, int64_t(16))));
  const int64_t group = i / kFp8Group;
  const bool some = group * kFp8Group < e.count;
  P* p = static_cast<P*>(e.p) + i;
  const G* g = static_cast<const G*>(e.g) + i;
  __nv_fp8_e4m3 *mq = static_cast<__nv_fp8_e4m3*>(e.m) + i, *vq = static_cast<__nv_fp8_e4m3*>(e.v) + i;
  const float ms = some ? e.ms[group] : 0.0f, vs = some ? e.vs[group] : 0.0f;
  const auto moments = [&](int j, float& m, float& r) {
    const float gj = to_f32(g[j]);
    m = first8(s, __fmul_rn(static_cast<float>(mq[j]), ms), gj);
    return root_far(s, __fmul_rn(static_cast<float>(vq[j]), vs), gj, r);
  };
  float top_m = 0.0f, top_r = 0.0f;
#pragma unroll 1
  for (int j = 0; j < count; ++j) {
    float m, r;
    const bool far = moments(j, m, r);
    const float pj = to_f32(p[j]);
    float a = update8(s, pj, m, r);
    if (far) {  // (a quarter of both sides where the sum could pass fp32's end)
      const float part = r > 1.0f ? 0.25f : 1.0f;
      a = fmaf(-s.rate, __fdiv_rn(part * m, fmaf(part * r, s.root, part * s.eps)), fmaf(-s.decay, pj, pj));
    }
    p[j] = from_f32<P>(a);
    top_m = max_mag(top_m, m), top_r = max_mag(top_r, r);
  }
  uint32_t am = __float_as_uint(top_m), av = __float_as_uint(top_r);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
    av = max(av, __shfl_xor_sync(0xffffffffu, av, o));
  }
  float mmul, mscale, vmul, vscale;
  state_scales(am, &mmul, &mscale);
  state_scales(av, &vmul, &vscale);
  const float mrest = mul_rest(am, mmul), vrest = mul_rest(av, vmul);
#pragma unroll 1
  for (int j = 0; j < count; ++j) {
    float m, r;
    moments(j, m, r);
    const uint2 w = philox(static_cast<uint32_t>((i + j) >> 1), low, s.key);
    const uint32_t random = (j & 1) ? w.y : w.x;
    mq[j].__x = static_cast<uint8_t>(e4m3x2(copysignf(round_exact(fabsf(m), mmul, mrest, random & 0xFFFFu, false), m), 0.0f));
    vq[j].__x = static_cast<uint8_t>(e4m3x2(round_exact(r, vmul, vrest, random >> 16, true), 0.0f));
  }
  if (some && (threadIdx.x & 7) == 0) e.ms[group] = mscale, e.vs[group] = vscale;
}

// Whether 16 elements from a 16-byte boundary are all 0.
template <class G>
__device__ __forceinline__ bool no_values(const G* g) {
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(G)); ++i) {
    const uint4 u = reinterpret_cast<const uint4*>(g)[i];
    any |= u.x | u.y | u.z | u.w;
  }
  return (any & (sizeof(G) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu)) == 0;
}
__device__ __forceinline__ bool no_codes(const uint8_t* q) {
  const uint4 u = *reinterpret_cast<const uint4*>(q);
  return ((u.x | u.y | u.z | u.w) & 0x7F7F7F7Fu) == 0;
}

// 8 lanes take a group, 16 consecutive elements each, which are held in
// registers between the update and the rounding.
constexpr int kOwn8 = 16;
constexpr int kTile8 = kAdamThreads * kOwn8;
constexpr int kChunk8 = 4 * kTile8;
template <class P, class G, int N>
__global__ void __launch_bounds__(kAdamThreads, 4) k_adamw8(const __grid_constant__ AdamwTable<N> T) {
  const int chunk = blockIdx.x, which = find_tensor(T, chunk);
  const AdamwEntry& e = T.t[which];
  const AdamwScalars s = T.s_dev ? *T.s_dev : T.s;
  const bool aligned = all_aligned(e, 16);
  const uint32_t low = s.low + static_cast<uint32_t>(e.id);
  const int64_t begin = static_cast<int64_t>(chunk - T.first[which]) * kChunk8, end = min(begin + kChunk8, e.count);
#pragma unroll 1
  for (int64_t tile = begin; tile < end; tile += kTile8) {
    const int64_t i = tile + threadIdx.x * kOwn8;
    const int64_t left = e.count - i;  // a group's first lane has an element where the group has one
    const bool vec = left >= kOwn8 && aligned;
    const int64_t group = i / kFp8Group;
    const bool some = group * kFp8Group < e.count;
    P* p = static_cast<P*>(e.p) + i;
    const G* g = static_cast<const G*>(e.g) + i;
    uint8_t *mq = static_cast<uint8_t*>(e.m) + i, *vq = static_cast<uint8_t*>(e.v) + i;

    float a[kOwn8], m[kOwn8], r[kOwn8];
    float top_r = 0.0f;  // (elements past the end are zeros: they change no maximum)
    bool far;
    {
      float b[kOwn8];
      uint4 cm = make_uint4(0, 0, 0, 0), cv = cm;
      if (vec) {
        float lo[8], hi[8];
        Pack<P> p0, p1;
        Pack<G> g0, g1;
        cm = *reinterpret_cast<const uint4*>(mq), cv = *reinterpret_cast<const uint4*>(vq);
        p0.load(p), p1.load(p + 8), g0.load(g), g1.load(g + 8);
        p0.unpack(lo), p1.unpack(hi);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = lo[j], a[8 + j] = hi[j];
        g0.unpack(lo), g1.unpack(hi);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = lo[j], b[8 + j] = hi[j];
      } else {
        uint32_t wm[4] = {}, wv[4] = {};
#pragma unroll
        for (int j = 0; j < kOwn8; ++j) {
          const bool in = j < left;
          a[j] = in ? to_f32(p[j]) : 0.0f;
          b[j] = in ? to_f32(g[j]) : 0.0f;
          if (in) {
            wm[j / 4] |= static_cast<uint32_t>(mq[j]) << (8 * (j % 4));
            wv[j / 4] |= static_cast<uint32_t>(vq[j]) << (8 * (j % 4));
          }
        }
        cm = make_uint4(wm[0], wm[1], wm[2], wm[3]), cv = make_uint4(wv[0], wv[1], wv[2], wv[3]);
      }
      const float ms = some ? e.ms[group] : 0.0f, vs = some ? e.vs[group] : 0.0f;
      const uint32_t wm[4] = {cm.x, cm.y, cm.z, cm.w}, wv[4] = {cv.x, cv.y, cv.z, cv.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) codes_to_f32(wm[j], m + 4 * j), codes_to_f32(wv[j], r + 4 * j);
      uint32_t least = ~0u;  // bits of the smallest root
#pragma unroll
      for (int j = 0; j < kOwn8; ++j) {
        m[j] = first8(s, __fmul_rn(m[j], ms), b[j]);
        r[j] = root_of(second8(s, __fmul_rn(r[j], vs), b[j]));
        a[j] = update8(s, a[j], m[j], r[j]);
        least = min(least, __float_as_uint(r[j]));
        top_r = max_mag(top_r, r[j]);
      }
      // an infinite v (its root came out as NaN), or a small one that is not the 0 of an element without gradient and
      // code (usual are lanes of nothing but those: rows of a table whose tokens did not occur)
      far = !(top_r < CUDART_INF_F);
      if (least < __float_as_uint(kFarRoot) && !(vec && no_values(g) && no_codes(vq))) {
#pragma unroll
        for (int j = 0; j < kOwn8; ++j)
          if (j < left && r[j] < kFarRoot) far = far || to_f32(g[j]) != 0.0f || (vq[j] & 0x7F) != 0;
      }
    }
    if (__any_sync(0xffffffffu, far)) {
      adamw8_far<P, G>(e, s, i, low);
      continue;
    }
    if (vec) {
      Pack<P> p0, p1;
      float lo[8], hi[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) lo[j] = a[j], hi[j] = a[8 + j];
      p0.pack(lo), p1.pack(hi);
      p0.store(p), p1.store(p + 8);
    } else {
#pragma unroll
      for (int j = 0; j < kOwn8; ++j)
        if (j < left) p[j] = from_f32<P>(a[j]);
    }

    float top_m = 0.0f;
#pragma unroll
    for (int j = 0; j < kOwn8; ++j) top_m = max_mag(top_m, m[j]);
    uint32_t am = __float_as_uint(top_m), av = __float_as_uint(top_r);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
      av = max(av, __shfl_xor_sync(0xffffffffu, av, o));
    }
    float mmul, mscale, vmul, vscale;
    state_scales(am, &mmul, &mscale);
    state_scales(av, &vmul, &vscale);
    uint32_t wm[4], wv[4];
    Doubt doubt;
#pragma unroll
    for (int j = 0; j < kOwn8; j += 4) {
      float qm[4], qv[4];
#pragma unroll
      for (int h = 0; h < 4; h += 2) {
        const uint2 w = philox(static_cast<uint32_t>((i + j + h) >> 1), low, s.key);
        qm[h] = round_code(m[j + h] * mmul, (w.x << 4) & 0xFFFF0u, doubt);
        qm[h + 1] = round_code(m[j + h + 1] * mmul, (w.y << 4) & 0xFFFF0u, doubt);
        qv[h] = round_code(r[j + h] * vmul, (w.x >> 12) & 0xFFFF0u, doubt);
        qv[h + 1] = round_code(r[j + h + 1] * vmul, (w.y >> 12) & 0xFFFF0u, doubt);
      }
      wm[j / 4] = e4m3x2(qm[0], qm[1]) | (e4m3x2(qm[2], qm[3]) << 16);
      wv[j / 4] = e4m3x2(qv[0], qv[1]) | (e4m3x2(qv[2], qv[3]) << 16);
    }
    // (a root whose share of the group's largest is below fp32's range is no zero, either)
    if (doubt.any() || av >= kWideRoots) {
      const float mrest = mul_rest(am, mmul), vrest = mul_rest(av, vmul);
#pragma unroll
      for (int j = 0; j < kOwn8; ++j) {
        const uint2 w = philox(static_cast<uint32_t>((i + j) >> 1), low, s.key);
        const uint32_t random = (j & 1) ? w.y : w.x;
        const uint32_t cm = e4m3x2(copysignf(round_exact(fabsf(m[j]), mmul, mrest, random & 0xFFFFu, false), m[j]), 0.0f) & 0xFFu;
        const uint32_t cv = e4m3x2(round_exact(r[j], vmul, vrest, random >> 16, true), 0.0f) & 0xFFu;
        const int at = 8 * (j % 4);
        wm[j / 4] = (wm[j / 4] & ~(0xFFu << at)) | (cm << at);
        wv[j / 4] = (wv[j / 4] & ~(0xFFu << at)) | (cv << at);
      }
    }
    if (vec) {
      *reinterpret_cast<uint4*>(mq) = make_uint4(wm[0], wm[1], wm[2], wm[3]);
      *reinterpret_cast<uint4*>(vq) = make_uint4(wv[0], wv[1], wv[2], wv[3]);
    } else {
#pragma unroll
      for (int j = 0; j < kOwn8; ++j) {
        if (j < left) {
          mq[j] = static_cast<uint8_t>(wm[j / 4] >> (8 * (j % 4)));
          vq[j] = static_cast<uint8_t>(wv[j / 4] >> (8 * (j % 4)));
        }
      }
    }
    if (some && (threadIdx.x & 7) == 0) e.ms[group] = mscale, e.vs[group] = vscale;
  }
}

// ------------------------------------------------------ step on the device
__global__ void k_adamw_clock(AdamwHyper h, const float* lr_dev, int64_t* step_dev, AdamwScalars* out) {
  const int64_t t = *step_dev + 1;
  *step_dev = t;
  if (lr_dev) h.lr = *lr_dev;
  *out = adamw_scalars(h, t);
}

template <class P, class G, int N>
cudaError_t launch_table(const AdamwEntry* e, int num, bool bits8, const AdamwScalars& s, const AdamwScalars* s_dev,
                         cudaStream_t st) {
  AdamwTable<N> T;
  T.s = s, T.s_dev = s_dev;
  const int64_t chunk = bits8 ? kChunk8 : kChunk32;
  for (int i = 0; i < num;) {
    // as many tensors as the table and the grid hold
    int64_t grid = 0;
    int k = 0;
    for (; i < num && k < N; ++i) {
      const int64_t c = lm_div_up(e[i].count, chunk);
      if (c == 0) continue;
      if (grid + c > 0x7FFFFFFF) break;
      T.t[k] = e[i], T.first[k] = static_cast<int32_t>(grid);
      grid += c, ++k;
    }
    T.num = k;
    if (k == 0) break;
    if (bits8)
      k_adamw8<P, G, N><<<static_cast<unsigned>(grid), kAdamThreads, 0, st>>>(T);
    else
      k_adamw32<P, G, N><<<static_cast<unsigned>(grid), kAdamThreads, 0, st>>>(T);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

template <class P, class G>
cudaError_t launch_typed(const AdamwEntry* e, int num, bool bits8, const AdamwScalars& s, const AdamwScalars* s_dev,
                         cudaStream_t st) {
  if (num <= kTableFew) return launch_table<P, G, kTableFew>(e, num, bits8, s, s_dev, st);
  return launch_table<P, G, kAdamwTable>(e, num, bits8, s, s_dev, st);
}

}  // namespace

cudaError_t launch_adamw(const AdamwEntry* e, int num, int param_dtype, int grad_dtype, bool bits8,
                         const AdamwScalars& s, const AdamwScalars* s_dev, cudaStream_t st) {
  typedef __nv_bfloat16 B;
  if (param_dtype == kDtF32)
    return grad_dtype == kDtF32 ? launch_typed<float, float>(e, num, bits8, s, s_dev, st)
                                : launch_typed<float, B>(e, num, bits8, s, s_dev, st);
  return grad_dtype == kDtF32 ? launch_typed<B, float>(e, num, bits8, s, s_dev, st)
                              : launch_typed<B, B>(e, num, bits8, s, s_dev, st);
}

cudaError_t launch_adamw_clock(const AdamwHyper& h, const float* lr_dev, int64_t* step_dev, AdamwScalars* out,
                               cudaStream_t st) {
  k_adamw_clock<<<1, 1, 0, st>>>(h, lr_dev, step_dev, out);
  return cudaGetLastError();
}

}  // namespace okls
