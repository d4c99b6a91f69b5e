// Sampling of a token from each row of logits with temperature, top-k, top-p
// and min-p, from given random numbers (sm_103a).
//
// With m = max z, the weights are w_j = e^((z_j - m) / T).  The tokens in
// falling order of (z, -id) are cut three times: to the first k; of those, to
// the shortest prefix whose mass is at least p of their mass; of those, to the
// ones with w_j >= min_p.  Each cut is a prefix of the same order, so the kept
// set is known by its last token: a least value and, among its equals, a last
// id (Cut).  The drawn token is the first, in the order of ids, at which the
// running sum of the kept weights is above u times their sum.
//
// Sums are whole numbers.  A weight is rounded to a multiple of 2^-(62 -
// log2 vocab), so a row's sum fits 63 bits and does not depend on the order in
// which threads add; a running sum past u W is found by exact comparisons.  What
// decides which token is drawn is then the weights' error alone: a hundred
// thousand tokens have as many borders, and with weights to fp32's 2^-24 one row
// in a thousand drew a neighbour.  So a weight is formed to about 2^-34:
//   z log2(e) 2048 / T = k + r, with k whole and r in two roundings (the factor in
//   two words, one fused product each);  k_m - k and r_m - r of the maximum are
//   the exponent in 2048ths;  2^-(j / 2048) comes from a table of 62 bits,
//   2^-((r_m - r) / 2048) = 1 - q with q of some 2^-11 from a polynomial, and one
//   32 x 32 + 64 bit product joins them.
//
// A row belongs to a cluster of 1 to 8 CTAs (few rows need many SMs), and a
// CTA to one row after the other.  The first pass over a row takes its maximum; what
// follows reads it again from L2.  A cut by count or mass is found from 2048
// bins of the order-preserving image of the values left in question; when the bin that holds the
// border has at most 512 values they are sorted, otherwise that bin is cut into 2048
// again (three times at most for 32 bits).
#include <cooperative_groups.h>
#include <math_constants.h>

#include "okls_internal.h"
#include "okls_lm.cuh"

namespace cg = cooperative_groups;

namespace okls {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kBinsThread = kBins / kThreads;
constexpr int kList = kThreads;  // values of a border bin that are sorted
constexpr int kSegs = 1024;      // segments of a CTA's part of a row
constexpr int kSteps = 2048;     // table entries in an octave
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: added to |x| <= 2^22, leaves x rounded in the low bits
constexpr double kLn2 = 0.6931471805599453094;

// ------------------------------------------------------------------ weights
// 2^62 * 2^(-j / 2048).
struct PowerTable {
  u64 v[kSteps];
};
constexpr u64 mul_high(u64 a, u64 b) {
  const u64 al = a & 0xFFFFFFFFull, ah = a >> 32, bl = b & 0xFFFFFFFFull, bh = b >> 32;
  const u64 mid = ah * bl + ((al * bl) >> 32), mid2 = al * bh + (mid & 0xFFFFFFFFull);
  return ah * bh + (mid >> 32) + (mid2 >> 32);
}
constexpr PowerTable make_powers() {
  PowerTable t{};
  u64 x = 1ull << 63;  // 2^63 * 2^(-j / 2048), each step cut off below 2^-63
  for (int j = 0; j < kSteps; ++j) {
    t.v[j] = (x + 1) >> 1;
    x = mul_high(x, 0xFFE9D2B2F7DB2755ull);  // 2^64 * 2^(-1 / 2048)
  }
  return t;
}
__device__ const PowerTable g_powers = make_powers();

// A row's temperature and maximum.
struct Heat {
  float base;    // taken from a value first: 0, or the maximum where that has many steps (then exact)
  float least;   // values below this have weight 0
  float ch, cl;  // 2048 log2(e) / T in two words
  int kb;        // bits of the maximum's k + kMagic
  float r;       // the maximum's r
  int shift;     // 62 bits to the row's unit, at least 1
};

__device__ __forceinline__ void steps_of(const Heat& h, float z, int& kb, float& r) {
  const float d = fmaxf(z - h.base, h.least);
  const float k = fmaf(d, h.ch, kMagic);
  r = fmaf(d, h.cl, fmaf(d, h.ch, -(k - kMagic)));
  kb = __float_as_int(k);
}

__device__ Heat make_heat(float m, float temperature, int shift) {
  Heat h;
  const double c = 2048.0 / kLn2 / static_cast<double>(temperature);
  h.ch = static_cast<float>(c), h.cl = static_cast<float>(c - static_cast<double>(h.ch));
  const bool far = fabs(static_cast<double>(m) * c) > 1900.0 * 2048.0;
  h.base = far ? m : 0.0f;
  // 70 octaves below the maximum there is nothing left of 62 bits
  h.least = static_cast<float>(fmax(static_cast<double>(far ? 0.0f : m) - 70.0 * 2048.0 / c, -3.4e38));
  h.shift = shift;
  steps_of(h, m, h.kb, h.r);
  return h;
}

__device__ __forceinline__ u64 weight(const Heat& h, const u64* powers, float z) {
  constexpr float a = 3.3845077175778578e-4f;  // ln 2 / 2048
  constexpr float s = 4294967296.0f;
  int kb;
  float r;
  steps_of(h, z, kb, r);
  const int k = h.kb - kb;
  const float d = h.r - r;
  // q 2^32 = (1 - 2^(-d / 2048)) 2^32, rounded
  const float q = fmaf(d, fmaf(d, fmaf(d, s * (a * a * a / 6.0f), -s * (a * a / 2.0f)), s * a), kMagic);
  const u64 p = powers[k & (kSteps - 1)];
  u64 w = p - static_cast<u64>(static_cast<long long>(static_cast<int>(p >> 32)) *
                               (__float_as_int(q) - __float_as_int(kMagic)));
  // (rounded: a hundred thousand weights cut off are half as many units)
  asm("shr.u64 %0, %1, %2;" : "=l"(w) : "l"(w), "r"((k >> 11) + h.shift - 1));
  return (w + 1) >> 1;
}

// floor(f * w) or ceil for a fraction f in [0, 1).
__device__ u64 fraction_of(float f, u64 w, bool up) {
  int e;
  const u64 mant = static_cast<u64>(ldexpf(frexpf(f, &e), 24));  // f = mant * 2^(e - 24)
  const int s = 24 - e;
  const u64 lo = w * mant, hi = __umul64hi(w, mant);
  if (mant == 0) return 0;
  if (s >= 128) return up ? 1 : 0;
  u64 v, rest;
  if (s >= 64) {
    v = s == 64 ? hi : hi >> (s - 64);
    rest = lo | (s == 64 ? 0 : hi << (128 - s));
  } else {
    v = (hi << (64 - s)) | (lo >> s);
    rest = lo << (64 - s);
  }
  return v + (up && rest != 0);
}

// ------------------------------------------------------------------ order
// fp32 order as unsigned order, -0 as 0 (no NaN).
__device__ __forceinline__ uint32_t ord_bits(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float ord_value(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u ^ 0x80000000u) : ~u);
}

// The last token that is kept: values above, and equal ones up to an id.
struct Cut {
  float value;
  int id;
};
constexpr int kAllIds = 0x7FFFFFFF;
__device__ __forceinline__ bool kept(const Cut& c, float z, int id) { return z > c.value || (z == c.value && id <= c.id); }
__device__ __forceinline__ Cut tighter(const Cut& a, const Cut& b) {
  if (a.value != b.value) return a.value > b.value ? a : b;
  return a.id < b.id ? a : b;
}

// ------------------------------------------------------------------ CTA
struct Shared {
  u64 powers[kSteps];
  union {
    struct {
      uint32_t count[kBins], low[kBins], high[kBins];
    } bin;
    struct {
      u64 mine[kList], all[kList];
    } list;
  };
  u64 seg[kSegs];
  u64 warp_sum[kWarps + 1];
  u64 total;
  float warp_max[kWarps], max;
  int listed, found;
  // the border bin
  u64 border_above;
  int border, border_count;
  Cut cut;
};

struct Group {  // a cluster, or a CTA alone
  cg::cluster_group c;
  int rank, size;
  __device__ void sync() const {
    if (size > 1)
      c.sync();
    else
      __syncthreads();
  }
  template <class T>
  __device__ T* of(T* p, int r) const {
    return size > 1 ? c.map_shared_rank(p, r) : p;
  }
};

// A CTA's part of a row.  Positions count from the 16-byte boundary at or
// before the row's first element.
template <class T>
struct Part {
  const T* base;
  int begin, end;  // positions of the row
  int from, segs;  // of this CTA: first position, segments
  int shift;       // position of id 0
  bool infinite;   // the maximum is +inf: only infinities count, equally
};

// 8 values from a position that is a multiple of 8; -inf outside the row.
template <class T>
__device__ __forceinline__ void load_block(const Part<T>& R, int q, float (&v)[8]) {
  if (q >= R.begin && q + 8 <= R.end) {
    Pack<T> p;
    p.load(R.base + q);
    p.unpack(v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = q + j >= R.begin && q + j < R.end ? to_f32(R.base[q + j]) : -CUDART_INF_F;
  }
}
template <class T>
__device__ __forceinline__ void load_finite(const Part<T>& R, int q, float (&v)[8]) {
  load_block(R, q, v);
  if (R.infinite) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] == CUDART_INF_F ? 0.0f : -CUDART_INF_F;
  }
}

__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}
__device__ __forceinline__ u64 warp_total(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Inclusive scan over the CTA's threads; the sum of all in S.warp_sum[kWarps].
__device__ u64 cta_scan(Shared& S, u64 v) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const u64 own = warp_scan(v, lane);
  __syncthreads();
  if (lane == 31) S.warp_sum[warp] = own;
  __syncthreads();
  u64 before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? S.warp_sum[w] : 0;
    all += S.warp_sum[w];
  }
  __syncthreads();
  if (threadIdx.x == 0) S.warp_sum[kWarps] = all;
  __syncthreads();
  return own + before;
}

// Sum of fn(value, id) over the row; segments' sums stay in S.seg and the CTA's in S.total.
template <int NV, class T, class Fn>
__device__ u64 sum_row(Shared& S, const Group& G, const Part<T>& R, Fn fn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 mine = 0;
  for (int s = warp; s < R.segs; s += kWarps) {
    u64 sum = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int q = R.from + (s * NV + v) * 256 + lane * 8;
      float z[8];
      load_finite(R, q, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += fn(z[j], q + j - R.shift);
    }
    sum = warp_total(sum);
    if (lane == 0) S.seg[s] = sum;
    mine += sum;
  }
  cta_scan(S, lane == 0 ? mine : 0);
  if (threadIdx.x == 0) S.total = S.warp_sum[kWarps];
  G.sync();
  u64 all = 0;
  for (int r = 0; r < G.size; ++r) all += *G.of(&S.total, r);
  return all;
}

// The first id at which the running sum of the last sum_row is above
// `target`; -1 in the CTAs that do not hold it (the same in all threads).
template <int NV, class T, class Fn>
__device__ int locate(Shared& S, const Group& G, const Part<T>& R, u64 target, Fn fn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 before = 0;
  for (int r = 0; r < G.rank; ++r) before += *G.of(&S.total, r);
  if (threadIdx.x == 0) S.found = -1;
  __syncthreads();
  if (warp == 0 && target >= before && target - before < S.total) {
    u64 left = target - before;
    // 32 segments a lane, then one lane's segments, then the segment's values
    u64 sum = 0;
    for (int i = 0; i < 32; ++i) {
      const int s = lane * 32 + i;
      sum += s < R.segs ? S.seg[s] : 0;
    }
    u64 run = warp_scan(sum, lane);
    int at = __ffs(__ballot_sync(0xffffffffu, run > left)) - 1;
    left -= __shfl_sync(0xffffffffu, run - sum, at);
    const int s0 = at * 32;
    sum = s0 + lane < R.segs ? S.seg[s0 + lane] : 0;
    run = warp_scan(sum, lane);
    at = __ffs(__ballot_sync(0xffffffffu, run > left)) - 1;
    left -= __shfl_sync(0xffffffffu, run - sum, at);
    const int s = s0 + at;
    for (int v = 0; v < NV; ++v) {
      const int q = R.from + (s * NV + v) * 256 + lane * 8;
      float z[8];
      u64 w[8];
      load_finite(R, q, z);
      sum = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += w[j] = fn(z[j], q + j - R.shift);
      run = warp_scan(sum, lane);
      const unsigned past = __ballot_sync(0xffffffffu, run > left);
      if (past == 0) {
        left -= __shfl_sync(0xffffffffu, run, 31);
        continue;
      }
      if (lane == __ffs(past) - 1) {
        left -= run - sum;
        int id = -1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (id < 0) {
            if (w[j] > left)
              id = q + j - R.shift;
            else
              left -= w[j];
          }
        }
        S.found = id;
      }
      break;
    }
  }
  __syncthreads();
  return S.found;
}

// The first token, in falling order of (value, -id) among those that `in`
// keeps, at which the running sum reaches `target` >= 1: of ones, or of weights
// (MASS).  False if the sum stays below.  `top` is the row's maximum.
template <bool MASS, int NV, class T>
__device__ bool select(Shared& S, const Group& G, const Part<T>& R, const Heat& h, u64 target, const Cut& in, float top,
                       Cut* out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t high = ord_bits(top), low = ord_bits(in.value);
  u64 above = 0;
  for (;;) {
    const uint32_t range = high - low;
    const int bits = 32 - __clz(range), shift = bits > 11 ? bits - 11 : 0;
    for (int i = threadIdx.x; i < kBins; i += kThreads) S.bin.count[i] = S.bin.low[i] = S.bin.high[i] = 0;
    __syncthreads();
    for (int s = warp; s < R.segs; s += kWarps) {
#pragma unroll 1
      for (int v = 0; v < NV; ++v) {
        const int q = R.from + (s * NV + v) * 256 + lane * 8;
        float z[8];
        load_finite(R, q, z);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (!kept(in, z[j], q + j - R.shift)) continue;
          const uint32_t key = ord_bits(z[j]);
          if (key > high || key < low) continue;
          const uint32_t b = (high - key) >> shift;
          atomicAdd(&S.bin.count[b], 1u);
          if (MASS) {
            const u64 w = weight(h, S.powers, z[j]);
            const uint32_t wl = static_cast<uint32_t>(w);
            const uint32_t old = atomicAdd(&S.bin.low[b], wl);
            const uint32_t wh = static_cast<uint32_t>(w >> 32) + (old > ~wl);
            if (wh) atomicAdd(&S.bin.high[b], wh);
          }
        }
      }
    }
    G.sync();
    // every CTA adds up the bins of all
    u64 mass[kBinsThread] = {}, sum = 0;
    const int b0 = threadIdx.x * kBinsThread;
    for (int r = 0; r < G.size; ++r) {
#pragma unroll
      for (int i = 0; i < kBinsThread; ++i) {
        if (MASS)
          mass[i] += (static_cast<u64>(*G.of(&S.bin.high[b0 + i], r)) << 32) + *G.of(&S.bin.low[b0 + i], r);
        else
          mass[i] += *G.of(&S.bin.count[b0 + i], r);
      }
    }
#pragma unroll
    for (int i = 0; i < kBinsThread; ++i) sum += mass[i];
    const u64 run = cta_scan(S, sum);
    const u64 need = target - above;
    if (S.warp_sum[kWarps] < need) {
      G.sync();
      return false;
    }
    if (run >= need && run - sum < need) {
      u64 before = run - sum;
      int b = 0;
      while (before + mass[b] < need) before += mass[b++];
      S.border = b0 + b;
      S.border_above = above + before;
      int n = 0;
      for (int r = 0; r < G.size; ++r) n += static_cast<int>(*G.of(&S.bin.count[b0 + b], r));
      S.border_count = n;
    }
    __syncthreads();
    const int border = S.border, count = S.border_count;
    above = S.border_above;
    G.sync();  // the bins are free
    const uint32_t first = high - (static_cast<uint32_t>(border) << shift);
    const uint32_t span = (1u << shift) - 1u;
    const uint32_t last = first - low > span ? first - span : low;
    high = first, low = last;
    if (shift == 0) {
      // one value: how many of its equals, in the order of their ids
      const float value = ord_value(high);
      u64 n = target - above;
      if (MASS) {
        const u64 w = weight(h, S.powers, value);
        n = (n + w - 1) / w;
      }
      int id = kAllIds;
      if (n < static_cast<u64>(count)) {
        const auto one = [&](float z, int at) { return static_cast<u64>(z == value && kept(in, z, at)); };
        sum_row<NV>(S, G, R, one);
        const int at = locate<NV>(S, G, R, n - 1, one);
        if (at >= 0 && threadIdx.x == 0)
          for (int r = 0; r < G.size; ++r) G.of(&S.cut, r)->id = at;
        G.sync();
        id = S.cut.id;
        G.sync();
      } else if (value == in.value) {
        id = in.id;
      }
      *out = {value, id};
      return true;
    }
    if (count <= kList) break;
  }
  // sort what lies in the border bin
  if (threadIdx.x == 0) S.listed = 0;
  __syncthreads();
  for (int s = warp; s < R.segs; s += kWarps) {
#pragma unroll 1
    for (int v = 0; v < NV; ++v) {
      const int q = R.from + (s * NV + v) * 256 + lane * 8;
      float z[8];
      load_finite(R, q, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int id = q + j - R.shift;
        if (!kept(in, z[j], id)) continue;
        const uint32_t key = ord_bits(z[j]);
        if (key > high || key < low) continue;
        S.list.mine[atomicAdd(&S.listed, 1)] = (static_cast<u64>(key) << 32) | static_cast<uint32_t>(~id);
      }
    }
  }
  G.sync();
  int n = 0;
  for (int r = 0; r < G.size; ++r) {
    const int c = *G.of(&S.listed, r);
    const u64* src = G.of(S.list.mine, r);
    for (int i = threadIdx.x; i < c; i += kThreads) S.list.all[n + i] = src[i];
    n += c;
  }
  int padded = 2;
  while (padded < n) padded <<= 1;
  for (int i = n + threadIdx.x; i < padded; i += kThreads) S.list.all[i] = 0;
  __syncthreads();
  for (int size = 2; size <= padded; size <<= 1) {
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      const int i = threadIdx.x, k = i ^ stride;
      if (i < padded && k > i) {
        const u64 a = S.list.all[i], b = S.list.all[k];
        if ((a < b) == ((i & size) == 0)) S.list.all[i] = b, S.list.all[k] = a;
      }
      __syncthreads();
    }
  }
  const u64 entry = threadIdx.x < n ? S.list.all[threadIdx.x] : 0;
  const float value = ord_value(static_cast<uint32_t>(entry >> 32));
  u64 a = 0;
  if (threadIdx.x < n) a = MASS ? weight(h, S.powers, value) : 1;
  const u64 run = cta_scan(S, a), need = target - above;
  if (threadIdx.x < n && run >= need && run - a < need) S.cut = {value, static_cast<int>(~static_cast<uint32_t>(entry))};
  __syncthreads();
  *out = S.cut;
  G.sync();
  return true;
}

template <class T, int NV>
__global__ void __launch_bounds__(kThreads) k_sample(const SampleArgs A) {
  extern __shared__ unsigned char raw[];
  Shared& S = *reinterpret_cast<Shared*>(raw);
  Group G = {cg::this_cluster(), 0, 1};
  G.rank = static_cast<int>(G.c.block_rank()), G.size = static_cast<int>(G.c.num_blocks());
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kSteps; i += kThreads) S.powers[i] = g_powers.v[i];
  const int vocab = static_cast<int>(A.vocab);

  for (int64_t row = blockIdx.x / G.size; row < A.rows; row += gridDim.x / G.size) {
    Part<T> R;
    const T* z0 = static_cast<const T*>(A.logits) + row * A.ldl;
    R.shift = static_cast<int>((reinterpret_cast<uintptr_t>(z0) & 15) / sizeof(T));
    R.base = z0 - R.shift;
    R.begin = R.shift, R.end = R.shift + vocab;
    const int unit = NV * 256, per = ((R.end + unit - 1) / unit + G.size - 1) / G.size;
    R.from = G.rank * per * unit;
    R.segs = min(per, max(0, (R.end - R.from + unit - 1) / unit));
    R.infinite = false;

    float top = -CUDART_INF_F;
    for (int s = warp; s < R.segs; s += kWarps) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float z[8];
        load_block(R, R.from + (s * NV + v) * 256 + lane * 8, z);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, z[j]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    __syncthreads();
    if (lane == 0) S.warp_max[warp] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, S.warp_max[w]);
      S.max = top;
    }
    G.sync();
    top = -CUDART_INF_F;
    for (int r = 0; r < G.size; ++r) top = fmaxf(top, *G.of(&S.max, r));
    if (top == -CUDART_INF_F) {  // no token is possible
      if (G.rank == 0 && threadIdx.x == 0) A.ids[row] = -1, A.logp[row] = -CUDART_INF_F;
      G.sync();
      continue;
    }
    if (top == CUDART_INF_F) R.infinite = true, top = 0.0f;

    float temperature = A.temperature ? A.temperature[row] : A.temperature_all;
    int64_t k = A.top_k ? A.top_k[row] : A.top_k_all;
    const float p = A.top_p ? A.top_p[row] : A.top_p_all;
    float least = A.min_p ? A.min_p[row] : A.min_p_all;
    // (a NaN fails the comparison that would turn its filter on)
    if (!(temperature >= kSampleColdest)) temperature = 1.0f, k = 1;
    if (p <= 0.0f) k = 1;
    const bool by_count = k > 0 && k < vocab, by_mass = p < 1.0f && p > 0.0f && k != 1;
    const Heat h = make_heat(top, temperature, A.shift);

    const Cut all = {-3.402823466e38f, kAllIds};  // every possible token
    Cut floor_cut = all;
    if (least > 0.0f) {
      // the least value is rounded up to fp32, so that comparing values is exact
      const double t = static_cast<double>(top) + static_cast<double>(temperature) * log(static_cast<double>(fminf(least, 1.0f)));
      float f = static_cast<float>(fmax(t, -3.402823466e38));
      if (static_cast<double>(f) < t) f = nextafterf(f, CUDART_INF_F);
      floor_cut.value = f;
    }
    const auto possible = [&](const Cut& c) {
      return [&](float z, int id) { return kept(c, z, id) ? weight(h, S.powers, z) : 0ull; };
    };
    Cut cut = all;
    if (by_count) {
      // (the mass of the first k is asked for where a cut by mass follows)
      const Cut in = by_mass ? all : floor_cut;
      if (!select<false, NV>(S, G, R, h, static_cast<u64>(k), in, top, &cut)) cut = in;
    }
    if (by_mass) {
      const u64 total = sum_row<NV>(S, G, R, possible(cut));
      const u64 target = fraction_of(p, total, true);
      Cut in = tighter(cut, floor_cut), c;
      G.sync();
      // tokens lighter than an equal share of what may be missing hold less than that together
      const u64 share = (total - target) / static_cast<u64>(vocab);
      if (share > 1) {
        const double t = static_cast<double>(top) + static_cast<double>(temperature) *
                         (log(static_cast<double>(share)) - kLn2 * (62 - A.shift));
        const float f = static_cast<float>(fmax(t - 1e-6 * fabs(t) - 1e-6 * temperature, -3.402823466e38));
        if (f > in.value) in = {f, kAllIds};
      }
      cut = tighter(cut, floor_cut);
      if (select<true, NV>(S, G, R, h, target < 1 ? 1 : target, in, top, &c)) cut = tighter(cut, c);
    } else {
      cut = tighter(cut, floor_cut);
    }

    float u = A.u[row];
    u = u > 0.0f ? fminf(u, 0.99999994f) : 0.0f;
    const u64 mass = sum_row<NV>(S, G, R, possible(cut));
    const int id = locate<NV>(S, G, R, fraction_of(u, mass, false), possible(cut));
    if (id >= 0 && threadIdx.x == 0) {
      A.ids[row] = id;
      const float z = R.infinite ? 0.0f : to_f32(z0[id]);
      // (a greedy row has one token: log 1)
      A.logp[row] = static_cast<float>((static_cast<double>(z) - static_cast<double>(top)) / static_cast<double>(temperature) -
                                       log(ldexp(static_cast<double>(mass), A.shift - 62)));
    }
    G.sync();
  }
}

template <class T, int NV>
cudaError_t launch_nv(const SampleArgs& A, int clusters, int size, cudaStream_t st) {
  static PerDevice pd;
  const cudaError_t e = once_per_device(pd, [](int) {
    return cudaFuncSetAttribute(k_sample<T, NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters) * size);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(size);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_sample<T, NV>, A);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& args, int dtype, int num_sms, cudaStream_t st) {
  if (args.rows == 0) return cudaSuccess;
  SampleArgs A = args;
  A.shift = 1;
  while ((int64_t(1) << A.shift) < A.vocab) ++A.shift;
  // a cluster for each row while the SMs last and a CTA has 2048 values
  int size = 1;
  while (size < 8 && A.rows * size * 2 <= num_sms && A.vocab >= size * 4096) size *= 2;
  // (what a CTA's segments hold)
  while (lm_div_up(A.vocab + 8, size) > (kSegs - 8) * 1024) size *= 2;
  const int64_t resident = static_cast<int64_t>(num_sms) * 2 / size;
  const int clusters = static_cast<int>(A.rows < resident ? A.rows : resident);
  const bool wide = lm_div_up(A.vocab, size) > 16384;
  if (dtype == kDtF32) return wide ? launch_nv<float, 4>(A, clusters, size, st) : launch_nv<float, 1>(A, clusters, size, st);
  return wide ? launch_nv<__nv_bfloat16, 4>(A, clusters, size, st) : launch_nv<__nv_bfloat16, 1>(A, clusters, size, st);
}

}  // namespace okls
