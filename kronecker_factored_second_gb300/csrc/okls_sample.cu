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
// Sums are whole numbers.  A weight is rounded down to a multiple of 2^-(63 -
// log2 vocab) of the largest, so a row's sum fits 63 bits and does not depend on
// the order in which threads add; a running sum past u W is found by exact
// comparisons.  What decides which token is drawn is then the weights' error
// alone: a hundred thousand tokens have as many borders, and with weights to
// fp32's 2^-24 one row in a thousand drew a neighbour.  So a weight is formed to
// about 2^-33:
//   z log2(e) 2048 / T = k + r, with k whole and r in two roundings (the factor in
//   two words, one fused product each);  k_m - k and r_m - r of the maximum are
//   the exponent in 2048ths;  2^-(j / 2048) comes from a table of 62 bits,
//   2^-((r_m - r) / 2048) = 1 - q with q of some 2^-11 from a polynomial, and one
//   32 x 32 + 64 bit product joins them.
//
// A row belongs to a cluster of 1 to 8 CTAs (few rows need many SMs), and a CTA
// to one row after the other. The first pass over a row takes the maxima of its
// segments; what follows reads it again from L2.
//   The best token is looked up there. The first k of few come from a bound that
// few values reach, the k-th largest of the segments' maxima.
//   Other cuts put the tokens into 2048 bins first, 64 to an octave of the
// weight: their number, or their weights to 14 bits; so the bin with the border
// is known, or the few bins among which it is. A second pass lists what lies in
// them (or, for a count that fits, everything from them on); for a mass it also
// weighs every token exactly and sums what lies above those bins by segments,
// which is what the drawing needs.
//   Lists are sorted, and the border, the mass and the segments' sums found from
// them.
//   Where bins hold too many tokens (runs of equal logits), the order-preserving
// image of the values is binned instead, and the border's bin again (three times
// at most for 32 bits).
//
// Measured (L2 flushed): 512 rows of 128257 fp32 with top-p in 258 us (1.0 TB/s),
// 1024 rows of 131072 bf16 without a filter in 213 to 238 us (39 instructions a
// token): 2.2 and 2.3 of four instructions a clock, with 29 of 64 warps an SM, a third of whose
// waiting is for logits from memory or L2; one row of 32000 in 18 us without its call
// (16 warps that wait for barriers, for code that is not in the instruction cache and for memory);
// 256 rows of 32000 with settings of their own in 66 to 78 us, the chain of the slowest row.
// At 64 registers a thread some 300 bytes are spilled, in the rare paths and around them.
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
constexpr int kList = 1024;  // tokens that are sorted
constexpr int kEach = kList / kThreads;
constexpr int kFewSegs = 320;        // segments whose maxima are ranked by counting
constexpr int kSegs = 1024;      // segments of a CTA's part of a row
constexpr int kSteps = 2048;     // table entries in an octave
constexpr float kLowest = -3.402823466e38f;  // the least possible logit
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: added to |x| <= 2^22, leaves x rounded in the low bits

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
  float least;   // lower values count as this: their weight is 0
  float ch, cl;  // 2048 log2(e) / T in two words
  int kb;        // bits of the maximum's k + kMagic, 62 bits to the row's unit in the octaves
  float r;       // the maximum's r
  float top, c;  // the maximum, 64 log2(e) / T
  bool zeros;    // a weight is 0 at `least` (a temperature past 1e36 leaves even impossible values one)
  int shift;     // 62 bits to the row's unit, at least 1
};

__device__ __forceinline__ void steps_of(const Heat& h, float z, int& kb, float& r) {
  const float d = fmaxf(z - h.base, h.least);
  const float k = fmaf(d, h.ch, kMagic);
  r = fmaf(d, h.cl, fmaf(d, h.ch, -(k - kMagic)));
  kb = __float_as_int(k);
}

__device__ Heat make_heat(float m, float temperature, int shift) {
  // 2048 log2(e) in two words, divided to two words (fp64 is slow here: a row's
  // few quotients and logarithms in it took longer than reading 32000 logits)
  constexpr float c_high = 2954.639404296875f, c_low = 3.9443722e-5f;
  Heat h;
  h.ch = __fdiv_rn(c_high, temperature);
  const float rest = isinf(temperature) ? 0.0f : fmaf(-h.ch, temperature, c_high) + c_low;
  h.cl = __fdiv_rn(rest, temperature);
  const bool far = fabsf(m * h.ch) > 1900.0f * 2048.0f;
  h.base = far ? m : 0.0f;
  // (64 - shift octaves below the maximum nothing is left of a weight)
  h.least = fmaxf((far ? 0.0f : m) - (63.9f - static_cast<float>(shift)) * 2048.0f / h.ch, -3.4e38f);
  h.zeros = h.least > -3.3e38f;
  h.shift = shift;
  h.top = m, h.c = h.ch * (1.0f / 32.0f);
  steps_of(h, m, h.kb, h.r);
  h.kb += (shift - 1) * kSteps;
  return h;
}

// -q 2^32 = (2^(-d / 2048) - 1) 2^32 for d steps, + kMagic
constexpr float kA = 3.3845077175778578e-4f;  // ln 2 / 2048
constexpr float kQ1 = -4294967296.0f * kA, kQ2 = 4294967296.0f * (kA * kA / 2.0f), kQ3 = -4294967296.0f * (kA * kA * kA / 6.0f);

__device__ __forceinline__ u64 weight(const Heat& h, const u64* powers, float z) {
  int kb;
  float r;
  steps_of(h, z, kb, r);
  const int k = h.kb - kb;
  const float d = h.r - r;
  const float q = fmaf(d, fmaf(d, fmaf(d, kQ3, kQ2), kQ1), kMagic);
  const u64 p = powers[k & (kSteps - 1)];
  u64 w = p + static_cast<u64>(static_cast<long long>(static_cast<int>(p >> 32)) *
                               (__float_as_int(q) - __float_as_int(kMagic)));
  // w >> n for n <= 63 (least sees to it), in funnel shifts: others look at
  // whether they reach past 31 bits
  const uint32_t n = static_cast<uint32_t>(k >> 11), wl = static_cast<uint32_t>(w), wh = static_cast<uint32_t>(w >> 32);
  const uint32_t low = __funnelshift_r(__funnelshift_rc(wl, wh, n), 0, static_cast<uint32_t>(max(static_cast<int>(n) - 32, 0)));
  const uint32_t high = __funnelshift_rc(wh, 0, n);
  u64 r64;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r64) : "r"(low), "r"(high));
  return r64;
}

// The bin of a value among 2048, 64 to an octave below the maximum: it does not
// fall when the value does.
__device__ __forceinline__ int bin_of(const Heat& h, float z) {
  return __float_as_int(fminf((h.top - z) * h.c, 2047.0f) + 8388608.0f) & (kBins - 1);
}
// And the weight in units of 2^-14 of its bin's octave, 2^-(bin / 64).
__device__ __forceinline__ uint32_t bin_weight(const Heat& h, float z, int& bin) {
  const float t = fminf((h.top - z) * h.c, 2047.0f), b = t + 8388608.0f;
  bin = __float_as_int(b) & (kBins - 1);
  const float octave = __int_as_float(__float_as_int(b) & ~63) - 8388608.0f;
  float w;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(fmaf(octave - t, 1.0f / 64.0f, 14.0f)));
  return __float_as_int(w + 8388608.0f) & 0xFFFFu;
}

// floor(f * w), or ceil, for a normal fraction f in [0, 1).
__device__ u64 fraction_of(float f, u64 w, bool up) {
  const uint32_t bits = __float_as_uint(f), mant = (bits & 0x7FFFFFu) | 0x800000u;  // f = mant * 2^-s
  const int s = 150 - static_cast<int>(bits >> 23);
  if (s >= 128) return up && f > 0.0f && w > 0 ? 1 : 0;
  const u64 lo = w * mant, hi = __umul64hi(w, mant);
  u64 v, rest;
  if (s < 64) {
    v = (hi << (64 - s)) | (lo >> s), rest = lo << (64 - s);
  } else {
    v = hi >> (s - 64), rest = lo | (hi & ((1ull << (s - 64)) - 1));
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
  float seg_max[kSegs];
  u64 warp_sum[2][kWarps];
  u64 total, rest;  // of this CTA: what is kept, everything
  float max;
  float warp_max[kWarps];
  int listed, found;
  // the border bin
  u64 border_above;
  int border, border_count;
  float bound, high, low;
  Cut cut;
  double floor_below;  // temperature * ln(min_p)
};

struct Group {  // a cluster, or a CTA alone
  cg::cluster_group c;
  int rank, size;
  mutable int turn;  // of the two rows of S.warp_sum
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
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ u64 warp_total(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Scan over the CTA's threads.  (Two rows of warps' sums in turn: one barrier a scan.)
struct Scan {
  u64 run, all;  // up to and with the thread, of all
};
__device__ Scan cta_scan(Shared& S, const Group& G, u64 v) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64* sums = S.warp_sum[G.turn ^= 1];
  const u64 own = warp_scan(v, lane);
  if (lane == 31) sums[warp] = own;
  __syncthreads();
  u64 before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) before = all;
    all += sums[w];
  }
  return {own + before, all};
}
// The sum over warps of what each of them has.
__device__ u64 cta_total(Shared& S, const Group& G, u64 of_warp) {
  u64* sums = S.warp_sum[G.turn ^= 1];
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = of_warp;
  __syncthreads();
  u64 all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) all += sums[w];
  return all;
}

// Inclusive scan over the list's entries, kEach of a thread; returns their sum.
__device__ __forceinline__ u64 list_scan(Shared& S, const Group& G, const u64 (&w)[kEach], u64 (&run)[kEach]) {
  u64 sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) sum += w[i];
  const Scan scan = cta_scan(S, G, sum);
  u64 at = scan.run - sum;
#pragma unroll
  for (int i = 0; i < kEach; ++i) run[i] = at += w[i];
  return scan.all;
}

// sum += w where z >= least.
__device__ __forceinline__ void add_from(u64& sum, u64 w, float z, float least) {
  asm("{\n\t.reg .pred p;\n\tsetp.ge.f32 p, %2, %3;\n\t@p add.u64 %0, %0, %1;\n\t}" : "+l"(sum) : "l"(w), "f"(z), "f"(least));
}
// Sum of fn(value, id) over the row; the segments' sums stay in S.seg and the CTA's in S.total.
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
  const u64 total = cta_total(S, G, mine);
  if (threadIdx.x == 0) S.total = total;
  G.sync();
  u64 all = 0;
  for (int r = 0; r < G.size; ++r) all += *G.of(&S.total, r);
  return all;
}

// The same of the weights of all values from `least` on.
template <int NV, class T>
__device__ u64 sum_above(Shared& S, const Group& G, const Part<T>& R, const Heat& h, float least) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool all_count = least <= kLowest && h.zeros;  // impossible values have weight 0
  u64 mine = 0;
  for (int s = warp; s < R.segs; s += kWarps) {
    u64 sum = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float z[8];
      load_finite(R, R.from + (s * NV + v) * 256 + lane * 8, z);
      if (all_count) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += weight(h, S.powers, z[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) add_from(sum, weight(h, S.powers, z[j]), z[j], least);
      }
    }
    sum = warp_total(sum);
    if (lane == 0) S.seg[s] = sum;
    mine += sum;
  }
  const u64 total = cta_total(S, G, mine);
  if (threadIdx.x == 0) S.total = total;
  G.sync();
  u64 all = 0;
  for (int r = 0; r < G.size; ++r) all += *G.of(&S.total, r);
  return all;
}

// The first id at which the running sum of the last sums by segments is above
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

// ------------------------------------------------------------------- list
__device__ __forceinline__ void list_begin(Shared& S) {
  if (threadIdx.x == 0) S.listed = 0;
  __syncthreads();
}
__device__ __forceinline__ void list_put(Shared& S, float z, int id) {
  const int at = atomicAdd(&S.listed, 1);
  if (at < kList) S.list.mine[at] = (static_cast<u64>(ord_bits(z)) << 32) | static_cast<uint32_t>(~id);
}
__device__ __forceinline__ float list_value(const Shared& S, int i) { return ord_value(static_cast<uint32_t>(S.list.all[i] >> 32)); }
__device__ __forceinline__ int list_id(const Shared& S, int i) { return static_cast<int>(~static_cast<uint32_t>(S.list.all[i])); }

// Joins the CTAs' lists in S.list.all and sorts them in falling order of (value,
// -id): every CTA the same.  Returns the number of tokens, or -1 if they are too many.
__device__ int list_sorted(Shared& S, const Group& G) {
  G.sync();
  int n = 0;
  for (int r = 0; r < G.size; ++r) n += *G.of(&S.listed, r);
  if (n > kList) return -1;
  for (int r = 0, at = 0; r < G.size; ++r) {
    const int c = *G.of(&S.listed, r);
    const u64* src = G.of(S.list.mine, r);
    for (int i = threadIdx.x; i < c; i += kThreads) S.list.all[at + i] = src[i];
    at += c;
  }
  int padded = 2;
  while (padded < n) padded <<= 1;
  for (int i = n + threadIdx.x; i < padded; i += kThreads) S.list.all[i] = 0;
  __syncthreads();
  const bool small = padded <= 64;  // one warp's work
  if (!small || threadIdx.x < 32) {
    for (int size = 2; size <= padded; size <<= 1) {
      for (int stride = size >> 1; stride > 0; stride >>= 1) {
        for (int t = threadIdx.x; 2 * t < padded; t += kThreads) {
          const int i = 2 * t - (t & (stride - 1)), k = i + stride;
          const u64 a = S.list.all[i], b = S.list.all[k];
          if ((a < b) == ((i & size) == 0)) S.list.all[i] = b, S.list.all[k] = a;
        }
        if (small)
          __syncwarp();
        else
          __syncthreads();
      }
    }
  }
  __syncthreads();
  return n;
}

// The first token, in falling order of (value, -id) among those that `in`
// keeps, at which the running sum reaches `target` >= 1: of ones, or of weights
// (MASS).  False if the sum stays below.  `top` is the row's maximum.
template <bool MASS, int NV, class T>
__device__ __noinline__ bool select(Shared& S, const Group& G, const Part<T>& R, const Heat& h, u64 target, const Cut& in, float top,
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
    const Scan scan = cta_scan(S, G, sum);
    const u64 run = scan.run, need = target - above;
    if (scan.all < need) {
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
  list_begin(S);
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
        if (key <= high && key >= low) list_put(S, z[j], id);
      }
    }
  }
  const int n = list_sorted(S, G);
  u64 w[kEach], run[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int at = kEach * threadIdx.x + i;
    w[i] = at >= n ? 0 : MASS ? weight(h, S.powers, list_value(S, at)) : 1;
  }
  list_scan(S, G, w, run);
  const u64 need = target - above;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int at = kEach * threadIdx.x + i;
    if (at < n && run[i] >= need && run[i] - w[i] < need) S.cut = {list_value(S, at), list_id(S, at)};
  }
  __syncthreads();
  *out = S.cut;
  G.sync();
  return true;
}

// Lists the tokens from `low` to below `high` (of a finite row's values).
template <int NV, class T, class Keep>
__device__ void list_between(Shared& S, const Group& G, const Part<T>& R, float low, float high, Keep keep) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  list_begin(S);
  const float least = R.infinite ? -CUDART_INF_F : low;
  for (int s = warp; s < R.segs; s += kWarps) {
    if (S.seg_max[s] < least) continue;
#pragma unroll 1
    for (int v = 0; v < NV; ++v) {
      const int q = R.from + (s * NV + v) * 256 + lane * 8;
      float z[8];
      load_finite(R, q, z);
      unsigned found = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) found |= z[j] >= low && z[j] < high ? 1u << j : 0u;
      if (found == 0) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if ((found >> j & 1) && keep(z[j], q + j - R.shift)) list_put(S, z[j], q + j - R.shift);
    }
  }
}

// A bound that the first k tokens reach, from the segments' maxima; -inf where
// that does not work out (too few or too many segments).
__device__ float bound_of_best(Shared& S, const Group& G, int k) {
  int all = 0;
  for (int r = 0; r < G.size; ++r) all += *G.of(&S.border_count, r);
  if (all > kFewSegs || 2 * k > all) return -CUDART_INF_F;
  // every CTA ranks all maxima; equal ones by their place
  float* maxima = reinterpret_cast<float*>(S.list.all);
  for (int r = 0, at = 0; r < G.size; ++r) {
    const int n = *G.of(&S.border_count, r);
    for (int i = threadIdx.x; i < n; i += kThreads) maxima[at + i] = G.of(S.seg_max, r)[i];
    at += n;
  }
  __syncthreads();
  for (int at = threadIdx.x; at < all; at += kThreads) {
    const float own = maxima[at];
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < all; ++i) rank += maxima[i] > own || (maxima[i] == own && i < at);
    if (rank == k - 1) S.bound = own;
  }
  __syncthreads();
  return S.bound;
}

// The values at which bins begin: S.high, from which on bins are below `first`,
// and S.low, from which on they are at most `last`.
__device__ void bins_to_values(Shared& S, const Heat& h, int first, int last) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp < 2) {
    // the least key whose bin is at most `most`, 32 places a time
    const int most = warp == 0 ? first - 1 : last;
    uint32_t low = ord_bits(kLowest), high = ord_bits(h.top) + 1;
    while (low < high) {
      const uint32_t step = (high - low + 31) / 32, at = low + lane * step;
      const unsigned reached = __ballot_sync(0xffffffffu, at >= high || at < low || bin_of(h, ord_value(at)) <= most);
      // (the last place may lie before the end)
      const int i = reached ? __ffs(reached) - 1 : 32;
      const uint32_t next = i == 32 || low + i * step < low ? high : min(high, low + i * step);
      low = i == 0 ? next : low + (i - 1) * step + 1;
      high = next;
    }
    const float v = low > ord_bits(h.top) ? CUDART_INF_F : ord_value(low);
    if (lane == 0) (warp == 0 ? S.high : S.low) = v;
  }
  __syncthreads();
}

// Fills the bins with the tokens that `keep` keeps: their number, or their weights.
template <bool MASS, int NV, class T, class Keep>
__device__ void fill_bins(Shared& S, const Group& G, const Part<T>& R, const Heat& h, Keep keep) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t bins = static_cast<uint32_t>(__cvta_generic_to_shared(S.bin.low));
  for (int i = threadIdx.x; i < kBins; i += kThreads) S.bin.low[i] = 0;
  __syncthreads();
  for (int s = warp; s < R.segs; s += kWarps) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int q = R.from + (s * NV + v) * 256 + lane * 8;
      float z[8];
      load_finite(R, q, z);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        int b;
        uint32_t n = 1;
        if (MASS)
          n = bin_weight(h, z[j], b);
        else
          b = bin_of(h, z[j]);
        // (a word of the lane's behind the bins takes the others: a branch around each addition costs more)
        b = keep(z[j], q + j - R.shift) ? b : kBins + lane;
        asm volatile("red.shared.add.u32 [%0], %1;" ::"r"(bins + 4 * b), "r"(n) : "memory");
      }
    }
  }
  G.sync();
}

// The first k tokens where they are many: a list that holds them (its length
// returned, sorted), or else the cut after the k-th (0 returned), or -1: bins that
// hold too many.
template <int NV, class T>
__device__ int list_by_count(Shared& S, const Group& G, const Part<T>& R, const Heat& h, int k, float least, Cut* out) {
  const auto every = [&](float z, int) { return z >= least; };
  fill_bins<false, NV>(S, G, R, h, every);
  u64 count[kBinsThread] = {}, sum = 0;
  const int b0 = threadIdx.x * kBinsThread;
#pragma unroll
  for (int i = 0; i < kBinsThread; ++i) {
    for (int r = 0; r < G.size; ++r) count[i] += *G.of(&S.bin.low[b0 + i], r);
    sum += count[i];
  }
  if (threadIdx.x == 0) S.border = kBins - 1, S.border_above = 0, S.border_count = kList + 1;
  const Scan scan = cta_scan(S, G, sum);
  const u64 need = static_cast<u64>(k), all = scan.all;
  u64 before = scan.run - sum;
#pragma unroll
  for (int i = 0; i < kBinsThread; ++i) {
    if (before < need && before + count[i] >= need) {
      S.border = b0 + i, S.border_above = before;
      S.border_count = static_cast<int>(min(count[i], static_cast<u64>(kList + 1)));
    }
    before += count[i];
  }
  __syncthreads();
  if (all <= need) {  // there are no more than k
    *out = {least, kAllIds};
    G.sync();
    if (all > kList) return 0;
    list_between<NV>(S, G, R, least, CUDART_INF_F, every);
    return list_sorted(S, G);
  }
  const int border = S.border, count_in = S.border_count;
  const u64 above = S.border_above;
  bins_to_values(S, h, border, border);
  const float high = S.high, low = fmaxf(S.low, least);
  G.sync();  // the bins are free
  if (count_in > kList) return -1;
  const bool whole = above + count_in <= kList;
  list_between<NV>(S, G, R, low, whole ? CUDART_INF_F : high, every);
  const int n = list_sorted(S, G);
  if (whole) return n;
  const int at = static_cast<int>(need - above) - 1;
  *out = {list_value(S, at), list_id(S, at)};
  G.sync();
  return 0;
}

// The listed tokens e < some, with weights w of this thread's two, join their
// segments' sums.  Returns their sum; S.total has grown by this CTA's.
template <int NV, class T>
__device__ u64 join_segments(Shared& S, const Group& G, const Part<T>& R, int some, const u64 (&w)[kEach]) {
  u64 more = 0, own = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = kEach * threadIdx.x + i;
    if (e >= some || w[i] == 0) continue;
    more += w[i];
    const int s = list_id(S, e) + R.shift - R.from;
    if (s >= 0 && s / (NV * 256) < R.segs) {
      atomicAdd(&S.seg[s / (NV * 256)], w[i]);
      own += w[i];
    }
  }
  const u64 all = cta_total(S, G, warp_total(more)), mine = G.size > 1 ? cta_total(S, G, warp_total(own)) : all;
  G.sync();
  if (threadIdx.x == 0) S.total += mine;
  G.sync();
  return all;
}

// Cuts a sorted list of n tokens, among them all that are kept: the first k, of
// those the prefix of at least p of their mass (p < 1), of those the values from `least` on.
template <int NV, class T>
__device__ u64 cut_list(Shared& S, const Group& G, const Part<T>& R, const Heat& h, int n, int k, float p, float least, Cut* out) {
  n = min(n, k);
  u64 w[kEach], run[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = kEach * threadIdx.x + i;
    w[i] = e < n ? weight(h, S.powers, list_value(S, e)) : 0;
  }
  const u64 sum = list_scan(S, G, w, run), target = p < 1.0f ? fraction_of(p, sum, true) : sum;
  for (int i = threadIdx.x; i < R.segs; i += kThreads) S.seg[i] = 0;
  if (threadIdx.x == 0) S.total = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = kEach * threadIdx.x + i;
    if (e >= n) continue;
    const bool stays = e == 0 || (run[i] - w[i] < target && list_value(S, e) >= least);
    const bool next = e + 1 < n && run[i] < target && list_value(S, e + 1) >= least;
    if (stays && !next) S.cut = {list_value(S, e), list_id(S, e)};
    if (!stays) w[i] = 0;
  }
  const u64 mass = join_segments<NV>(S, G, R, n, w);
  *out = S.cut;
  return mass;
}

// Cut by mass: the shortest prefix of the tokens that `of` keeps whose mass is
// at least p of theirs, and that `in` keeps (tighter than `of`).  Leaves in S.seg
// and S.total the sums by segments of what is kept, and returns their sum; 0
// where the border's bins hold too many tokens.
// Without TIES `of` are all possible tokens (the others have weight 0), `in` those
// from a value on.
template <bool TIES, int NV, class T>
__device__ u64 cut_by_mass(Shared& S, const Group& G, const Part<T>& R, const Heat& h, float p, const Cut& of, const Cut& in,
                           Cut* out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const auto of_these = [&](float z, int id) { return TIES ? kept(of, z, id) : z >= of.value; };
  const auto in_these = [&](float z, int id) { return TIES ? kept(in, z, id) : z >= in.value; };
  fill_bins<true, NV>(S, G, R, h, of_these);
  // in units of 2^-40 of the largest weight
  uint32_t mass[kBinsThread];
  u64 sum = 0;
  const int b0 = threadIdx.x * kBinsThread, octave = b0 >> 6;  // (a thread's bins lie in one octave)
  const auto scaled = [octave](u64 n) { return octave < 26 ? n << (26 - octave) : n >> (octave - 26); };
#pragma unroll
  for (int i = 0; i < kBinsThread; ++i) mass[i] = S.bin.low[b0 + i];
  for (int r = 1; r < G.size; ++r) {
    // (Not past 32 bits here.  A CTA's own sum wraps around past 2^18 tokens of the largest weight: the exact masses
    // below then find the border to be wrong, or too many tokens at it, and `select` takes over.)
    const uint32_t* other = G.of(S.bin.low, (G.rank + r) % G.size);
#pragma unroll
    for (int i = 0; i < kBinsThread; ++i) mass[i] = min(mass[i], 0x7FFFFFFFu) + min(other[b0 + i], 0x7FFFFFFFu);
  }
#pragma unroll
  for (int i = 0; i < kBinsThread; ++i) sum += mass[i];
  sum = scaled(sum);
  if (threadIdx.x == 0) S.border = 0, S.border_count = kBins - 1;
  const Scan scan = cta_scan(S, G, sum);
  const u64 goal = fraction_of(p, scan.all, true), margin = scan.all >> 12;
  u64 at = scan.run - sum;
  if (at < goal + margin && scan.run + margin >= goal) {
#pragma unroll
    for (int i = 0; i < kBinsThread; ++i) {
      const u64 next = at + scaled(mass[i]);
      if (at + margin < goal && next + margin >= goal) S.border = b0 + i;
      if (at < goal + margin && next >= goal + margin) S.border_count = b0 + i;
      at = next;
    }
  }
  __syncthreads();
  bins_to_values(S, h, S.border, S.border_count);
  const float high = S.high, low = S.low;
  G.sync();  // the bins are free

  // exact masses: of all, of what lies above the border's bins by segments; the border's bins are listed
  list_begin(S);
  const float upper = fmaxf(high, in.value), lower = fmaxf(low, in.value);
  u64 above = 0, all = 0;
  for (int s = warp; s < R.segs; s += kWarps) {
    u64 part = 0;
#pragma unroll 1
    for (int v = 0; v < NV; ++v) {
      const int q = R.from + (s * NV + v) * 256 + lane * 8;
      float z[8];
      load_finite(R, q, z);
      unsigned listed = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int id = q + j - R.shift;
        const u64 w = weight(h, S.powers, z[j]);
        if (TIES) {
          const bool takes = z[j] >= upper && in_these(z[j], id);
          if (of_these(z[j], id)) all += w;
          if (takes) part += w;
          listed |= z[j] >= lower && !takes ? 1u << j : 0u;
        } else {
          all += w;
          add_from(part, w, z[j], upper);
          listed |= z[j] >= lower && z[j] < upper ? 1u << j : 0u;
        }
      }
      if (listed != 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if ((listed >> j & 1) && in_these(z[j], q + j - R.shift)) list_put(S, z[j], q + j - R.shift);
      }
    }
    part = warp_total(part);
    if (lane == 0) S.seg[s] = part;
    above += part;
  }
  const u64 total = cta_total(S, G, above), total_all = cta_total(S, G, warp_total(all));
  if (threadIdx.x == 0) S.total = total, S.rest = total_all;
  const int n = list_sorted(S, G);
  u64 mass_above = 0;
  all = 0;
  for (int r = 0; r < G.size; ++r) mass_above += *G.of(&S.total, r), all += *G.of(&S.rest, r);
  if (n < 0) {
    G.sync();
    return 0;
  }
  u64 w[kEach], at_run[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = kEach * threadIdx.x + i;
    w[i] = e < n ? weight(h, S.powers, list_value(S, e)) : 0;
  }
  const u64 listed = list_scan(S, G, w, at_run);
  const u64 target = max(fraction_of(p, all, true), static_cast<u64>(1));
  if (threadIdx.x == 0) S.cut = in, S.found = n;
  __syncthreads();
  // the border lies above the bins: they were chosen wrongly; or below: `in` ends before it, or wrongly
  const bool wrong = mass_above >= target || (mass_above + listed < target && in.value < low);
  const u64 need = target - mass_above;
  if (!wrong && listed >= need) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      if (at_run[i] >= need && at_run[i] - w[i] < need) {
        const int e = kEach * threadIdx.x + i;
        S.cut = {list_value(S, e), list_id(S, e)}, S.found = e + 1;
      }
    }
  }
  __syncthreads();
  *out = S.cut;
  const int some = S.found;
  if (wrong) {
    G.sync();
    return 0;
  }
  return mass_above + join_segments<NV>(S, G, R, some, w);
}

template <class T, int NV>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) k_sample(const SampleArgs A) {
  extern __shared__ unsigned char raw[];
  Shared& S = *reinterpret_cast<Shared*>(raw);
  Group G = {cg::this_cluster(), 0, 1, 0};
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

    float temperature = A.temperature ? A.temperature[row] : A.temperature_all;
    int64_t k = A.top_k ? A.top_k[row] : A.top_k_all;
    const float p = A.top_p ? A.top_p[row] : A.top_p_all;
    const float least = A.min_p ? A.min_p[row] : A.min_p_all;
    // (a NaN fails the comparison that would turn its filter on)
    if (!(temperature >= kSampleColdest) || p <= 0.0f) k = 1;
    if (least > 0.0f && threadIdx.x == kThreads - 1)
      S.floor_below = static_cast<double>(temperature) * log(static_cast<double>(fminf(least, 1.0f)));

    float top = -CUDART_INF_F;
    constexpr int kTogether = 4 / NV;  // segments on their way together
    for (int s0 = warp; s0 < R.segs; s0 += kWarps * kTogether) {
      float z[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i) load_block(R, R.from + ((s0 + i / NV * kWarps) * NV + i % NV) * 256 + lane * 8, z[i]);
#pragma unroll
      for (int i = 0; i < kTogether; ++i) {
        float best = -CUDART_INF_F;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < 8; ++j) best = fmaxf(best, z[i * NV + v][j]);
        best = warp_max(best);
        const int s = s0 + i * kWarps;
        if (lane == 0 && s < R.segs) S.seg_max[s] = best;
        // (a segment behind this CTA's is another's, or -inf)
        if (s < R.segs) top = fmaxf(top, best);
      }
    }
    if (lane == 0) S.warp_max[warp] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, S.warp_max[w]);
      S.max = top, S.border_count = R.segs;
    }
    G.sync();
    top = -CUDART_INF_F;
    for (int r = 0; r < G.size; ++r) top = fmaxf(top, *G.of(&S.max, r));
    if (top == -CUDART_INF_F) {  // no token is possible
      if (G.rank == 0 && threadIdx.x == 0) A.ids[row] = -1, A.logp[row] = -CUDART_INF_F;
      G.sync();
      continue;
    }

    if (k == 1) {
      // the first token of the largest value
      if (threadIdx.x == 0) S.found = kAllIds;
      __syncthreads();
      for (int s = warp; s < R.segs; s += kWarps) {
        if (S.seg_max[s] != top) continue;
#pragma unroll 1
        for (int v = 0; v < NV; ++v) {
          const int q = R.from + (s * NV + v) * 256 + lane * 8;
          float z[8];
          load_block(R, q, z);
          int id = kAllIds;
#pragma unroll
          for (int j = 7; j >= 0; --j)
            if (z[j] == top) id = q + j - R.shift;
          if (id != kAllIds) atomicMin(&S.found, id);
        }
      }
      G.sync();
      if (G.rank == 0 && threadIdx.x == 0) {
        int id = kAllIds;
        for (int r = 0; r < G.size; ++r) id = min(id, *G.of(&S.found, r));
        A.ids[row] = id, A.logp[row] = 0.0f;
      }
      G.sync();
      continue;
    }
    if (top == CUDART_INF_F) R.infinite = true, top = 0.0f;
    const bool by_count = k > 0 && k < vocab, by_mass = p < 1.0f;
    const Heat h = make_heat(top, temperature, A.shift);

    float floor = kLowest;  // every possible token
    if (least > 0.0f) {
      // the least value is rounded up to fp32, so that comparing values is exact
      if (threadIdx.x == 0) {
        const double t = static_cast<double>(top) + S.floor_below;
        float f = static_cast<float>(fmax(t, -3.402823466e38));
        if (static_cast<double>(f) < t) f = nextafterf(f, CUDART_INF_F);
        S.bound = f;
      }
      __syncthreads();
      floor = fmaxf(floor, S.bound);
      __syncthreads();
    }
    const Cut floor_cut = {floor, kAllIds};
    const auto possible = [&](const Cut& c) {
      return [&](float z, int id) { return kept(c, z, id) ? weight(h, S.powers, z) : 0ull; };
    };

    // (the mass of the first k, whatever their weights, is asked for where a cut by mass follows)
    const float least_counted = by_mass ? kLowest : floor;
    Cut cut = {least_counted, kAllIds};
    u64 mass = 0;
    if (by_count) {
      int n = -1;
      const float bound = k <= kFewSegs / 2 ? bound_of_best(S, G, static_cast<int>(k)) : -CUDART_INF_F;
      if (bound > -CUDART_INF_F) {
        const float from = R.infinite ? 0.0f : bound;
        list_between<NV>(S, G, R, from, CUDART_INF_F, [&](float, int) { return true; });
        n = list_sorted(S, G);
      }
      // (too many: many tokens at the bound)
      if (n <= 0) {
        G.sync();
        n = list_by_count<NV>(S, G, R, h, static_cast<int>(k), least_counted, &cut);
      }
      if (n > 0) {
        mass = cut_list<NV>(S, G, R, h, n, static_cast<int>(k), p, floor, &cut);
      } else if (n < 0) {
        const Cut in = {least_counted, kAllIds};
        if (!select<false, NV>(S, G, R, h, static_cast<u64>(k), in, top, &cut)) cut = in;
      }
    }
    if (by_mass && mass == 0) {
      const Cut of = cut, in = tighter(cut, floor_cut);
      Cut c;
      mass = of.id == kAllIds && in.id == kAllIds && of.value <= kLowest && h.zeros ? cut_by_mass<false, NV>(S, G, R, h, p, of, in, &c)
                                                  : cut_by_mass<true, NV>(S, G, R, h, p, of, in, &c);
      if (mass == 0) {
        const u64 target = fraction_of(p, sum_row<NV>(S, G, R, possible(of)), true);
        G.sync();
        if (!select<true, NV>(S, G, R, h, max(target, static_cast<u64>(1)), in, top, &c)) c = in;
      }
      cut = c;
    }
    cut = tighter(cut, floor_cut);
    if (mass == 0) mass = cut.id == kAllIds ? sum_above<NV>(S, G, R, h, cut.value) : sum_row<NV>(S, G, R, possible(cut));

    float u = A.u[row];
    u = u > 0.0f ? fminf(u, 0.99999994f) : 0.0f;
    const int id = locate<NV>(S, G, R, fraction_of(u, mass, false), possible(cut));
    if (id >= 0 && threadIdx.x == 0) {
      const float z = R.infinite ? 0.0f : to_f32(z0[id]);
      // ln(w / mass), w relative to the largest weight: two terms that are not positive
      const u64 most = weight(h, S.powers, top);
      A.ids[row] = id;
      A.logp[row] = __fdiv_rn(z - top, temperature) - log1pf(static_cast<float>(mass - most) / static_cast<float>(most));
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
  // more CTAs for a row while the SMs last and a CTA keeps 32768 values: below
  // that the cluster's barriers cost more (one row of 32000 with all filters: 18 us in
  // one CTA, 23 in eight; of 128256 with top-p: 94 in one, 45 in the four that it gets, 41 in eight).
  // Many rows, 1024 of 131072: 234 us with a CTA for a row, 270 with two, 507 with four.
  int size = 1;
  while (size < 8 && A.rows * size * 2 <= num_sms && A.vocab >= size * 32768) size *= 2;
  // (what a CTA's segments hold)
  while (lm_div_up(A.vocab + 8, size) > (kSegs - 8) * 1024) size *= 2;
  const int64_t resident = static_cast<int64_t>(num_sms) * (1024 / kThreads) / size;
  const int clusters = static_cast<int>(A.rows < resident ? A.rows : resident);
  // segments of 256 values, and of 1024 where that would be more than kFewSegs
  const bool wide = lm_div_up(A.vocab, size) > 65536;
  if (dtype == kDtF32) return wide ? launch_nv<float, 4>(A, clusters, size, st) : launch_nv<float, 1>(A, clusters, size, st);
  return wide ? launch_nv<__nv_bfloat16, 4>(A, clusters, size, st) : launch_nv<__nv_bfloat16, 1>(A, clusters, size, st);
}

}  // namespace okls
