// 8-bit matrix product with a scale for each block of 128 along the sum
// (sm_103a):
//
//   out[i, j] = sum_kb sa[i, kb] sb[j, kb] sum_{p in kb} a[i, p] b[j, p].
//
// The inner sums run on the tensor cores (tcgen05 kind::f8f6f4, both operands
// e4m3, fp32 accumulators in TMEM); the scales change with every 128 of the
// sum, so each partial product is taken out of TMEM, scaled and added to a
// running sum in fp32 registers.  A persistent CTA per SM:
//   warp 0 / lane 0  TMA producer: 128 x 128 A and BN x 128 B boxes (BN 64 or
//                    128 columns of the output; one 128-byte swizzle row per
//                    matrix row) into a ring;
//   warp 1 / lane 0  MMA issuer: four K32 MMAs per stage into one of the TMEM
//                    buffers in turn, overwriting it;
//   warp 2           copies each step's scales into a ring of their own, with
//                    asynchronous copies that take any layout;
//   warps 4-11       scale and add (add_square, add_rows), then store.
// The TMEM buffers let the additions of one step overlap the MMAs of the
// next.  The running sums of 128 x 256 results (CTA pairs, below) take half of
// the SM's registers, so the first four warps hand theirs to the other eight.
//
// Every wait is bounded; when one expires the CTA raises kStTimeout and runs to
// its end without further waits, apart from the bounded ones for its own copies
// and MMAs.  The CTA's waits look at a word in its shared memory, which joins
// the caller's status word at the end: a timeout that an earlier product left
// there must not make this one give up.
#include <cuda_fp16.h>

#include "okls_fp8_layout.h"
#include "okls_internal.h"
#include "okls_lm.cuh"
#include "okls_ptx.cuh"

namespace okls {
namespace {

__device__ __forceinline__ uint8_t* smem_base(uint8_t* raw) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + kSmemAlign - 1) & ~uintptr_t(kSmemAlign - 1));
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}

// The four K32 MMAs of one 128-deep step (32 bytes apart in each operand's
// swizzled rows); the first one overwrites the accumulator.
__device__ __forceinline__ void umma_f8_step(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "setp.ne.b32 p, %3, %3;\n\t"
      "setp.eq.b32 q, %3, %3;\n\t"
      "add.s64 a1, %1, 2;\n\t"
      "add.s64 b1, %2, 2;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
      "add.s64 a2, %1, 4;\n\t"
      "add.s64 b2, %2, 4;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, q;\n\t"
      "add.s64 a3, %1, 6;\n\t"
      "add.s64 b3, %2, 6;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, q;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, q;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc)
      : "memory");
}

// 4 bytes into shared memory without registers, zeros where !valid.
__device__ __forceinline__ void copy4(float* dst, const float* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(valid ? 4 : 0)
               : "memory");
}
// One arrival on `bar` when this thread's copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 32 fp32 columns of this thread's TMEM lane on their way into v; usable
// after tmem_ld_wait(v), which waits for every load of this thread.
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&v)[32]) {
  // the registers are operands so that no use of them moves above the wait
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                 "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]),
                 "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}

// 16 TMEM lanes x 32 fp32 columns in the 16x256b shape: of each 8 columns i,
// v[4 i + {0, 1}] are lane / 4's columns 2 (lane % 4) + {0, 1}, and
// v[4 i + {2, 3}] those of the TMEM lane 8 further.
__device__ __forceinline__ void tmem_ld16x256_start(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16x256_wait(uint32_t (&v)[16], uint32_t (&w)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                 "+r"(w[0]), "+r"(w[1]), "+r"(w[2]), "+r"(w[3]), "+r"(w[4]), "+r"(w[5]), "+r"(w[6]), "+r"(w[7]),
                 "+r"(w[8]), "+r"(w[9]), "+r"(w[10]), "+r"(w[11]), "+r"(w[12]), "+r"(w[13]), "+r"(w[14]), "+r"(w[15])
               :
               : "memory");
}

// Two fp32 values in a 64-bit register, with one instruction for both.
__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ void fma_pair(uint64_t& acc, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t pick4(const uint32_t (&w)[4], int i) {
  const uint32_t a = i & 1 ? w[1] : w[0], b = i & 1 ? w[3] : w[2];
  return i & 2 ? b : a;
}

// The 4 x 4 words of a quad transposed: each lane then has 8 consecutive
// columns (w[i]: columns 8 i + 2 p and + 1 of quad position p) and the quad 64
// bytes.
__device__ __forceinline__ uint4 quad_transpose(const uint32_t (&w)[4], int p) {
  uint32_t u[4];
  u[0] = pick4(w, p);
#pragma unroll
  for (int e = 1; e < 4; ++e) u[e] = __shfl_xor_sync(0xffffffffu, pick4(w, p ^ e), e);
  // u[e] came from quad position p ^ e
  return make_uint4(pick4(u, p), pick4(u, p ^ 1), pick4(u, p ^ 2), pick4(u, p ^ 3));
}

struct TileAt {
  int tm, tn;
};

// Tiles in groups of kGroup row blocks, column by column inside a group, so
// that the A panels of a group and the B panel in turn stay in L2.
constexpr int kGroup = 16;
__device__ __forceinline__ TileAt tile_at(int t, int tiles_m, int tiles_n) {
  const int per = kGroup * tiles_n;
  const int g = t / per, in = t - g * per;
  const int h = min(kGroup, tiles_m - g * kGroup);
  return {g * kGroup + in % h, in / h};
}

// An arrival on a barrier of either CTA of a pair.  What it hands over is TMEM
// (ordered by the tcgen05 fences around it), not memory, so it needs no
// release at cluster scope, which would wait for the thread's outstanding
// memory accesses every step.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Results of a warp's 32 rows x 128 columns in bf16 on their way out: two boxes
// of 64 columns (128 bytes a row, 128-byte swizzle) in shared memory, which the
// copy engine stores while the warp goes on with the next tile.
__device__ __forceinline__ void out_chunk(uint8_t* mine, int row, int chunk, uint4 v) {
  // chunk: 8 columns; the 16-byte positions of a row are permuted by the row
  *reinterpret_cast<uint4*>(mine + (chunk >> 3) * kOutBox + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)) = v;
}
// The warp's earlier stores have read their boxes.
__device__ __forceinline__ void out_free(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}
// Stores the boxes, rows row .. row + 31 and columns col .. col + 127 of the
// output; what lies outside it is left out.
__device__ __forceinline__ void out_store(const Fp8GemmArgs& A, const uint8_t* mine, int row, int col, int lane) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0 && row < A.m) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
      if (col + b * 64 < A.n)
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(&A.omap),
                     "r"(smem_u32(mine + b * kOutBox)), "r"(col + b * 64), "r"(row)
                     : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

// What the adding warps share with the others, and the CTA's walk over the
// tiles.  PAIR: the two CTAs of a cluster hold the halves of 256-row tiles.
template <int BN, bool PAIR>
struct Adder {
  int first, stride;        // tiles first, first + stride, ...
  int row_step, row0;       // rows of a tile, and this CTA's first of them
  uint32_t tmem;
  const float* scales;  // ring of slots: the tile's rows' scales, then its columns' (or square blocks')
  int slot_floats, slots;
  uint64_t *acc_full, *acc_empty, *sempty;
  uint32_t acc_empty_lead;  // PAIR: acc_empty of the cluster's first CTA
  uint8_t* out;             // PAIR: the warps' output boxes
  uint32_t* stop;           // the CTA's status word
};

// Per-step bookkeeping of an adding warp: waits for a TMEM buffer and hands it
// and the scales back.
template <int BN, bool PAIR>
struct Steps {
  uint32_t it = 0, slot = 0;
  bool ok = true, ready;
  // The first look at a step's barrier is taken before the last additions of
  // the step before, so that its latency passes under them (a test, not a
  // try: a try holds the warp until the barrier turns or a time limit passes).
  __device__ __forceinline__ explicit Steps(const Adder<BN, PAIR>& R) { ready = mbar_test(&R.acc_full[0], 0); }
  __device__ __forceinline__ uint32_t buf() const { return Buffers<BN>::at(it); }
  __device__ __forceinline__ const float* begin(const Adder<BN, PAIR>& R) {
    if (!ready) ok = ok && mbar_wait(&R.acc_full[buf()], Buffers<BN>::parity(it), R.stop);
    __syncwarp();
    tc_fence_after();
    return R.scales + slot * R.slot_floats;
  }
  __device__ __forceinline__ void loaded(const Adder<BN, PAIR>& R, int lane) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      if (PAIR)
        mbar_arrive_pair(R.acc_empty_lead + buf() * 8);
      else
        mbar_arrive(&R.acc_empty[buf()]);
    }
    ready = mbar_test(&R.acc_full[Buffers<BN>::at(it + 1)], Buffers<BN>::parity(it + 1));
  }
  __device__ __forceinline__ void end(const Adder<BN, PAIR>& R, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&R.sempty[slot]);
    if (static_cast<int>(++slot) == R.slots) slot = 0;
    ++it;
  }
};

// 16 bf16 or 8 fp32 results of one row (left: how many of them exist), 32 bytes
// a store where the address allows: whole memory sectors, although neighbouring
// lanes write different rows.  vec: the address is 16-byte aligned.
__device__ __forceinline__ void store_bf16x16(const Fp8GemmArgs& A, __nv_bfloat16* p, int left, bool vec, float (&v)[16]) {
  if (vec && left >= 16) {
    if (A.accumulate) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float old[8];
        load8(p + 8 * h, old);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * h + j] += old[j];
      }
    }
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
    if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
      store32(p, w);
    } else {
      reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < left) p[j] = __float2bfloat16_rn(A.accumulate ? v[j] + __bfloat162float(p[j]) : v[j]);
  }
}
__device__ __forceinline__ void store_f32x8(const Fp8GemmArgs& A, float* p, int left, bool vec, float (&v)[8]) {
  if (vec && left >= 8) {
    if (A.accumulate) {
      float old[8];
      load8(p, old);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += old[j];
    }
    store8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) p[j] = A.accumulate ? v[j] + p[j] : v[j];
  }
}

// B in square blocks: a thread owns one output row and BN / 2 columns; one
// block's scale covers 32 or more of them, so an addition is one fused
// multiply-add.
template <int BN, bool PAIR>
__device__ __forceinline__ void add_square(const Fp8GemmArgs& A, const Adder<BN, PAIR>& R, int tiles_m, int tiles_n, int nkb) {
  constexpr int kCols = BN / 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3;  // TMEM lane quarter of this warp
  const int half = (warp - 4) >> 2;
  const uint32_t tbase = R.tmem + (static_cast<uint32_t>(q * 32) << 16) + half * kCols;
  const int tiles = tiles_m * tiles_n;
  Steps<BN, PAIR> S(R);
  for (int t = R.first; t < tiles; t += R.stride) {
    const TileAt at = tile_at(t, tiles_m, tiles_n);
    const int row = at.tm * R.row_step + R.row0 + q * 32 + lane;
    const int col0 = at.tn * BN + half * kCols;
    float acc[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) acc[j] = 0.0f;
    for (int kb = 0; kb < nkb; ++kb) {
      const float* sc = S.begin(R);
      const uint32_t d = tbase + S.buf() * BN;
      const float s = sc[q * 32 + lane];
      const float* sb = sc + kTM - (at.tn * BN) / kFp8Group;
      if constexpr (kCols <= 64) {
        // one CTA's 32 or 64 columns, the whole step at once: the buffer is free
        // before the additions
        uint32_t v[kCols / 32][32];
#pragma unroll
        for (int c = 0; c < kCols; c += 32) tmem_ld32_start(d + c, v[c / 32]);
#pragma unroll
        for (int c = 0; c < kCols; c += 32) tmem_ld_wait(v[c / 32]);
        S.loaded(R, lane);
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          const float x = s * sb[(col0 + c) / kFp8Group];
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[c + j] = fmaf(__uint_as_float(v[c / 32][j]), x, acc[c + j]);
        }
      } else {
        // 32 columns are loaded while the 32 before them are added
        uint32_t v[2][32];
        tmem_ld32_start(d, v[0]);
        const float x = s * sb[col0 / kFp8Group];  // 128 columns of one block
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          tmem_ld_wait(v[(c / 32) & 1]);
          if (c + 32 < kCols)
            tmem_ld32_start(d + c + 32, v[(c / 32 + 1) & 1]);
          else
            S.loaded(R, lane);
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[c + j] = fmaf(__uint_as_float(v[(c / 32) & 1][j]), x, acc[c + j]);
        }
      }
      S.end(R, lane);
    }
    if (PAIR && A.tma_out) {
      uint8_t* mine = R.out + (warp - 4) * kOutWarp;
      out_free(lane);
#pragma unroll
      for (int c = 0; c < kCols; c += 8)
        out_chunk(mine, lane, c / 8,
                  make_uint4(pack_bf16(acc[c], acc[c + 1]), pack_bf16(acc[c + 2], acc[c + 3]),
                             pack_bf16(acc[c + 4], acc[c + 5]), pack_bf16(acc[c + 6], acc[c + 7])));
      out_store(A, mine, row - lane, col0, lane);
      continue;
    }
    if (row >= A.m) continue;
    const int eb = A.out_dtype == kDtBf16 ? 2 : 4;
    char* o = static_cast<char*>(A.out) + (static_cast<int64_t>(row) * A.ldo + col0) * eb;
    const bool vec = (reinterpret_cast<uintptr_t>(o) & 15) == 0;
    if (A.out_dtype == kDtBf16) {
#pragma unroll
      for (int c = 0; c < kCols; c += 16) {
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = acc[c + j];
        store_bf16x16(A, reinterpret_cast<__nv_bfloat16*>(o) + c, A.n - col0 - c, vec, v);
      }
    } else {
#pragma unroll
      for (int c = 0; c < kCols; c += 8) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = acc[c + j];
        store_f32x8(A, reinterpret_cast<float*>(o) + c, A.n - col0 - c, vec, v);
      }
    }
  }
}

// B in row groups: every column has a scale of its own.  With a row a thread,
// each thread would read all of them from shared memory every step (128
// floats, four clocks of the read path per 16 bytes and warp: twice the MMAs'
// time).  In the 16x256b shape a thread owns 4 rows and a quarter of the
// columns, so it reads 32; a product and a fused multiply-add per value are
// left.  Column c of a 32-column chunk: pair i of lane quad position p holds
// columns 8 i + 2 p and + 1; rows: half h (16 TMEM lanes), r: lane / 4 + 8 r.
template <int BN, bool PAIR>
__device__ __forceinline__ void add_rows(const Fp8GemmArgs& A, const Adder<BN, PAIR>& R, int tiles_m, int tiles_n, int nkb) {
  constexpr int kCols = BN / 2;
  constexpr int kChunks = kCols / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3, p = lane & 3;
  const int half = (warp - 4) >> 2;
  const uint32_t tbase = R.tmem + (static_cast<uint32_t>(q * 32) << 16) + half * kCols;
  const int tiles = tiles_m * tiles_n;
  Steps<BN, PAIR> S(R);
  for (int t = R.first; t < tiles; t += R.stride) {
    const TileAt at = tile_at(t, tiles_m, tiles_n);
    const int row0 = at.tm * R.row_step + R.row0 + q * 32 + (lane >> 2);
    const int col0 = at.tn * BN + half * kCols;
    uint64_t acc[kChunks][4][2][2];  // [chunk][i][h][r], two columns each
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[c][i][0][0] = acc[c][i][0][1] = acc[c][i][1][0] = acc[c][i][1][1] = 0;
    for (int kb = 0; kb < nkb; ++kb) {
      const float* sc = S.begin(R);
      const uint32_t d = tbase + S.buf() * BN;
      // [chunk, or in turn][half][4 i + 2 r + column]: one CTA's 32 or 64 columns
      // at once (the buffer is then free before the additions), a pair's 128 a
      // chunk ahead
      constexpr int kHeld = kChunks <= 2 ? kChunks : 2;
      uint32_t v[kHeld][2][16];
#pragma unroll
      for (int c = 0; c < (kChunks <= 2 ? kChunks : 1); ++c) {
        tmem_ld16x256_start(d + c * 32, v[c][0]);
        tmem_ld16x256_start(d + (16u << 16) + c * 32, v[c][1]);
      }
      uint64_t sa[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float x = sc[q * 32 + h * 16 + r * 8 + (lane >> 2)];
          sa[h][r] = pair_of(__float_as_uint(x), __float_as_uint(x));
        }
      const uint64_t* sb = reinterpret_cast<const uint64_t*>(sc + kTM + half * kCols) + p;
      if (kChunks <= 2) {
#pragma unroll
        for (int c = 0; c < kHeld; ++c) tmem_ld16x256_wait(v[c][0], v[c][1]);
        S.loaded(R, lane);
      }
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        uint32_t(&x)[2][16] = v[c % kHeld];
        if (kChunks > 2) {
          tmem_ld16x256_wait(x[0], x[1]);
          if (c + 1 < kChunks) {
            tmem_ld16x256_start(d + (c + 1) * 32, v[(c + 1) % kHeld][0]);
            tmem_ld16x256_start(d + (16u << 16) + (c + 1) * 32, v[(c + 1) % kHeld][1]);
          } else {
            S.loaded(R, lane);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t w = sb[c * 16 + i * 4];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              fma_pair(acc[c][i][h][r], mul_pair(pair_of(x[h][4 * i + 2 * r], x[h][4 * i + 2 * r + 1]), w), sa[h][r]);
        }
      }
      S.end(R, lane);
    }
    if (PAIR && A.tma_out) {
      uint8_t* mine = R.out + (warp - 4) * kOutWarp;
      out_free(lane);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float lo, hi;
              unpair(acc[c][i][h][r], lo, hi);
              w[i] = pack_bf16(lo, hi);
            }
            out_chunk(mine, h * 16 + r * 8 + (lane >> 2), c * 4 + p, quad_transpose(w, p));
          }
      out_store(A, mine, row0 - (lane >> 2), col0, lane);
      continue;
    }
    const int eb = A.out_dtype == kDtBf16 ? 2 : 4;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = row0 + h * 16 + r * 8;
        char* o = static_cast<char*>(A.out) + (static_cast<int64_t>(row) * A.ldo + col0) * eb;
        // one answer for the warp: lanes hold different rows, and the quads trade values
        const bool in = row < A.m, vec = __all_sync(0xffffffffu, (reinterpret_cast<uintptr_t>(o) & 15) == 0);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const int left = A.n - col0 - c * 32;  // columns of this chunk that exist
          float v[4][2];
#pragma unroll
          for (int i = 0; i < 4; ++i) unpair(acc[c][i][h][r], v[i][0], v[i][1]);
          if (A.out_dtype == kDtBf16) {
            __nv_bfloat16* b = reinterpret_cast<__nv_bfloat16*>(o) + c * 32;
            if (vec && left >= 32 && !A.accumulate) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[i][0], v[i][1]);
              const uint4 z = quad_transpose(w, p);
              if (in) *reinterpret_cast<uint4*>(b + 8 * p) = z;
            } else if (in) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const int col = 8 * i + 2 * p + j;
                  if (col < left)
                    b[col] = __float2bfloat16_rn(A.accumulate ? v[i][j] + __bfloat162float(b[col]) : v[i][j]);
                }
            }
          } else if (in) {
            float* f = reinterpret_cast<float*>(o) + c * 32;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int col = 8 * i + 2 * p;
              if (vec && col + 2 <= left) {
                float2 z = make_float2(v[i][0], v[i][1]);
                if (A.accumulate) {
                  const float2 old = *reinterpret_cast<const float2*>(f + col);
                  z.x += old.x, z.y += old.y;
                }
                *reinterpret_cast<float2*>(f + col) = z;
              } else {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  if (col + j < left) f[col + j] = A.accumulate ? v[i][j] + f[col + j] : v[i][j];
              }
            }
          }
        }
      }
  }
}

// 16 bytes, of which the first `bytes` come from global memory and the rest
// are zeros.
__device__ __forceinline__ void copy16(float* dst, const float* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}

// Rows `row0 ..` of a matrix of scales, N of them, of one group: where they
// lie group by group (as the quantiser writes them), four rows a copy.
template <int N>
struct ScaleRows {
  const float* at;  // this lane's first row in group 0
  int64_t step;     // to the next group
  int64_t ld;
  int left;         // rows from this lane's first to the end
  bool fast;
  __device__ __forceinline__ void set(const float* p, int64_t ld_row, int64_t ld_group, int row0, int rows, int lane) {
    fast = ld_row == 1 && (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld_group & 3) == 0;
    const int r = row0 + lane * (fast ? 4 : 1);
    at = p + static_cast<int64_t>(min(r, fast ? (rows - 1) & ~3 : rows - 1)) * ld_row;
    step = ld_group;
    ld = ld_row;
    left = rows - r;
  }
  __device__ __forceinline__ void copy(float* dst, int lane) {
    if (fast) {
#pragma unroll
      for (int i = 0; i < (N + 127) / 128; ++i) {
        const int n = min(4, left - i * 128);
        if (N % 128 == 0 || i * 128 + lane * 4 < N) copy16(dst + i * 128 + lane * 4, n > 0 ? at + i * 128 : at, n > 0 ? 4 * n : 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < (N + 31) / 32; ++i) {
        const bool in = left > i * 32;
        if (N % 32 == 0 || i * 32 + lane < N) copy4(dst + i * 32 + lane, in ? at + i * 32 * ld : at, in);
      }
    }
    at += step;
  }
};

// The scale warp: the tile's rows of A, then its rows of B, or the one or two
// square blocks its columns meet, of every step; zeros outside.  It is one
// warp with a step's time for a step, so it takes four rows a copy where they
// lie next to each other (row groups, 11008 x 4096 x 8192: 441 us, with scales
// that lie row by row 855; square blocks, 8192 x 11008 x 4096: 305 and 320).
template <int BN>
__device__ __forceinline__ void copy_scales(const Fp8GemmArgs& A, float* ring, int slot_floats, int slots, uint64_t* sfull,
                                            uint64_t* sempty, int first, int stride, int row_step, int row0, int tiles_m,
                                            int tiles_n, int nkb, uint32_t* stop) {
  constexpr int kBlocks = (BN + kFp8Group - 1) / kFp8Group;
  const int lane = threadIdx.x & 31, tiles = tiles_m * tiles_n;
  int slot = 0;
  uint32_t phase = 0;
  for (int t = first; t < tiles; t += stride) {
    const TileAt at = tile_at(t, tiles_m, tiles_n);
    ScaleRows<kTM> a;
    a.set(A.a_scale, A.lda_row, A.lda_group, at.tm * row_step + row0, A.m, lane);
    ScaleRows<BN> b;
    ScaleRows<kBlocks> sq;
    if (A.b_square) {
      sq.set(A.b_scale, A.ldb_row, A.ldb_group, at.tn * BN / kFp8Group, (A.n + kFp8Group - 1) / kFp8Group, lane);
      if (sq.fast) {  // a block a lane: the tile's first need not be a multiple of four
        sq.fast = false;
        const int blocks = (A.n + kFp8Group - 1) / kFp8Group, r = at.tn * BN / kFp8Group + lane;
        sq.at = A.b_scale + min(r, blocks - 1);
        sq.left = blocks - r;
      }
    } else {
      b.set(A.b_scale, A.ldb_row, A.ldb_group, at.tn * BN, A.n, lane);
    }
    for (int kb = 0; kb < nkb; ++kb) {
      if (__any_sync(0xffffffffu, !mbar_wait(&sempty[slot], phase ^ 1u, stop))) goto out;
      float* sc = ring + slot * slot_floats;
      a.copy(sc, lane);
      if (A.b_square)
        sq.copy(sc + kTM, lane);
      else
        b.copy(sc + kTM, lane);
      copy_arrive(&sfull[slot]);
      if (++slot == slots) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
out:
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int BN>
__global__ void __launch_bounds__(kThreads, 1) k_fp8_gemm(const __grid_constant__ Fp8GemmArgs A) {
  using C = Tile<BN>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t stop;  // the CTA's status word
  uint8_t* smem = smem_base(smem_raw);
  uint8_t* scales = smem + C::kRing * C::kBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + C::kSlots * C::kScaleBytes);
  uint64_t* empty = full + C::kRing;
  uint64_t* sfull = empty + C::kRing;
  uint64_t* sempty = sfull + C::kSlots;
  uint64_t* acc_full = sempty + C::kSlots;
  uint64_t* acc_empty = acc_full + Buffers<BN>::kCount;
  uint64_t* drain = acc_empty + Buffers<BN>::kCount;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kRing; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&sfull[s], 32);
      mbar_init(&sempty[s], 8);
    }
    for (int b = 0; b < Buffers<BN>::kCount; ++b) {
      mbar_init(&acc_full[b], 2);   // the MMAs, and the issuer, which has seen the step's scales
      mbar_init(&acc_empty[b], 8);
    }
    mbar_init(drain, 1);
    stop = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int tiles_m = (A.m + kTM - 1) / kTM, tiles_n = (A.n + BN - 1) / BN;
  const int tiles = tiles_m * tiles_n;
  const int nkb = (A.k + kTK - 1) / kTK;

  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtlRegs));
  if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(&A.amap);
      prefetch_tmap(&A.bmap);
      uint32_t stage = 0, phase = 0;
      int64_t issued = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const TileAt at = tile_at(t, tiles_m, tiles_n);
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, &stop)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * C::kBytes;
          mbar_expect_tx(&full[stage], C::kBytes);
          tma_load_2d(sa, &A.amap, &full[stage], kb * kTK, at.tm * kTM);
          tma_load_2d(sa + kABytes, &A.bmap, &full[stage], kb * kTK, at.tn * BN);
          ++issued;
          if (++stage == C::kRing) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // no copy may still be landing in shared memory at exit
      const int64_t back = issued < C::kRing ? issued : C::kRing;
      for (int64_t q = 1; q <= back; ++q) {
        const int64_t idx = issued - q;
        if (!mbar_wait_own(&full[idx % C::kRing], static_cast<uint32_t>((idx / C::kRing) & 1), &stop)) break;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_f16_f32(kTM, BN);  // fp32 accumulators; format code 0 is e4m3 here
      const uint32_t s0 = smem_u32(smem);
      const uint64_t adesc0 = sw128_desc(s0), bdesc0 = sw128_desc(s0 + kABytes);
      constexpr uint64_t kStep = C::kBytes >> 4;
      uint32_t stage = 0, phase = 0, slot = 0, sphase = 0, it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const uint32_t buf = Buffers<BN>::at(it);
          if (!mbar_wait(&full[stage], phase, &stop) || !mbar_wait(&sfull[slot], sphase, &stop) ||
              !mbar_wait(&acc_empty[buf], Buffers<BN>::parity(it) ^ 1u, &stop)) {
            ok = false;
            break;
          }
          tc_fence_after();
          umma_f8_step(tmem + buf * BN, adesc0 + stage * kStep, bdesc0 + stage * kStep, idesc);
          umma_commit(&acc_full[buf]);
          umma_commit(&empty[stage]);
          mbar_arrive(&acc_full[buf]);
          if (++stage == C::kRing) {
            stage = 0;
            phase ^= 1u;
          }
          if (++slot == C::kSlots) {
            slot = 0;
            sphase ^= 1u;
          }
        }
      }
      umma_commit(drain);
      mbar_wait_own(drain, 0, &stop);
    }
    __syncwarp();
  } else if (warp == 2) {
    copy_scales<BN>(A, reinterpret_cast<float*>(scales), C::kScaleBytes / 4, C::kSlots, sfull, sempty, blockIdx.x,
                    gridDim.x, kTM, 0, tiles_m, tiles_n, nkb, &stop);
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAddRegs));
    const Adder<BN, false> R = {static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), kTM, 0, tmem,
                                reinterpret_cast<const float*>(scales), C::kScaleBytes / 4, C::kSlots,
                                acc_full, acc_empty, sempty, 0, nullptr, &stop};
    if (A.b_square)
      add_square<BN, false>(A, R, tiles_m, tiles_n, nkb);
    else
      add_rows<BN, false>(A, R, tiles_m, tiles_n, nkb);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kCols);
  if (threadIdx.x == 0 && stop) atomicOr(A.status, stop);
}

// ------------------------------------------------------------- CTA pairs
// The same over clusters of two CTAs on two SMs: one tcgen05.mma.cta_group::2
// multiplies 256 rows of A (128 from each CTA's shared memory) with 256 rows
// of B (128 from each), so a CTA loads and the tensor cores read 32 KB a step
// instead of 48 (operands written and read at 128 bytes a clock take 1.5 times
// the MMAs of a 128 x 256 tile).  Each CTA adds the 128 rows in its own TMEM.
//
// What bounds it: the way of a TMEM buffer, MMAs (512 clocks), commit, loads
// by the adding warps (about 370), hand-over, and back; with two buffers a
// step takes about 1000 clocks.  bf16 results leave through the copy engine
// from shared memory, a tile's 64 KB under the next tile's first steps (threads
// storing their rows took 2.7 us a tile).  8192 x 11008 x 4096 with square
// blocks: 305 us, 2.42 PFLOP/s (threads storing 330, one CTA a tile 353);
// 8192 x 4096 x 11008: 295 us, 2.50; 8192 x 5504 x 2048: 93 us, 1.99; with row
// groups, 11008 x 4096 x 8192: 441 us, 1.68.  Narrower tiles with more buffers
// cost more operand traffic than they save (before the change of stores): 256
// x 192 388 us, 256 x 128 with four buffers 488 us.  With row groups a step takes
// about 1400 clocks: its additions are 512 of them on the fp32 units, and wait,
// TMEM loads and hand-over are not hidden under another step's.
//
// Differences to the kernel above: the first CTA issues the MMAs for both; its `full` barriers count both CTAs' copies; commits
// arrive on both CTAs' `empty` and `acc_full`; both CTAs' adding warps hand
// buffers back on the first one's `acc_empty`.  Two issuers take every other
// step each: one waits for its barriers while the other's MMAs run.

__device__ __forceinline__ uint32_t steps_of(int first, int stride, int tiles, int nkb) {
  return first < tiles ? static_cast<uint32_t>((tiles - 1 - first) / stride + 1) * static_cast<uint32_t>(nkb) : 0u;
}

__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar_cluster, int32_t c0,
                                                 int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar_cluster), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ void umma_f8_step_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "setp.ne.b32 p, %3, %3;\n\t"
      "setp.eq.b32 q, %3, %3;\n\t"
      "add.s64 a1, %1, 2;\n\t"
      "add.s64 b1, %2, 2;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
      "add.s64 a2, %1, 4;\n\t"
      "add.s64 b2, %2, 4;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a1, b1, %3, q;\n\t"
      "add.s64 a3, %1, 6;\n\t"
      "add.s64 b3, %2, 6;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a2, b2, %3, q;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a3, b3, %3, q;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc)
      : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_fp8_gemm_pair(const __grid_constant__ Fp8GemmArgs A) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t stop;  // the CTA's status word
  uint8_t* smem = smem_base(smem_raw);
  uint8_t* out = smem + kPairRing * kPairStage;
  uint8_t* scales = out + 8 * kOutWarp;
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + kPairSlots * kPairScaleBytes);
  uint64_t* empty = full + kPairRing;
  uint64_t* sfull = empty + kPairRing;
  uint64_t* sempty = sfull + kPairSlots;
  uint64_t* acc_full = sempty + kPairSlots;
  uint64_t* acc_empty = acc_full + Buffers<kPN>::kCount;
  uint64_t* drain = acc_empty + Buffers<kPN>::kCount;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairRing; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kPairSlots; ++s) {
      mbar_init(&sfull[s], 32);
      mbar_init(&sempty[s], 8);
    }
    for (int b = 0; b < Buffers<kPN>::kCount; ++b) {
      mbar_init(&acc_full[b], 2);    // the MMAs, and a thread that has seen the step's scales
      mbar_init(&acc_empty[b], 16);  // the adding warps of both CTAs
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    stop = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int tiles_m = (A.m + 2 * kTM - 1) / (2 * kTM), tiles_n = (A.n + kPN - 1) / kPN;
  const int tiles = tiles_m * tiles_n;
  const int nkb = (A.k + kTK - 1) / kTK;
  const int first = blockIdx.x / 2, stride = gridDim.x / 2;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtlRegs));
    if (warp == 0) {
      if (lane == 0) {
        prefetch_tmap(&A.amap);
        prefetch_tmap(&A.bmap);
        uint32_t stage = 0, phase = 0;
        int64_t issued = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += stride) {
          const TileAt at = tile_at(t, tiles_m, tiles_n);
          for (int kb = 0; kb < nkb; ++kb) {
            if (!mbar_wait(&empty[stage], phase ^ 1u, &stop)) {
              ok = false;
              break;
            }
            uint8_t* sa = smem + stage * kPairStage;
            if (rank == 0) mbar_expect_tx(&full[stage], 2 * kPairStage);
            const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
            tma_load_2d_pair(sa, &A.amap, bar, kb * kTK, at.tm * 2 * kTM + rank * kTM);
            tma_load_2d_pair(sa + kABytes, &A.bmap, bar, kb * kTK, at.tn * kPN + rank * (kPN / 2));
            ++issued;
            if (++stage == kPairRing) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        // no copy of either CTA may still be landing at exit (the first CTA
        // sees them all; the other leaves after the cluster's last barrier)
        if (rank == 0) {
          const int64_t back = issued < kPairRing ? issued : kPairRing;
          for (int64_t q = 1; q <= back; ++q) {
            const int64_t idx = issued - q;
            if (!mbar_wait_own_cluster(&full[idx % kPairRing], static_cast<uint32_t>((idx / kPairRing) & 1), &stop)) break;
          }
        }
      }
      __syncwarp();
    } else if ((warp == 1 || warp == 3) && rank == 0) {
      if (lane == 0) {
        constexpr uint32_t idesc = idesc_f16_f32(2 * kTM, kPN);  // format code 0 is e4m3 here
        const uint32_t s0 = smem_u32(smem);
        const uint64_t adesc0 = sw128_desc(s0), bdesc0 = sw128_desc(s0 + kABytes);
        constexpr uint64_t kStep = kPairStage >> 4;
        const uint32_t mine = warp >> 1;  // steps mine, mine + 2, ...
        const uint32_t total = steps_of(first, stride, tiles, nkb);
        for (uint32_t it = mine; it < total; it += 2) {
          const uint32_t buf = Buffers<kPN>::at(it), stage = it % kPairRing, slot = it % kPairSlots;
          if (!mbar_wait(&full[stage], (it / kPairRing) & 1u, &stop) ||
              !mbar_wait(&sfull[slot], (it / kPairSlots) & 1u, &stop) ||
              !mbar_wait(&acc_empty[buf], Buffers<kPN>::parity(it) ^ 1u, &stop))
            break;
          mbar_arrive(&acc_full[buf]);
          tc_fence_after();
          umma_f8_step_pair(tmem + buf * kPN, adesc0 + stage * kStep, bdesc0 + stage * kStep, idesc);
          umma_commit_pair(&acc_full[buf], 3);
          umma_commit_pair(&empty[stage], 3);
        }
        umma_commit_pair(&drain[mine], 1);
        mbar_wait_own_cluster(&drain[mine], 0, &stop);
      }
      __syncwarp();
    } else if (warp == 2) {
      copy_scales<kPN>(A, reinterpret_cast<float*>(scales), kPairScaleBytes / 4, kPairSlots, sfull, sempty, first, stride,
                       2 * kTM, rank * kTM, tiles_m, tiles_n, nkb, &stop);
    } else if (warp == 1) {
      if (lane == 0) {
        // one arrival a step and buffer, after the buffer's step before is over
        uint32_t slot = 0, sphase = 0, it = 0;
        bool ok = true;
        for (int t = first; t < tiles && ok; t += stride) {
          for (int kb = 0; kb < nkb; ++kb, ++it) {
            constexpr uint32_t kBufs = Buffers<kPN>::kCount;
            const uint32_t buf = Buffers<kPN>::at(it);
            if ((it >= kBufs && !mbar_wait(&acc_full[buf], Buffers<kPN>::parity(it - kBufs), &stop)) ||
                !mbar_wait(&sfull[slot], sphase, &stop)) {
              ok = false;
              break;
            }
            mbar_arrive(&acc_full[buf]);
            if (++slot == kPairSlots) {
              slot = 0;
              sphase ^= 1u;
            }
          }
        }
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAddRegs));
    const Adder<kPN, true> R = {first, stride, 2 * kTM, rank * kTM, tmem,
                                reinterpret_cast<const float*>(scales), kPairScaleBytes / 4, kPairSlots,
                                acc_full, acc_empty, sempty, mapa_shared(smem_u32(acc_empty), 0), out, &stop};
    if (A.b_square)
      add_square<kPN, true>(A, R, tiles_m, tiles_n, nkb);
    else
      add_rows<kPN, true>(A, R, tiles_m, tiles_n, nkb);
    // shared memory is read until the stores are done
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
  if (threadIdx.x == 0 && stop) atomicOr(A.status, stop);
}

// ------------------------------------------------------------ a few tokens
// Up to 32 rows of A: the bytes of B bound the product, and a 128-row tile
// would be mostly padding.  A CTA takes 16 rows of B (output columns); its 8
// warps split the sum's groups of 128 and join through shared memory.  Codes
// become binary16 (exact), and mma.sync m16n8k16 multiplies them with fp32
// sums: B's rows are its 16-row operand, A's rows its 8 columns.  Within a
// group the order of the sum is free, so a lane's operand values are 16
// consecutive bytes of its row on both sides.  5504 x 2048 in a graph: one to 8
// tokens 5.1 us a product, 16 6.3, 32 9.6; 33 and more take a 128-row tile
// (10 us up to 64), so 32 is where the two meet.
constexpr int kSkinnyMax = 32;
constexpr int kSkinnyWarps = 8;

__device__ __forceinline__ uint32_t f16x2_of(uint32_t two_codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two_codes)));
  return r;
}

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes of a row at offset p, zeros at and past k (rows are 16-byte
// aligned; a row's last bytes are read one by one)
__device__ __forceinline__ uint4 load16(const uint8_t* row, bool valid, int p, int k) {
  uint4 r = make_uint4(0, 0, 0, 0);
  if (!valid || p >= k) return r;
  if (p + 16 <= k) return *reinterpret_cast<const uint4*>(row + p);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (p + j < k) w[j >> 2] |= static_cast<uint32_t>(row[p + j]) << (8 * (j & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int MT>
__global__ void __launch_bounds__(kSkinnyWarps * 32) k_fp8_skinny(const __grid_constant__ Fp8GemmArgs A) {
  __shared__ float part[kSkinnyWarps][16][MT * 8 + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16;
  const int nkb = (A.k + kFp8Group - 1) / kFp8Group;
  const bool ok0 = n0 + g < A.n, ok1 = n0 + g + 8 < A.n;
  const uint8_t* w0 = A.b + static_cast<int64_t>(n0 + g) * A.ldb;
  const uint8_t* w1 = w0 + 8 * A.ldb;
  const int r0 = min(n0 + g, A.n - 1), r1 = min(n0 + g + 8, A.n - 1);
  const float* sb0 = A.b_scale + static_cast<int64_t>(A.b_square ? r0 / kFp8Group : r0) * A.ldb_row;
  const float* sb1 = A.b_scale + static_cast<int64_t>(A.b_square ? r1 / kFp8Group : r1) * A.ldb_row;
  float acc[MT][4] = {};
  for (int kb = warp; kb < nkb; kb += kSkinnyWarps) {
    uint4 wa[2], wb[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int p = kb * kFp8Group + h * 64 + t * 16;
      wa[h] = load16(w0, ok0, p, A.k);
      wb[h] = load16(w1, ok1, p, A.k);
    }
    const float s0 = sb0[kb * A.ldb_group], s1 = sb1[kb * A.ldb_group];
    float c[MT][4] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int p = kb * kFp8Group + h * 64 + t * 16;
      const uint32_t a0[4] = {wa[h].x, wa[h].y, wa[h].z, wa[h].w};
      const uint32_t a1[4] = {wb[h].x, wb[h].y, wb[h].z, wb[h].w};
      uint4 x[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int tok = i * 8 + g;
        x[i] = load16(A.a + static_cast<int64_t>(tok) * A.lda, tok < A.m, p, A.k);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t f0 = f16x2_of(a0[u]), f1 = f16x2_of(a1[u]);
        const uint32_t f2 = f16x2_of(a0[u] >> 16), f3 = f16x2_of(a1[u] >> 16);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const uint32_t xw = u == 0 ? x[i].x : u == 1 ? x[i].y : u == 2 ? x[i].z : x[i].w;
          mma_16x8x16(c[i], f0, f1, f2, f3, f16x2_of(xw), f16x2_of(xw >> 16));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int tok = i * 8 + t * 2;
      const float x0 = A.a_scale[static_cast<int64_t>(min(tok, A.m - 1)) * A.lda_row + kb * A.lda_group];
      const float x1 = A.a_scale[static_cast<int64_t>(min(tok + 1, A.m - 1)) * A.lda_row + kb * A.lda_group];
      acc[i][0] = fmaf(c[i][0], s0 * x0, acc[i][0]);
      acc[i][1] = fmaf(c[i][1], s0 * x1, acc[i][1]);
      acc[i][2] = fmaf(c[i][2], s1 * x0, acc[i][2]);
      acc[i][3] = fmaf(c[i][3], s1 * x1, acc[i][3]);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int tok = i * 8 + t * 2;
    part[warp][g][tok] = acc[i][0];
    part[warp][g][tok + 1] = acc[i][1];
    part[warp][g + 8][tok] = acc[i][2];
    part[warp][g + 8][tok + 1] = acc[i][3];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 16 * A.m; e += kSkinnyWarps * 32) {
    const int tok = e >> 4, col = n0 + (e & 15);
    if (col >= A.n) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kSkinnyWarps; ++w) v += part[w][e & 15][tok];
    const int64_t at = static_cast<int64_t>(tok) * A.ldo + col;
    if (A.out_dtype == kDtBf16) {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(A.out) + at;
      *o = __float2bfloat16_rn(A.accumulate ? v + __bfloat162float(*o) : v);
    } else {
      float* o = static_cast<float*>(A.out) + at;
      *o = A.accumulate ? v + *o : v;
    }
  }
}

template <int BN>
cudaError_t run_gemm(const Fp8GemmArgs& A, int num_sms, cudaStream_t st) {
  static PerDevice pd;
  const cudaError_t e = once_per_device(pd, [](int) {
    return cudaFuncSetAttribute(k_fp8_gemm<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tile<BN>::kSmem);
  });
  if (e != cudaSuccess) return e;
  const int64_t tiles = lm_div_up(A.m, kTM) * lm_div_up(A.n, BN);
  k_fp8_gemm<BN><<<static_cast<int>(tiles < num_sms ? tiles : num_sms), kThreads, Tile<BN>::kSmem, st>>>(A);
  return cudaGetLastError();
}

cudaError_t run_gemm_pair(const Fp8GemmArgs& A, int num_sms, cudaStream_t st) {
  static PerDevice pd;
  const cudaError_t e = once_per_device(pd, [](int) {
    return cudaFuncSetAttribute(k_fp8_gemm_pair, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
  });
  if (e != cudaSuccess) return e;
  const int64_t tiles = lm_div_up(A.m, 2 * kTM) * lm_div_up(A.n, kPN);
  const int clusters = static_cast<int>(tiles < num_sms / 2 ? tiles : num_sms / 2);
  k_fp8_gemm_pair<<<2 * clusters, kThreads, kPairSmem, st>>>(A);
  return cudaGetLastError();
}

}  // namespace

// A step of a tile takes about the same time whatever its width, and a launch
// as many tiles' times as its busiest SM (or pair) has tiles.  Measured at K =
// 2048, us a step of one round, square blocks / row groups: CTA pairs 0.54 /
// 0.77, 128 columns 0.47 / 0.52, 64 columns 0.40 / 0.42 (one CTA with 256
// columns was never the best: 0.62 / 0.9).  512 x 5504 x 2048: pairs 13.6 us, 128
// columns 18.8, 64 columns 22.8; 128 x 5504 x 2048: 13.3, 11.0, 10.0.
Fp8Plan fp8_plan(int64_t m, int64_t n, bool b_square, int num_sms) {
  Fp8Plan P = {};
  P.skinny = m <= kSkinnyMax;
  P.box_a = kTM;
  auto cost = [&](int64_t tiles, int units, double square, double rows) {
    return static_cast<double>(lm_div_up(tiles, units)) * (b_square ? square : rows);
  };
  const int64_t tm = lm_div_up(m, kTM);
  const double pair = cost(lm_div_up(m, 2 * kTM) * lm_div_up(n, kPN), num_sms / 2, 0.54, 0.77);
  const double wide = cost(tm * lm_div_up(n, 128), num_sms, 0.47, 0.52);
  const double narrow = cost(tm * lm_div_up(n, 64), num_sms, 0.40, 0.42);
  P.pair = pair <= wide && pair <= narrow;
  P.box_b = P.pair ? kPN / 2 : wide <= narrow ? 128 : 64;
  return P;
}

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& A, const Fp8Plan& P, int num_sms, cudaStream_t st) {
  if (P.skinny) {
    const int grid = static_cast<int>(lm_div_up(A.n, 16)), threads = kSkinnyWarps * 32;
    if (A.m <= 8)
      k_fp8_skinny<1><<<grid, threads, 0, st>>>(A);
    else if (A.m <= 16)
      k_fp8_skinny<2><<<grid, threads, 0, st>>>(A);
    else
      k_fp8_skinny<4><<<grid, threads, 0, st>>>(A);
    return cudaGetLastError();
  }
  if (P.pair) return run_gemm_pair(A, num_sms, st);
  if (P.box_b == 128) return run_gemm<128>(A, num_sms, st);
  return run_gemm<64>(A, num_sms, st);
}

}  // namespace okls
