// Tile sizes of the 8-bit matrix product and the shared memory that its
// kernels lay out: rings, output boxes, barriers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace okls {
namespace {

constexpr int kTM = 128;         // output rows of a tile
constexpr int kTK = 128;         // depth of a stage: one scale group
constexpr int kThreads = 384;    // 4 control warps, 8 that scale and add
constexpr int kCtlRegs = 40, kAddRegs = 232;
static_assert(128 * kCtlRegs + 256 * kAddRegs <= kThreads * 168, "more registers than the launch holds");
constexpr int kABytes = kTM * kTK;

// The swizzled boxes start at a multiple of 1024 bytes; dynamic shared memory
// is only known to start at a multiple of 16 (the kernels' static variables
// come before it), so a launch asks for what the rounding up may take.
constexpr int kSmemAlign = 1024;

// 8-byte barriers, and the word that takes the TMEM address.
constexpr int ctl_bytes(int barriers) { return barriers * 8 + 8; }

// TMEM buffers of a BN-column step: a power of two, as many as the 512 columns
// hold, at most 4.
template <int BN>
struct Buffers {
  static constexpr int kLog = BN > 128 ? 1 : 2;
  static constexpr int kCount = 1 << kLog;
  __host__ __device__ static constexpr uint32_t at(uint32_t it) { return it & (kCount - 1); }
  __host__ __device__ static constexpr uint32_t parity(uint32_t it) { return (it >> kLog) & 1u; }
};

template <int BN>
struct Tile {
  static constexpr int kBBytes = BN * kTK;
  static constexpr int kBytes = kABytes + kBBytes;
  static constexpr int kRing = BN == 128 ? 6 : 8;
  static constexpr int kCols = BN == 64 ? 256 : 512;  // TMEM columns: the buffers', up to a power of two
  static constexpr int kSlots = 8;                             // scale ring
  static constexpr int kScaleBytes = (kTM + BN) * 4;           // of one step
  // full and empty of both rings and of the TMEM buffers, and the last MMAs'
  static constexpr int kBars = 2 * (kRing + kSlots + Buffers<BN>::kCount) + 1;
  static constexpr int kSmem = kRing * kBytes + kSlots * kScaleBytes + ctl_bytes(kBars) + kSmemAlign;
};

// CTA pairs
constexpr int kOutBox = 32 * 128;  // 32 rows of 64 bf16 results
constexpr int kOutWarp = 2 * kOutBox;
constexpr int kPN = 256;
constexpr int kPairStage = kABytes + kPN / 2 * kTK;
constexpr int kPairRing = 4, kPairSlots = 8, kPairScaleBytes = (kTM + kPN) * 4;
constexpr int kPairBars = 2 * (kPairRing + kPairSlots + Buffers<kPN>::kCount) + 2;
constexpr int kPairSmem =
    kPairRing * kPairStage + 8 * kOutWarp + kPairSlots * kPairScaleBytes + ctl_bytes(kPairBars) + kSmemAlign;

constexpr int kMaxSmem = 227 * 1024;  // of one CTA
static_assert(Tile<64>::kSmem <= kMaxSmem && Tile<128>::kSmem <= kMaxSmem && kPairSmem <= kMaxSmem,
              "more shared memory than a CTA has");

}  // namespace
}  // namespace okls
