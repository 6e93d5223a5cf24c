// Device code that the LM-head operators' kernels share (flce_score.h).
#pragma once
#include <stdint.h>

#include "flce_internal.h"
#include "flce_score.h"
#include "ptx.cuh"

namespace flce {

// ------------------------------------------------------------- arithmetic

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// the larger, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// What a group's logits are taken relative to: its largest, or where all are -inf (the
// columns of masked tokens) nothing, so that -inf stays what they are
__device__ __forceinline__ float group_base(float largest) { return largest == -INFINITY ? 0.f : largest; }

// The gradient of one fp32 logit in column j: p from the natural exponential, whose
// argument has no factor to round
__device__ __forceinline__ float dlogit_f32(float z, int64_t j, float c, float inv_t, const ScoreRow& q) {
  const float u = z - q.largest;
  const float t = max_nan(fmaf(u, c, -q.log2_total), -1000.f);
  const float d = expf(max_nan(u * inv_t, -700.f)) * q.inv_total * fmaf(q.b, t, q.a);
  // a row without a gradient has none, whatever its logits are
  return j == q.target ? q.at : q.a == 0.f && q.b == 0.f ? 0.f : d;
}

// ---------------------------------------------------------------- products

// The ring of a CTA of a pair on 256 x 512 tiles: four 64-deep k-blocks of its 128
// rows of A and its 256 columns of B, and a staging tile for each epilogue warpgroup.
constexpr int kRing = 4;
constexpr uint32_t kRingA = kBM * kBK * 2;
constexpr uint32_t kRingB = kBN * kBK * 2;
constexpr uint32_t kRingHalfB = kRingB / 2;
constexpr uint32_t kStagingBytes = 128 * 128;  // 128 rows x 128 bytes
// Each warp stages and copies out its own 32 rows: no warp waits for another
constexpr uint32_t kWarpStaging = kStagingBytes / 4;
constexpr uint32_t kAccumulatorColumns = 512;
// warpgroup 0 loads and issues; two epilogue warpgroups of 128 threads
constexpr int kPairThreads = 384;
constexpr int kWarpgroup = 128;
// registers move from the loading and issuing warpgroup to the epilogues; the split
// must fit what the launch holds (checked on the host)
constexpr uint32_t kRegsControl = 40, kRegsEpilogue = 232;
constexpr int kRegsLaunch = 168;
static_assert(128 * kRegsControl + 256 * kRegsEpilogue <= kPairThreads * kRegsLaunch, "register split");

// Rows of a chunk (off .. off + rows - 1 of the rows that count, of which there are
// *live; live null: all count) that there are.
__device__ __forceinline__ int chunk_rows(const uint32_t* live, int64_t off, int rows) {
  if (!live) return rows;
  const int64_t left = static_cast<int64_t>(*live) - off;
  return static_cast<int>(left < 0 ? 0 : (left < rows ? left : rows));
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint64_t timeout_ns) {
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > timeout_ns) return;
}

// Eight 16-bit columns, the j-th such piece of a row of a 128-row x 128-byte staging
// tile (or a warp's 32 rows of it) in the 128-byte swizzle. Each piece is staged as it is computed: a group's 32
// words at once would take registers that three groups of sums leave no room for.
__device__ __forceinline__ void stage_piece(uint8_t* buf, int row, int j, const uint32_t (&w)[4]) {
  reinterpret_cast<uint4*>(buf + row * 128)[j ^ (row & 7)] = make_uint4(w[0], w[1], w[2], w[3]);
}

// Arrives on a barrier of the pair's even CTA
__device__ __forceinline__ void arrive_even(uint32_t bar, uint32_t rank) {
  if (rank == 0)
    mbar_arrive(bar);
  else
    mbar_arrive_cluster(mapa_shared(bar, 0));
}

// An increase of registers waits until the block's pool holds them
template <class Kernel>
bool registers_fit(Kernel k) {
  cudaFuncAttributes at;
  return cudaFuncGetAttributes(&at, k) == cudaSuccess &&
         at.numRegs * kPairThreads >= static_cast<int>(128 * kRegsControl + 256 * kRegsEpilogue);
}

}  // namespace flce
