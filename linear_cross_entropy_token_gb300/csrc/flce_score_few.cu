// The product z = x Wt of a few tokens (a decoding batch) with the statistics of each
// row's softmax and entropy: what flce_score_gemm.cu does for many.
//
// W's bytes are all there is to it (1.05 GB at 128256 x 4096, 155 us at the measured
// copy rate), so the operands change sides: 128 rows of W are the 128 rows of a
// tcgen05.mma, the tokens (padded to 16) its columns. A CTA streams its tiles of W
// through a ring that takes all the shared memory (some 190 KB in flight on each SM),
// x comes from L2 with every block of W, and a product costs the tensor cores next to
// nothing. On 256 x 512 tiles of CTA pairs the same call computes 256 rows of tokens,
// waits for its products as much as for W and leaves a fifth of the pairs idle in
// its last round.
//
// The k-blocks of a sum go to up to four accumulators in turn: the tensor cores cut
// running sums off, the less the smaller they are, and fp32 adds the parts: log
// probabilities of 65 rows of 5608 columns are 2.5e-7 off instead of 8e-7, in the same
// time.
//
// A tile's accumulator has a column of W a lane and a token a register; the epilogue
// turns it over in shared memory, and four threads take 64 columns of a token.
//
// Measured at 4096 x 128256: one token 180 us (5.8 TB/s) where the pair tiles take 238,
// 128 tokens 193 where they take 200. Time grows with W's bytes at 6.5 TB/s, above some
// 20 us that a cold start takes (much of it the write-back of what L2 held). Even shares
// of k-blocks a CTA instead of whole tiles, joined where two meet, gained nothing: 181
// us, and at 64 tokens 7 more.
#include <cuda_fp16.h>

#include <algorithm>

#include "flce_score.cuh"

namespace flce {
namespace {

constexpr int kTileRows = 128;                    // of W
constexpr uint32_t kWBytes = kTileRows * kBK * 2;
constexpr int kFewThreads = 192;                  // loads, products, four epilogue warps
constexpr int kMaxStages = 12;
constexpr int kTurnStride = kTileRows + 4;        // floats between tokens: 16-byte rows, no bank twice
constexpr uint32_t kMostSmem = 232448;

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void regs_ready(uint32_t (&r)[16]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

// M 128, N tokens (a multiple of 16, at most 256), both operands along K
__device__ __forceinline__ uint32_t few_idesc(int tokens) {
  return idesc_bf16_f32(kTileRows, 0, 0, 0) | (static_cast<uint32_t>(tokens >> 3) << 17);
}

template <bool STORE>
__global__ void __launch_bounds__(kFewThreads, 1)
    score_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const ScoreFewArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t x_bytes = static_cast<uint32_t>(a.padded) * kBK * 2, stage_bytes = kWBytes + x_bytes;
  const uint32_t stages = static_cast<uint32_t>(a.stages);
  float* turn = reinterpret_cast<float*>(smem + stages * stage_bytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(turn + a.padded * kTurnStride);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxStages + 5);

  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (kMaxStages + s); };
  auto tfull_bar = [&](int acc) { return bar0 + 8u * (2 * kMaxStages + acc); };
  auto tempty_bar = [&](int acc) { return bar0 + 8u * (2 * kMaxStages + 2 + acc); };
  const uint32_t drain_bar = bar0 + 8u * (2 * kMaxStages + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int acc = 0; acc < 2; ++acc) {
      mbar_init(tfull_bar(acc), 1);
      mbar_init(tempty_bar(acc), kWarpgroup);
    }
    mbar_init(drain_bar, 1);
    fence_mbar_init();
    fence_proxy_async_smem();
    tma_prefetch_map(&tmW);
    tma_prefetch_map(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), static_cast<uint32_t>(a.tmem_columns));
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------- loads
      uint32_t stage = 0, phase = 1, issued = 0;
      bool failed = false;
      for (int u = blockIdx.x; u < a.tiles && !failed; u += gridDim.x)
        for (int kb = 0; kb < a.kb_total; ++kb) {
          if (!mbar_wait_bounded(empty_bar(stage), phase, a.ctrl, a.timeout_ns)) {
            failed = true;
            break;
          }
          mbar_arrive_expect_tx(full_bar(stage), stage_bytes);
          const uint32_t at = smem_u32(smem + stage * stage_bytes);
          tma_load_2d(at, &tmW, full_bar(stage), kb * kBK, u * kTileRows);
          tma_load_2d(at + kWBytes, &tmX, full_bar(stage), kb * kBK, 0);
          ++issued;
          if (++stage == stages) stage = 0, phase ^= 1u;
        }
      if (failed)  // the loads in flight land before the CTA goes away
        for (uint32_t i = issued > stages ? issued - stages : 0; i < issued; ++i)
          drain_wait(full_bar(i % stages), (i / stages) & 1u, a.timeout_ns);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------- products
      const uint32_t idesc = few_idesc(a.padded);
      uint32_t stage = 0, phase = 0;
      bool issued = false, failed = false;
      int it = 0;
      for (int u = blockIdx.x; u < a.tiles && !failed; u += gridDim.x, ++it) {
        const int acc = it & 1;
        if (!mbar_wait_bounded(tempty_bar(acc), ((it >> 1) & 1u) ^ 1u, a.ctrl, a.timeout_ns)) {
          failed = true;
          break;
        }
        tc_fence_after();
        int part = 0;
        for (int kb = 0; kb < a.kb_total; ++kb) {
          if (!mbar_wait_bounded(full_bar(stage), phase, a.ctrl, a.timeout_ns)) {
            failed = true;
            break;
          }
          tc_fence_after();
          const uint32_t at = smem_u32(smem + stage * stage_bytes);
          const uint32_t to = tmem_base + static_cast<uint32_t>((acc * a.parts + part) * a.padded);
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            tc_mma_bf16(to, smem_desc_sw128(at + 32u * k, 16u, 1024u), smem_desc_sw128(at + kWBytes + 32u * k, 16u, 1024u), idesc,
                        (kb >= a.parts || k > 0) ? 1u : 0u);
          issued = true;
          tc_commit(empty_bar(stage));
          if (++stage == stages) stage = 0, phase ^= 1u;
          if (++part == a.parts) part = 0;
        }
        if (failed) break;
        tc_commit(tfull_bar(acc));
      }
      if (failed && issued) {
        tc_commit(drain_bar);
        drain_wait(drain_bar, 0, a.timeout_ns);
      }
    }
  } else {
    // ---------------------------------------------------------- epilogue
    const int wq = warp & 3;  // TMEM lanes 32 wq .. 32 wq + 31
    const int thread = threadIdx.x - 64;
    const int q = thread & 3;  // of the four threads of a token's 64 columns
    int it = 0;
    for (int u = blockIdx.x; u < a.tiles; u += gridDim.x, ++it) {
      const int acc = it & 1;
      const bool ok = mbar_wait_bounded(tfull_bar(acc), (it >> 1) & 1u, a.ctrl, a.timeout_ns);
      if (named_bar_or(1, kWarpgroup, !ok)) break;  // and the last tile's have been read
      tc_fence_after();
      const uint32_t from = tmem_base + (static_cast<uint32_t>(wq * 32) << 16) + static_cast<uint32_t>(acc * a.parts * a.padded);
      for (int n = 0; n < a.padded; n += 16) {
        uint32_t r[16];
        tmem_ld_x16(from + n, r);
        tmem_ld_wait();
        regs_ready(r);
        for (int part = 1; part < a.parts; ++part) {
          uint32_t more[16];
          tmem_ld_x16(from + part * a.padded + n, more);
          tmem_ld_wait();
          regs_ready(more);
#pragma unroll
          for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) + __uint_as_float(more[i]));
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) turn[(n + i) * kTurnStride + wq * 32 + lane] = __uint_as_float(r[i]);
      }
      tc_fence_before();
      mbar_arrive(tempty_bar(acc));
      named_bar_sync(1, kWarpgroup);
      const int tasks = 2 * a.rows;  // (token, 64 columns)
      // the threads of a warp stay together: shuffles below
      for (int first = 0; first < tasks; first += kWarpgroup / 4) {
        const int task = first + (thread >> 2), token = task >> 1, g = u * 2 + (task & 1);
        const int64_t col = static_cast<int64_t>(g) * kScoreGroup + 16 * q;
        const bool there = task < tasks && g < a.groups;
        float z[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = there ? *reinterpret_cast<const float4*>(turn + token * kTurnStride + (task & 1) * kScoreGroup + 16 * q + 4 * i)
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
          z[4 * i] = v.x, z[4 * i + 1] = v.y, z[4 * i + 2] = v.z, z[4 * i + 3] = v.w;
        }
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (col + i >= a.cols) z[i] = -INFINITY;  // adds nothing
          m = max_nan(m, z[i]);
        }
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const float base = group_base(m);
        float l = 0.f, s = 0.f;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float d0 = z[i] - base, d1 = z[i + 1] - base;
          const float y0 = max_nan(d0 * a.c, -1000.f), y1 = max_nan(d1 * a.c, -1000.f);
          const float e0 = ex2(y0), e1 = ex2(y1);
          l += e0 + e1;
          s = fmaf(y0, e0, fmaf(y1, e1, s));
          const __half2 h = __floats2half2_rn(d0, d1);
          w[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          l += __shfl_xor_sync(0xffffffffu, l, o);
          s += __shfl_xor_sync(0xffffffffu, s, o);
        }
        if (!there) continue;
        if (STORE) {  // the padding behind the last column is the row's own (ldv)
          uint4* to = reinterpret_cast<uint4*>(a.z + token * a.ldv + col);
          to[0] = make_uint4(w[0], w[1], w[2], w[3]);
          to[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
        if (q == 0) {
          const int64_t at = static_cast<int64_t>(token) * a.groups + g;
          a.partials[at] = make_float2(m, l);
          a.part_s[at] = s;
        }
      }
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, static_cast<uint32_t>(a.tmem_columns));
  }
}

template <bool STORE>
cudaError_t launch(const CUtensorMap& w, const CUtensorMap& x, const ScoreFewArgs& args, uint32_t bytes, int blocks,
                   cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(score_few_kernel<STORE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kMostSmem));
  if (e != cudaSuccess) return e;
  score_few_kernel<STORE><<<blocks, kFewThreads, bytes, s>>>(w, x, args);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_score_few(const CUtensorMap& w, const CUtensorMap& x, ScoreFewArgs args, int sms, cudaStream_t s) {
  const uint32_t stage = kWBytes + static_cast<uint32_t>(args.padded) * kBK * 2;
  const uint32_t rest = 1024 + static_cast<uint32_t>(args.padded) * kTurnStride * 4 + (2 * kMaxStages + 5) * 8 + 16;
  args.stages = static_cast<int32_t>(std::min<uint32_t>(kMaxStages, (kMostSmem - rest) / stage));
  args.tmem_columns = 32;
  while (args.tmem_columns < 2 * args.parts * args.padded) args.tmem_columns *= 2;
  args.tiles = (args.cols + kTileRows - 1) / kTileRows;
  const uint32_t bytes = rest + static_cast<uint32_t>(args.stages) * stage;
  const int blocks = std::min(args.tiles, sms);
  return args.z ? launch<true>(w, x, args, bytes, blocks, s) : launch<false>(w, x, args, bytes, blocks, s);
}

}  // namespace flce
