// The product z = x Wt of the LM-head operators (flce_score.h) on tcgen05, with
// what becomes of z in its epilogue: the statistics of each row's softmax and
// entropy (and z at picked columns), or the gradient of the logits.
//
// 256 x 512 tiles on CTA pairs, as the loss runs them: per 16-deep step two
// tcgen05.mma.cta_group::2 (M 256, N 256) share A through the collector, a
// four-stage ring of TMA loads, the 512 accumulator columns filling TMEM. The
// accumulator is handed back in two halves of 256 columns. An epilogue warpgroup has
// two groups of 64 columns in each half. For the statistics alone and the gradient it
// takes three of the four into registers (192 of its 232 a thread), hands the first
// half back, computes the first group's exponentials, takes the fourth into its
// registers and hands the second half back: so the accumulator is held for a quarter
// of the arithmetic, while the next tile's first products run on the half that is
// free. (Two groups at a time held it for half of it: 104 us instead of 90 at 2048 x
// 1024 x 32000.) The loss's epilogue rounds z to bf16 to hold all four at once; here
// every sum is of the fp32 accumulators, since log probabilities are compared with
// each other. What is stored goes out by the warp: 32 rows of 64 columns in its own
// staging tile, one TMA store, no barrier among warps (by the warpgroup the gradient
// at 2048 x 64 x 32000 took 90 us instead of 49, at 1024 columns of x 121 instead of
// 96, the stored statistics 106 instead of 104).
//
// Measured, us for 2048 rows x H x 32000 columns, H = 64 / 1024 / 4096: statistics 45 /
// 90 / 282, with the logits stored 57 / 104 / 295, with 64 picked columns 59 at 64, the
// gradient 49 / 96 / 290; 4096 x 4096 x 128256: 2190 / 2400 / 2380 (1.96 to 1.8
// PFLOP/s, the power cap).
//
// Mathematics. With c = log2(e) / temperature and, per 64 columns, the largest m:
// y = (z - m) c, and the sums l of 2^y and s of y 2^y give the log-sum-exp and
// E[y] of the row (joined over the columns by flce_score.cu). The gradient of a
// row is d = p (a + b log2 p) with p = 2^((z - M) c - log2 L), but for the target's
// column: ScoreRow.
//
// What bounds it: the tensor cores (and the power cap) from some 256 rows on,
// below that the reads of W. The exponentials take 4096 of a tile's cycles at 16 a
// clock, against some 1060 for each 64 of H.
//
// Every wait is bounded (ScoreGemmArgs.timeout_ns); one that runs out records
// FLCE_ERR_TIMEOUT, the CTA waits for its own loads and products in flight, frees
// its TMEM and returns.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "flce_score.cuh"

namespace flce {
namespace {

constexpr uint32_t kSmemBytes = 1024 + kRing * (kRingA + kRingB) + 2 * kStagingBytes + (2 * kRing + 4) * 8 + 16;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

// 64 columns from two 32-register loads
struct Group {
  uint32_t (&lo)[32];
  uint32_t (&hi)[32];
};

// -inf, which adds nothing, in this thread's lane of a column of the accumulator
__device__ __forceinline__ void tmem_clear(uint32_t taddr) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(0xFF800000u) : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The largest of 64 columns of this thread's row
__device__ __forceinline__ float group_max(Group g) {
  float m4[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) m4[j] = max_nan(__uint_as_float(g.lo[j]), __uint_as_float(g.hi[j]));
#pragma unroll
  for (int i = 4; i < 32; ++i)
    m4[i & 3] = max_nan(m4[i & 3], max_nan(__uint_as_float(g.lo[i]), __uint_as_float(g.hi[i])));
  return max_nan(max_nan(m4[0], m4[1]), max_nan(m4[2], m4[3]));
}

// Their statistics relative to it, and z - m staged as fp16
template <bool STORE>
__device__ __forceinline__ void group_stats(Group g, float m, float c, float2* part, float* part_s, bool rvalid,
                                            uint8_t* buf, int row) {
  float l[4] = {0.f, 0.f, 0.f, 0.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  const float base = group_base(m);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t (&r)[32] = half ? g.hi : g.lo;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int i = 8 * j; i < 8 * j + 8; i += 2) {
        const float d0 = __uint_as_float(r[i]) - base, d1 = __uint_as_float(r[i + 1]) - base;
        // at -1000 the exponential is 0 and y 2^y is too, which -inf would make NaN
        const float y0 = max_nan(d0 * c, -1000.f), y1 = max_nan(d1 * c, -1000.f);
        const float e0 = ex2(y0), e1 = ex2(y1);
        l[i & 3] += e0;
        l[(i + 1) & 3] += e1;
        s[i & 3] = fmaf(y0, e0, s[i & 3]);
        s[(i + 1) & 3] = fmaf(y1, e1, s[(i + 1) & 3]);
        // 11 bits of a distance to the group's largest: what the gradient's
        // exponentials and the search for alternatives need of it
        const __half2 h = __floats2half2_rn(d0, d1);
        w[(i & 7) / 2] = *reinterpret_cast<const uint32_t*>(&h);
      }
      if (STORE) stage_piece(buf, row, 4 * half + j, w);
    }
  }
  if (rvalid) {
    *part = make_float2(m, (l[0] + l[1]) + (l[2] + l[3]));
    *part_s = (s[0] + s[1]) + (s[2] + s[3]);
  }
}

// The gradient of 64 columns of this thread's row staged as bf16 (but for the target's
// entry, which launch_score_target writes: found here, it took code that the
// instruction cache did not hold)
__device__ __forceinline__ void group_gradient(Group g, const ScoreRow& q, float c, uint8_t* buf, int row) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t (&r)[32] = half ? g.hi : g.lo;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = max_nan(fmaf(__uint_as_float(r[8 * j + i]) - q.largest, c, -q.log2_total), -1000.f);
        v[i] = ex2(t) * fmaf(q.b, t, q.a);
      }
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      stage_piece(buf, row, 4 * half + j, w);
    }
  }
  // a row without a gradient, whatever its logits are: 0 times them may be NaN
  if (q.a == 0.f && q.b == 0.f) {
    const uint32_t zero[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
    for (int j = 0; j < 8; ++j) stage_piece(buf, row, j, zero);
  }
}

// This thread's value of column i of its group, i by thread: registers cannot be
// indexed, so halves are chosen between bit by bit (63 selections).
template <int N>
__device__ __forceinline__ uint32_t column_of(const uint32_t* r, int i) {
  if constexpr (N == 1) {
    return r[0];
  } else {
    const uint32_t lo = column_of<N / 2>(r, i), hi = column_of<N / 2>(r + N / 2, i);
    return (i & (N / 2)) ? hi : lo;
  }
}

// z at the picked ones of this thread's 64 columns from cg on: entries first .. end - 1
// are its part's, of which few are in it (64 a row of 128256: one in 30 threads has one).
__device__ __forceinline__ void pick_columns(Group g, const ScoreGemmArgs& a, int first, int end, int64_t grow, int cg) {
  for (int e = first; __any_sync(0xffffffffu, e < end); ++e) {
    const int2 en = e < end ? a.entries[grow * a.k + e] : make_int2(-1, 0);
    const bool here = en.x >= cg && en.x < cg + 64;
    if (!__any_sync(0xffffffffu, here)) continue;
    const int i = en.x - cg;
    const uint32_t lo = column_of<32>(g.lo, i), hi = column_of<32>(g.hi, i);
    if (here) a.picked[grow * a.k + en.y] = __uint_as_float((i & 32) ? hi : lo);
  }
}

template <int MODE, bool STORE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    score_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmO, const ScoreGemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kRing * kRingA;
  uint8_t* sE = sB + kRing * kRingB;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sE + 2 * kStagingBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kRing + 4);

  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kRing + s); };
  const uint32_t tfull_bar = bar0 + 8u * (2 * kRing);
  const uint32_t tempty0_bar = bar0 + 8u * (2 * kRing + 1);
  const uint32_t tempty1_bar = bar0 + 8u * (2 * kRing + 2);
  const uint32_t drain_bar = bar0 + 8u * (2 * kRing + 3);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: the CTA that issues the products
  const int pair = static_cast<int>(cluster_id_x());
  const int npairs = static_cast<int>(num_clusters_x());

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(full_bar(s), 1);   // used in CTA 0: both CTAs' loads land here
      mbar_init(empty_bar(s), 1);  // each CTA's own, released by the products' commit
    }
    mbar_init(tfull_bar, 1);
    mbar_init(tempty0_bar, 2 * 2 * kWarpgroup);  // used in CTA 0: both CTAs' two epilogues
    mbar_init(tempty1_bar, 2 * 2 * kWarpgroup);
    mbar_init(drain_bar, 1);
    fence_mbar_init();
    fence_proxy_async_smem();
    tma_prefetch_map(&tmA);
    tma_prefetch_map(&tmB);
    tma_prefetch_map(&tmO);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kAccumulatorColumns);
    tmem_relinquish_pair();
  }
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are there before the other uses them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // rows fastest: the pairs that run together share columns of W
  const int rows = max(chunk_rows(a.live, a.off, a.rows), a.least);
  const int num_m = (rows + 2 * kBM - 1) / (2 * kBM);
  const int units = num_m * a.num_n;
  if (warp < 4) {
    warpgroup_regs_dec<kRegsControl>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- loads
      uint32_t n_issued = 0;
      bool failed = false;
      for (int u = pair; u < units && !failed; u += npairs) {
        const int mA = (u % num_m) * 2 * kBM + static_cast<int>(rank) * kBM;
        const int nB = (u / num_m) * 2 * kBN + static_cast<int>(rank) * (kBN / 2);
        for (int kb = 0; kb < a.kb_total; ++kb) {
          const uint32_t stage = n_issued % kRing;
          if (!mbar_wait_bounded_cluster(empty_bar(stage), ((n_issued / kRing) & 1u) ^ 1u, a.ctrl, a.timeout_ns)) {
            failed = true;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2 * (kRingA + kRingB));
          const uint32_t fb = mapa_shared(full_bar(stage), 0);
          const uint32_t sb = smem_u32(sB + stage * kRingB);
          tma_load_2d_pair(smem_u32(sA + stage * kRingA), &tmA, fb, kb * kBK, mA);
          tma_load_2d_pair(sb, &tmB, fb, kb * kBK, nB);
          tma_load_2d_pair(sb + kRingHalfB, &tmB, fb, kb * kBK, nB + kBN);
          ++n_issued;
        }
      }
      if (failed && rank == 0) {
        const uint32_t first = n_issued > kRing ? n_issued - kRing : 0;
        for (uint32_t i = first; i < n_issued; ++i) drain_wait(full_bar(i % kRing), (i / kRing) & 1u, a.timeout_ns);
      }
    } else if (warp == 1 && lane == 0 && rank == 0) {
      // ------------------------------------------------------- products
      constexpr uint32_t idesc = idesc_bf16_f32(2 * kBM, kBN, 0, 0);
      uint32_t n_consumed = 0;
      bool issued = false, failed = false;
      // the four steps of a k-block: both halves sharing A (half < 0), or one half
      auto products = [&](int stage, int half, bool first) {
        const uint32_t sa = smem_u32(sA + stage * kRingA);
        const uint32_t sb = smem_u32(sB + stage * kRingB);
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k) {
          const uint64_t ad = smem_desc_sw128(sa + 32u * k, 16u, 1024u);
          const uint64_t bd0 = smem_desc_sw128(sb + 32u * k, 16u, 1024u);
          const uint64_t bd1 = smem_desc_sw128(sb + kRingHalfB + 32u * k, 16u, 1024u);
          const uint32_t add = (!first || k > 0) ? 1u : 0u;
          if (half < 0) {
            tc_mma_bf16_pair_a_fill(tmem_base, ad, bd0, idesc, add);
            tc_mma_bf16_pair_a_lastuse(tmem_base + kBN, ad, bd1, idesc, add);
          } else {
            tc_mma_bf16_pair(tmem_base + half * kBN, ad, half ? bd1 : bd0, idesc, add);
          }
        }
      };
      int it = 0;
      for (int u = pair; u < units && !failed; u += npairs, ++it) {
        const uint32_t tph = (it & 1) ^ 1u;
        if (!mbar_wait_bounded_cluster(tempty0_bar, tph, a.ctrl, a.timeout_ns)) {
          failed = true;
          break;
        }
        tc_fence_after();
        // while the second half is still being read, the first half's products
        // of the k-blocks that are there (their stages stay until the second
        // half's products have read them too)
        int ahead = 0;
        const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
        for (uint32_t spin = 0; !mbar_try_wait_cluster(tempty1_bar, tph); ++spin) {
          if (ahead < kRing && ahead < a.kb_total) {
            const uint32_t n = n_consumed + static_cast<uint32_t>(ahead);
            if (mbar_try_wait_cluster(full_bar(n % kRing), (n / kRing) & 1u)) {
              tc_fence_after();
              products(n % kRing, 0, ahead == 0);
              issued = true;
              ++ahead;
              continue;
            }
          }
          if ((spin & 63u) == 0u && (ld_volatile_u32(a.ctrl) != 0u || globaltimer_ns() - t0 > a.timeout_ns)) {
            atomicCAS(a.ctrl, 0u, kErrTimeout);
            failed = true;
            break;
          }
        }
        if (failed) break;
        tc_fence_after();
        for (int j = 0; j < ahead; ++j) {
          const int stage = (n_consumed + static_cast<uint32_t>(j)) % kRing;
          products(stage, 1, j == 0);
          tc_commit_pair_multicast(empty_bar(stage), 0x3);
        }
        n_consumed += static_cast<uint32_t>(ahead);
        for (int kb = ahead; kb < a.kb_total; ++kb) {
          const int stage = n_consumed % kRing;
          if (!mbar_wait_bounded_cluster(full_bar(stage), (n_consumed / kRing) & 1u, a.ctrl, a.timeout_ns)) {
            failed = true;
            break;
          }
          tc_fence_after();
          products(stage, -1, kb == 0);
          issued = true;
          tc_commit_pair_multicast(empty_bar(stage), 0x3);
          ++n_consumed;
        }
        if (failed) break;
        tc_commit_pair_multicast(tfull_bar, 0x3);
      }
      if (failed && issued) {
        tc_commit_pair(drain_bar);
        drain_wait(drain_bar, 0, a.timeout_ns);
      }
    }
  } else {
    warpgroup_regs_inc<kRegsEpilogue>();
    // ---------------------------------------------------------- epilogue
    const int grp = (warp - 4) >> 2;
    const int wq = warp & 3;               // TMEM lanes 32 wq .. 32 wq + 31
    const int row = wq * 32 + lane;
    const uint32_t bar = 1u + static_cast<uint32_t>(grp);
    uint8_t* buf = sE + (warp - 4) * kWarpStaging;
    const float c = a.c;
    int it = 0;
    for (int u = pair; u < units; u += npairs, ++it) {
      const int m0 = (u % num_m) * 2 * kBM + static_cast<int>(rank) * kBM;
      const int n0 = (u / num_m) * 2 * kBN;
      const int grow = m0 + row;
      const bool rvalid = grow < rows;
      ScoreRow q{0.f, 0.f, 0.f, 0.f, 0.f, -1, 0.f};
      if (MODE == kScoreGradient && rvalid) q = a.row[grow];
      int first[2] = {0, 0}, end[2] = {0, 0};  // this warpgroup's part of either half
      if (MODE == kScorePick && rvalid) {
        const uint2 pp = a.parts[static_cast<int64_t>(grow) * a.num_n + u / num_m];
        const uint64_t at = static_cast<uint64_t>(pp.x) | (static_cast<uint64_t>(pp.y) << 32);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          first[half] = static_cast<int>(at >> (9 * (2 * half + grp))) & 511;
          end[half] = static_cast<int>(at >> (9 * (2 * half + grp + 1))) & 511;
        }
      }
      const bool ok = mbar_wait_bounded_cluster(tfull_bar, it & 1, a.ctrl, a.timeout_ns);
      if (named_bar_or(bar, kWarpgroup, !ok)) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(wq * 32) << 16);
      const size_t prow = static_cast<size_t>(grow) * a.groups;
      // tile column of group i: two in each half
      auto col_of = [&](int i) { return (i < 2 ? 0 : kBN) + grp * 128 + (i & 1) * 64; };
      // two ahead where storing or picking takes registers too: three left too few for
      // the arithmetic to overlap itself (68 us instead of 56 at 2048 x 64 x 32000)
      constexpr int kAhead = MODE == kScoreGradient || (MODE == kScoreStats && !STORE) ? 3 : 2;
      uint32_t r[kAhead][2][32];
      auto load = [&](int i, uint32_t (&to)[2][32]) {
        if (n0 + col_of(i) < a.cols) {  // uniform
          tmem_ld_32x32b_x32(tbase + col_of(i), to[0]);
          tmem_ld_32x32b_x32(tbase + col_of(i) + 32, to[1]);
        }
      };
      auto release = [&](uint32_t b) {
        tc_fence_before();
        arrive_even(b, rank);
      };
      auto process = [&](int i, uint32_t (&from)[2][32]) {
        const int cg = n0 + col_of(i);
        if (cg >= a.cols) return;  // uniform
        const Group v{from[0], from[1]};
        if constexpr (MODE == kScorePick) pick_columns(v, a, first[i >> 1], end[i >> 1], grow, cg);
        float m = 0.f;
        if constexpr (MODE != kScoreGradient) m = group_max(v);
        if constexpr (STORE) {
          // the copy that still reads the warp's staging tile
          if (lane == 0) bulk_wait_group_read<0>();
          __syncwarp();
        }
        if constexpr (MODE == kScoreGradient) {
          group_gradient(v, q, c, buf, lane);
        } else {
          group_stats<STORE>(v, m, c, a.partials + prow + cg / 64, a.part_s + prow + cg / 64, rvalid, buf, lane);
        }
        if constexpr (STORE) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmO, smem_u32(buf), cg, m0 + 32 * wq);
            bulk_commit_group();
          }
          __syncwarp();
        }
      };
      if (MODE != kScoreGradient && n0 + 2 * kBN > a.cols) {
        // a ragged last group: its columns past the last become -inf in place (masks
        // on registers would be code in every tile's way)
#pragma unroll 1
        for (int i = 0; i < 4; ++i)
#pragma unroll 1
          for (int col = max(a.cols - n0, col_of(i)); col < col_of(i) + 64 && n0 + col_of(i) < a.cols; ++col)
            tmem_clear(tbase + col);
        tmem_st_wait();
      }
      auto ready = [&](uint32_t (&v)[2][32]) {
        tmem_regs_ready(v[0]);
        tmem_regs_ready(v[1]);
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) load(i, r[i]);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < kAhead; ++i) ready(r[i]);
      release(tempty0_bar);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        process(i, r[i % kAhead]);
        if (i + kAhead < 4) {
          load(i + kAhead, r[i % kAhead]);
          tmem_ld_wait();
          ready(r[i % kAhead]);
          if (i + kAhead == 3) release(tempty1_bar);
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();
  }

  __syncwarp();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the pair's products may touch its memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kAccumulatorColumns);
  }
}

template <int MODE, bool STORE>
cudaError_t launch(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& to, const ScoreGemmArgs& args,
                   int pairs, cudaStream_t s) {
  auto kern = score_gemm_kernel<MODE, STORE>;
  static const bool fits = registers_fit(kern);
  if (!fits) return cudaErrorInvalidConfiguration;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
  if (e != cudaSuccess) return e;
  kern<<<2 * pairs, kPairThreads, kSmemBytes, s>>>(ta, tb, to, args);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_score_gemm(int mode, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o,
                              const ScoreGemmArgs& args, int pairs, cudaStream_t s) {
  switch (mode) {
    case kScoreStats:
      return args.store ? launch<kScoreStats, true>(a, b, o, args, pairs, s)
                        : launch<kScoreStats, false>(a, b, o, args, pairs, s);
    case kScorePick:
      return args.store ? launch<kScorePick, true>(a, b, o, args, pairs, s)
                        : launch<kScorePick, false>(a, b, o, args, pairs, s);
    case kScoreGradient: return launch<kScoreGradient, true>(a, b, o, args, pairs, s);
    default: return cudaErrorInvalidValue;
  }
}

int score_gemm_max_clusters() {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kPairThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaFuncSetAttribute(score_gemm_kernel<kScoreStats, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kSmemBytes)) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, score_gemm_kernel<kScoreStats, false>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

}  // namespace flce
