// The backward products of the LM-head operators (flce_score.h): from a chunk's
// gradient of the logits d (rows x V, bf16), dx = d W and dW (+)= dt x, in one
// persistent launch on 256 x 512 tiles of CTA pairs.
//
// Units of work are tiles: dx's first (long: a part of V's k-blocks each), then dW's
// (short: the chunk's rows), handed out from a counter, so pairs that run out of long
// ones fill in with short ones, as in the loss's backward. What is different here:
//
// - How many rows count is read on the device. Rows that do not (ignored tokens)
//   have been left out of d and x, and the products are as much smaller; a chunk
//   without any is no work at all. 16384 x 4096 x 128256 with every other token
//   ignored: 20.4 ms a policy step instead of 36.5.
// - dW may be bf16. The last chunk's tiles then add what the earlier chunks summed
//   in fp32, round once and store, instead of adding to the fp32 sum for a pass over
//   all of it to read and round: 10 bytes an element less.
// - A tile whose second 256 columns lie beyond the last is computed on its first half
//   alone (H up to 256, or a ragged end).
// - Either product alone, where only one gradient is wanted.
//
// What bounds it: the tensor cores under the power cap; for short chunks dW's bytes.
// Every wait is bounded, as in flce_score_gemm.cu.
#include <algorithm>

#include <cuda_bf16.h>

#include "flce_score.cuh"

namespace flce {
namespace {

constexpr int kUnitDepth = 4;   // units published ahead
// who reads a published unit: the even CTA's issuer, the odd CTA's loader and the
// leaders of four epilogue warpgroups
constexpr int kUnitReaders = 6;
constexpr uint32_t kSmemBytes = 1024 + kRing * (kRingA + kRingB) + 2 * kStagingBytes + (2 * kRing + 3 + 2 * kUnitDepth) * 8 +
                                16 + 4 * kUnitDepth;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

struct Unit {
  int dw;      // 0: dx
  int m, n, s;
};

// Everything that follows from how many rows there are
struct Shape {
  int rows, units0, units;
  int m0, n;          // dx: tiles of rows; both: tiles of columns
  int kb_rows;        // k-blocks of dW
  bool last;          // dW: no later chunk has rows
};

__device__ __forceinline__ Unit unit_of(const ScoreBackwardArgs& a, const Shape& p, int u) {
  Unit r;
  r.dw = u >= p.units0;
  if (r.dw) {
    u -= p.units0;
    r.n = u % p.n;
    r.m = u / p.n;
    r.s = 0;
    return r;
  }
  // groups of group_m tile rows sweep the columns, rows fastest: units that run
  // together share both operands
  const int mn = p.m0 * p.n;
  r.s = u / mn;
  const int w = u - r.s * mn, per = a.group_m * p.n, g = w / per, i = w - g * per;
  const int rows = min(a.group_m, p.m0 - g * a.group_m);
  r.m = g * a.group_m + i % rows;
  r.n = i / rows;
  return r;
}

// fp32 out: 32 columns at a time, read six such groups ahead of the copies
__device__ __forceinline__ void epilogue_f32(const CUtensorMap* map, bool add, int cols, uint32_t tbase, int m0, int n0,
                                             int s, uint8_t* buf, int row, bool leader, uint32_t bar, uint32_t free_bar,
                                             uint32_t rank) {
  constexpr int kGroups = kBN / 32, kAhead = 6;
  if (n0 >= cols) {  // uniform
    tc_fence_before();
    arrive_even(free_bar, rank);
    return;
  }
  uint32_t r[kAhead][32];
#pragma unroll
  for (int g = 0; g < kAhead; ++g) tmem_ld_32x32b_x32(tbase + g * 32, r[g]);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    uint32_t (&cur)[32] = r[g % kAhead];
    tmem_ld_wait();
    tmem_regs_ready(cur);
    if (g == kGroups - kAhead) {
      tc_fence_before();
      arrive_even(free_bar, rank);
    }
    const int c0 = n0 + g * 32;
    if (c0 < cols) {  // uniform
      if (leader) bulk_wait_group_read<0>();
      named_bar_sync(bar, kWarpgroup);
#pragma unroll
      for (int j = 0; j < 8; ++j) stage_piece(buf, row, j, *reinterpret_cast<const uint32_t(*)[4]>(&cur[4 * j]));
      fence_proxy_async_smem();
      named_bar_sync(bar, kWarpgroup);
      if (leader) {
        if (add)
          tma_reduce_add_3d(map, smem_u32(buf), c0, m0, s);
        else
          tma_store_3d(map, smem_u32(buf), c0, m0, s);
        bulk_commit_group();
      }
      __syncwarp();
    }
    if (g + kAhead < kGroups) tmem_ld_32x32b_x32(tbase + (g + kAhead) * 32, cur);
  }
}

// bf16 out: acc (+ the earlier chunks' fp32 sum), rounded once; 64 columns at a time.
// The earlier sum is fetched to L2 while the products still run (prefetch_sum), and
// its reads are all under way before a group's first is needed: read piece by piece
// from HBM it held the accumulator for 30 us a tile.
__device__ __forceinline__ const float* sum_row(const float* prior, int rows, int64_t H, int m) {
  return prior != nullptr && m < rows ? prior + static_cast<int64_t>(m) * H : nullptr;
}

__device__ __forceinline__ void prefetch_sum(const float* from, int n0, int cols) {
  if (from == nullptr) return;
#pragma unroll
  for (int c = 0; c < kBN; c += 32)
    if (n0 + c < cols) asm volatile("prefetch.global.L2 [%0];" ::"l"(from + n0 + c));
}

__device__ __forceinline__ void epilogue_bf16(const CUtensorMap* map, const float* from, int cols, uint32_t tbase, int m0,
                                              int n0, uint8_t* buf, int row, bool leader, uint32_t bar, uint32_t free_bar,
                                              uint32_t rank) {
  constexpr int kGroups = kBN / 64;
  auto release = [&] {
    tc_fence_before();
    arrive_even(free_bar, rank);
  };
  if (n0 >= cols) {  // uniform
    release();
    return;
  }
  uint32_t r[2][2][32];
  auto load = [&](int g, uint32_t (&to)[2][32]) {
    tmem_ld_32x32b_x32(tbase + g * 64, to[0]);
    tmem_ld_32x32b_x32(tbase + g * 64 + 32, to[1]);
  };
  auto process = [&](int g, uint32_t (&v)[2][32]) {
    const int c0 = n0 + g * 64;
    if (c0 >= cols) return;  // uniform
    if (from != nullptr) {
      float4 p[16];
#pragma unroll
      for (int j = 0; j < 16; ++j)  // cols is a multiple of 8
        p[j] = c0 + 4 * j < cols ? __ldcs(reinterpret_cast<const float4*>(from + c0 + 4 * j)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        uint32_t* at = &v[j >> 3][4 * (j & 7)];
        at[0] = __float_as_uint(__uint_as_float(at[0]) + p[j].x);
        at[1] = __float_as_uint(__uint_as_float(at[1]) + p[j].y);
        at[2] = __float_as_uint(__uint_as_float(at[2]) + p[j].z);
        at[3] = __float_as_uint(__uint_as_float(at[3]) + p[j].w);
      }
    }
    if (leader) bulk_wait_group_read<0>();
    named_bar_sync(bar, kWarpgroup);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 8 * j + 2 * i;
        const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(v[e >> 5][e & 31]),
                                                       __uint_as_float(v[(e + 1) >> 5][(e + 1) & 31]));
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      stage_piece(buf, row, j, w);
    }
    fence_proxy_async_smem();
    named_bar_sync(bar, kWarpgroup);
    if (leader) {
      tma_store_2d(map, smem_u32(buf), c0, m0);
      bulk_commit_group();
    }
    __syncwarp();
  };
  auto ready = [&](uint32_t (&v)[2][32]) {
    tmem_ld_wait();
    tmem_regs_ready(v[0]);
    tmem_regs_ready(v[1]);
  };
  load(0, r[0]);
  ready(r[0]);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    if (g + 1 < kGroups) {
      load(g + 1, r[(g + 1) & 1]);
      ready(r[(g + 1) & 1]);
      if (g + 2 == kGroups) release();
    }
    process(g, r[g & 1]);
  }
}

// The loads of a unit's k-blocks: this CTA's 128 rows of A (d along its rows, or its
// columns for dW) and its 128 columns of either half of B.
template <bool DW, bool BOTH>
__device__ __forceinline__ bool load_unit(const ScoreBackwardMaps& maps, int kb0, int kb1, int mA, int nB, uint32_t rank,
                                          const uint8_t* sA, const uint8_t* sB, uint32_t full0, uint32_t empty0,
                                          uint32_t& n_issued, uint32_t* ctrl, uint64_t timeout_ns) {
  const CUtensorMap* ma = DW ? &maps.dt : &maps.d;
  const CUtensorMap* mb = DW ? &maps.x : &maps.w;
  for (int kb = kb0; kb < kb1; ++kb) {
    const uint32_t stage = n_issued % kRing;
    if (!mbar_wait_bounded_cluster(empty0 + 8u * stage, ((n_issued / kRing) & 1u) ^ 1u, ctrl, timeout_ns)) return false;
    const uint32_t full = full0 + 8u * stage;
    if (rank == 0) mbar_arrive_expect_tx(full, 2 * (kRingA + (BOTH ? kRingB : kRingHalfB)));
    const uint32_t fb = mapa_shared(full, 0);
    const uint32_t sa = smem_u32(sA + stage * kRingA), sb = smem_u32(sB + stage * kRingB);
    const int k0 = kb * kBK;
    if (DW) {
      tma_load_2d_pair(sa, ma, fb, mA, k0);
      tma_load_2d_pair(sa + 8192, ma, fb, mA + 64, k0);
    } else {
      tma_load_2d_pair(sa, ma, fb, k0, mA);
    }
    tma_load_2d_pair(sb, mb, fb, nB, k0);
    tma_load_2d_pair(sb + 8192, mb, fb, nB + 64, k0);
    if (BOTH) {
      tma_load_2d_pair(sb + kRingHalfB, mb, fb, nB + kBN, k0);
      tma_load_2d_pair(sb + kRingHalfB + 8192, mb, fb, nB + kBN + 64, k0);
    }
    ++n_issued;
  }
  return true;
}

// Its products
template <bool DW, bool BOTH>
__device__ __forceinline__ bool issue_unit(int blocks, uint32_t tmem_base, const uint8_t* sA, const uint8_t* sB, uint32_t full0,
                                           uint32_t empty0, uint32_t& n_consumed, uint32_t* ctrl, uint64_t timeout_ns) {
  constexpr uint32_t idesc = idesc_bf16_f32(2 * kBM, kBN, DW ? 1 : 0, 1);
  for (int i = 0; i < blocks; ++i) {
    const uint32_t stage = n_consumed % kRing;
    if (!mbar_wait_bounded_cluster(full0 + 8u * stage, (n_consumed / kRing) & 1u, ctrl, timeout_ns)) return false;
    tc_fence_after();
    const uint32_t sa = smem_u32(sA + stage * kRingA), sb = smem_u32(sB + stage * kRingB);
#pragma unroll
    for (int k = 0; k < kBK / 16; ++k) {
      const uint64_t ad = DW ? smem_desc_sw128(sa + 2048u * k, 8192u, 1024u) : smem_desc_sw128(sa + 32u * k, 16u, 1024u);
      const uint64_t bd = smem_desc_sw128(sb + 2048u * k, 8192u, 1024u);
      const uint32_t add = (i > 0 || k > 0) ? 1u : 0u;
      if (BOTH) {
        tc_mma_bf16_pair_a_fill(tmem_base, ad, bd, idesc, add);
        tc_mma_bf16_pair_a_lastuse(tmem_base + kBN, ad, smem_desc_sw128(sb + kRingHalfB + 2048u * k, 8192u, 1024u), idesc, add);
      } else {
        tc_mma_bf16_pair(tmem_base, ad, bd, idesc, add);
      }
    }
    tc_commit_pair_multicast(empty0 + 8u * stage, 0x3);
    ++n_consumed;
  }
  return true;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    score_backward_kernel(const __grid_constant__ ScoreBackwardMaps maps, const __grid_constant__ ScoreBackwardArgs a) {
  Shape p;
  p.rows = chunk_rows(a.live, a.off, a.rows);
  if (p.rows == 0) {
    if (a.off > 0) return;  // no row of this chunk counts (the same in all threads)
    p.rows = 1;             // none of the call's does: zeros, from a row of zeros
  }
  p.last = a.live ? static_cast<int64_t>(*a.live) <= a.off + a.rows : a.last != 0;
  p.n = (a.H + 2 * kBN - 1) / (2 * kBN);
  p.m0 = (p.rows + 2 * kBM - 1) / (2 * kBM);
  p.units0 = a.dx ? p.m0 * p.n * a.splits : 0;
  p.units = p.units0 + (a.dw ? (a.V + 2 * kBM - 1) / (2 * kBM) * p.n : 0);
  p.kb_rows = (p.rows + kBK - 1) / kBK;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kRing * kRingA;
  uint8_t* sE = sB + kRing * kRingB;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sE + 2 * kStagingBytes);
  uint64_t* ubars = bars + 2 * kRing + 3;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ubars + 2 * kUnitDepth);
  int32_t* published = reinterpret_cast<int32_t*>(tmem_slot + 1);

  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kRing + s); };
  const uint32_t tfull_bar = bar0 + 8u * (2 * kRing);
  const uint32_t tempty_bar = bar0 + 8u * (2 * kRing + 1);
  const uint32_t drain_bar = bar0 + 8u * (2 * kRing + 2);
  const uint32_t ubar0 = smem_u32(ubars);
  auto ufull_bar = [&](int i) { return ubar0 + 8u * i; };
  auto uempty_bar = [&](int i) { return ubar0 + 8u * (kUnitDepth + i); };
  const uint32_t published0 = smem_u32(published);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: the CTA that claims units and issues the products

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(full_bar(s), 1);   // used in CTA 0: both CTAs' loads land here
      mbar_init(empty_bar(s), 1);  // each CTA's own, released by the products' commit
    }
    mbar_init(tfull_bar, 1);
    mbar_init(tempty_bar, 2 * 2 * kWarpgroup);  // used in CTA 0: both CTAs' two epilogues
    mbar_init(drain_bar, 1);
    for (int i = 0; i < kUnitDepth; ++i) {
      mbar_init(ufull_bar(i), 1);
      mbar_init(uempty_bar(i), kUnitReaders);  // used in CTA 0
    }
    fence_mbar_init();
    fence_proxy_async_smem();
    tma_prefetch_map(&maps.d);
    tma_prefetch_map(&maps.w);
    tma_prefetch_map(&maps.dt);
    tma_prefetch_map(&maps.x);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kAccumulatorColumns);
    tmem_relinquish_pair();
  }
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are there before the other uses them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // the unit of step i (-1: no more); false if the wait ran out
  auto next_unit = [&](int i, int& u, bool release) {
    const int slot = i % kUnitDepth;
    if (!mbar_wait_bounded_cluster(ufull_bar(slot), (i / kUnitDepth) & 1u, a.ctrl, a.timeout_ns)) return false;
    u = ld_shared_s32(published0 + 4u * slot);
    if (release) arrive_even(uempty_bar(slot), rank);
    return true;
  };
  // k-blocks of a unit, and whether its second 256 columns are there
  auto extent = [&](const Unit& t, int& kb0, int& kb1) {
    kb0 = t.dw ? 0 : t.s * a.kb_per_split;
    kb1 = t.dw ? p.kb_rows : min(a.kb_v, kb0 + a.kb_per_split);
  };
  auto both_halves = [&](const Unit& t) { return t.n * 2 * kBN + kBN < a.H; };

  if (warp < 4) {
    warpgroup_regs_dec<kRegsControl>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------- loads
      uint32_t n_issued = 0;
      bool failed = false;
      for (int i = 0; !failed; ++i) {
        int u;
        if (rank == 0) {
          // claims the next unit and tells both CTAs
          const int slot = i % kUnitDepth;
          if (!mbar_wait_bounded_cluster(uempty_bar(slot), ((i / kUnitDepth) & 1u) ^ 1u, a.ctrl, a.timeout_ns)) {
            failed = true;
            break;
          }
          u = atomicAdd(a.claims, 1);
          if (u >= p.units) u = -1;
          published[slot] = u;
          st_shared_cluster_u32(mapa_shared(published0 + 4u * slot, 1), static_cast<uint32_t>(u));
          mbar_arrive(ufull_bar(slot));
          mbar_arrive_cluster(mapa_shared(ufull_bar(slot), 1));
        } else if (!next_unit(i, u, true)) {
          failed = true;
          break;
        }
        if (u < 0) break;
        const Unit t = unit_of(a, p, u);
        int kb0, kb1;
        extent(t, kb0, kb1);
        const bool both = both_halves(t);
        const int mA = t.m * 2 * kBM + static_cast<int>(rank) * kBM;
        const int nB = t.n * 2 * kBN + static_cast<int>(rank) * (kBN / 2);
        const bool ok = t.dw ? (both ? load_unit<true, true>(maps, kb0, kb1, mA, nB, rank, sA, sB, full_bar(0), empty_bar(0),
                                                             n_issued, a.ctrl, a.timeout_ns)
                                     : load_unit<true, false>(maps, kb0, kb1, mA, nB, rank, sA, sB, full_bar(0), empty_bar(0),
                                                              n_issued, a.ctrl, a.timeout_ns))
                             : (both ? load_unit<false, true>(maps, kb0, kb1, mA, nB, rank, sA, sB, full_bar(0), empty_bar(0),
                                                              n_issued, a.ctrl, a.timeout_ns)
                                     : load_unit<false, false>(maps, kb0, kb1, mA, nB, rank, sA, sB, full_bar(0), empty_bar(0),
                                                               n_issued, a.ctrl, a.timeout_ns));
        if (!ok) failed = true;
      }
      if (failed && rank == 0) {
        const uint32_t first = n_issued > kRing ? n_issued - kRing : 0;
        for (uint32_t i = first; i < n_issued; ++i) drain_wait(full_bar(i % kRing), (i / kRing) & 1u, a.timeout_ns);
      }
    } else if (warp == 1 && lane == 0 && rank == 0) {
      // ------------------------------------------------------- products
      uint32_t n_consumed = 0;
      bool issued = false, failed = false;
      for (int it = 0; !failed; ++it) {
        int u;
        if (!next_unit(it, u, true)) {
          failed = true;
          break;
        }
        if (u < 0) break;
        const Unit t = unit_of(a, p, u);
        int kb0, kb1;
        extent(t, kb0, kb1);
        const bool both = both_halves(t);
        if (!mbar_wait_bounded_cluster(tempty_bar, (it & 1) ^ 1u, a.ctrl, a.timeout_ns)) {
          failed = true;
          break;
        }
        tc_fence_after();
        const bool ok = t.dw ? (both ? issue_unit<true, true>(kb1 - kb0, tmem_base, sA, sB, full_bar(0), empty_bar(0), n_consumed,
                                                              a.ctrl, a.timeout_ns)
                                     : issue_unit<true, false>(kb1 - kb0, tmem_base, sA, sB, full_bar(0), empty_bar(0),
                                                               n_consumed, a.ctrl, a.timeout_ns))
                             : (both ? issue_unit<false, true>(kb1 - kb0, tmem_base, sA, sB, full_bar(0), empty_bar(0),
                                                               n_consumed, a.ctrl, a.timeout_ns)
                                     : issue_unit<false, false>(kb1 - kb0, tmem_base, sA, sB, full_bar(0), empty_bar(0),
                                                                n_consumed, a.ctrl, a.timeout_ns));
        issued = true;
        if (!ok) failed = true;
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
    // one warpgroup for each 256 columns
    const int grp = (warp - 4) >> 2;
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const bool leader = threadIdx.x == (grp + 1) * kWarpgroup;
    const uint32_t bar = 1u + static_cast<uint32_t>(grp);
    uint8_t* buf = sE + grp * kStagingBytes;
    const uint32_t tbase = tmem_base + (static_cast<uint32_t>(wq * 32) << 16) + grp * kBN;
    for (int it = 0;; ++it) {
      int u = -1;
      const bool got = next_unit(it, u, false);
      // all have read the slot (or given up) before one releases it
      if (named_bar_or(bar, kWarpgroup, !got)) break;
      if (leader) arrive_even(uempty_bar(it % kUnitDepth), rank);
      if (u < 0) break;
      const Unit t = unit_of(a, p, u);
      const int m0 = t.m * 2 * kBM + static_cast<int>(rank) * kBM;
      const int n0 = t.n * 2 * kBN + grp * kBN;
      const bool to16 = t.dw && a.dw_bf16 && p.last;
      const float* from = sum_row(to16 && a.off > 0 ? a.dw_sum : nullptr, a.V, a.H, m0 + row);
      prefetch_sum(from, n0, a.H);
      const bool ok = mbar_wait_bounded_cluster(tfull_bar, it & 1, a.ctrl, a.timeout_ns);
      if (named_bar_or(bar, kWarpgroup, !ok)) break;
      tc_fence_after();
      if (to16)
        epilogue_bf16(&maps.dw16, from, a.H, tbase, m0, n0, buf, row, leader, bar, tempty_bar, rank);
      else
        epilogue_f32(t.dw ? &maps.dw32 : &maps.part, t.dw && a.off > 0, a.H, tbase, m0, n0, t.s, buf, row, leader, bar,
                     tempty_bar, rank);
    }
    if (leader) bulk_wait_group<0>();
  }

  __syncwarp();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the pair's products may touch its memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kAccumulatorColumns);
  }
}

}  // namespace

cudaError_t launch_score_backward(const ScoreBackwardMaps& maps, const ScoreBackwardArgs& args, int pairs, cudaStream_t s) {
  static const bool fits = registers_fit(score_backward_kernel);
  if (!fits) return cudaErrorInvalidConfiguration;
  const cudaError_t e = cudaFuncSetAttribute(score_backward_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kSmemBytes));
  if (e != cudaSuccess) return e;
  score_backward_kernel<<<2 * pairs, kPairThreads, kSmemBytes, s>>>(maps, args);
  return cudaGetLastError();
}

}  // namespace flce
