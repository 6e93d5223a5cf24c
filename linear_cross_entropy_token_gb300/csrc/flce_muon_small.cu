// The orthogonalised momentum update of matrices whose short side is at most
// 128, in one launch: momentum, norm, all Newton-Schulz steps and the result.
// (flce_muon.cu has the formulas and the choice of fp16 parts.)
//
// Such a matrix is bound by latency: a step's products take well under a
// microsecond, and as 17 launches that pass X, A and B through global memory a
// 128 x 128 matrix took 95 us. Here one cluster of C CTAs holds the matrix on
// chip from the load to the result, each CTA a slab of up to 256 of its columns:
//
//   shared memory  X hi and lo, [64-column chunk][128 rows][128 bytes] with the
//                  128-byte swizzle; that one copy is the K-major operand of
//                  X Xt and the MN-major right operand of B X
//                  A and B, [64-column chunk][128 rows][128 bytes]
//   TMEM           columns 0..127 the accumulator of X Xt, then of A A;
//                  columns 128.. the accumulator of B X
//
// X Xt sums over the slabs: each CTA leaves its partial product in global memory
// (L2), adds its share of the 128 x 128 elements over the C partial products in
// order, leaves the rounded values as the image of A's tile, and loads that
// whole; cluster barriers order the three. (An SM sends only about 15 bytes per
// clock to its peers' shared memories: the same exchange that way, by stores or
// bulk copies, took 8.6 and 7.6 us a step at 128 x 1024, this 7.0.) A A and
// B are the same small work in every CTA. Rows past the short side are zero.
//
// A short side up to kMuonPairSide (BOTH) runs each product as three, high x high, low
// x high and high x low parts, into one accumulator: A and B are one block of 32 x
// 32 then, their low part where otherwise B is, and take 32 of 128 columns and of
// the depth, so that this costs no more (32 x 32: 19.3 us, one product of whole
// tiles each 19.7). Their partial products are 4 KB, which every CTA adds for itself,
// behind one cluster barrier instead of two (32 x 1024: 28 us, 43).
//
// 512 threads; thread t works on row 32 (warp % 4) + lane of an accumulator,
// and on one quarter of its columns. Every wait is bounded: one that runs out is
// recorded, and the kernel goes on to its end (no CTA leaves a cluster barrier
// waiting).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "flce_muon.cuh"

namespace flce {
namespace {

constexpr int kSmallThreads = 512;
constexpr int kSmallWarps = kSmallThreads / 32;
constexpr uint32_t kChunkBytes = 128 * 128;   // 128 rows x 64 fp16
constexpr uint32_t kPanelBytes = 2 * kChunkBytes;

__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

// 32 lanes x 16 consecutive fp32 columns
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// as tmem_regs_ready: no use of the registers moves above the wait
__device__ __forceinline__ void tmem_regs_ready16(uint32_t (&r)[16]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

// bulk copy from global to this CTA's shared memory, completing on its barrier
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}

// byte offset of 16-byte chunk j (8 fp16) of row r in a [128 rows][128 bytes] tile
__device__ __forceinline__ uint32_t tile16(int r, int j) { return r * 128 + ((j ^ (r & 7)) << 4); }

template <int NCH, bool BOTH>
__global__ void __launch_bounds__(kSmallThreads, 1)
    muon_small_kernel(const __grid_constant__ MuonArgs a, const __grid_constant__ MuonSteps steps) {
  constexpr int kSlab = 64 * NCH;
  constexpr uint32_t kCols = NCH <= 2 ? 256 : 512;   // TMEM: 128 + the slab
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_word[2];   // products done; A loaded
  __shared__ uint32_t tmem_slot;
  __shared__ float diag[128];
  __shared__ double norm_warp[kSmallWarps], norm_part[16];
  __shared__ float factor[2];

  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sHi = smem;
  uint8_t* sLo = sHi + NCH * kChunkBytes;
  uint8_t* sA = sLo + NCH * kChunkBytes;
  uint8_t* sB = sA + kPanelBytes;
  const int C = static_cast<int>(a.cluster);
  const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const MuonMat& t = a.mat[blockIdx.x / C];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = 32 * (warp & 3) + lane, quarter = warp >> 2;   // of the accumulators
  const int slab0 = rank * kSlab;
  const uint32_t bar = smem_u32(&bar_word[0]), bar_gram = smem_u32(&bar_word[1]);
  // this matrix's partial products [C][16 warps][8][32 lanes] of four, and A's image
  float4* partials = reinterpret_cast<float4*>(a.sums) + static_cast<int64_t>(blockIdx.x / C) * (C * 4096 + 2048);
  uint8_t* image = reinterpret_cast<uint8_t*>(partials + C * 4096);
  uint32_t parity = 0;
  auto wait_for = [&](uint32_t b, uint32_t par) {
    if (!wait_limited(b, par, a.timeout_ns)) *reinterpret_cast<volatile uint32_t*>(a.host_error) = kErrTimeout;
  };
  auto wait_products = [&] {
    wait_for(bar, parity);
    parity ^= 1u;
    tc_fence_after();
  };

  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    mbar_init(bar_gram, 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&tmem_slot), kCols);
    tmem_relinquish();
  }

  if (C > 1) cluster_arrive();   // waited for before the first access to another CTA

  // u of the slab, as fp32, to where X will be. A thread takes 16 neighbouring
  // columns of one row of X per chunk. The rows of X are the rows of u, four
  // threads per row, or its columns, a warp per 32 neighbours: either way
  // global memory sees runs. (The loops are unrolled no further than their
  // loads need: each instruction runs once or five times, and fetching a
  // fully unrolled body was the kernel's bound.)
  const int lrow = a.transposed ? (threadIdx.x & 127) : (threadIdx.x >> 2);
  const int lq = a.transposed ? (threadIdx.x >> 7) : (threadIdx.x & 3);
  // fp32 staging: the thread's 16 values of a chunk fill its 32 bytes of the hi
  // tile and its 32 bytes of the lo tile, so no other thread's
  auto staged = [&](int ch, int v4) {   // the v4-th of 4 vectors of four
    return reinterpret_cast<float4*>((v4 < 2 ? sHi : sLo) + ch * kChunkBytes + tile16(lrow, lq * 2 + (v4 & 1)));
  };
  SquareSum q;
#pragma unroll 1
  for (int ch = 0; ch < NCH; ++ch) {
    const int j0 = slab0 + ch * 64 + lq * 16;
    const bool in = lrow < a.m && j0 < a.n;
    if (!a.transposed && a.vec) {
      float g[4][4];
      float4 m[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g[e][0] = g[e][1] = g[e][2] = g[e][3] = 0.f;
        if (in && j0 + 4 * e < a.n) {
          load4(t.grad, a.grad_dtype, lrow * t.ld_grad + j0 + 4 * e, g[e]);
          if (t.momentum) m[e] = *reinterpret_cast<const float4*>(t.momentum + lrow * t.ld_momentum + j0 + 4 * e);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (t.momentum && in && j0 + 4 * e < a.n) {
          momentum4(a, m[e], g[e]);
          *reinterpret_cast<float4*>(t.momentum + lrow * t.ld_momentum + j0 + 4 * e) = m[e];
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) q.add(g[e][x]);
        *staged(ch, e) = make_float4(g[e][0], g[e][1], g[e][2], g[e][3]);
      }
    } else {
      const int64_t step = a.transposed ? 1 : 0;   // along u's rows or columns
      const int64_t gs = step ? t.ld_grad : 1, ms = step ? t.ld_momentum : 1;
      const int64_t g0 = step ? j0 * t.ld_grad + lrow : lrow * t.ld_grad + j0;
      float* m0 = t.momentum + (step ? j0 * t.ld_momentum + lrow : lrow * t.ld_momentum + j0);
      float g[16], m[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        g[x] = m[x] = 0.f;
        if (in && j0 + x < a.n) {
          g[x] = load1(t.grad, a.grad_dtype, g0 + x * gs);
          if (t.momentum) m[x] = m0[x * ms];
        }
      }
      if (t.momentum) {
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          m[x] = m[x] * a.beta + g[x] * a.one_minus_beta;
          g[x] = a.nesterov ? m[x] * a.beta + g[x] * a.one_minus_beta : m[x];
          if (in && j0 + x < a.n) m0[x * ms] = m[x];
        }
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) q.add(g[x]);
#pragma unroll
      for (int e = 0; e < 4; ++e) *staged(ch, e) = make_float4(g[4 * e], g[4 * e + 1], g[4 * e + 2], g[4 * e + 3]);
    }
  }
  q.reduce_warp();
  if (lane == 0) norm_warp[warp] = q.total();
  __syncthreads();
  if (C > 1) cluster_wait();
  if (threadIdx.x == 0) {
    double s = 0.0;
#pragma unroll 1
    for (int w = 0; w < kSmallWarps; ++w) s += norm_warp[w];
    if (C == 1) {
      norm_part[0] = s;
    } else {
#pragma unroll 1
      for (int c = 0; c < C; ++c) st_cluster_f64(mapa_shared(smem_u32(&norm_part[rank]), c), s);
    }
  }
  if (C > 1) {
    cluster_sync();
  } else {
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    double s = 0.0;
#pragma unroll 1
    for (int c = 0; c < C; ++c) s += norm_part[c];
    norm_factors(s, a.eps, factor);
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const uint32_t tmem_row = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
  {
    const float f1 = factor[0], f2 = factor[1];
#pragma unroll 1
    for (int ch = 0; ch < NCH; ++ch) {   // in place: a thread's values lie in its own bytes
      float4 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = *staged(ch, e);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t h[4], l[4];
        split_half2(v[2 * j].x * f1 * f2, v[2 * j].y * f1 * f2, h[0], l[0]);
        split_half2(v[2 * j].z * f1 * f2, v[2 * j].w * f1 * f2, h[1], l[1]);
        split_half2(v[2 * j + 1].x * f1 * f2, v[2 * j + 1].y * f1 * f2, h[2], l[2]);
        split_half2(v[2 * j + 1].z * f1 * f2, v[2 * j + 1].w * f1 * f2, h[3], l[3]);
        const uint32_t at = ch * kChunkBytes + tile16(lrow, lq * 2 + j);
        *reinterpret_cast<uint4*>(sHi + at) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(sLo + at) = make_uint4(l[0], l[1], l[2], l[3]);
      }
    }
  }
  fence_proxy_async_smem();
  __syncthreads();

  const uint32_t aHi = smem_u32(sHi), aLo = smem_u32(sLo), aA = smem_u32(sA), aB = smem_u32(sB);
  // BOTH: the terms' products of `steps` 16-deep slices, `a` and `b` the operands' slices (part, slice)
  auto terms = [&](uint32_t d, uint32_t idesc, auto count, auto&& da, auto&& db) {
#pragma unroll 1
    for (int term = 0; term < 3; ++term) {
#pragma unroll
      for (int i = 0; i < decltype(count)::value; ++i)
        tc_mma_bf16(d, da(term == 1, i), db(term == 2, i), idesc, term > 0 || i > 0 ? 1u : 0u);
    }
  };
  // BOTH: this lane's row of A or B, four values from column c on, to its place in either part
  auto put_pair4 = [&](int c, float v0, float v1, float v2, float v3) {
    uint2 h, l;
    split_half2(v0, v1, h.x, l.x);
    split_half2(v2, v3, h.y, l.y);
    const uint32_t at = tile16(lane, c >> 3) + (c & 4) * 2;
    *reinterpret_cast<uint2*>(sA + at) = h;
    *reinterpret_cast<uint2*>(sB + at) = l;
  };
#pragma unroll 1
  for (int k = 0; k < steps.count; ++k) {
    const float ca = steps.c[k][0], cb = steps.c[k][1], cc = steps.c[k][2];
    // ---- A = X Xt
    if (threadIdx.x == 0) {
      tc_fence_after();
      if constexpr (BOTH) {
        auto slice = [&](bool low, int i) {
          return smem_desc_sw128((low ? aLo : aHi) + (i >> 2) * kChunkBytes + 32u * (i & 3), 16u, 1024u);
        };
        terms(tmem, idesc_f16_f32(128, kMuonPairSide, 0, 0), std::integral_constant<int, 4 * NCH>(), slice, slice);
      } else {
        constexpr uint32_t idesc = idesc_f16_f32(128, 128, 0, 0);
#pragma unroll
        for (int i = 0; i < 4 * NCH; ++i) {
          const uint64_t d = smem_desc_sw128(aHi + (i >> 2) * kChunkBytes + 32u * (i & 3), 16u, 1024u);
          tc_mma_bf16(tmem, d, d, idesc, i > 0 ? 1u : 0u);
        }
      }
      tc_commit(bar);
    }
    wait_products();
    if constexpr (BOTH) {
      // a step's partial products in one half of their room, the next step's in the other:
      // a CTA writes a half again only behind a barrier that all readers have passed
      float4* mine = partials + (k & 1) * C * 256;
      if (warp == 0) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tmem_row, r);
        tmem_ld_wait();
        tmem_regs_ready(r);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v[4] = {__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]), __uint_as_float(r[4 * j + 2]),
                              __uint_as_float(r[4 * j + 3])};
          if (C == 1)
            put_pair4(4 * j, v[0] * kGramScale, v[1] * kGramScale, v[2] * kGramScale, v[3] * kGramScale);
          else
            __stcg(mine + rank * 256 + j * 32 + lane, make_float4(v[0], v[1], v[2], v[3]));
        }
      }
      tc_fence_before();
      if (C > 1) {
        cluster_sync();
        if (warp < 8) {   // columns 4 warp .. of a row per lane, over the CTAs in order
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
          for (int src = 0; src < C; ++src) {
            const float4 v = __ldcg(mine + src * 256 + warp * 32 + lane);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
          }
          put_pair4(4 * warp, s.x * kGramScale, s.y * kGramScale, s.z * kGramScale, s.w * kGramScale);
        }
      }
      fence_proxy_async_smem();
      __syncthreads();
    } else if (C == 1) {
      uint32_t r[32];
      __syncwarp();
      tmem_ld_32x32b_x32(tmem_row + quarter * 32, r);
      tmem_ld_wait();
      tmem_regs_ready(r);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = pack_half2(__uint_as_float(r[8 * j + 2 * e]) * kGramScale,
                            __uint_as_float(r[8 * j + 2 * e + 1]) * kGramScale);
        *reinterpret_cast<uint4*>(sA + (quarter >> 1) * kChunkBytes + tile16(row, (quarter & 1) * 4 + j)) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
    } else {
      {
        uint32_t r[32];
        __syncwarp();
        tmem_ld_32x32b_x32(tmem_row + quarter * 32, r);
        tmem_ld_wait();
        tmem_regs_ready(r);
        float4* to = partials + rank * 4096 + warp * 256 + lane;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          __stcg(to + j * 32, make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                          __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])));
      }
      tc_fence_before();
      cluster_sync();
      // 128 runs of 32 lanes: run b is warp b / 8's vector b % 8, columns 4 (b % 8)
      // of that warp's quarter, a row per lane
      for (int b = rank * (128 / C) + warp; b < (rank + 1) * (128 / C); b += kSmallWarps) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4* from = partials + b * 32 + lane;
#pragma unroll 8
        for (int src = 0; src < C; ++src) {
          const float4 v = __ldcg(from + src * 4096);
          s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        const int w = b >> 3, grow = 32 * (w & 3) + lane, col = (w >> 2) * 32 + (b & 7) * 4;
        const uint32_t at = (col >> 6) * kChunkBytes + tile16(grow, (col & 63) >> 3) + (col & 4) * 2;
        __stcg(reinterpret_cast<uint2*>(image + at), make_uint2(pack_half2(s.x * kGramScale, s.y * kGramScale),
                                                                pack_half2(s.z * kGramScale, s.w * kGramScale)));
      }
      fence_proxy_async_all();
      cluster_sync();
      if (threadIdx.x == 0) {
        fence_proxy_async_all();
        mbar_arrive_expect_tx(bar_gram, kPanelBytes);
        bulk_load(smem_u32(sA), image, kPanelBytes, bar_gram);
      }
      wait_for(bar_gram, k & 1u);
    }
    // ---- B = b A + c A A
    if (threadIdx.x == 0) {
      tc_fence_after();
      if constexpr (BOTH) {
        auto slice = [&](bool low, int i) { return smem_desc_sw128((low ? aB : aA) + 32u * i, 16u, 1024u); };
        terms(tmem, idesc_f16_f32(128, kMuonPairSide, 0, 0), std::integral_constant<int, kMuonPairSide / 16>(), slice, slice);
      } else {
        constexpr uint32_t idesc = idesc_f16_f32(128, 128, 0, 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint64_t d = smem_desc_sw128(aA + (i >> 2) * kChunkBytes + 32u * (i & 3), 16u, 1024u);
          tc_mma_bf16(tmem, d, d, idesc, i > 0 ? 1u : 0u);
        }
      }
      tc_commit(bar);
    }
    wait_products();
    if constexpr (BOTH) {
      if (warp == 0) {   // B in A's place
        uint32_t r[32];
        tmem_ld_32x32b_x32(tmem_row, r);
        tmem_ld_wait();
        tmem_regs_ready(r);
        float on_diag = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t at = tile16(lane, j >> 1) + (j & 1) * 8;
          const uint2 h = *reinterpret_cast<const uint2*>(sA + at), l = *reinterpret_cast<const uint2*>(sB + at);
          const float2 h0 = unpack_half2(h.x), h1 = unpack_half2(h.y), l0 = unpack_half2(l.x), l1 = unpack_half2(l.y);
          float v[4] = {h0.x + l0.x, h0.y + l0.y, h1.x + l1.x, h1.y + l1.y};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = cb * kPolyB * v[e] + cc * kPolyC * __uint_as_float(r[4 * j + e]);
            on_diag = 4 * j + e == lane ? v[e] : on_diag;   // the diagonal stays in fp32, apart
            v[e] = 4 * j + e == lane ? 0.f : v[e];
          }
          put_pair4(4 * j, v[0], v[1], v[2], v[3]);
        }
        diag[lane] = on_diag * kPolyInv;
      }
    } else {
      uint32_t r[32];
      __syncwarp();
      tmem_ld_32x32b_x32(tmem_row + quarter * 32, r);
      tmem_ld_wait();
      tmem_regs_ready(r);
      float on_diag = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t at = (quarter >> 1) * kChunkBytes + tile16(row, (quarter & 1) * 4 + j);
        const uint4 av = *reinterpret_cast<const uint4*>(sA + at);
        const uint32_t aw[4] = {av.x, av.y, av.z, av.w};
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack_half2(aw[e]);
          v[2 * e] = cb * kPolyB * f.x + cc * kPolyC * __uint_as_float(r[8 * j + 2 * e]);
          v[2 * e + 1] = cb * kPolyB * f.y + cc * kPolyC * __uint_as_float(r[8 * j + 2 * e + 1]);
        }
        const int d = row - (quarter * 32 + 8 * j);   // the diagonal stays in fp32, apart
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          on_diag = e == d ? v[e] : on_diag;
          v[e] = e == d ? 0.f : v[e];
        }
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack_half2(v[2 * e], v[2 * e + 1]);
        *reinterpret_cast<uint4*>(sB + at) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if ((row >> 5) == quarter) diag[row] = on_diag * kPolyInv;
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    // ---- X = a X + B X
    if (threadIdx.x == 0) {
      tc_fence_after();
      constexpr uint32_t idesc = idesc_f16_f32(128, kSlab, 0, 1);
      if constexpr (BOTH) {
        terms(tmem + 128, idesc, std::integral_constant<int, kMuonPairSide / 16>(),
              [&](bool low, int i) { return smem_desc_sw128((low ? aB : aA) + 32u * i, 16u, 1024u); },
              [&](bool low, int i) { return smem_desc_sw128((low ? aLo : aHi) + 2048u * i, kChunkBytes, 1024u); });
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint64_t da = smem_desc_sw128(aB + (i >> 2) * kChunkBytes + 32u * (i & 3), 16u, 1024u);
          const uint64_t db = smem_desc_sw128(aHi + 2048u * i, kChunkBytes, 1024u);
          tc_mma_bf16(tmem + 128, da, db, idesc, i > 0 ? 1u : 0u);
        }
      }
      tc_commit(bar);
    }
    wait_products();
    const bool last = k == steps.count - 1;
    const float2 f = BOTH ? make_float2(ca + diag[lane], ca + diag[lane])
                          : part_factors(ca, diag[row], 32 * (warp & 3) + 32 <= a.m);
    const float sc = a.scale * kXInv;
#pragma unroll 1
    for (int g = 0; g < NCH; ++g) {   // the thread's quarter of the slab, 16 columns at a time
      if (BOTH && (warp & 3) != 0) break;   // (rows past the matrix)
      const int col = (quarter * NCH + g) * 16;
      uint32_t r[16];
      __syncwarp();
      tmem_ld_32x32b_x16(tmem_row + 128 + col, r);
      const uint32_t at0 = (col >> 6) * kChunkBytes + tile16(row, (col & 63) >> 3);
      const uint32_t at1 = (col >> 6) * kChunkBytes + tile16(row, ((col & 63) >> 3) + 1);
      const uint4 h0 = *reinterpret_cast<const uint4*>(sHi + at0), h1 = *reinterpret_cast<const uint4*>(sHi + at1);
      const uint4 l0 = *reinterpret_cast<const uint4*>(sLo + at0), l1 = *reinterpret_cast<const uint4*>(sLo + at1);
      uint32_t h[8] = {h0.x, h0.y, h0.z, h0.w, h1.x, h1.y, h1.z, h1.w};
      uint32_t l[8] = {l0.x, l0.y, l0.z, l0.w, l1.x, l1.y, l1.z, l1.w};
      tmem_ld_wait();
      tmem_regs_ready16(r);
      float o[16];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 fh = unpack_half2(h[e]), fl = unpack_half2(l[e]);
        o[2 * e] = f.x * fh.x + (f.y * fl.x + __uint_as_float(r[2 * e]) * kPolyInv);
        o[2 * e + 1] = f.x * fh.y + (f.y * fl.y + __uint_as_float(r[2 * e + 1]) * kPolyInv);
        split_half2(o[2 * e], o[2 * e + 1], h[e], l[e]);
      }
      if (!last) {
        *reinterpret_cast<uint4*>(sHi + at0) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(sHi + at1) = make_uint4(h[4], h[5], h[6], h[7]);
        *reinterpret_cast<uint4*>(sLo + at0) = make_uint4(l[0], l[1], l[2], l[3]);
        *reinterpret_cast<uint4*>(sLo + at1) = make_uint4(l[4], l[5], l[6], l[7]);
        continue;
      }
      // ---- the result
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] *= sc;
      const int j0 = slab0 + col, cols = min(16, a.n - j0);
      if (a.transposed) {
        if (row < a.m && cols > 0)
          with_result(a, t, [&](auto* out, auto W, int64_t ld) {
            write_columns<decltype(W)::value>(out + j0 * ld + row, ld, cols, a.decay, a.lr, o);
          });
      } else {
        // the warp's 32 x 16 block as fp32 where A was (2 KB per warp, 16-byte
        // chunks swizzled by the row), then two rows at a time, a column per lane
        float* block = reinterpret_cast<float*>(sA + warp * 2048);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float4*>(block + lane * 16 + ((j ^ ((lane >> 1) & 3)) << 2)) =
              make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        __syncwarp();
        const int rows = min(32, a.m - 32 * (warp & 3));
        const int c = lane & 15, r1 = lane >> 4;
        if (c < cols)
          with_result(a, t, [&](auto* out, auto W, int64_t ld) {
            constexpr bool kW = decltype(W)::value;
            auto* p = out + (static_cast<int64_t>(32 * (warp & 3)) + r1) * ld + j0 + c;
#pragma unroll 1
            for (int r0 = r1; r0 < rows; r0 += 16, p += 16 * ld) {
              std::remove_pointer_t<decltype(p)> w[8];
              if (kW) {
#pragma unroll
                for (int x = 0; x < 8; ++x)
                  if (r0 + 2 * x < rows) w[x] = p[2 * x * ld];
              }
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const int rr = r0 + 2 * x;
                if (rr < rows) {
                  const float v = block[rr * 16 + (((c >> 2) ^ ((rr >> 1) & 3)) << 2) + (c & 3)];
                  put(p + 2 * x * ld, kW ? to_float(w[x]) * a.decay - a.lr * v : v);
                }
              }
            }
          });
        __syncwarp();
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

template <int NCH, bool BOTH>
cudaError_t launch_small_t(const MuonArgs& a, const MuonSteps& steps, cudaStream_t s, int* fits) {
  constexpr size_t smem = 1024 + 2 * NCH * kChunkBytes + 2 * kPanelBytes;   // X, A, B
  auto kern = muon_small_kernel<NCH, BOTH>;
  // at every launch: the attributes belong to the current device, and a process may use several
  cudaError_t opted = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (opted == cudaSuccess && a.cluster > 8)
    opted = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (opted != cudaSuccess) return opted;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.count * a.cluster);
  cfg.blockDim = dim3(kSmallThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = a.cluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (fits) return cudaOccupancyMaxActiveClusters(fits, kern, &cfg);
  return cudaLaunchKernelEx(&cfg, kern, a, steps);
}

template <bool BOTH>
cudaError_t launch_small(const MuonArgs& a, const MuonSteps& steps, int chunks, cudaStream_t s, int* fits) {
  switch (chunks) {
    case 1: return launch_small_t<1, BOTH>(a, steps, s, fits);
    case 2: return launch_small_t<2, BOTH>(a, steps, s, fits);
    case 3: return launch_small_t<3, BOTH>(a, steps, s, fits);
    default: return launch_small_t<4, BOTH>(a, steps, s, fits);
  }
}

}  // namespace

int muon_small_cluster(int64_t m, int64_t n) {
  if (m > 128 || n > 16 * 256) return 0;
  int c = 1;
  while (c * 256 < n) c *= 2;
  return c;
}

int muon_small_chunks(int64_t n, int cluster) { return static_cast<int>(((n + cluster - 1) / cluster + 63) / 64); }

cudaError_t launch_muon_small(const MuonArgs& a, const MuonSteps& steps, int chunks, cudaStream_t s) {
  return a.m <= kMuonPairSide ? launch_small<true>(a, steps, chunks, s, nullptr)
                              : launch_small<false>(a, steps, chunks, s, nullptr);
}

// Clusters of this size that fit the device at once
int muon_small_clusters(int cluster, int chunks, bool pairs) {
  MuonArgs a{};
  a.cluster = cluster;
  a.count = 1;
  int n = 0;
  if ((pairs ? launch_small<true>(a, MuonSteps{}, chunks, nullptr, &n)
             : launch_small<false>(a, MuonSteps{}, chunks, nullptr, &n)) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

}  // namespace flce
