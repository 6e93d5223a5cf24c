// The orthogonalised momentum update of weight matrices (Newton-Schulz).
//
//   buf = beta buf + (1 - beta) g,  u = nesterov ? beta buf + (1 - beta) g : buf
//   X = u / (|u|_F + eps), taken as its transpose when it has more rows than
//       columns, so that X is m x n with m <= n
//   per step: A = X Xt, B = b A + c A^2, X = a X + B X
//   O = scale X;  W = (1 - lr wd) W - lr O, or the update O itself
//
// The three products run on tcgen05 (fp16 operands, fp32 accumulators). A and
// A^2 are symmetric: only the tiles on and above the diagonal are computed,
// and an epilogue writes a tile and its mirror image.
//
// Why fp16 and not bf16: both run at the same rate, and the norms are known (X
// starts with Frobenius norm 1 and the map keeps its singular values near 1),
// so the range of fp16 suffices once X and A are scaled by 2^12 and B by 2^11,
// and three more mantissa bits remain. Why X is kept as two fp16 parts (hi and
// lo, 22 bits together): the map multiplies small singular values by a = 3.4
// per step, 480 times in five steps, and with them whatever rounding put into
// those directions. B X is small there (B is), so B may meet the rounded hi;
// a X must not. The same holds for the diagonal of B, the largest part of it:
// it multiplies the whole X in fp32 in the epilogue, and the product runs on B
// with a zero diagonal. In a float emulation this leaves 2e-4 to 2.5e-3
// relative error (rank 1, rank 16, 1/i and 1/i^2 spectra, Gaussian), of the
// order of one bf16 rounding of the result (1.7e-3); iterates rounded to bf16
// are 1e-2 off on Gaussian matrices and 0.15 to 1 on the others.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "flce_internal.h"
#include "flce_train.h"
#include "ptx.cuh"

namespace flce {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kXScale = 4096.f;           // hi + lo = 2^12 X
constexpr float kXInv = 1.f / 4096.f;
constexpr float kGramScale = 1.f / 4096.f;  // (2^12 X)(2^12 X)t -> 2^12 A
constexpr float kPolyB = 0.5f;              // 2^12 A -> 2^11 A
constexpr float kPolyC = 1.f / 8192.f;      // (2^12 A)^2 -> 2^11 A^2
constexpr float kPolyInv = 1.f / 2048.f;    // 2^11 B -> B; (2^11 B)(2^12 X) -> 2^12 B X

// ------------------------------------------------- momentum and norm

__device__ __forceinline__ void load4(const void* p, int dtype, int64_t i, float (&v)[4]) {
  if (dtype == 1) {
    const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + i);
    v[0] = __uint_as_float(w.x << 16), v[1] = __uint_as_float(w.x & 0xFFFF0000u);
    v[2] = __uint_as_float(w.y << 16), v[3] = __uint_as_float(w.y & 0xFFFF0000u);
  }
}

__device__ __forceinline__ float load1(const void* p, int dtype, int64_t i) {
  return dtype == 1 ? static_cast<const float*>(p)[i]
                    : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// The squares of a thread's elements in three ranges of fp32, so that no sum
// over- or underflows unnoticed; joined in fp64.
struct SquareSum {
  float mid = 0.f, big = 0.f, small = 0.f;
  __device__ __forceinline__ void add(float v) {
    mid = fmaf(v, v, mid);
    const float b = v * 0x1p-64f, s = v * 0x1p64f;
    big = fmaf(b, b, big);
    small = fmaf(s, s, small);
  }
  __device__ __forceinline__ double total() const {
    if (!(mid <= 3e38f)) return static_cast<double>(big) * 0x1p128;  // inf, or NaN (then big is too)
    return mid < 0x1p-90f ? static_cast<double>(small) * 0x1p-128 : static_cast<double>(mid);
  }
};

__global__ void __launch_bounds__(256) muon_momentum_kernel(const __grid_constant__ MuonArgs a) {
  __shared__ double sh[8];
  const MuonMat& t = a.mat[blockIdx.y];
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.ctrl[kCtrlError] = 0;
  const uint32_t step = a.norm_blocks * 256u;
  const uint32_t first = blockIdx.x * 256u + threadIdx.x;
  SquareSum q;
  if (a.vec) {
    const uint32_t per_row = a.cols / 4, total = per_row * static_cast<uint32_t>(a.rows);
    for (uint32_t i = first; i < total; i += step) {
      const uint32_t row = i / per_row, col = (i - row * per_row) * 4;
      float g[4];
      load4(t.grad, a.grad_dtype, row * t.ld_grad + col, g);
      if (t.momentum) {
        float4* mp = reinterpret_cast<float4*>(t.momentum + row * t.ld_momentum + col);
        float4 m = *mp;
        m.x = m.x * a.beta + g[0] * a.one_minus_beta;
        m.y = m.y * a.beta + g[1] * a.one_minus_beta;
        m.z = m.z * a.beta + g[2] * a.one_minus_beta;
        m.w = m.w * a.beta + g[3] * a.one_minus_beta;
        *mp = m;
        if (a.nesterov) {
          g[0] = m.x * a.beta + g[0] * a.one_minus_beta;
          g[1] = m.y * a.beta + g[1] * a.one_minus_beta;
          g[2] = m.z * a.beta + g[2] * a.one_minus_beta;
          g[3] = m.w * a.beta + g[3] * a.one_minus_beta;
        } else {
          g[0] = m.x, g[1] = m.y, g[2] = m.z, g[3] = m.w;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) q.add(g[j]);
    }
  } else {
    const uint64_t total = static_cast<uint64_t>(a.rows) * a.cols;
    for (uint64_t i = first; i < total; i += step) {
      const uint32_t row = static_cast<uint32_t>(i / static_cast<uint32_t>(a.cols));
      const uint32_t col = static_cast<uint32_t>(i - static_cast<uint64_t>(row) * a.cols);
      float g = load1(t.grad, a.grad_dtype, row * t.ld_grad + col);
      if (t.momentum) {
        float* mp = t.momentum + row * t.ld_momentum + col;
        const float m = *mp * a.beta + g * a.one_minus_beta;
        *mp = m;
        g = a.nesterov ? m * a.beta + g * a.one_minus_beta : m;
      }
      q.add(g);
    }
  }
  double s = q.total();
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int w = 0; w < 8; ++w) s += sh[w];
    a.norm[blockIdx.y * kMuonNormBlocks + blockIdx.x] = s;
  }
}

// ------------------------------------- X = u / (|u| + eps) in two fp16 parts

constexpr int kTile = 64;

__global__ void __launch_bounds__(256) muon_prepare_kernel(const __grid_constant__ MuonArgs a) {
  __shared__ float tile[kTile][kTile + 1];
  __shared__ double sh[8];
  const MuonMat& t = a.mat[blockIdx.y];
  const int tiles_c = (a.cols + kTile - 1) / kTile;
  const int r0 = (blockIdx.x / tiles_c) * kTile, c0 = (blockIdx.x % tiles_c) * kTile;
  // u of this tile, unscaled
  const int tc = threadIdx.x & (kTile - 1), tr = threadIdx.x / kTile;
  for (int r = tr; r < kTile; r += 256 / kTile) {
    float u = 0.f;
    if (r0 + r < a.rows && c0 + tc < a.cols) {
      const int64_t row = r0 + r, col = c0 + tc;
      if (t.momentum) {
        u = t.momentum[row * t.ld_momentum + col];
        if (a.nesterov) u = u * a.beta + load1(t.grad, a.grad_dtype, row * t.ld_grad + col) * a.one_minus_beta;
      } else {
        u = load1(t.grad, a.grad_dtype, row * t.ld_grad + col);
      }
    }
    tile[r][tc] = u;
  }
  double s = threadIdx.x < a.norm_blocks ? a.norm[blockIdx.y * kMuonNormBlocks + threadIdx.x] : 0.0;
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.0;
  for (int w = 0; w < 8; ++w) s += sh[w];
  const double inv = static_cast<double>(kXScale) / (sqrt(s) + a.eps);
  // in two factors, so that neither leaves fp32's normal range
  const float f1 = inv < 1e-30 ? 0x1p-64f : 1.f;
  const float f2 = static_cast<float>(inv < 1e-30 ? inv * 0x1p64 : inv);
  const int64_t base = static_cast<int64_t>(blockIdx.y) * a.m * a.ldx;
  for (int r = tr; r < kTile; r += 256 / kTile) {
    const float x = (a.transposed ? tile[tc][r] : tile[r][tc]) * f1 * f2;
    const int i = (a.transposed ? c0 : r0) + r, j = (a.transposed ? r0 : c0) + tc;
    if (i < a.m && j < a.n) {
      const __half h = __float2half_rn(x);
      const __half l = __float2half_rn(x - __half2float(h));
      const int64_t o = base + static_cast<int64_t>(i) * a.ldx + j;
      a.hi[0][o] = __half_as_ushort(h);
      a.lo[o] = __half_as_ushort(l);
    }
  }
}

// ------------------------------------------------------- the products

constexpr int kTM = 256, kTN = 256;
constexpr int kStages = 6;
constexpr uint32_t kABytes = 128 * kBK * 2;    // 16 KB: a CTA's 128 rows of A
constexpr uint32_t kBBytes = 128 * kBK * 2;    // 16 KB: its 128 columns of B
constexpr uint32_t kStageBytes = kABytes + kBBytes;
constexpr uint32_t kSmemBytes = 1024 + kStages * kStageBytes + (2 * kStages + 5) * 8 + 16;
constexpr uint32_t kTmemCols = 512;
constexpr int kThreads = 192;
constexpr int kEpiThreads = 128;
constexpr uint32_t kEpiBar = 1;

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t c0,
                                                 int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// fp16 operands: the type fields (bits 7-9 and 10-12) are 0
__host__ __device__ constexpr uint32_t idesc_f16_f32(uint32_t M, uint32_t N, uint32_t a_mn, uint32_t b_mn) {
  return (1u << 4) | (a_mn << 15) | (b_mn << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float2 unpack_half2(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, uint64_t timeout_ns) {
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > timeout_ns) return;
  }
}

struct MuonUnit {
  int mat, tm, tn;
};

// Work units: per matrix the tiles of the output, for the symmetric products
// only those with tm <= tn (column by column: column tn has tn + 1 of them).
template <int PHASE>
__device__ __forceinline__ MuonUnit muon_unit(int u, int tiles_m, int tiles_n) {
  MuonUnit r;
  if (PHASE == kMuonGram || PHASE == kMuonPoly) {
    const int per = tiles_m * (tiles_m + 1) / 2;
    r.mat = u / per;
    const int w = u - r.mat * per;
    int tn = static_cast<int>((sqrtf(8.f * w + 1.f) - 1.f) * 0.5f);
    while (tn * (tn + 1) / 2 > w) --tn;
    while ((tn + 1) * (tn + 2) / 2 <= w) ++tn;
    r.tn = tn;
    r.tm = w - tn * (tn + 1) / 2;
  } else {
    const int per = tiles_m * tiles_n;
    r.mat = u / per;
    const int w = u - r.mat * per;
    r.tm = w % tiles_m;
    r.tn = w / tiles_m;
  }
  return r;
}

// A row of 32 fp16 values as 16 words (16-byte aligned)
__device__ __forceinline__ void load_half32(const uint16_t* p, uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 v = *reinterpret_cast<const uint4*>(p + 8 * j);
    w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
  }
}
__device__ __forceinline__ void store_half32(uint16_t* p, const uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(p + 8 * j) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}

// One element of the result: the weight's update in place, or the update.
__device__ __forceinline__ void write_result(const MuonArgs& a, const MuonMat& t, int i, int j, float o) {
  const int64_t row = a.transposed ? j : i, col = a.transposed ? i : j;
  if (t.weight) {
    const int64_t at = row * t.ld_weight + col;
    if (a.weight_dtype == 1) {
      float* w = static_cast<float*>(t.weight) + at;
      *w = *w * a.decay - a.lr * o;
    } else {
      __nv_bfloat16* w = static_cast<__nv_bfloat16*>(t.weight) + at;
      *w = __float2bfloat16_rn(__bfloat162float(*w) * a.decay - a.lr * o);
    }
  } else {
    const int64_t at = row * t.ld_update + col;
    if (a.update_dtype == 1)
      static_cast<float*>(t.update)[at] = o;
    else
      static_cast<__nv_bfloat16*>(t.update)[at] = __float2bfloat16_rn(o);
  }
}

// The epilogue of 128 rows x 256 columns of an accumulator, one row per
// thread; `release` hands the accumulator back after its last read.
template <int PHASE, class Release>
__device__ __forceinline__ void muon_epilogue(const MuonArgs& a, const MuonStep& st, int mat, int m0, int n0,
                                              bool mirror, int row, uint32_t tbase, Release&& release) {
  const int i = m0 + row;
  const bool rvalid = i < a.m;
  constexpr bool kSym = PHASE == kMuonGram || PHASE == kMuonPoly;
  const int ncols = kSym ? a.m : a.n;
  float factor = 0.f;
  if (!kSym && rvalid) factor = st.a + a.diag[static_cast<int64_t>(mat) * a.m + i];
#pragma unroll 1
  for (int g = 0; g < kTN / 32; ++g) {
    __syncwarp();  // rows past the last leave the loop body early; the TMEM read is the whole warp's
    uint32_t r[32];
    tmem_ld_32x32b_x32(tbase + g * 32, r);
    tmem_ld_wait();
    tmem_regs_ready(r);
    const int c0 = n0 + g * 32;
    if (g == kTN / 32 - 1) release();
    if (!rvalid || c0 >= ncols) continue;
    if constexpr (kSym) {
      const int64_t base = static_cast<int64_t>(mat) * a.m * a.lda;
      uint16_t* out = (PHASE == kMuonGram ? a.gram : a.poly) + base;
      float v[32];
      if constexpr (PHASE == kMuonGram) {
#pragma unroll
        for (int q = 0; q < 32; ++q) v[q] = __uint_as_float(r[q]) * kGramScale;
      } else {
        uint32_t w[16];
        load_half32(a.gram + base + static_cast<int64_t>(i) * a.lda + c0, w);
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const float2 f = unpack_half2(w[q]);
          v[2 * q] = st.b * kPolyB * f.x + st.c * kPolyC * __uint_as_float(r[2 * q]);
          v[2 * q + 1] = st.b * kPolyB * f.y + st.c * kPolyC * __uint_as_float(r[2 * q + 1]);
        }
        if (i >= c0 && i < c0 + 32) {  // the diagonal stays in fp32, apart
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            if (c0 + q == i) {
              a.diag[static_cast<int64_t>(mat) * a.m + i] = v[q] * kPolyInv;
              v[q] = 0.f;
            }
          }
        }
      }
      uint32_t w[16];
#pragma unroll
      for (int q = 0; q < 16; ++q) w[q] = pack_half2(v[2 * q], v[2 * q + 1]);
      store_half32(out + static_cast<int64_t>(i) * a.lda + c0, w);
      if (mirror) {
#pragma unroll
        for (int q = 0; q < 32; ++q)
          if (c0 + q < a.m)
            out[static_cast<int64_t>(c0 + q) * a.lda + i] = static_cast<uint16_t>(w[q / 2] >> (16 * (q & 1)));
      }
    } else {
      const int64_t at = (static_cast<int64_t>(mat) * a.m + i) * a.ldx + c0;
      uint32_t h[16], l[16];
      load_half32(a.hi[st.src] + at, h);
      load_half32(a.lo + at, l);
      float x[32];
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const float2 fh = unpack_half2(h[q]), fl = unpack_half2(l[q]);
        x[2 * q] = factor * (fh.x + fl.x) + __uint_as_float(r[2 * q]) * kPolyInv;
        x[2 * q + 1] = factor * (fh.y + fl.y) + __uint_as_float(r[2 * q + 1]) * kPolyInv;
      }
      if constexpr (PHASE == kMuonApply) {
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          h[q] = pack_half2(x[2 * q], x[2 * q + 1]);
          const float2 f = unpack_half2(h[q]);
          l[q] = pack_half2(x[2 * q] - f.x, x[2 * q + 1] - f.y);
        }
        store_half32(a.hi[1 - st.src] + at, h);
        store_half32(a.lo + at, l);
      } else {
        const float sc = a.scale * kXInv;
#pragma unroll
        for (int q = 0; q < 32; ++q)
          if (c0 + q < a.n) write_result(a, a.mat[mat], i, c0 + q, x[q] * sc);
      }
    }
  }
}

// A persistent kernel of CTA pairs on 256 x 256 tiles (tcgen05 cta_group::2,
// each CTA holding its 128 rows of A and 128 columns of B per 64-deep
// k-block), the accumulator double-buffered in TMEM so that the epilogue of a
// tile overlaps the next tile's products. Warp 0 loads by TMA, warp 1 issues,
// warps 2..5 run the epilogue. Every wait is bounded.
template <int PHASE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    muon_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ MuonArgs a, const MuonStep st) {
  constexpr bool kSym = PHASE == kMuonGram || PHASE == kMuonPoly;
  constexpr int BMN = kSym ? 0 : 1;   // X as the right operand is contiguous along its columns
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kStages * kABytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sB + kStages * kBBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 5);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
  auto tfull_bar = [&](int acc) { return bar0 + 8u * (2 * kStages + acc); };
  auto tempty_bar = [&](int acc) { return bar0 + 8u * (2 * kStages + 2 + acc); };
  const uint32_t drain_bar = bar0 + 8u * (2 * kStages + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(cluster_id_x()), npairs = static_cast<int>(num_clusters_x());
  uint32_t* err = a.ctrl + kCtrlError;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int acc = 0; acc < 2; ++acc) {
      mbar_init(tfull_bar(acc), 1);
      mbar_init(tempty_bar(acc), 2 * kEpiThreads);
    }
    mbar_init(drain_bar, 1);
    fence_mbar_init();
    fence_proxy_async_smem();
    tma_prefetch_map(&tmA);
    tma_prefetch_map(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int tiles_m = (a.m + kTM - 1) / kTM;
  const int tiles_n = kSym ? tiles_m : (a.n + kTN - 1) / kTN;
  const int num_units = a.count * (kSym ? tiles_m * (tiles_m + 1) / 2 : tiles_m * tiles_n);
  const int num_kb = ((PHASE == kMuonGram ? a.n : a.m) + kBK - 1) / kBK;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t n_issued = 0;
      bool failed = false;
      for (int u = pair; u < num_units && !failed; u += npairs) {
        const MuonUnit t = muon_unit<PHASE>(u, tiles_m, tiles_n);
        const int mA = t.tm * kTM + static_cast<int>(rank) * 128;
        const int nB = t.tn * kTN + static_cast<int>(rank) * 128;
        for (int kb = 0; kb < num_kb; ++kb) {
          const int stage = n_issued % kStages;
          const uint32_t phase = (n_issued / kStages) & 1u;
          if (!mbar_wait_bounded_cluster(empty_bar(stage), phase ^ 1u, err, a.timeout_ns)) {
            failed = true;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2 * kStageBytes);
          const uint32_t fb = mapa_shared(full_bar(stage), 0);
          const uint32_t sa = smem_u32(sA + stage * kABytes);
          const uint32_t sb = smem_u32(sB + stage * kBBytes);
          const int k0 = kb * kBK;
          tma_load_3d_pair(sa, &tmA, fb, k0, mA, t.mat);
          if (BMN == 0) {
            tma_load_3d_pair(sb, &tmB, fb, k0, nB, t.mat);
          } else {
            tma_load_3d_pair(sb, &tmB, fb, nB, k0, t.mat);
            tma_load_3d_pair(sb + 8192, &tmB, fb, nB + 64, k0, t.mat);
          }
          ++n_issued;
        }
      }
      if (failed && rank == 0) {
        const uint32_t first = n_issued > kStages ? n_issued - kStages : 0;
        for (uint32_t i = first; i < n_issued; ++i)
          drain_wait(full_bar(i % kStages), (i / kStages) & 1u, a.timeout_ns);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_f16_f32(kTM, kTN, 0, BMN);
      uint32_t n_consumed = 0;
      bool issued = false, failed = false;
      int it = 0;
      for (int u = pair; u < num_units && !failed; u += npairs, ++it) {
        const int acc = it & 1;
        const uint32_t acc_phase = (it >> 1) & 1;
        if (!mbar_wait_bounded_cluster(tempty_bar(acc), acc_phase ^ 1u, err, a.timeout_ns)) {
          failed = true;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * kTN;
        for (int kb = 0; kb < num_kb; ++kb) {
          const int stage = n_consumed % kStages;
          const uint32_t phase = (n_consumed / kStages) & 1u;
          if (!mbar_wait_bounded_cluster(full_bar(stage), phase, err, a.timeout_ns)) {
            failed = true;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(sA + stage * kABytes);
          const uint32_t sb = smem_u32(sB + stage * kBBytes);
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k) {
            const uint64_t ad = smem_desc_sw128(sa + 32u * k, 16u, 1024u);
            const uint64_t bd = BMN ? smem_desc_sw128(sb + 2048u * k, 8192u, 1024u)
                                    : smem_desc_sw128(sb + 32u * k, 16u, 1024u);
            tc_mma_bf16_pair(d_tmem, ad, bd, idesc, (kb > 0 || k > 0) ? 1u : 0u);
          }
          issued = true;
          tc_commit_pair_multicast(empty_bar(stage), 0x3);
          ++n_consumed;
        }
        if (failed) break;
        tc_commit_pair_multicast(tfull_bar(acc), 0x3);
      }
      if (failed && issued) {
        tc_commit_pair(drain_bar);
        drain_wait(drain_bar, 0, a.timeout_ns);
      }
    }
  } else {
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    int it = 0;
    for (int u = pair; u < num_units; u += npairs, ++it) {
      const int acc = it & 1;
      const uint32_t acc_phase = (it >> 1) & 1;
      const bool ok = mbar_wait_bounded_cluster(tfull_bar(acc), acc_phase, err, a.timeout_ns);
      if (named_bar_or(kEpiBar, kEpiThreads, !ok)) break;
      tc_fence_after();
      const MuonUnit t = muon_unit<PHASE>(u, tiles_m, tiles_n);
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(wq * 32) << 16) + acc * kTN;
      muon_epilogue<PHASE>(a, st, t.mat, t.tm * kTM + static_cast<int>(rank) * 128, t.tn * kTN,
                           kSym && t.tm != t.tn, row, tbase, [&] {
                             tc_fence_before();
                             if (rank == 0)
                               mbar_arrive(tempty_bar(acc));
                             else
                               mbar_arrive_cluster(mapa_shared(tempty_bar(acc), 0));
                           });
    }
  }

  __syncwarp();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
  if (threadIdx.x == 0) {
    const uint32_t code = ld_volatile_u32(err);
    if (code != 0) *reinterpret_cast<volatile uint32_t*>(a.host_error) = code;
  }
}

template <int PHASE>
cudaError_t launch_phase(const CUtensorMap& ta, const CUtensorMap& tb, const MuonArgs& a, const MuonStep& st,
                         int pairs, cudaStream_t s) {
  auto kern = muon_gemm_kernel<PHASE>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmemBytes));
  if (e != cudaSuccess) return e;
  const int tiles_m = (a.m + kTM - 1) / kTM, tiles_n = (a.n + kTN - 1) / kTN;
  const bool sym = PHASE == kMuonGram || PHASE == kMuonPoly;
  const int64_t units = static_cast<int64_t>(a.count) * (sym ? tiles_m * (tiles_m + 1) / 2 : tiles_m * tiles_n);
  if (units < pairs) pairs = static_cast<int>(units);
  kern<<<2 * pairs, kThreads, kSmemBytes, s>>>(ta, tb, a, st);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_muon_momentum(const MuonArgs& a, cudaStream_t s) {
  muon_momentum_kernel<<<dim3(a.norm_blocks, a.count), 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_muon_prepare(const MuonArgs& a, cudaStream_t s) {
  const int tiles = ((a.rows + kTile - 1) / kTile) * ((a.cols + kTile - 1) / kTile);
  muon_prepare_kernel<<<dim3(tiles, a.count), 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_muon_gemm(int phase, const CUtensorMap& ta, const CUtensorMap& tb, const MuonArgs& a,
                             const MuonStep& st, int pairs, cudaStream_t s) {
  switch (phase) {
    case kMuonGram: return launch_phase<kMuonGram>(ta, tb, a, st, pairs, s);
    case kMuonPoly: return launch_phase<kMuonPoly>(ta, tb, a, st, pairs, s);
    case kMuonApply: return launch_phase<kMuonApply>(ta, tb, a, st, pairs, s);
    case kMuonLast: return launch_phase<kMuonLast>(ta, tb, a, st, pairs, s);
    default: return cudaErrorInvalidValue;
  }
}

// Clusters of two that fit on the device at once
int muon_max_clusters() {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto kern = muon_gemm_kernel<kMuonApply>;
  int n = 0;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes)) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

}  // namespace flce
