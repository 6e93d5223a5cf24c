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
// a X must not. The diagonal of B, the largest part of it, multiplies X's high
// part in fp32 in the epilogue, and of the low part what is common to 32 rows
// (part_factors; all of B meets the same matrix), and the product runs on B
// with a zero diagonal. So what the roundings of A, B and X's high part add
// stays in the row and column spaces that X has, and is not raised. This leaves
// 1e-4 to 4.3e-3 relative error (Gaussian, decaying and low-rank spectra), of the order
// of one bf16 rounding of the result (1.7e-3); iterates rounded to bf16 are
// 1e-2 off on Gaussian matrices and 0.15 to 1 on the others.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "flce_muon.cuh"

namespace flce {
namespace {

// ------------------------------------------------- momentum and norm

// One pass over gradient and momentum: bound by HBM (10 or 12 bytes read and
// written per element). Four vectors of four elements are in flight per
// thread: 4096 x 16384 in bf16 moves 671 MB in 121 us, 5.5 TB/s.
__global__ void __launch_bounds__(256) muon_momentum_kernel(const __grid_constant__ MuonArgs a) {
  __shared__ double sh[8];
  const MuonMat& t = a.mat[blockIdx.y];
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (blockIdx.y == 0) a.ctrl[kCtrlError] = 0;
    a.done[blockIdx.y] = 0;
    a.partial[blockIdx.y] = 0;
  }
  const uint32_t step = a.norm_blocks * 256u;
  const uint32_t first = blockIdx.x * 256u + threadIdx.x;
  SquareSum q;
  if (a.vec) {
    constexpr int kAhead = 4;
    const uint32_t per_row = a.cols / 4, total = per_row * static_cast<uint32_t>(a.rows);
    for (uint32_t i0 = first; i0 < total; i0 += kAhead * step) {
      float g[kAhead][4];
      float4 m[kAhead];
      int64_t at[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const uint32_t i = i0 + j * step;
        if (i < total) {
          uint32_t row = 0, col = i;  // a matrix without gaps is one long row
          if (!a.flat) {
            row = i / per_row;
            col = i - row * per_row;
          }
          load4(t.grad, a.grad_dtype, row * t.ld_grad + 4 * static_cast<int64_t>(col), g[j]);
          if (t.momentum) {
            at[j] = row * t.ld_momentum + 4 * static_cast<int64_t>(col);
            m[j] = *reinterpret_cast<const float4*>(t.momentum + at[j]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (i0 + j * step < total) {
          if (t.momentum) {
            momentum4(a, m[j], g[j]);
            *reinterpret_cast<float4*>(t.momentum + at[j]) = m[j];
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) q.add(g[j][e]);
        }
      }
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
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  q.reduce_warp();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = q.total();
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < 8; ++w) s += sh[w];
    a.norm[blockIdx.y * kMuonNormBlocks + blockIdx.x] = pack_sum(s);
  }
}

// ------------------------------------- X = u / (|u| + eps) in two fp16 parts

constexpr int kTile = 64;

// Where rows stay rows (and are aligned), 16 rows x 256 columns per turn of a
// block, 8 neighbours per thread. Else 64 x 64 tiles through shared memory,
// which transposes them where X is the transpose. Whole 16-byte stores either
// way: a row of X has room to a multiple of 64 elements, and what lies past the
// matrix is zero. Bound by HBM (10 or 8 bytes read, 4 written per element).
__global__ void __launch_bounds__(256) muon_prepare_kernel(const __grid_constant__ MuonArgs a) {
  __shared__ float tile[kTile][kTile + 1];
  __shared__ float sh[2], sh_m[8];
  __shared__ int sh_e[8];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const MuonMat& t = a.mat[blockIdx.y];
  // Every block takes the factor from the partial sums itself, once, in 32-bit
  // arithmetic: fp64 runs at a sixty-fourth of fp32's rate (a block per 64 x 64
  // tile, each with one warp's fp64 sum, took 163 us at 4096 x 16384; this 140,
  // where HBM's bound is 99).
  float mant[kMuonNormBlocks / 256];
  int expo[kMuonNormBlocks / 256], top = -30000;
#pragma unroll
  for (int j = 0; j < kMuonNormBlocks / 256; ++j) {
    const int i = threadIdx.x + 256 * j;
    const float2 v =
        i < a.norm_blocks ? a.norm[blockIdx.y * kMuonNormBlocks + i] : make_float2(0.f, __int_as_float(-30000));
    mant[j] = v.x;
    expo[j] = __float_as_int(v.y);
    top = max(top, expo[j]);
  }
  top = __reduce_max_sync(kAll, top);
  if ((threadIdx.x & 31) == 0) sh_e[threadIdx.x >> 5] = top;
  __syncthreads();
  top = __reduce_max_sync(kAll, sh_e[threadIdx.x & 7]);
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < kMuonNormBlocks / 256; ++j) s += mant[j] * exp2f(static_cast<float>(max(expo[j] - top, -200)));
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
  if ((threadIdx.x & 31) == 0) sh_m[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.f;
    for (int w = 0; w < 8; ++w) s += sh_m[w];
    norm_factors(ldexp(static_cast<double>(s), top), a.eps, sh);
  }
  __syncthreads();
  const float f1 = sh[0], f2 = sh[1];

  // four neighbours of u at (row, col), unscaled
  auto u4 = [&](int64_t row, int64_t col, float (&u)[4]) {
    u[0] = u[1] = u[2] = u[3] = 0.f;
    if (row < a.rows && col < a.cols) {
      if (!t.momentum || a.nesterov) load4(t.grad, a.grad_dtype, row * t.ld_grad + col, u);
      if (t.momentum) {
        const float4 m = *reinterpret_cast<const float4*>(t.momentum + row * t.ld_momentum + col);
        const float mv[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = a.nesterov ? mv[e] * a.beta + u[e] * a.one_minus_beta : mv[e];
      }
    }
  };
  // eight neighbours of X at (i, j)
  const int64_t base = static_cast<int64_t>(blockIdx.y) * a.m * a.ldx;
  auto x8 = [&](int i, int j, const float (&u)[8]) {
    if (i >= a.m || j >= a.ldx) return;
    uint32_t h[4], l[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) split_half2(u[2 * q] * f1 * f2, u[2 * q + 1] * f1 * f2, h[q], l[q]);
    const int64_t o = base + static_cast<int64_t>(i) * a.ldx + j;
    *reinterpret_cast<uint4*>(a.hi[0] + o) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(a.lo + o) = make_uint4(l[0], l[1], l[2], l[3]);
  };

  if (a.vec && !a.transposed) {
    const int tiles_c = (a.cols + 255) / 256, tiles = tiles_c * ((a.rows + 15) / 16);
    for (int tl = blockIdx.x; tl < tiles; tl += gridDim.x) {
      const int r = (tl / tiles_c) * 16 + (threadIdx.x >> 5), c = (tl % tiles_c) * 256 + (threadIdx.x & 31) * 8;
      float u[2][2][4];
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        u4(r + 8 * it, c, u[it][0]);
        u4(r + 8 * it, c + 4, u[it][1]);
      }
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        const float v[8] = {u[it][0][0], u[it][0][1], u[it][0][2], u[it][0][3],
                            u[it][1][0], u[it][1][1], u[it][1][2], u[it][1][3]};
        x8(r + 8 * it, c, v);
      }
    }
    return;
  }
  const int tiles_c = (a.cols + kTile - 1) / kTile, tiles = tiles_c * ((a.rows + kTile - 1) / kTile);
  for (int tl = blockIdx.x; tl < tiles; tl += gridDim.x) {
    const int r0 = (tl / tiles_c) * kTile, c0 = (tl % tiles_c) * kTile;
    if (a.vec) {
      const int c = 4 * (threadIdx.x & 15);
      float u[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) u4(r0 + (threadIdx.x >> 4) + 16 * j, c0 + c, u[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) tile[(threadIdx.x >> 4) + 16 * j][c + e] = u[j][e];
    } else {
      const int tc = threadIdx.x & (kTile - 1), tr = threadIdx.x / kTile;
#pragma unroll 8
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
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      const int idx = threadIdx.x + 256 * it, r = idx >> 3, c = (idx & 7) * 8;
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = a.transposed ? tile[c + q][r] : tile[r][c + q];
      x8((a.transposed ? c0 : r0) + r, (a.transposed ? r0 : c0) + c, v);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------- the products

// Output tiles. SINGLE: 128 x 128 on one CTA. PAIR: 256 x 256 on a CTA pair
// (tcgen05 cta_group::2, each CTA holding its 128 rows of A and 128 columns of
// B). WIDE: 256 x 512 on a CTA pair, two products per k-step that share their A
// operand through the tensor core's collector buffer. kBufs: 32-column groups
// that an epilogue warp holds at once. PAIR has all its four, so that all loads
// run while the products do, for two stages less (2048 x 2048: 317 us, with two
// groups and five stages 322; 4096 x 4096, which is WIDE's: 1214 and 1142).
template <int SHAPE>
struct MuonTile;
template <>
struct MuonTile<kMuonSingle> {
  static constexpr int kM = 128, kN = 128, kAccs = 2, kStages = 5, kBufs = 2;
};
template <>
struct MuonTile<kMuonPair> {
  static constexpr int kM = 256, kN = 256, kAccs = 2, kStages = 3, kBufs = 4;
};
template <>
struct MuonTile<kMuonWide> {
  static constexpr int kM = 256, kN = 512, kAccs = 1, kStages = 3, kBufs = 2;
};

constexpr uint32_t kPartBytes = 128 * kBK * 2;  // 16 KB: 128 rows or columns of a 64-deep k-block
constexpr int kThreads = 384;                   // warp 0 loads, warp 1 issues, warps 4..11 run the epilogue
constexpr int kEpiThreads = 256;
constexpr uint32_t kEpiBar = 1;                 // their named barrier
// per epilogue warp kBufs buffers of 32 rows x 32 fp16 columns, twice (X hi and
// lo; a tile and its mirror image; one fp32 tile)
constexpr uint32_t kEpiPart = 32 * 64;
template <int SHAPE>
constexpr uint32_t epi_bytes() {
  return 8 * MuonTile<SHAPE>::kBufs * 2 * kEpiPart;
}
template <int SHAPE>
constexpr uint32_t stage_bytes() {
  return (SHAPE == kMuonWide ? 3 : 2) * kPartBytes;
}
template <int SHAPE>
constexpr uint32_t smem_bytes() {
  constexpr int stages = MuonTile<SHAPE>::kStages;
  return 1024 + stages * stage_bytes<SHAPE>() + epi_bytes<SHAPE>() + (2 * stages + 5 + 8 * MuonTile<SHAPE>::kBufs) * 8 + 16;
}
static_assert(smem_bytes<kMuonSingle>() <= 232448 && smem_bytes<kMuonPair>() <= 232448 && smem_bytes<kMuonWide>() <= 232448, "shared memory per CTA");

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t c0,
                                                 int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

struct MuonUnit {
  int mat, tm, tn;
};

// Work units: per matrix the tiles of the output. Of the symmetric products
// only the tiles that reach the diagonal or lie above it, column by column:
// tile column tn has the rows 0 .. R (tn + 1) - 1, R tile rows to a tile
// column's width, but no more than there are (the last column).
template <int SHAPE>
__host__ __device__ __forceinline__ int muon_units_per_matrix(bool sym, int tiles_m, int tiles_n) {
  if (!sym) return tiles_m * tiles_n;
  constexpr int R = MuonTile<SHAPE>::kN / MuonTile<SHAPE>::kM;
  return R * tiles_n * (tiles_n + 1) / 2 - (R * tiles_n - tiles_m);
}

// The work of one launch, as one sequence: steps, in each the three products,
// in each the matrices one after another, and their tiles. Unit g of it is
// slot g mod (number of slots)'s. Every role of a CTA walks it by itself.
template <int SHAPE>
struct MuonWalk {
  using Tile = MuonTile<SHAPE>;
  int tiles_m, tiles_s, tiles_n;   // tile rows; tile columns of the symmetric products and of B X
  int per_s, per_x;                // tiles per matrix of either
  int count, slots, steps, splits;
  int step = 0, phase = 0, u;
  int mat, tile, split, tm, tn;

  __device__ __forceinline__ MuonWalk(const MuonArgs& a, int steps_, int slot, int slots_)
      : count(a.count), slots(slots_), steps(steps_), splits(a.splits), u(slot) {
    tiles_m = (a.m + Tile::kM - 1) / Tile::kM;
    tiles_s = (a.m + Tile::kN - 1) / Tile::kN;
    tiles_n = (a.n + Tile::kN - 1) / Tile::kN;
    per_s = muon_units_per_matrix<SHAPE>(true, tiles_m, tiles_s);
    per_x = muon_units_per_matrix<SHAPE>(false, tiles_m, tiles_n);
  }
  __device__ __forceinline__ bool symmetric() const { return phase < kMuonApply; }
  // Units of a matrix: X Xt, whose sum may be split over several units per
  // tile, has its tiles once per split, the last split (which adds the others)
  // last.
  __device__ __forceinline__ int per_matrix() const {
    return phase == kMuonGram ? per_s * splits : phase == kMuonPoly ? per_s : per_x;
  }
  // to the unit at u; false past the last
  __device__ __forceinline__ bool locate() {
    for (;;) {
      const int units = count * per_matrix();
      if (u < units) break;
      u -= units;
      if (++phase == 3) {
        phase = 0;
        if (++step == steps) return false;
      }
    }
    const int per = per_matrix();
    mat = u / per;
    int w = u - mat * per;
    split = splits - 1;
    if (phase == kMuonGram && splits > 1) {
      split = w / per_s;
      w -= split * per_s;
    }
    tile = w;
    if (symmetric()) {
      // columns before tn hold R tn (tn + 1) / 2 tiles
      constexpr int R = Tile::kN / Tile::kM;
      tn = static_cast<int>((sqrtf(8.f / R * w + 1.f) - 1.f) * 0.5f);
      while (R * tn * (tn + 1) / 2 > w) --tn;
      while (R * (tn + 1) * (tn + 2) / 2 <= w) ++tn;
      tm = w - R * tn * (tn + 1) / 2;
    } else {
      tm = w % tiles_m;
      tn = w / tiles_m;
    }
    return true;
  }
  __device__ __forceinline__ void advance() { u += slots; }
  // tiles of this matrix that come before this product: all of them are read by it
  __device__ __forceinline__ uint32_t needed() const {
    return static_cast<uint32_t>(step * (2 * per_s + per_x) + phase * per_s);
  }
};

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void add_release(uint32_t* p, uint32_t v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Waits until a matrix's count of finished tile parts has reached `target`
// (it only grows), bounded like every other wait; then later TMA accesses of
// this thread are ordered behind what the count stands for.
__device__ __forceinline__ bool wait_done(const uint32_t* done, uint32_t target, uint32_t* err, uint64_t timeout_ns) {
  if (ld_acquire(done) < target) {
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    for (uint32_t it = 0; ld_acquire(done) < target; ++it) {
      if ((it & 31u) != 31u) continue;
      if (ld_volatile_u32(err) != 0u) return false;
      if (globaltimer_ns() - t0 > timeout_ns) {
        atomicCAS(err, 0u, kErrTimeout);
        return false;
      }
    }
  }
  asm volatile("fence.proxy.async;" ::: "memory");
  return true;
}

// `rows` rows of 32 result columns from a warp's staged fp32 block [32][32]
// (16-byte chunks swizzled by the row): half a warp per row, two columns per
// lane; a weight's eight rows are read before the first is written.
template <bool W, class T>
__device__ __forceinline__ void write_rows(T* out, int64_t ld, int rows, int cols, bool pairs, float decay, float lr,
                                           const float* block, int lane) {
  using T2 = typename PairOf<T>::type;
  const int c = 2 * (lane & 15), r1 = lane >> 4;
  if (c >= cols) return;
  auto staged = [&](int r) {
    return *reinterpret_cast<const float2*>(block + r * 32 + (((c >> 2) ^ (r & 7)) << 2) + (c & 3));
  };
  T* p = out + r1 * ld + c;
  if (pairs && c + 1 < cols) {
#pragma unroll
    for (int r0 = 0; r0 < 32; r0 += 16) {
      T2 w[8];
      if (W) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (r0 + r1 + 2 * j < rows) w[j] = *reinterpret_cast<const T2*>(p + (r0 + 2 * j) * ld);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = r0 + r1 + 2 * j;
        if (r < rows) {
          float2 o = staged(r);
          if (W) {
            const float2 v = to_float2(w[j]);
            o = make_float2(v.x * decay - lr * o.x, v.y * decay - lr * o.y);
          }
          put(reinterpret_cast<T2*>(p + (r0 + 2 * j) * ld), o);
        }
      }
    }
  } else {
    for (int r = r1; r < rows; r += 2) {
      const float2 o = staged(r);
      T* q = p + (r - r1) * ld;
      put(q, W ? to_float(q[0]) * decay - lr * o.x : o.x);
      if (c + 1 < cols) put(q + 1, W ? to_float(q[1]) * decay - lr * o.y : o.y);
    }
  }
}

// The epilogue of one warp: 32 rows (TMEM lanes) of one half of a tile's
// columns, in groups of 32. What a group reads (X hi and lo, or A) comes by TMA
// into the warp's own buffers, for a tile's first groups before its products
// are done; what it writes leaves the same buffers by TMA stores. So global
// memory sees runs of 64 bytes and more, and no warp waits for another. (With
// each thread reading and writing its own row in global memory every access
// touched 32 lines: B X of 8 x 1024 x 1024 took 36.8 us, its products 8.7.)
// BOTH: A and B are one block of 32 x 32, in two parts as X is.
template <uint32_t BUFS, bool BOTH>
struct MuonEpilogue {
  const MuonArgs& a;
  uint8_t* buf;        // this warp's BUFS x 2 x kEpiPart
  uint32_t bar;        // this warp's BUFS load barriers
  int lane;
  uint32_t loads = 0, uses = 0;   // groups loaded, groups taken

  // TMA loads of the group at column c0 into the next buffer: X hi and lo, or A
  __device__ __forceinline__ void load(const CUtensorMap* e0, const CUtensorMap* e1, int mat, int row0, int c0) {
    __syncwarp();   // every lane has read what the buffer held
    if (lane == 0) {
      bulk_wait_group_read<0>();  // the buffer's last stores have read it
      const uint32_t b = loads % BUFS;
      const uint32_t dst = smem_u32(buf + b * 2 * kEpiPart), bb = bar + 8u * b;
      mbar_arrive_expect_tx(bb, e1 ? 2 * kEpiPart : kEpiPart);
      tma_load_3d(dst, e0, bb, c0, row0, mat);
      if (e1) tma_load_3d(dst + kEpiPart, e1, bb, c0, row0, mat);
    }
    ++loads;
  }

  // a weight's lines under this warp's rows and columns into L2, while the
  // products run
  __device__ __forceinline__ void prefetch_weight(int mat, int row0, int c0, int width) {
    const MuonMat& t = a.mat[mat];
    if (!t.weight) return;
    const int es = a.weight_dtype == 1 ? 4 : 2;
    const char* w = static_cast<const char*>(t.weight);
    const int cols = min(width, a.n - c0), rows = min(32, a.m - row0);
    if (a.transposed) {  // `cols` rows of `rows` elements
      for (int r = lane; r < cols; r += 32)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(w + ((c0 + r) * t.ld_weight + row0) * es));
    } else if (lane < rows) {
      const char* p = w + ((row0 + lane) * t.ld_weight + c0) * es;
      for (int b = 0; b < cols * es; b += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + b));
    }
  }

  // columns c0 .. c0 + 31 of the warp's rows, accumulator values in r; written
  // to o0 and, a mirror image or the low part, to o1
  template <int PHASE>
  __device__ __forceinline__ bool group(const MuonStep& st, const CUtensorMap* o0, const CUtensorMap* o1, int g, int mat,
                                        int row0, int c0, bool mirror, float2 factor, const uint32_t (&r)[32]) {
    constexpr bool kSym = PHASE == kMuonGram || PHASE == kMuonPoly;
    const uint32_t b = PHASE == kMuonGram ? g % BUFS : uses % BUFS;
    uint8_t* p0 = buf + b * 2 * kEpiPart;
    uint8_t* p1 = p0 + kEpiPart;
    if (PHASE != kMuonGram) {
      if (!__all_sync(kAll, mbar_wait_bounded(bar + 8u * b, (uses / BUFS) & 1u, a.ctrl + kCtrlError, a.timeout_ns)))
        return false;
      ++uses;
    } else {
      // the buffer's last stores have read it (other products left either buffer's)
      if (lane == 0) {
        if (g == 0)
          bulk_wait_group_read<0>();
        else
          bulk_wait_group_read<BUFS - 1>();
      }
      __syncwarp();
    }
    uint4* q0 = reinterpret_cast<uint4*>(p0 + lane * 64);
    uint4* q1 = reinterpret_cast<uint4*>(p1 + lane * 64);
    const int sw = (lane >> 1) & 3;   // 64-byte swizzle: chunk j of a row sits at chunk j ^ (row / 2 % 4)
    auto acc = [&](int i) { return __uint_as_float(r[i]); };
    if constexpr (kSym) {
      const int i = row0 + lane;
      float on_diag = 0.f;
      uint16_t* mir = reinterpret_cast<uint16_t*>(p1) + lane;   // [32][32], its columns are this tile's rows
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[8];
        if constexpr (PHASE == kMuonGram) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = acc(8 * j + e) * kGramScale;
        } else {
          const uint4 w = q0[j ^ sw];
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
          uint4 wl = make_uint4(0, 0, 0, 0);
          if constexpr (BOTH) wl = q1[j ^ sw];
          const uint32_t wwl[4] = {wl.x, wl.y, wl.z, wl.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 f = unpack_half2(ww[e]);
            if constexpr (BOTH) {
              const float2 fl = unpack_half2(wwl[e]);
              f.x += fl.x, f.y += fl.y;
            }
            v[2 * e] = st.b * kPolyB * f.x + st.c * kPolyC * acc(8 * j + 2 * e);
            v[2 * e + 1] = st.b * kPolyB * f.y + st.c * kPolyC * acc(8 * j + 2 * e + 1);
          }
          // the diagonal stays in fp32, apart (by selects: a branch per element
          // costs more than the rest of the epilogue)
          if (c0 == row0) {
            const int d = lane - 8 * j;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              on_diag = e == d ? v[e] : on_diag;
              v[e] = e == d ? 0.f : v[e];
            }
          }
        }
        uint32_t w[4];
        if constexpr (BOTH) {
          uint32_t l[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) split_half2(v[2 * e], v[2 * e + 1], w[e], l[e]);
          q1[j ^ sw] = make_uint4(l[0], l[1], l[2], l[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = pack_half2(v[2 * e], v[2 * e + 1]);
        }
        q0[j ^ sw] = make_uint4(w[0], w[1], w[2], w[3]);
        if (!BOTH && mirror) {
#pragma unroll
          for (int e = 0; e < 8; ++e) mir[(8 * j + e) * 32] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
        }
      }
      if (PHASE == kMuonPoly && c0 == row0 && i < a.m)
        a.diag[static_cast<int64_t>(mat) * a.m + i] = on_diag * kPolyInv;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d(o0, smem_u32(p0), c0, row0, mat);
        if (BOTH)
          tma_store_3d(o1, smem_u32(p1), c0, row0, mat);
        else if (mirror)
          tma_store_3d(o1, smem_u32(p1), row0, c0, mat);
        bulk_commit_group();
      }
      __syncwarp();
    } else {
      float x[32];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 wh = q0[j ^ sw], wl = q1[j ^ sw];
        uint32_t h[4] = {wh.x, wh.y, wh.z, wh.w}, l[4] = {wl.x, wl.y, wl.z, wl.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 fh = unpack_half2(h[e]), fl = unpack_half2(l[e]);
          float* y = x + 8 * j + 2 * e;
          y[0] = factor.x * fh.x + (factor.y * fl.x + acc(8 * j + 2 * e) * kPolyInv);
          y[1] = factor.x * fh.y + (factor.y * fl.y + acc(8 * j + 2 * e + 1) * kPolyInv);
          if constexpr (PHASE == kMuonApply) split_half2(y[0], y[1], h[e], l[e]);
        }
        if constexpr (PHASE == kMuonApply) {
          q0[j ^ sw] = make_uint4(h[0], h[1], h[2], h[3]);
          q1[j ^ sw] = make_uint4(l[0], l[1], l[2], l[3]);
        }
      }
      if constexpr (PHASE == kMuonApply) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(o0, smem_u32(p0), c0, row0, mat);
          tma_store_3d(o1, smem_u32(p1), c0, row0, mat);
          bulk_commit_group();
        }
        __syncwarp();
      } else {
        const float sc = a.scale * kXInv;
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] *= sc;
        if (a.transposed) {
          // out[c0 + ..][row0 + lane]: the lanes' columns are neighbours
          with_result(a, a.mat[mat], [&](auto* out, auto W, int64_t ld) {
            if (row0 + lane < a.m)
              write_columns<decltype(W)::value>(out + c0 * ld + row0 + lane, ld, min(32, a.n - c0), a.decay, a.lr, x);
          });
        } else {
          // as fp32 where hi and lo were (every lane has read its own)
          float* block = reinterpret_cast<float*>(p0);
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float4*>(block + lane * 32 + ((j ^ (lane & 7)) << 2)) =
                make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
          __syncwarp();
          with_result(a, a.mat[mat], [&](auto* out, auto W, int64_t ld) {
            write_rows<decltype(W)::value>(out + row0 * ld + c0, ld, min(32, a.m - row0), min(32, a.n - c0), a.pairs,
                                           a.decay, a.lr, block, lane);
          });
          fence_proxy_async_smem();  // the next load overwrites what was written here
          __syncwarp();
        }
      }
    }
    return true;
  }
};

// All steps of a group of matrices in one persistent launch. PAIR and SINGLE
// tiles have two accumulators in TMEM, so that the epilogue of a tile overlaps
// the next tile's products; a WIDE tile fills TMEM, and the next tile's
// products wait until its columns have been read.
//
// A product reads what the products before it wrote for the same matrix. A CTA
// adds to the matrix's counter when its part of a tile is in global memory, and
// a tile's loads wait for the counter to reach all earlier tiles of that matrix.
// So one matrix's tiles fill the time in which another's are still to finish,
// and a product starts a flag's latency after its predecessor instead of a
// launch's. Every slot takes its units in the order of the sequence and all slots
// are resident (a cooperative launch), so a unit only ever waits for units that
// run. Every wait is bounded.
//
// Small and middle sizes are bound by that chain: 8 x 1024 x 1024 takes 43 us a
// step, of which its products need 17 (as a launch per product it took 57); 256 x
// 256 takes 16. Large ones by the tensor cores: 4096 x 4096, five steps of 1.37
// TFLOP together, in 1.0 ms (80 % of the library's sustained bf16 rate), 4096 x
// 16384 in 3.07 ms (85 %).
//
// BOTH (a short side up to kMuonPairSide): each product is three, high x high, low
// x high and high x low parts, into one accumulator. X Xt and A A take them from
// one loaded k-block, high part as A and low part as B (X and A are one tile high);
// B X, which is a single k-block, loads it three times. 32 x 8192: 156 us, with one
// product each 119 and 1e-3 more error. (Shorter matrices run in one launch.)
template <int SHAPE, bool BOTH>
__global__ void __cluster_dims__(SHAPE == kMuonSingle ? 1 : 2, 1, 1) __launch_bounds__(kThreads, 1)
    muon_steps_kernel(const __grid_constant__ std::conditional_t<BOTH, MuonPairMaps, MuonMaps> maps,
                      const __grid_constant__ MuonArgs a, const __grid_constant__ MuonSteps steps) {
  using Tile = MuonTile<SHAPE>;
  constexpr bool kPaired = SHAPE != kMuonSingle, kWide = SHAPE == kMuonWide;
  constexpr int kStages = Tile::kStages, kAccs = Tile::kAccs, kBufs = Tile::kBufs;
  constexpr uint32_t kStageBytes = stage_bytes<SHAPE>();
  constexpr uint32_t kTmemCols = kAccs * Tile::kN;
  constexpr uint32_t kParts = kPaired ? 2 : 1;   // CTAs of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sE = smem + kStages * kStageBytes;   // a stage: A, B (wide: B of either half)
  uint64_t* bars = reinterpret_cast<uint64_t*>(sE + epi_bytes<SHAPE>());
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 5 + 8 * kBufs);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
  auto tfull_bar = [&](int acc) { return bar0 + 8u * (2 * kStages + acc); };
  auto tempty_bar = [&](int acc) { return bar0 + 8u * (2 * kStages + 2 + acc); };
  const uint32_t drain_bar = bar0 + 8u * (2 * kStages + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kPaired ? cluster_ctarank() : 0u;
  const int slot = kPaired ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int slots = kPaired ? static_cast<int>(num_clusters_x()) : static_cast<int>(gridDim.x);
  uint32_t* err = a.ctrl + kCtrlError;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return kPaired ? mbar_wait_bounded_cluster(bar, parity, err, a.timeout_ns)
                   : mbar_wait_bounded(bar, parity, err, a.timeout_ns);
  };
  // an arrival, when the products issued so far are done, in every CTA of the unit
  auto commit = [&](uint32_t bar) {
    if (kPaired)
      tc_commit_pair_multicast(bar, 0x3);
    else
      tc_commit(bar);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int acc = 0; acc < kAccs; ++acc) {
      mbar_init(tfull_bar(acc), 1);
      mbar_init(tempty_bar(acc), (kPaired ? 2 : 1) * kEpiThreads);
    }
    mbar_init(drain_bar, 1);
    for (int i = 0; i < 8 * kBufs; ++i) mbar_init(drain_bar + 8u * (1 + i), 1);  // the epilogue warps' loads
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    if (kPaired) {
      tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), kTmemCols);
      tmem_relinquish();
    }
  }
  if (warp == 2 && lane < static_cast<int>(sizeof(maps) / sizeof(CUtensorMap)))
    tma_prefetch_map(reinterpret_cast<const CUtensorMap*>(&maps) + lane);
  __syncthreads();
  if (kPaired) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // k-blocks of X Xt, of one of its splits, of the other products
  const int kb_n = (a.n + kBK - 1) / kBK, kb_split = (kb_n + a.splits - 1) / a.splits, kb_m = (a.m + kBK - 1) / kBK;
  auto gram_blocks = [&](int split) { return min(kb_split, kb_n - split * kb_split); };
  MuonWalk<SHAPE> w(a, steps.count, slot, slots);

  if (warp == 0) {
    if (lane == 0) {
      uint32_t n_issued = 0;
      bool failed = false;
      int seen_mat = -1;
      uint32_t seen = 0;
      for (; !failed && w.locate(); w.advance()) {
        const int src = w.step & 1;
        const CUtensorMap* ma = w.phase == kMuonGram ? &maps.xk[src] : w.phase == kMuonPoly ? &maps.gk : &maps.pk;
        const CUtensorMap* mb = w.phase == kMuonGram ? &maps.xk[src] : w.phase == kMuonPoly ? &maps.gk : &maps.xn[src];
        const uint32_t needed = w.needed() * kParts;
        if (w.mat != seen_mat || needed != seen) {
          if (needed > 0 && !wait_done(a.done + w.mat, needed + a.hold, err, a.timeout_ns)) {
            failed = true;
            break;
          }
          seen_mat = w.mat;
          seen = needed;
        }
        const int mA = w.tm * Tile::kM + static_cast<int>(rank) * 128;
        const int nB = w.tn * Tile::kN + static_cast<int>(rank) * 128;
        const int num_kb = w.phase == kMuonGram ? gram_blocks(w.split) : kb_m;
        const int k_first = w.phase == kMuonGram ? w.split * kb_split * kBK : 0;
        for (int kb = 0, blocks = num_kb * (BOTH && !w.symmetric() ? 3 : 1); kb < blocks; ++kb) {
          const int stage = n_issued % kStages;
          const uint32_t phase = (n_issued / kStages) & 1u;
          if (!wait(empty_bar(stage), phase ^ 1u)) {
            failed = true;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), (kPaired ? 2 : 1) * kStageBytes);
          const uint32_t fb = kPaired ? mapa_shared(full_bar(stage), 0) : full_bar(stage);
          const uint32_t sa = smem_u32(smem + stage * kStageBytes);
          const int k0 = k_first + (BOTH && !w.symmetric() ? 0 : kb) * kBK;
          const CUtensorMap *pa = ma, *pb = mb;
          if constexpr (BOTH) {
            if (w.symmetric())
              pb = w.phase == kMuonGram ? &maps.lk : &maps.glk;
            else
              pa = kb == 1 ? &maps.plk : ma, pb = kb == 2 ? &maps.ln : mb;
          }
          auto load = [&](uint32_t dst, const CUtensorMap* m, int c0, int c1) {
            if (kPaired)
              tma_load_3d_pair(dst, m, fb, c0, c1, w.mat);
            else
              tma_load_3d(dst, m, fb, c0, c1, w.mat);
          };
          load(sa, pa, k0, mA);
#pragma unroll
          for (int h = 0; h < (kWide ? 2 : 1); ++h) {
            const uint32_t sb = sa + (1 + h) * kPartBytes;
            const int n = nB + 256 * h;
            if (w.symmetric()) {
              load(sb, pb, k0, n);
            } else {   // X as the right operand is contiguous along its columns
              load(sb, pb, n, k0);
              load(sb + 8192, pb, n + 64, k0);
            }
          }
          ++n_issued;
        }
      }
      if (failed && rank == 0) {
        const uint32_t first = n_issued > kStages ? n_issued - kStages : 0;
        for (uint32_t i = first; i < n_issued; ++i)
          wait_limited(full_bar(i % kStages), (i / kStages) & 1u, a.timeout_ns);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      uint32_t n_consumed = 0;
      bool issued = false, failed = false;
      int it = 0;
      // the k-blocks of one tile; kind::f16, the descriptor's type fields say fp16
      auto products = [&](auto mn, int num_kb, uint32_t d_tmem) {
        constexpr int BMN = decltype(mn)::value;
        constexpr uint32_t idesc = idesc_f16_f32(Tile::kM, kWide ? 256 : Tile::kN, 0, BMN);
        for (int kb = 0; kb < num_kb; ++kb) {
          const int stage = n_consumed % kStages;
          const uint32_t phase = (n_consumed / kStages) & 1u;
          if (!wait(full_bar(stage), phase)) {
            failed = true;
            return;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * kStageBytes);
          const uint32_t sb = sa + kPartBytes;
          if constexpr (BOTH && !BMN) {
#pragma unroll
            for (int i = 0; i < 3 * (kBK / 16); ++i) {
              const int term = i / (kBK / 16), k = i % (kBK / 16);
              tc_mma_bf16(d_tmem, smem_desc_sw128((term == 1 ? sb : sa) + 32u * k, 16u, 1024u),
                          smem_desc_sw128((term == 2 ? sb : sa) + 32u * k, 16u, 1024u), idesc, kb > 0 || i > 0 ? 1u : 0u);
            }
          }
#pragma unroll
          for (int k = 0; k < (BOTH && !BMN ? 0 : kBK / 16); ++k) {
            const uint32_t in = (kb > 0 || k > 0) ? 1u : 0u;
            const uint64_t ad = smem_desc_sw128(sa + 32u * k, 16u, 1024u);
            auto bdesc = [&](uint32_t at) {
              return BMN ? smem_desc_sw128(at + 2048u * k, 8192u, 1024u) : smem_desc_sw128(at + 32u * k, 16u, 1024u);
            };
            if (kWide) {
              tc_mma_bf16_pair_a_fill(d_tmem, ad, bdesc(sb), idesc, in);
              tc_mma_bf16_pair_a_lastuse(d_tmem + 256, ad, bdesc(sb + kPartBytes), idesc, in);
            } else if (kPaired) {
              tc_mma_bf16_pair(d_tmem, ad, bdesc(sb), idesc, in);
            } else {
              tc_mma_bf16(d_tmem, ad, bdesc(sb), idesc, in);
            }
          }
          issued = true;
          commit(empty_bar(stage));
          ++n_consumed;
        }
      };
      for (; !failed && w.locate(); w.advance(), ++it) {
        const int acc = it % kAccs;
        const uint32_t acc_phase = (it / kAccs) & 1;
        if (!wait(tempty_bar(acc), acc_phase ^ 1u)) {
          failed = true;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * Tile::kN;
        if (w.symmetric())
          products(std::integral_constant<int, 0>(), w.phase == kMuonGram ? gram_blocks(w.split) : kb_m, d_tmem);
        else
          products(std::integral_constant<int, 1>(), BOTH ? 3 : kb_m, d_tmem);
        if (failed) break;
        commit(tfull_bar(acc));
      }
      if (failed && issued) {
        if (kPaired)
          tc_commit_pair(drain_bar);
        else
          tc_commit(drain_bar);
        wait_limited(drain_bar, 0, a.timeout_ns);
      }
    }
  } else if (warp >= 4) {
    constexpr int kHalf = Tile::kN / 2;                     // columns of an epilogue warp
    constexpr int kBlock = SHAPE == kMuonSingle ? 128 : 256;  // the symmetric products' unit of "above the diagonal"
    const int wq = warp & 3, half = (warp - 4) >> 2;
    MuonEpilogue<kBufs, BOTH> epi{a, sE + (warp - 4) * kBufs * 2 * kEpiPart, drain_bar + 8u * (1 + kBufs * (warp - 4)), lane};
    bool ok = true;
    int it = 0;
    const CUtensorMap *gram_lo = nullptr, *poly_lo = nullptr;
    if constexpr (BOTH) gram_lo = &maps.gle, poly_lo = &maps.ple;
    auto unit = [&](auto phase_c) {
      constexpr int PHASE = decltype(phase_c)::value;
      constexpr bool kSym = PHASE == kMuonGram || PHASE == kMuonPoly;
      const int src = w.step & 1;
      const MuonStep st{steps.c[w.step][0], steps.c[w.step][1], steps.c[w.step][2]};
      const CUtensorMap* e0 = PHASE == kMuonPoly ? &maps.ge : &maps.xe[src];
      const CUtensorMap* e1 = PHASE == kMuonPoly ? gram_lo : &maps.lo;
      const CUtensorMap* o0 = PHASE == kMuonGram ? &maps.ge : PHASE == kMuonPoly ? &maps.pe : &maps.xe[1 - src];
      const CUtensorMap* o1 = PHASE == kMuonGram   ? (BOTH ? gram_lo : &maps.gm)
                              : PHASE == kMuonPoly ? (BOTH ? poly_lo : &maps.pm)
                                                   : &maps.lo;
      const int acc = it % kAccs;
      const uint32_t acc_phase = (it / kAccs) & 1;
      const int ncols = kSym ? a.m : a.n;
      const int row0 = w.tm * Tile::kM + static_cast<int>(rank) * 128 + wq * 32;
      const int col0 = w.tn * Tile::kN + half * kHalf;
      // below the diagonal blocks a tile of a symmetric product repeats what
      // another tile mirrors
      const int block_m = w.tm * Tile::kM / kBlock, block_n = col0 / kBlock;
      const bool skip = row0 >= a.m || col0 >= ncols || (kSym && block_n < block_m);
      const int groups = skip ? 0 : min(kHalf / 32, (ncols - col0 + 31) / 32);
      float2 factor = make_float2(0.f, 0.f);
      bool good = true;
      if (PHASE != kMuonGram && groups > 0) {
        if (lane == 0) good = wait_done(a.done + w.mat, w.needed() * kParts + a.hold, err, a.timeout_ns);
        good = __all_sync(kAll, good);
        if (good) {
          for (int g = 0; g < min(groups, kBufs); ++g) epi.load(e0, e1, w.mat, row0, col0 + g * 32);
          if (!kSym) {   // (behind lane 0's wait, by the loads' barrier)
            const float d = row0 + lane < a.m ? __ldcg(a.diag + static_cast<int64_t>(w.mat) * a.m + row0 + lane) : 0.f;
            factor = BOTH ? make_float2(st.a + d, st.a + d) : part_factors(st.a, d, row0 + 32 <= a.m);
          }
          if (PHASE == kMuonLast) epi.prefetch_weight(w.mat, row0, col0, kHalf);
        }
      }
      if (good) good = wait(tfull_bar(acc), acc_phase);
      good = __all_sync(kAll, good);
      // X Xt in splits: every split but the last leaves its fp32 sums, a 32 x 32
      // block per warp and group as [8][lane][4], where the last split's same
      // warps and lanes read them, in the order of the splits
      const bool partial = PHASE == kMuonGram && w.split + 1 < w.splits;
      const bool joins = PHASE == kMuonGram && w.splits > 1 && !partial;
      if (good && joins && groups > 0) {
        const uint32_t parts = static_cast<uint32_t>((w.step + 1) * (w.splits - 1) * w.per_s) * kParts;
        if (lane == 0) good = wait_done(a.partial + w.mat, parts, err, a.timeout_ns);
        good = __all_sync(kAll, good);
      }
      if (good) {
        tc_fence_after();
        const uint32_t tbase = tmem_base + (static_cast<uint32_t>(wq * 32) << 16) + acc * Tile::kN + half * kHalf;
        auto release = [&] {
          tc_fence_before();
          if (rank == 0)
            mbar_arrive(tempty_bar(acc));
          else
            mbar_arrive_cluster(mapa_shared(tempty_bar(acc), 0));
        };
        float4* sums = nullptr;
        if (partial || joins) {
          const int64_t tile =
              (static_cast<int64_t>(w.mat) * (w.splits - 1) + (partial ? w.split : 0)) * w.per_s + w.tile;
          const int block = ((static_cast<int>(rank) * 4 + wq) * 2 + half) * (kHalf / 32);
          sums = reinterpret_cast<float4*>(a.sums) + (tile * (Tile::kM * Tile::kN / 1024) + block) * 256 + lane;
        }
        if (groups == 0) release();
#pragma unroll 1
        for (int g = 0; g < groups && good; ++g) {
          __syncwarp();
          uint32_t r[32];
          tmem_ld_32x32b_x32(tbase + g * 32, r);
          tmem_ld_wait();
          tmem_regs_ready(r);
          if (g == groups - 1) release();
          if constexpr (PHASE == kMuonGram) {
            if (partial) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                __stcg(sums + g * 256 + j * 32,
                       make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                   __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3])));
              continue;
            }
            if (joins) {
              for (int s = 0; s + 1 < w.splits; ++s) {   // onto this split's own, in order
                float4 v[8];
                const float4* from = sums + static_cast<int64_t>(s) * w.per_s * (Tile::kM * Tile::kN / 4) + g * 256;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __ldcg(from + j * 32);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  r[4 * j] = __float_as_uint(__uint_as_float(r[4 * j]) + v[j].x);
                  r[4 * j + 1] = __float_as_uint(__uint_as_float(r[4 * j + 1]) + v[j].y);
                  r[4 * j + 2] = __float_as_uint(__uint_as_float(r[4 * j + 2]) + v[j].z);
                  r[4 * j + 3] = __float_as_uint(__uint_as_float(r[4 * j + 3]) + v[j].w);
                }
              }
            }
          }
          good = epi.template group<PHASE>(st, o0, o1, g, w.mat, row0, col0 + g * 32, kSym && block_n > block_m, factor, r);
          if (PHASE != kMuonGram && good && g + kBufs < groups) epi.load(e0, e1, w.mat, row0, col0 + (g + kBufs) * 32);
        }
      }
      if (PHASE != kMuonLast) {
        // This CTA's part of the tile is in global memory: say so, once for its
        // eight warps (an atomic per warp queues a hundred on one counter). All
        // eight come here whatever happened, and leave together if a wait failed.
        __syncwarp();
        if (lane == 0) bulk_wait_group<0>();
        ok = !named_bar_or(kEpiBar, kEpiThreads, !good);
        if (ok && warp == 4 && lane == 0) add_release((partial ? a.partial : a.done) + w.mat, 1);
      } else {
        ok = good;
      }
    };
    for (; ok && w.locate(); w.advance(), ++it) {
      if (w.phase == kMuonGram)
        unit(std::integral_constant<int, kMuonGram>());
      else if (w.phase == kMuonPoly)
        unit(std::integral_constant<int, kMuonPoly>());
      else if (w.step + 1 < steps.count)
        unit(std::integral_constant<int, kMuonApply>());
      else
        unit(std::integral_constant<int, kMuonLast>());
    }
    if (lane == 0) bulk_wait_group<0>();
    // a load that is still in flight lands before the CTA leaves
    if (!ok && lane == 0)
      for (; epi.uses < epi.loads; ++epi.uses)
        wait_limited(epi.bar + 8u * (epi.uses % kBufs), (epi.uses / kBufs) & 1u, a.timeout_ns);
  }

  __syncwarp();
  __syncthreads();
  if (kPaired) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if (kPaired)
      tmem_dealloc_pair(tmem_base, kTmemCols);
    else
      tmem_dealloc(tmem_base, kTmemCols);
  }
  if (threadIdx.x == 0) {
    const uint32_t code = ld_volatile_u32(err);
    if (code != 0) *reinterpret_cast<volatile uint32_t*>(a.host_error) = code;
  }
}

template <int SHAPE>
int64_t muon_units(int phase, const MuonArgs& a) {
  using Tile = MuonTile<SHAPE>;
  const bool sym = phase == kMuonGram || phase == kMuonPoly;
  const int tm = (a.m + Tile::kM - 1) / Tile::kM, tn = ((sym ? a.m : a.n) + Tile::kN - 1) / Tile::kN;
  return static_cast<int64_t>(a.count) * muon_units_per_matrix<SHAPE>(sym, tm, tn);
}

// A launch that may start while the one before it drains
template <class... P, class... A>
cudaError_t launch_chained(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int SHAPE, bool BOTH, class Maps>
cudaError_t launch_steps(const Maps& maps, const MuonArgs& a, const MuonSteps& steps, int slots, cudaStream_t s) {
  auto kern = muon_steps_kernel<SHAPE, BOTH>;
  // at every launch: the attribute belongs to the current device, and a process may use several
  const cudaError_t opted = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(smem_bytes<SHAPE>()));
  if (opted != cudaSuccess) return opted;
  const int64_t most = std::max(a.splits * muon_units<SHAPE>(kMuonGram, a), muon_units<SHAPE>(kMuonApply, a));
  const int n = static_cast<int>(std::min<int64_t>(most, slots));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(SHAPE == kMuonSingle ? n : 2 * n);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<SHAPE>();
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeCooperative;
  attr.val.cooperative = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, maps, a, steps);
}

}  // namespace

// Tile shape and splits of X Xt: those that take least by this model of a
// step, in nanoseconds. A unit costs its k-blocks (more per block the more of
// the GPU reads L2 at once); a product follows its predecessor after its
// epilogue and a flag's latency, with one matrix in whole rounds of units,
// while several matrices fill each other's rounds; a wide tile's epilogue is
// not overlapped. Splitting X Xt shortens its units where there are few of
// them (a long X), and costs the last split the reading of the others' sums.
MuonPlan muon_plan(const MuonArgs& a, int fixed_shape, int pairs, int sms) {
  struct Cost {
    double per_kb, full, epilogue;
    bool overlapped;
    int groups;   // 32-column groups of an epilogue warp
  };
  static const Cost costs[3] = {{270, 180, 2000, true, 2}, {330, 60, 4500, true, 4}, {540, 20, 9000, false, 8}};
  const double latency = 3500, join = 1200, join_group = 600;
  const int kb_n = (a.n + kBK - 1) / kBK, kb_m = (a.m + kBK - 1) / kBK;
  MuonPlan best;
  double best_ns = 0;
  for (int shape = 0; shape < 3; ++shape) {
    if (fixed_shape >= 0 && shape != fixed_shape) continue;
    const Cost& c = costs[shape];
    const double slots = shape == kMuonSingle ? sms : pairs;
    const int64_t sym = shape == kMuonSingle ? muon_units<kMuonSingle>(kMuonGram, a)
                        : shape == kMuonPair ? muon_units<kMuonPair>(kMuonGram, a)
                                             : muon_units<kMuonWide>(kMuonGram, a);
    const int64_t full = shape == kMuonSingle ? muon_units<kMuonSingle>(kMuonApply, a)
                         : shape == kMuonPair ? muon_units<kMuonPair>(kMuonApply, a)
                                              : muon_units<kMuonWide>(kMuonApply, a);
    auto product = [&](double units, double kb) {
      const double unit = kb * (c.per_kb + c.full * std::min(1.0, units / slots)) + (c.overlapped ? 0 : c.epilogue);
      const double rounds = a.count > 1 ? std::max(1.0, units / slots) : std::ceil(units / slots);
      return rounds * unit + (c.overlapped ? c.epilogue : 0) + latency;
    };
    for (int splits = 1; splits <= kMuonMaxSplits; ++splits) {
      const int kb = (kb_n + splits - 1) / splits;
      if (splits > 1 && (kb < kMuonMinSplitBlocks || (kb_n + kb - 1) / kb != splits || sym * splits > slots)) continue;
      const int64_t tile_bytes = 4ll * (shape == kMuonSingle ? 128 * 128 : shape == kMuonPair ? 256 * 256 : 256 * 512);
      if ((splits - 1) * sym * tile_bytes > a.sums_bytes) continue;
      const double ns = product(static_cast<double>(sym) * splits, kb) +
                        (splits > 1 ? join + (splits - 1) * join_group * c.groups : 0) +
                        product(static_cast<double>(sym), kb_m) + product(static_cast<double>(full), kb_m);
      if (best.shape < 0 || ns < best_ns) {
        best.shape = shape;
        best.splits = splits;
        best_ns = ns;
      }
    }
  }
  return best;
}

cudaError_t launch_muon_momentum(const MuonArgs& a, cudaStream_t s) {
  muon_momentum_kernel<<<dim3(a.norm_blocks, a.count), 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_muon_prepare(const MuonArgs& a, int sms, cudaStream_t s) {
  // eight blocks of 256 threads per SM, each over many tiles
  const int64_t tiles = a.vec && !a.transposed
                            ? static_cast<int64_t>((a.rows + 15) / 16) * ((a.cols + 255) / 256)
                            : static_cast<int64_t>((a.rows + kTile - 1) / kTile) * ((a.cols + kTile - 1) / kTile);
  const int64_t most = std::max<int64_t>(1, 8ll * sms / a.count);
  return launch_chained(muon_prepare_kernel, dim3(static_cast<unsigned>(std::min(tiles, most)), a.count), 256, 0, s, a);
}

cudaError_t launch_muon_steps(int shape, const MuonMaps& maps, const MuonArgs& a, const MuonSteps& steps, int slots,
                              cudaStream_t s) {
  return shape == kMuonSingle ? launch_steps<kMuonSingle, false>(maps, a, steps, slots, s)
         : shape == kMuonPair ? launch_steps<kMuonPair, false>(maps, a, steps, slots, s)
                              : launch_steps<kMuonWide, false>(maps, a, steps, slots, s);
}

cudaError_t launch_muon_steps_pairs(const MuonPairMaps& maps, const MuonArgs& a, const MuonSteps& steps, int slots,
                                    cudaStream_t s) {
  return launch_steps<kMuonSingle, true>(maps, a, steps, slots, s);
}

// CTA pairs that fit on the device at once (the three shapes take an SM each)
int muon_max_clusters() {
  auto kern = muon_steps_kernel<kMuonPair, false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem_bytes<kMuonPair>();
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem_bytes<kMuonPair>())) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

}  // namespace flce
