// The products of the LM-head operators for fp32 inputs, on the CUDA cores (TF32
// cannot hold fp32 inputs' gradients): C (+)= A B, and z = x Wt with the statistics
// of its 64-column groups as epilogue, where a row's group is one block's.
//
// 64 x 64 tiles, 128 threads of 8 x 4 outputs: for 32 multiply-adds a thread reads
// 12 floats from shared memory, so the FMA pipes bound a long sum. fp32 inputs are
// small models' (256 x 128 x 4096), where latency does: k-blocks of 32 come
// through a three-deep ring of asynchronous copies, and a sum with few tiles of
// output is split over idle SMs. The copies are of single elements: x, W and their
// rows may start anywhere, and whichever way an operand lies it is turned to
// [k][row] on the way.
//
// Measured against the loss's kernel for such inputs (64 x 64 tiles, 4 x 4 a
// thread, one k-block of 16 in flight), 256 x 128 x 4096: see launch_score_f32.
#include <algorithm>

#include "flce_score.cuh"

namespace flce {
namespace {

constexpr int kTile = 64, kDeep = 32, kRing3 = 3, kThreads = 128;
constexpr int kStride = kTile + 4;                    // floats between k's: rows of 16 bytes
constexpr uint32_t kOperand = kDeep * kStride * 4;
constexpr uint32_t kSmem = kRing3 * 2 * kOperand;

__device__ __forceinline__ void copy4(uint32_t to, const float* from, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(there ? 4 : 0) : "memory");
}

// rows o0 .. o0 + 63 of an operand at k0 .. k0 + 31 to [k][row]; so, sk: strides.
// Consecutive threads follow the unit stride.
__device__ __forceinline__ void fetch(uint32_t to, const float* p, int64_t so, int64_t sk, int64_t o0, int64_t outer, int64_t k0,
                                      int64_t kend) {
  constexpr int kCopies = kTile * kDeep / kThreads;
  const int t = static_cast<int>(threadIdx.x);
  const bool along_k = sk == 1;
  // the thread's first element, and its steps of rows or k's
  const int k = along_k ? t % kDeep : t / kTile, o = along_k ? t / kDeep : t % kTile;
  const int step_k = along_k ? 0 : kThreads / kTile, step_o = along_k ? kThreads / kDeep : 0;
  const float* from = p + (o0 + o) * so + (k0 + k) * sk;
  const int64_t step = step_o * so + step_k * sk;
  to += 4u * (k * kStride + o);
#pragma unroll 4
  for (int i = 0; i < kCopies; ++i) {
    const bool there = o0 + o + i * step_o < outer && k0 + k + i * step_k < kend;
    copy4(to, there ? from : p, there);
    from += step;
    to += 4u * (step_k * kStride + step_o);
  }
}

template <bool STATS>
__global__ void __launch_bounds__(kThreads, 4) score_f32_kernel(const ScoreF32Args a) {
  extern __shared__ __align__(16) float smem[];
  const uint32_t base = smem_u32(smem);
  const int64_t tiles_n = (a.N + kTile - 1) / kTile, group = blockIdx.x % tiles_n;
  const int64_t m0 = blockIdx.x / tiles_n * kTile, n0 = group * kTile;
  const int64_t kbeg = static_cast<int64_t>(blockIdx.y) * a.k_per_split, kend = min(a.K, kbeg + a.k_per_split);
  const int blocks = static_cast<int>((kend - kbeg + kDeep - 1) / kDeep);
  auto load = [&](int i) {
    if (i < blocks) {
      const uint32_t to = base + (i % kRing3) * 2 * kOperand;
      fetch(to, a.A, a.sam, a.sak, m0, a.M, kbeg + i * kDeep, kend);
      fetch(to + kOperand, a.B, a.sbn, a.sbk, n0, a.N, kbeg + i * kDeep, kend);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  load(0);
  load(1);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[8][4] = {};
  for (int i = 0; i < blocks; ++i) {
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();  // block i is there for all, and block i - 1 has been read
    load(i + 2);
    const float* as = smem + (i % kRing3) * 2 * (kOperand / 4) + 8 * ty;
    const float* bs = smem + (i % kRing3) * 2 * (kOperand / 4) + kOperand / 4 + 4 * tx;
#pragma unroll 8
    for (int k = 0; k < kDeep; ++k) {
      const float4 lo = *reinterpret_cast<const float4*>(as + k * kStride), hi = *reinterpret_cast<const float4*>(as + k * kStride + 4);
      const float4 bv = *reinterpret_cast<const float4*>(bs + k * kStride);
      const float av[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}, b[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
      for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][c] = fmaf(av[r], b[c], acc[r][c]);
    }
  }
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int64_t m = m0 + 8 * ty + r;
    if (m < a.M) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int64_t n = n0 + 4 * tx + c;
        if (n >= a.N) continue;
        if (a.part) {
          a.part[(static_cast<int64_t>(blockIdx.y) * a.M + m) * a.N + n] = acc[r][c];
        } else {
          float* at = a.C + m * a.ldc + n;
          *at = a.accumulate ? *at + acc[r][c] : acc[r][c];
        }
      }
    }
    if constexpr (STATS) {
      // the 16 threads of a row: half a warp
      float z[4], mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        z[c] = n0 + 4 * tx + c < a.N ? acc[r][c] : -INFINITY;
        mx = max_nan(mx, z[c]);
      }
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      float l = 0.f, s = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        // the natural exponential's argument has no factor to round; NaN stays NaN
        const float d = z[c] - mx, e = expf(max_nan(d * a.inv_temperature, -700.f));
        l += e;
        s = fmaf(max_nan(d * a.c, -1000.f), e, s);
      }
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, o);
        s += __shfl_xor_sync(0xffffffffu, s, o);
      }
      if (tx == 0 && m < a.M) {
        a.partials[m * a.groups + group] = make_float2(mx, l);
        a.part_s[m * a.groups + group] = s;
      }
    }
  }
}

// The splits' sums added in their order
__global__ void __launch_bounds__(256) score_f32_join_kernel(const float* __restrict__ part, int splits, int64_t M, int64_t N,
                                                             float* __restrict__ C, int64_t ldc, int accumulate) {
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, MN = M * N;
  if (e >= MN) return;
  float v = 0.f;
  for (int s = 0; s < splits; s += 8) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = s + i < splits ? part[(s + i) * MN + e] : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += q[i];
  }
  float* at = C + e / N * ldc + e % N;
  *at = accumulate ? *at + v : v;
}

}  // namespace

// As many parts of at least 64 of K as give every SM two blocks, within `most`
int score_f32_splits(int64_t M, int64_t N, int64_t K, int sms, int64_t most) {
  const int64_t tiles = ((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile);
  const int64_t fill = 2 * sms / std::max<int64_t>(tiles, 1);
  return static_cast<int>(std::max<int64_t>(1, std::min({fill, K / 64, most, static_cast<int64_t>(64)})));
}

cudaError_t launch_score_f32(ScoreF32Args a, int splits, cudaStream_t s) {
  if (splits > 1 && a.part) {
    a.k_per_split = ((a.K + splits - 1) / splits + kDeep - 1) / kDeep * kDeep;
    splits = static_cast<int>((a.K + a.k_per_split - 1) / a.k_per_split);
  } else {
    splits = 1;
    a.part = nullptr;
    a.k_per_split = a.K;
  }
  auto kern = a.partials ? score_f32_kernel<true> : score_f32_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>((a.N + kTile - 1) / kTile * ((a.M + kTile - 1) / kTile)), static_cast<unsigned>(splits));
  kern<<<grid, kThreads, kSmem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.part) return e;
  score_f32_join_kernel<<<static_cast<unsigned>((a.M * a.N + 255) / 256), 256, 0, s>>>(a.part, splits, a.M, a.N, a.C, a.ldc,
                                                                                    a.accumulate);
  return cudaGetLastError();
}

}  // namespace flce
