// The products of the LM-head operators for fp32 inputs, on the CUDA cores (TF32
// cannot hold fp32 inputs' gradients): C (+)= A B, and z = x Wt with the statistics
// of its 64-column groups as epilogue, where a row's group is one block's.
//
// 64 x 64 tiles, 128 threads of 8 x 4 outputs: for 32 multiply-adds a thread reads
// 12 floats from shared memory. Operands lie there as [k][row], whichever way they
// come: a k-block of 32 is read in vectors of four along the unit stride (single
// elements at ragged ends, and where x, W or their rows do not start on 16 bytes)
// while the one before is multiplied, and turned as it is stored; rows are swapped in
// fours by k, so that neither the turned stores nor the reads meet a bank twice.
// A sum with few tiles of output is split over idle SMs.
//
// What bounds it: issue (the multiply-adds are four fifths of its instructions) for
// long sums; fp32 inputs are small models', where latency does. 256 x 128 x 4096, us
// a product under a profiler: 14 to 18; with element-wise asynchronous copies instead
// of vectors half of the instructions were theirs; the loss's kernel for such inputs
// (4 x 4 outputs a thread, blocks of 16) 20.
#include <algorithm>

#include "flce_score.cuh"

namespace flce {
namespace {

constexpr int kTile = 64, kDeep = 32, kThreads = 128;
constexpr int kStride = kTile + 4;                    // floats between k's: rows of 16 bytes
constexpr int kVectors = kTile * kDeep / 4 / kThreads;  // a thread's, of an operand's block

struct Operand {
  const float* p;
  int64_t so, sk;      // strides of rows and k's, one of them 1
  int64_t o0, outer;   // first row, rows there are
  bool vectors;        // of four are aligned
};

// where row o of k lies in its [k][row] line
__device__ __forceinline__ int swapped(int o, int k) { return o ^ (k & 28); }

__device__ __forceinline__ void fetch(const Operand& q, int64_t k0, int64_t kend, float4 (&v)[kVectors]) {
  const bool along_k = q.sk == 1;
#pragma unroll
  for (int i = 0; i < kVectors; ++i) {
    const int e = i * kThreads + static_cast<int>(threadIdx.x);
    const int64_t o = q.o0 + (along_k ? e / (kDeep / 4) : e % (kTile / 4) * 4);
    const int64_t k = k0 + (along_k ? e % (kDeep / 4) * 4 : e / (kTile / 4));
    const float* at = q.p + o * q.so + k * q.sk;
    const int64_t left = along_k ? kend - k : q.outer - o;  // elements from here on
    const bool line = along_k ? o < q.outer : k < kend;
    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (line && left >= 4 && q.vectors) {
      v[i] = *reinterpret_cast<const float4*>(at);
    } else if (line) {
      if (left > 0) v[i].x = at[0];
      if (left > 1) v[i].y = at[1];
      if (left > 2) v[i].z = at[2];
      if (left > 3) v[i].w = at[3];
    }
  }
}

__device__ __forceinline__ void put(float* to, bool along_k, const float4 (&v)[kVectors]) {
#pragma unroll
  for (int i = 0; i < kVectors; ++i) {
    const int e = i * kThreads + static_cast<int>(threadIdx.x);
    if (along_k) {
      const int o = e / (kDeep / 4), k = e % (kDeep / 4) * 4;
      float* at = to + k * kStride + swapped(o, k);  // the same place for four k's
      at[0] = v[i].x;
      at[kStride] = v[i].y;
      at[2 * kStride] = v[i].z;
      at[3 * kStride] = v[i].w;
    } else {
      const int o = e % (kTile / 4) * 4, k = e / (kTile / 4);
      *reinterpret_cast<float4*>(to + k * kStride + swapped(o, k)) = v[i];
    }
  }
}

enum Epilogue : int { kPlain, kStats, kGradient };

template <int EPILOGUE>
__global__ void __launch_bounds__(kThreads, 4) score_f32_kernel(const __grid_constant__ ScoreF32Pair pair) {
  const bool second = static_cast<int64_t>(blockIdx.x) >= pair.blocks0;
  const ScoreF32Args& a = pair.p[EPILOGUE == kPlain && second ? 1 : 0];
  __shared__ __align__(16) float smem[2][2][kDeep * kStride];
  const int64_t tiles_n = (a.N + kTile - 1) / kTile, tiles = tiles_n * ((a.M + kTile - 1) / kTile);
  const int64_t unit = blockIdx.x - (EPILOGUE == kPlain && second ? pair.blocks0 : 0);
  const int64_t split = unit / tiles, tile = unit - split * tiles, group = tile % tiles_n;
  const int64_t m0 = tile / tiles_n * kTile, n0 = group * kTile;
  const int64_t kbeg = split * a.k_per_split, kend = min(a.K, kbeg + a.k_per_split);
  const Operand qa{a.A, a.sam, a.sak, m0, a.M, a.vectors_a != 0}, qb{a.B, a.sbn, a.sbk, n0, a.N, a.vectors_b != 0};
  float4 va[kVectors], vb[kVectors];
  fetch(qa, kbeg, kend, va);
  fetch(qb, kbeg, kend, vb);
  put(smem[0][0], qa.sk == 1, va);
  put(smem[0][1], qb.sk == 1, vb);
  __syncthreads();
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[8][4] = {};
  int turn = 0;
  for (int64_t k0 = kbeg; k0 < kend; k0 += kDeep, turn ^= 1) {
    const bool more = k0 + kDeep < kend;
    if (more) {
      fetch(qa, k0 + kDeep, kend, va);
      fetch(qb, k0 + kDeep, kend, vb);
    }
    const float* as = smem[turn][0];
    const float* bs = smem[turn][1];
#pragma unroll
    for (int k4 = 0; k4 < kDeep; k4 += 4) {
      const int oa = swapped(8 * ty, k4), ob = swapped(4 * tx, k4);
#pragma unroll
      for (int k = k4; k < k4 + 4; ++k) {
        // the second four rows lie where the swap takes them
        const float4 lo = *reinterpret_cast<const float4*>(as + k * kStride + oa);
        const float4 hi = *reinterpret_cast<const float4*>(as + k * kStride + (oa ^ 4));
        const float4 bv = *reinterpret_cast<const float4*>(bs + k * kStride + ob);
        const float av[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}, b[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[r][c] = fmaf(av[r], b[c], acc[r][c]);
      }
    }
    if (more) {  // the other buffer was read before the last barrier
      put(smem[turn ^ 1][0], qa.sk == 1, va);
      put(smem[turn ^ 1][1], qb.sk == 1, vb);
    }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int64_t m = m0 + 8 * ty + r;
    if constexpr (EPILOGUE == kGradient) {
      if (m >= a.M) continue;
      const ScoreRow q = a.row[m];
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[r][c] = dlogit_f32(acc[r][c], n0 + 4 * tx + c, a.c, a.inv_temperature, q);
    }
    if (m < a.M) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int64_t n = n0 + 4 * tx + c;
        if (n >= a.N) continue;
        if (a.part) {
          a.part[(split * a.M + m) * a.N + n] = acc[r][c];
        } else {
          float* at = a.C + m * a.ldc + n;
          *at = a.accumulate ? *at + acc[r][c] : acc[r][c];
        }
      }
    }
    if constexpr (EPILOGUE == kStats) {
      // the 16 threads of a row: half a warp
      float z[4], mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        z[c] = n0 + 4 * tx + c < a.N ? acc[r][c] : -INFINITY;
        mx = max_nan(mx, z[c]);
      }
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float base = group_base(mx);
      float l = 0.f, s = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        // the natural exponential's argument has no factor to round; NaN stays NaN
        const float d = z[c] - base, e = expf(max_nan(d * a.inv_temperature, -700.f));
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
__global__ void __launch_bounds__(256) score_f32_join_kernel(const float* __restrict__ part, int splits, int64_t MN,
                                                             float* __restrict__ C) {
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (e >= MN) return;
  float v = 0.f;
  for (int s = 0; s < splits; s += 16) {
    float q[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = s + i < splits ? part[(s + i) * MN + e] : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += q[i];
  }
  C[e] = v;
}

int64_t tiles_of(const ScoreF32Args& a) { return (a.M + kTile - 1) / kTile * ((a.N + kTile - 1) / kTile); }

void finish(ScoreF32Args& a) {
  auto aligned = [](const float* p, int64_t so, int64_t sk) {
    return reinterpret_cast<uint64_t>(p) % 16 == 0 && (sk == 1 ? so : sk) % 4 == 0;
  };
  a.vectors_a = aligned(a.A, a.sam, a.sak);
  a.vectors_b = aligned(a.B, a.sbn, a.sbk);
  if (a.part == nullptr) a.k_per_split = a.K;
}

}  // namespace

// As many parts of at least 64 of K as give every SM two blocks, within `most`
int score_f32_splits(int64_t M, int64_t N, int64_t K, int sms, int64_t most) {
  const int64_t tiles = ((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile);
  const int64_t fill = 2 * sms / std::max<int64_t>(tiles, 1);
  return static_cast<int>(std::max<int64_t>(1, std::min({fill, K / 64, most, static_cast<int64_t>(64)})));
}

cudaError_t launch_score_f32(ScoreF32Args a, cudaStream_t s) {
  finish(a);
  const unsigned blocks = static_cast<unsigned>(tiles_of(a));
  const ScoreF32Pair pair{{a, a}, static_cast<int64_t>(blocks)};
  if (a.row)
    score_f32_kernel<kGradient><<<blocks, kThreads, 0, s>>>(pair);
  else
    score_f32_kernel<kStats><<<blocks, kThreads, 0, s>>>(pair);
  return cudaGetLastError();
}

cudaError_t launch_score_f32_backward(const ScoreF32Args* dx, int splits, const ScoreF32Args* dw, cudaStream_t s) {
  ScoreF32Pair pair{};
  int64_t blocks = 0;
  if (dx) {
    ScoreF32Args a = *dx;
    if (splits > 1) {
      a.k_per_split = ((a.K + splits - 1) / splits + kDeep - 1) / kDeep * kDeep;
      splits = static_cast<int>((a.K + a.k_per_split - 1) / a.k_per_split);
    } else {
      splits = 1;
      a.part = nullptr;
    }
    finish(a);
    pair.p[0] = a;
    blocks = tiles_of(a) * splits;
  }
  pair.blocks0 = blocks;
  if (dw) {
    pair.p[1] = *dw;
    pair.p[1].part = nullptr;
    finish(pair.p[1]);
    blocks += tiles_of(pair.p[1]);
  }
  score_f32_kernel<kPlain><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(pair);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !dx || !pair.p[0].part) return e;
  const int64_t n = dx->M * dx->N;  // rows of dx lie side by side
  score_f32_join_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(pair.p[0].part, splits, n, dx->C);
  return cudaGetLastError();
}

}  // namespace flce
