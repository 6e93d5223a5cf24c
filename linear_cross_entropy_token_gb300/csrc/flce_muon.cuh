// What the kernels of the orthogonalised momentum update share: scales, fp16
// parts, momentum, norms, result writes.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "flce_internal.h"
#include "flce_train.h"
#include "ptx.cuh"

namespace flce {

constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kXScale = 4096.f;           // hi + lo = 2^12 X
constexpr float kXInv = 1.f / 4096.f;
constexpr float kGramScale = 1.f / 4096.f;  // (2^12 X)(2^12 X)t -> 2^12 A
constexpr float kPolyB = 0.5f;              // 2^12 A -> 2^11 A
constexpr float kPolyC = 1.f / 8192.f;      // (2^12 A)^2 -> 2^11 A^2
constexpr float kPolyInv = 1.f / 2048.f;    // 2^11 B -> B; (2^11 B)(2^12 X) -> 2^12 B X

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float2 unpack_half2(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// hi = fp16(x), lo = fp16(x - hi), two values at once
__device__ __forceinline__ void split_half2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_half2(x0, x1);
  const float2 f = unpack_half2(hi);
  lo = pack_half2(x0 - f.x, x1 - f.y);
}

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
    const float b = v * 0x1p-80f, s = v * 0x1p80f;
    big = fmaf(b, b, big);
    small = fmaf(s, s, small);
  }
  // the sum over the warp, valid in every lane; fp64 in lane 0's hands alone
  // (fp64 runs at a sixty-fourth of fp32's rate)
  __device__ __forceinline__ void reduce_warp() {
    for (int o = 16; o > 0; o >>= 1) {
      mid += __shfl_xor_sync(kAll, mid, o);
      big += __shfl_xor_sync(kAll, big, o);
      small += __shfl_xor_sync(kAll, small, o);
    }
  }
  __device__ __forceinline__ double total() const {
    if (!(mid <= 3e38f)) return static_cast<double>(big) * 0x1p160;  // inf, or NaN (then big is too)
    return mid < 0x1p-90f ? static_cast<double>(small) * 0x1p-160 : static_cast<double>(mid);
  }
};

// Four elements of u from the gradient (and the momentum, updated in place).
__device__ __forceinline__ void momentum4(const MuonArgs& a, float4& m, float (&g)[4]) {
  m.x = m.x * a.beta + g[0] * a.one_minus_beta;
  m.y = m.y * a.beta + g[1] * a.one_minus_beta;
  m.z = m.z * a.beta + g[2] * a.one_minus_beta;
  m.w = m.w * a.beta + g[3] * a.one_minus_beta;
  if (a.nesterov) {
    g[0] = m.x * a.beta + g[0] * a.one_minus_beta;
    g[1] = m.y * a.beta + g[1] * a.one_minus_beta;
    g[2] = m.z * a.beta + g[2] * a.one_minus_beta;
    g[3] = m.w * a.beta + g[3] * a.one_minus_beta;
  } else {
    g[0] = m.x, g[1] = m.y, g[2] = m.z, g[3] = m.w;
  }
}

// The factor 2^12 / (|u| + eps) of X from |u|^2, as two, so that neither leaves
// fp32's normal range.
__device__ __forceinline__ void norm_factors(double square_sum, double eps, float* f) {
  const float s = static_cast<float>(square_sum);
  if (s > 1e-30f && s < 1e38f) {  // fp32's own square root and quotient: exact to its last bits
    f[0] = 1.f;
    f[1] = kXScale / (sqrtf(s) + static_cast<float>(eps));
    return;
  }
  const double inv = static_cast<double>(kXScale) / (sqrt(square_sum) + eps);
  f[0] = inv < 1e-30 ? 0x1p-64f : 1.f;
  f[1] = static_cast<float>(inv < 1e-30 ? inv * 0x1p64 : inv);
}

// A sum of squares as mantissa and exponent (int bits in y): 32-bit values that
// neither over- nor underflow, for a sum that many blocks repeat.
__device__ __forceinline__ float2 pack_sum(double s) {
  int e = -30000;
  double m = s;
  if (s > 0.0 && s < 1e300) m = frexp(s, &e);
  return make_float2(static_cast<float>(m), __int_as_float(e));
}

// The factors of X's two parts in a X + B X, for a warp of 32 rows with B's
// diagonal d: the high part meets all of B, the low part only a and what the
// rows' diagonals have in common. Applied to the low part alone, without the
// rest of B, a diagonal that varies puts rounding noise into every direction,
// and the small ones are raised up to 3.4 times a step (rank one on 3 x 3
// entries: 5.6e-2 off, 7e-4 without); left off the low part altogether, it costs
// Gaussian matrices half of their accuracy (128 x 128: 1.5e-3, 1.0e-3 with what
// is common). `whole`: the warp's rows all lie in the matrix.
__device__ __forceinline__ float2 part_factors(float a, float d, bool whole) {
  float least, most;
  asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(least) : "f"(d));
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(most) : "f"(d));
  const float common = !whole ? 0.f : least > 0.f ? least : most < 0.f ? most : 0.f;
  return make_float2(a + d, a + common);
}

// fp16 operands: the type fields (bits 7-9 and 10-12) are 0
__host__ __device__ constexpr uint32_t idesc_f16_f32(uint32_t M, uint32_t N, uint32_t a_mn, uint32_t b_mn) {
  return (1u << 4) | (a_mn << 15) | (b_mn << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// mbar_try_wait until the phase is done or the limit has passed
__device__ __forceinline__ bool wait_limited(uint32_t bar, uint32_t parity, uint64_t timeout_ns) {
#pragma unroll 1
  for (int i = 0; i < 128; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > timeout_ns) return false;
  return true;
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float2 to_float2(float2 v) { return v; }
__device__ __forceinline__ float2 to_float2(__nv_bfloat162 v) { return __bfloat1622float2(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(float2* p, float2 v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat162* p, float2 v) { *p = __floats2bfloat162_rn(v.x, v.y); }
template <class T>
struct PairOf;
template <>
struct PairOf<float> {
  using type = float2;
};
template <>
struct PairOf<__nv_bfloat16> {
  using type = __nv_bfloat162;
};

// f(T*, W) for the result tensor of a matrix: its element type, whether it is
// a weight to be updated (true) or the update itself (false), its row stride
template <class F>
__device__ __forceinline__ void with_result(const MuonArgs& a, const MuonMat& t, F&& f) {
  if (t.weight) {
    if (a.weight_dtype == 1)
      f(static_cast<float*>(t.weight), std::true_type(), t.ld_weight);
    else
      f(static_cast<__nv_bfloat16*>(t.weight), std::true_type(), t.ld_weight);
  } else {
    if (a.update_dtype == 1)
      f(static_cast<float*>(t.update), std::false_type(), t.ld_update);
    else
      f(static_cast<__nv_bfloat16*>(t.update), std::false_type(), t.ld_update);
  }
}

// The transpose: the lane's row of N values down one column of the result
// (the lanes' columns are neighbours).
template <bool W, class T, int N>
__device__ __forceinline__ void write_columns(T* out, int64_t ld, int rows, float decay, float lr,
                                              const float (&o)[N]) {
#pragma unroll
  for (int r0 = 0; r0 < N; r0 += 16) {
    T w[16];
    if (W) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (r0 + j < rows) w[j] = out[(r0 + j) * ld];
    }
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (r0 + j < rows) put(out + (r0 + j) * ld, W ? to_float(w[j]) * decay - lr * o[r0 + j] : o[r0 + j]);
  }
}

}  // namespace flce
