// Expert routing with its balance and z losses, forward and backward.
//
// Per token row of E logits z: p = softmax(z), lse = log sum exp z, the k
// experts of largest z (ties to the lowest index) with their probabilities as
// weights (divided by their sum if asked). Per document d with n_d live
// tokens, c_de chosen slots and P_de = sum of p_e over its tokens, and n live
// tokens in all:
//   balance = sum_d (n_d / n) sum_e (E c_de / (k n_d)) (P_de / n_d)
//   z       = (1 / n) sum lse^2
// The counts carry no gradient, so with slope_de = E c_de / (k n_d n)
//   d z_e = p_e (u_e - sum_j p_j u_j) + g_z 2 lse / n p_e,
//   u_e = g_balance slope_de + (the gradient of the chosen weights).
//
// A row is held by G lanes with NPL consecutive experts each, in registers,
// from the one load to the last use; the sums over tokens stay in registers
// too (an expert's column belongs to one lane) until a block's piece of a
// document ends. Sums over tokens are taken in a fixed order (per piece, then
// over the pieces), so results repeat bit for bit; only integer counts use
// atomics. All arithmetic is fp32, but for a thread's share of the documents'
// terms in the closing pass, and the terms of the one-cluster form (fp64).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "flce_train.h"
#include "ptx.cuh"

namespace flce {
namespace {

constexpr int kWarps = kRouteThreads / 32;
// Blocks resident per SM. Forward: two with 16 experts a lane, one with 32; and
// three for fp32 rows of 129 to 256 experts (131072 x 256: 76 us, with four 80;
// x 128: 63 and 61).
constexpr int kBackwardBlocks = 4;
constexpr int forward_blocks(int element_bytes, int lanes, int per_lane) {
  return per_lane == 32 ? 1 : per_lane == 16 ? 2 : element_bytes == 4 && lanes == 32 ? 3 : 4;
}
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xFF800000); }

// max that keeps a NaN, so that a row with one is not taken for a dead row
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// within 1 ulp; sums of exp lie in [1, 1024]
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// NPL consecutive elements of a row from column c0 on; `fill` past column E.
// 16-byte loads where the caller found the rows aligned and the whole vector
// lies inside the row.
template <class T, int NPL>
__device__ __forceinline__ void load_row(const T* row, int c0, int E, bool vec, float fill, float (&z)[NPL]) {
  constexpr int V = 16 / sizeof(T);
#pragma unroll
  for (int c = 0; c < NPL; c += V) {
    if (vec && c0 + c + V <= E) {
      union {
        uint4 u;
        T t[V];
      } w;
      w.u = *reinterpret_cast<const uint4*>(row + c0 + c);
#pragma unroll
      for (int i = 0; i < V; ++i) z[c + i] = to_f(w.t[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) z[c + i] = c0 + c + i < E ? to_f(row[c0 + c + i]) : fill;
    }
  }
}

// The same as they are in memory, for a row that waits a turn.
template <class T, int NPL>
struct RawRow {
  static constexpr int V = 16 / sizeof(T);
  union Vector {
    uint4 u;
    uint16_t h[8];
    uint32_t w[4];
  };
  Vector v[NPL / V];

  __device__ __forceinline__ void load(const T* row, int c0, int E, bool vec, T fill) {
#pragma unroll
    for (int c = 0; c < NPL; c += V) {
      if (vec && c0 + c + V <= E) {
        v[c / V].u = *reinterpret_cast<const uint4*>(row + c0 + c);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const T x = c0 + c + i < E ? row[c0 + c + i] : fill;
          if constexpr (sizeof(T) == 2)
            v[c / V].h[i] = reinterpret_cast<const uint16_t&>(x);
          else
            v[c / V].w[i] = reinterpret_cast<const uint32_t&>(x);
        }
      }
    }
  }

  __device__ __forceinline__ float operator[](int i) const {
    T x;
    if constexpr (sizeof(T) == 2)
      reinterpret_cast<uint16_t&>(x) = v[i / V].h[i % V];
    else
      reinterpret_cast<uint32_t&>(x) = v[i / V].w[i % V];
    return to_f(x);
  }
};

template <class T, int NPL>
__device__ __forceinline__ void store_row(T* row, int c0, int E, bool vec, const float (&z)[NPL]) {
  constexpr int V = 16 / sizeof(T);
#pragma unroll
  for (int c = 0; c < NPL; c += V) {
    if (vec && c0 + c + V <= E) {
      union {
        uint4 u;
        T t[V];
      } w;
#pragma unroll
      for (int i = 0; i < V; ++i) w.t[i] = from_f<T>(z[c + i]);
      *reinterpret_cast<uint4*>(row + c0 + c) = w.u;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c0 + c + i < E) row[c0 + c + i] = from_f<T>(z[c + i]);
    }
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

template <int G>
__device__ __forceinline__ float group_max_nan(float v) {
  if (G == 32) {
    float r;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
  }
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

template <int G>
__device__ __forceinline__ int32_t group_max_s32(int32_t v) {
  if (G == 32) return __reduce_max_sync(kAll, v);
  if (G == 16) {  // a warp's maximum twice, with the other half out of it: a third of the
    // shuffles' latency (16384 x 128 call: 18.7 -> 17.3 us; four of 8 lanes: slower)
    const bool upper = threadIdx.x & 16;
    const int32_t a = __reduce_max_sync(kAll, upper ? INT32_MIN : v);
    const int32_t b = __reduce_max_sync(kAll, upper ? v : INT32_MIN);
    return upper ? b : a;
  }
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

constexpr int log2_of(int v) { return v <= 1 ? 0 : 1 + log2_of(v / 2); }

// A key that orders a row's experts: the leading bits of the logit (as an
// ordered integer), then the expert, the lower the larger. 16-bit types fit
// whole; of an fp32 logit the last IDX bits are cut.
template <int IDX>
__device__ __forceinline__ int32_t expert_key(float z, int e) {
  const int32_t b = __float_as_int(z + 0.0f);   // -0 ties with 0
  constexpr int32_t low = (1 << IDX) - 1;
  return ((b ^ ((b >> 31) & 0x7FFFFFFF)) & ~low) | (low - e);
}

// N values, largest first: Batcher's odd-even merge sort (8: 19 exchanges, 16: 63, 32: 191)
template <int N>
__device__ __forceinline__ void sort_down(int32_t (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int d = p; d >= 1; d /= 2)
#pragma unroll
      for (int i = 0; i + d < N; ++i)
        if (i >= d % p && (i - d % p) / d % 2 == 0 && i / (2 * p) == (i + d) / (2 * p)) {
          const int32_t hi = max(v[i], v[i + d]), lo = min(v[i], v[i + d]);
          v[i] = hi;
          v[i + d] = lo;
        }
}

// The largest keys of a group of G lanes, each lane's NPL sorted: a round
// takes the largest of the lanes' heads, and its lane moves up the next of its
// first D. G = 32: round j's key goes to lane j (`mine`), otherwise its expert
// to slot[j]. Returns whether a lane gave all its D and had more.
template <int G, int IDX, int D, int NPL>
__device__ __forceinline__ bool take_largest(const int32_t (&sorted)[NPL], int k, int rounds, int32_t* slot, int32_t& mine,
                                             int32_t& last, bool& unsure) {
  constexpr int32_t kNone = INT32_MIN;
  const int lane = threadIdx.x & 31;
  int32_t h[D];
#pragma unroll
  for (int i = 0; i < D; ++i) h[i] = sorted[i];
  last = 0x7FFFFFFF;
  unsure = false;
  for (int j = 0; j < rounds; ++j) {
    const int32_t best = group_max_s32<G>(h[0]);
    if (h[0] == best) {
#pragma unroll
      for (int i = 0; i + 1 < D; ++i) h[i] = h[i + 1];
      h[D - 1] = kNone;
    }
    if (G == 32) {
      if (lane == j) mine = best;
    } else {
      if (j > 0) unsure |= ((best ^ last) >> IDX) == 0;
      if (j < k && (lane % G) == 0) slot[j] = ((1 << IDX) - 1) - (best & ((1 << IDX) - 1));
    }
    last = best;
  }
  return D < NPL && h[0] == kNone;
}

// The first document whose end lies past row r (documents: none does), by whole
// warps with one r: 32 ends a step, since the loads' latency is all of it. The
// index stays in [0, documents] whatever the offsets hold.
__device__ __forceinline__ int first_document(const int64_t* offsets, int documents, int64_t r) {
  if (!offsets) return 0;
  int lo = 0, hi = documents;
  while (lo < hi) {
    const int stride = (hi - lo + 31) / 32;
    const int probe = lo + static_cast<int>(threadIdx.x & 31) * stride;
    const uint32_t past = __ballot_sync(kAll, probe < hi && offsets[probe + 1] > r);
    const int first = past ? __ffs(past) - 1 : 32;
    const int probes = (hi - lo + stride - 1) / stride;
    if (first < probes) hi = lo + first * stride;
    if (first > 0) lo += (min(first, probes) - 1) * stride + 1;
  }
  return lo;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// ONE: the grid is one cluster and there is one document without offsets: the
// blocks' sums meet in the first block over distributed shared memory, which
// closes the call. Otherwise the sums go to the workspace for the second launch.
//
// Bound by issue and by the rounds' latency, not by memory: at 131072 x 256
// fp32, k = 8 this takes 66 us where HBM needs 21 (bf16: 57 and 11). Sorting a
// lane's keys once and taking heads costs a third of searching all keys in
// every round (83 us); rows whose largest all lie in one lane take both (81).
template <class T, int G, int NPL, bool ONE>
__global__ void __launch_bounds__(kRouteThreads, forward_blocks(sizeof(T), G, NPL)) route_forward_kernel(const RouteArgs a) {
  constexpr int RPW = 32 / G;          // rows a warp holds at once
  constexpr int kTurns = RPW >= 4 ? 1 : 4 / RPW;   // of such, before the slots of all are worked out
  constexpr int kRows = RPW * kTurns;
  constexpr int kCols = G * NPL;
  extern __shared__ uint8_t smem[];
  float* red = reinterpret_cast<float*>(smem);                        // [kWarps * RPW][kCols]
  int32_t* cnt = reinterpret_cast<int32_t*>(red + kWarps * RPW * kCols);  // [kCols]
  float* stage_v = reinterpret_cast<float*>(cnt + kCols);             // [kWarps][kRows][k]
  int32_t* stage_i = reinterpret_cast<int32_t*>(stage_v + kWarps * kRows * a.k);
  __shared__ float2 sh_row[kWarps * kRows];    // the rows' largest logit and sum of exp (-1 where not live)
  __shared__ float sh_z[kWarps];
  __shared__ int32_t sh_live[kWarps];
  __shared__ float sh_sum[ONE ? kCols : 1];    // ONE: this block's sums, read by the first block
  __shared__ float sh_block_z;
  __shared__ int32_t sh_block_live;
  __shared__ double sh_term[kWarps];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = lane % G, gr = lane / G;
  const uint32_t gmask = (G == 32 ? kAll : ((1u << G) - 1u)) << (G == 32 ? 0 : gr * G);
  const int c0 = gl * NPL;
  const int k = a.k;
  const T* logits = static_cast<const T*>(a.logits);
  const bool vec = ((reinterpret_cast<uintptr_t>(logits) | (a.ld * sizeof(T))) & 15u) == 0;
  float* my_v = stage_v + warp * kRows * k;
  int32_t* my_i = stage_i + warp * kRows * k;
  float2* my_row = sh_row + warp * kRows;
  const uint32_t inv_k = 65536u / k + 1u;      // t / k as t inv_k / 2^16, exact for t < 2048

  if (!ONE && blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  if (ONE && static_cast<int64_t>(blockIdx.x) * a.rows_per_block >= a.N) {  // a block without rows
    for (int e = threadIdx.x; e < kCols; e += kRouteThreads) {
      cnt[e] = 0;
      sh_sum[e] = 0.f;
    }
    if (threadIdx.x == 0) {
      sh_block_z = 0.f;
      sh_block_live = 0;
    }
  }

  const int64_t r0 = blockIdx.x * a.rows_per_block;
  const int64_t r1 = min(a.N, r0 + a.rows_per_block);
  int doc = first_document(a.offsets, a.documents, r0);
  int64_t r = r0;
  while (r < r1) {
    // the piece [r, end): of document doc, or between documents (dead rows)
    int64_t end = r1;
    bool outside = false;
    if (a.offsets) {
      while (doc < a.documents && a.offsets[doc + 1] <= r) ++doc;
      if (doc == a.documents) {
        outside = true;
      } else {
        const int64_t begin = a.offsets[doc];
        outside = begin > r;
        end = min(r1, outside ? begin : a.offsets[doc + 1]);
      }
    }
    for (int e = threadIdx.x; e < kCols; e += kRouteThreads) cnt[e] = 0;
    float acc[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) acc[i] = 0.f;
    float zacc = 0.f;
    int live_rows = 0;
    __syncthreads();

    constexpr bool kAhead = NPL == 8;
    RawRow<T, NPL> next;   // the row after this one, loaded a turn ahead
    if (kAhead && r + warp * kRows + gr < end)
      next.load(logits + (r + warp * kRows + gr) * a.ld, c0, a.E, vec, from_f<T>(neg_inf()));
    for (int64_t base = r + warp * kRows; base < end; base += kWarps * kRows) {
#pragma unroll 1
      for (int turn = 0; turn < kTurns && base + turn * RPW < end; ++turn) {
        const int64_t row = base + turn * RPW + gr;
        const bool in = row < end;
        float z[NPL];
        if (kAhead) {
#pragma unroll
          for (int i = 0; i < NPL; ++i) z[i] = in ? next[i] : neg_inf();
          const int64_t then = turn + 1 < kTurns ? row + RPW : row - turn * RPW + kWarps * kRows;
          if (then < end) next.load(logits + then * a.ld, c0, a.E, vec, from_f<T>(neg_inf()));
        } else if (in) {
          load_row<T, NPL>(logits + row * a.ld, c0, a.E, vec, neg_inf(), z);
        } else {
#pragma unroll
          for (int i = 0; i < NPL; ++i) z[i] = neg_inf();
        }
        bool live = in && !outside && (!a.valid || a.valid[row] != 0);
        float m = z[0];
#pragma unroll
        for (int i = 1; i < NPL; ++i) m = max_nan(m, z[i]);
        m = group_max_nan<G>(m);
        live = live && !(m == neg_inf());
        const float mm = live ? m : 0.f;
        float p[NPL], sum = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          p[i] = exp2_approx((z[i] - mm) * kLog2e);
          sum += p[i];
        }
        sum = group_sum<G>(sum);
        if (live) {
          const float inv = rcp_approx(sum);   // one more error of 2^-23, as in each exp
#pragma unroll
          for (int i = 0; i < NPL; ++i) acc[i] = fmaf(p[i], inv, acc[i]);
        }
        // The k largest by keys, all distinct.
        constexpr int IDX = log2_of(kCols);
        int32_t* slot = my_i + (turn * RPW + gr) * k;
        // fp32: two keys alike in what they keep of the logit, and some logit of
        // the lane's with bits in what they cut (logits rounded to 16 bits have
        // none: their ties are true ties, in the keys' order)
        bool unsure = false;
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) bits |= __float_as_uint(z[i]);
        const int rounds = sizeof(T) == 4 && k < a.E ? k + 1 : k;
        int32_t key[NPL];
        if (a.E == kCols) {
#pragma unroll
          for (int i = 0; i < NPL; ++i) key[i] = expert_key<IDX>(z[i], c0 + i);
        } else {
#pragma unroll
          for (int i = 0; i < NPL; ++i)
            key[i] = c0 + i < a.E ? expert_key<IDX>(z[i], c0 + i) : INT32_MIN + (kCols - 1 - c0 - i);
        }
        sort_down(key);
        if constexpr (G == 1) {
#pragma unroll
          for (int j = 0; j < NPL; ++j) {
            if (j < k) slot[j] = (kCols - 1) - (key[j] & (kCols - 1));
            if (j > 0 && j < rounds) unsure |= ((key[j] ^ key[j - 1]) >> IDX) == 0;
          }
        } else {
          // Few lanes give more than four of the k, so a round moves four; a
          // warp with one that does starts again with all.
          constexpr int D = G >= 16 ? 4 : NPL;
          int32_t mine = 0, last;
          const bool more = take_largest<G, IDX, D>(key, k, rounds, slot, mine, last, unsure);
          if (D < NPL && __any_sync(kAll, more)) take_largest<G, IDX, NPL>(key, k, rounds, slot, mine, last, unsure);
          if (G == 32) {
            const int32_t below = __shfl_down_sync(kAll, mine, 1);
            unsure = lane + 1 < rounds && (((lane == 31 ? last : below) ^ mine) >> IDX) == 0;
            if (lane < k) slot[lane] = (kCols - 1) - (mine & (kCols - 1));
          }
        }
        if (sizeof(T) == 4 && __any_sync(kAll, unsure) && __any_sync(kAll, (bits & ((2u << IDX) - 1u)) != 0)) {
          // (the fast rounds' slots were written by other lanes than these will be)
          __syncwarp();
          // exact: the group's largest logit, the lowest lane that has it (its
          // experts come before the others'), the first of that lane's
          for (int j = 0; j < k; ++j) {
            float bv = neg_inf();
            int bi = 0;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
              const float v = z[i] != z[i] ? __int_as_float(0x7F800000) : z[i];   // NaN before all, as in the keys
              if (v > bv) {
                bv = v;
                bi = i;
              }
            }
            const uint32_t who = __ballot_sync(kAll, bv == group_max<G>(bv)) & gmask;
            if (__ffs(who) - 1 == lane) {
              slot[j] = bv > neg_inf() ? c0 + bi : 0;
#pragma unroll
              for (int i = 0; i < NPL; ++i)
                if (i == bi) z[i] = neg_inf();
            }
            // a row without a logit left: its slots read a -inf again below
            if (bv == neg_inf() && who == gmask && gl == 0) slot[j] = -1;
          }
        }
        if (gl == 0) my_row[turn * RPW + gr] = make_float2(live ? m : neg_inf(), live ? sum : -1.f);
      }
      __syncwarp();
      // these rows' statistics, a lane per row
      const int rows = static_cast<int>(min(static_cast<int64_t>(kRows), end - base));
      if (lane < rows) {
        const float2 rw = my_row[lane];
        const bool live = rw.y != -1.f;
        const float log_sum = live ? logf(rw.y) : 0.f;
        // apart: their sum would lose log_sum's last bits where |m| is large,
        // and with them the backward's softmax
        a.stats[base + lane] = make_float2(rw.x, log_sum);
        if (live) {
          const float lse = rw.x + log_sum;
          zacc = fmaf(lse, lse, zacc);
          ++live_rows;
        }
      }
      // and their slots, a lane per slot: exp, then the weights
      const int slots = rows * k;
      for (int t = lane; t < slots; t += 32) {
        const int b = (t * inv_k) >> 16;
        const float2 rw = my_row[b];
        const int e = my_i[t];
        float ex = 0.f;
        int keep = -1;
        if (e >= 0 && rw.y != -1.f) {   // live
          const float v = to_f(logits[(base + b) * a.ld + e]);
          if (v != neg_inf()) {
            ex = exp2_approx((v - rw.x) * kLog2e);
            keep = e;
            atomicAdd(&cnt[e], 1);
          }
        }
        my_v[t] = ex;
        my_i[t] = keep;
      }
      __syncwarp();
      for (int t = lane; t < slots; t += 32) {
        const int b = (t * inv_k) >> 16;
        float share = my_row[b].y;
        if (a.renormalize) {
          share = 0.f;
          for (int j = 0; j < k; ++j) share += my_v[b * k + j];
        }
        const int e = my_i[t];
        a.weights[base * k + t] = e >= 0 ? my_v[t] * (1.0f / share) : 0.f;
        a.experts[base * k + t] = e;
      }
      __syncwarp();
    }

    // the piece's sums, in a fixed order
#pragma unroll
    for (int i = 0; i < NPL; ++i) red[(warp * RPW + gr) * kCols + c0 + i] = acc[i];
    for (int o = 16; o > 0; o >>= 1) {
      zacc += __shfl_xor_sync(kAll, zacc, o);
      live_rows += __shfl_xor_sync(kAll, live_rows, o);
    }
    if (lane == 0) {
      sh_z[warp] = zacc;
      sh_live[warp] = live_rows;
    }
    __syncthreads();
    if (!outside) {
      const int64_t unit = static_cast<int64_t>(blockIdx.x) + doc;
      for (int e = threadIdx.x; e < a.E; e += kRouteThreads) {
        float s = 0.f;
        for (int w = 0; w < kWarps * RPW; ++w) s += red[w * kCols + e];
        if (ONE) {
          sh_sum[e] = s;
        } else {
          a.unit_p[unit * a.E + e] = s;
          a.unit_c[unit * a.E + e] = cnt[e];
        }
      }
      if (threadIdx.x == 0) {
        float s = 0.f;
        int n = 0;
        for (int w = 0; w < kWarps; ++w) {
          s += sh_z[w];
          n += sh_live[w];
        }
        if (ONE) {
          sh_block_z = s;
          sh_block_live = n;
        } else {
          a.unit_z[unit] = s;
          a.unit_live[unit] = n;
        }
      }
    }
    __syncthreads();
    r = end;
  }
  if constexpr (ONE) {
    cluster_sync();
    if (blockIdx.x == 0) {
      float zs = 0.f;
      int n = 0;
      for (uint32_t b = 0; b < gridDim.x; ++b) {
        zs += __uint_as_float(ld_cluster_u32(mapa_shared(smem_u32(&sh_block_z), b)));
        n += static_cast<int>(ld_cluster_u32(mapa_shared(smem_u32(&sh_block_live), b)));
      }
      const float slope_n = n > 0 ? static_cast<float>(a.E) / (static_cast<float>(a.k) * static_cast<float>(n)) : 0.f;
      double term = 0.0;
      for (int e = threadIdx.x; e < a.E; e += kRouteThreads) {
        float p = 0.f;
        int c = 0;
        for (uint32_t b = 0; b < gridDim.x; ++b) {
          p += __uint_as_float(ld_cluster_u32(mapa_shared(smem_u32(sh_sum + e), b)));
          c += static_cast<int>(ld_cluster_u32(mapa_shared(smem_u32(cnt + e), b)));
        }
        a.counts[e] = c;
        const float slope = slope_n * static_cast<float>(c);
        a.slope[e] = slope;
        term += static_cast<double>(slope * p);
      }
      for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(kAll, term, o);
      if (lane == 0) sh_term[warp] = term;
      __syncthreads();
      if (threadIdx.x == 0) {
        term = 0.0;
        for (int w = 0; w < kWarps; ++w) term += sh_term[w];
        const double inv = n > 0 ? 1.0 / n : 0.0;
        a.result[0] = static_cast<float>(term * inv);
        a.result[1] = static_cast<float>(zs * inv);
        a.result[2] = static_cast<float>(inv);
        a.result[3] = __int_as_float(n);
      }
    }
    cluster_sync();  // the first block reads the others' shared memory until here
  } else {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
}

// The blocks whose rows meet document d: [*b0, *b1), empty if it has none.
__device__ __forceinline__ void document_blocks(const RouteArgs& a, int d, int* b0, int* b1) {
  int64_t lo = 0, hi = a.N;
  if (a.offsets) {
    lo = a.offsets[d];
    hi = a.offsets[d + 1];
  }
  lo = max(lo, static_cast<int64_t>(0));
  hi = min(hi, a.N);
  if (lo >= hi) {
    *b0 = *b1 = 0;
    return;
  }
  *b0 = static_cast<int>(lo / a.rows_per_block);
  *b1 = static_cast<int>((hi - 1) / a.rows_per_block) + 1;
}

// One block of R warps per (document, chunk of experts): counts, slopes and
// the balance term of its experts from the units, in order. The last block to
// finish adds the terms, in order, and writes the losses. Bound by the latency
// of its chain (loads, three barriers, a counter): about 7 us after the
// forward at 456 units of 256 experts, whose 0.9 MB are nothing. It starts while
// the forward drains.
template <int R>
__global__ void __launch_bounds__(32 * R) route_finish_kernel(const RouteArgs a, int chunks, int chunk_size) {
  __shared__ float sh_p[32][R + 1];
  __shared__ int32_t sh_c[32][R + 1];
  // launched while the forward still runs: its results from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float sh_z[R];
  __shared__ int32_t sh_n[R];
  __shared__ float sh_t[2][R];
  __shared__ bool last;
  const int d = blockIdx.x / chunks, chunk = blockIdx.x - d * chunks;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  int b0, b1;
  document_blocks(a, d, &b0, &b1);

  int n = 0;
  float zs = 0.f;  // (fp64 on every thread would be the bound: 36 us at 608 units of 128 experts)
  for (int b = b0 + threadIdx.x; b < b1; b += 32 * R) {
    n += a.unit_live[static_cast<int64_t>(b) + d];
    zs += a.unit_z[static_cast<int64_t>(b) + d];
  }
  for (int o = 16; o > 0; o >>= 1) {
    n += __shfl_xor_sync(kAll, n, o);
    zs += __shfl_xor_sync(kAll, zs, o);
  }
  if (tx == 0) {
    sh_n[ty] = n;
    sh_z[ty] = zs;
  }
  // a lane's share of the units of expert e (a tree over the lanes follows:
  // fp32 in both); the first ones are on their way over the barrier
  const int e_end = min(a.E, (chunk + 1) * chunk_size);
  float p = 0.f;
  int c = 0;
  auto load_share = [&](int e) {
    p = 0.f;
    c = 0;
    if (e >= e_end) return;
#pragma unroll 16
    for (int b = b0 + ty; b < b1; b += R) {
      const int64_t u = (static_cast<int64_t>(b) + d) * a.E + e;
      p += a.unit_p[u];
      c += a.unit_c[u];
    }
  };
  load_share(chunk * chunk_size + tx);
  __syncthreads();
  n = tx < R ? sh_n[tx] : 0;
  zs = tx < R ? sh_z[tx] : 0.f;
  for (int o = 16; o > 0; o >>= 1) {
    n += __shfl_xor_sync(kAll, n, o);
    zs += __shfl_xor_sync(kAll, zs, o);
  }
  const float slope_n = n > 0 ? static_cast<float>(a.E) / (static_cast<float>(a.k) * static_cast<float>(n)) : 0.f;

  float term = 0.f;
  for (int e0 = chunk * chunk_size; e0 < e_end; e0 += 32) {
    if (e0 != chunk * chunk_size) load_share(e0 + tx);
    sh_p[tx][ty] = p;
    sh_c[tx][ty] = c;
    __syncthreads();
    for (int x = ty; x < 32 && e0 + x < e_end; x += R) {  // a warp per expert, its lanes over the shares
      p = tx < R ? sh_p[x][tx] : 0.f;
      c = tx < R ? sh_c[x][tx] : 0;
      for (int o = 16; o > 0; o >>= 1) {
        p += __shfl_xor_sync(kAll, p, o);
        c += __shfl_xor_sync(kAll, c, o);
      }
      if (tx == 0) {
        const int64_t o = static_cast<int64_t>(d) * a.E + e0 + x;
        const float slope = slope_n * static_cast<float>(c);
        a.counts[o] = c;
        a.slope[o] = slope;
        term = fmaf(slope, p, term);
      }
    }
    __syncthreads();
  }
  if (tx == 0) sh_z[ty] = term;
  __syncthreads();
  if (ty == 0) {
    term = tx < R ? sh_z[tx] : 0.f;
    for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(kAll, term, o);
    if (tx == 0) {
      a.terms[blockIdx.x] = term;
      if (chunk == 0) {
        a.doc_live[d] = n;
        a.doc_z[d] = zs;
      }
      __threadfence();   // these three are all the last block reads
      last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();

  // fixed order: a thread's stride, then the tree
  // (the strides in fp64: a thread has many only where there are many documents)
  double bal_sum = 0.0, z_sum = 0.0;
  int live = 0;
  const int64_t terms = static_cast<int64_t>(a.documents) * chunks;
  for (int64_t i = threadIdx.x; i < terms; i += 32 * R) bal_sum += __ldcg(a.terms + i);
  for (int i = threadIdx.x; i < a.documents; i += 32 * R) {
    live += __ldcg(a.doc_live + i);
    z_sum += __ldcg(a.doc_z + i);
  }
  // (few documents fill few warps: the others have nothing to add)
  const int busy = static_cast<int>(min(static_cast<int64_t>(R), (terms + 31) / 32));
  float bal = static_cast<float>(bal_sum), z = static_cast<float>(z_sum);
  if (ty < busy) {
    for (int o = 16; o > 0; o >>= 1) {
      bal += __shfl_xor_sync(kAll, bal, o);
      z += __shfl_xor_sync(kAll, z, o);
      live += __shfl_xor_sync(kAll, live, o);
    }
    if (tx == 0) {
      sh_t[0][ty] = bal;
      sh_t[1][ty] = z;
      sh_n[ty] = live;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < busy; ++w) {
      bal += sh_t[0][w];
      z += sh_t[1][w];
      live += sh_n[w];
    }
    const double inv = live > 0 ? 1.0 / live : 0.0;
    a.result[0] = static_cast<float>(bal * inv);
    a.result[1] = static_cast<float>(z * inv);
    a.result[2] = static_cast<float>(inv);
    a.result[3] = __int_as_float(live);
  }
}

// d z of every row, as the formula at the top has it: one read of the logits, one
// write of the gradient, the row in registers in between. What the chosen
// weights add is scattered into a row of shared memory per group of lanes, the
// one place where an expert's lane is not known before. Bound by HBM: 131072 x
// 256 fp32 moves 282 MB in 47 us, 6.0 TB/s, 89 % of what a copy reaches.
template <class T, int G, int NPL>
__global__ void __launch_bounds__(kRouteThreads)
    route_backward_kernel(const RouteArgs a, const float* d_weights, const float* d_balance, const float* d_z,
                          T* d_logits, int64_t ldd) {
  constexpr int RPW = 32 / G;
  constexpr int kCols = G * NPL;
  extern __shared__ uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = lane % G, gr = lane / G;
  const int c0 = gl * NPL;
  const int k = a.k;
  // what the chosen weights add to d_logits of this group's row
  float* extra = reinterpret_cast<float*>(smem) + (warp * RPW + gr) * kCols;
#pragma unroll
  for (int i = 0; i < NPL; ++i) extra[c0 + i] = 0.f;
  __syncwarp();
  const T* logits = static_cast<const T*>(a.logits);
  const bool vec = ((reinterpret_cast<uintptr_t>(logits) | (a.ld * sizeof(T))) & 15u) == 0;
  const bool vec_d = ((reinterpret_cast<uintptr_t>(d_logits) | (ldd * sizeof(T))) & 15u) == 0;
  const float inv_n = a.result[2];
  const float gb = d_balance ? *d_balance * inv_n : 0.f;
  const float gz = d_z ? 2.0f * *d_z * inv_n : 0.f;

  const int64_t r0 = blockIdx.x * a.rows_per_block;
  const int64_t r1 = min(a.N, r0 + a.rows_per_block);
  int doc = first_document(a.offsets, a.documents, r0), held = -1;
  float slope[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) slope[i] = 0.f;
  // A round ahead: the row and what belongs to it. The loads of one row alone
  // left the kernel waiting for memory (70 us at 131072 x 256 fp32).
  constexpr bool kAhead = NPL == 8;
  float next[NPL];
  float2 next_stat = make_float2(neg_inf(), 0.f);
  int next_e = -1;
  float next_w = 0.f, next_d = 0.f;
  auto fetch = [&](int64_t row) {
    next_stat = make_float2(neg_inf(), 0.f);
    if (row < r1) {
      next_stat = a.stats[row];
      load_row<T, NPL>(logits + row * a.ld, c0, a.E, vec, neg_inf(), next);
      if (d_weights && gl < k) {
        next_e = a.experts[row * k + gl];
        next_w = a.weights[row * k + gl];
        next_d = d_weights[row * k + gl];
      }
    }
  };
  if (kAhead) fetch(r0 + warp * RPW + gr);
  for (int64_t base = r0 + warp * RPW; base < r1; base += kWarps * RPW) {
    const int64_t row = base + gr;
    const bool in = row < r1;
    if (!kAhead) fetch(row);
    const float2 stat = next_stat;
    const int slot_e = next_e;
    const float slot_w = next_w, slot_d = next_d;
    float z[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) z[i] = next[i];
    if (kAhead) fetch(row + kWarps * RPW);
    const bool live = !(stat.x == neg_inf());
    if (in && a.offsets)
      while (doc < a.documents && a.offsets[doc + 1] <= row) ++doc;
    if (live && doc != held && doc < a.documents) {
      load_row<float, NPL>(a.slope + static_cast<int64_t>(doc) * a.E, c0, a.E, false, 0.f, slope);
#pragma unroll
      for (int i = 0; i < NPL; ++i) slope[i] *= gb;
      held = doc;
    }
    // chosen slots: w (g - [renormalised] sum g w) lands on the slot's expert
    float gw = 0.f;
    if (d_weights && live) {
      // (a slot without an expert has weight 0, whatever gradient came for it)
      if (gl < k && slot_e >= 0) gw = slot_d * slot_w;
      for (int j = gl + G; j < k; j += G)
        if (a.experts[row * k + j] >= 0) gw = fmaf(d_weights[row * k + j], a.weights[row * k + j], gw);
    }
    gw = group_sum<G>(gw);
    if (d_weights && live) {
      const float off = a.renormalize ? gw : 0.f;
      if (gl < k && slot_e >= 0 && slot_e < a.E) extra[slot_e] = slot_w * (slot_d - off);
      for (int j = gl + G; j < k; j += G) {
        const int e = a.experts[row * k + j];
        if (e >= 0 && e < a.E) extra[e] = a.weights[row * k + j] * (d_weights[row * k + j] - off);
      }
    }
    __syncwarp();
    float p[NPL], dot = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      p[i] = live ? exp2_approx(((z[i] - stat.x) - stat.y) * kLog2e) : 0.f;
      dot = fmaf(p[i], slope[i], dot);
    }
    dot = group_sum<G>(dot) + (a.renormalize ? 0.f : gw);
    const float shift = live ? gz * (stat.x + stat.y) - dot : 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      p[i] = fmaf(p[i], slope[i] + shift, extra[c0 + i]);
      extra[c0 + i] = 0.f;
    }
    if (in) store_row<T, NPL>(d_logits + row * ldd, c0, a.E, vec_d, p);
    __syncwarp();
  }
}

template <class T, int G, int NPL>
cudaError_t forward_t(const RouteArgs& a, cudaStream_t s) {
  const size_t rows = kWarps * (32 / G), cols = G * NPL;
  // at most 8 x 32 x 32 + 1024 floats and 8 x 4 x 32 slots, 44 KB (beside 4 KB of static memory)
  const size_t smem = rows * cols * 4 + cols * 4 + std::max<size_t>(rows, 4 * kWarps) * a.k * 8;
  // only with the static memory can that pass the default 48 KB; per launch,
  // since the attribute belongs to the current device
  if (smem > 40960) {
    auto kern = a.one_launch ? route_forward_kernel<T, G, NPL, true> : route_forward_kernel<T, G, NPL, false>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 45056);
    if (e != cudaSuccess) return e;
  }
  if (!a.one_launch) {
    route_forward_kernel<T, G, NPL, false><<<a.blocks, kRouteThreads, smem, s>>>(a);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.blocks);
  cfg.blockDim = dim3(kRouteThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = a.blocks;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, route_forward_kernel<T, G, NPL, true>, a);
}

template <class T, int G, int NPL>
cudaError_t backward_t(const RouteArgs& a, const float* dw, const float* db, const float* dz, void* out, int64_t ldd,
                       cudaStream_t s) {
  const size_t smem = kWarps * (32 / G) * static_cast<size_t>(G * NPL) * 4;
  route_backward_kernel<T, G, NPL><<<a.blocks, kRouteThreads, smem, s>>>(a, dw, db, dz, static_cast<T*>(out), ldd);
  return cudaGetLastError();
}

// f(G, NPL) for the geometry's instantiation, as integral constants
template <class T, class F>
cudaError_t for_geometry(const RouteGeometry& g, F&& f) {
  if (g.per_lane == 8) {
    switch (g.lanes) {
      case 1: return f(std::integral_constant<int, 1>(), std::integral_constant<int, 8>());
      case 2: return f(std::integral_constant<int, 2>(), std::integral_constant<int, 8>());
      case 4: return f(std::integral_constant<int, 4>(), std::integral_constant<int, 8>());
      case 8: return f(std::integral_constant<int, 8>(), std::integral_constant<int, 8>());
      case 16: return f(std::integral_constant<int, 16>(), std::integral_constant<int, 8>());
      default: return f(std::integral_constant<int, 32>(), std::integral_constant<int, 8>());
    }
  }
  if (g.per_lane == 16) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>(), std::integral_constant<int, 32>());
}

}  // namespace

RouteGeometry route_geometry(int64_t N, int64_t E, int element_bytes, int64_t documents, bool offsets, bool backward,
                             int num_sms) {
  RouteGeometry g;
  g.per_lane = E <= 256 ? 8 : (E <= 512 ? 16 : 32);
  g.lanes = 1;
  while (g.lanes < 32 && static_cast<int64_t>(g.lanes) * g.per_lane < E) g.lanes *= 2;
  const int64_t step = std::max(32 / g.lanes, 4);   // a warp's rows before their slots
  // Short batches run as one cluster of up to 8 blocks that closes the call
  // itself: one launch instead of two. Past 8 turns of rows per warp the
  // whole GPU's width is worth the second launch.
  g.one_launch = !backward && !offsets && N > 0 && N <= 8 * 8 * kWarps * (32 / g.lanes);
  // as many blocks as are resident
  const int resident = backward ? kBackwardBlocks : forward_blocks(element_bytes, g.lanes, g.per_lane);
  const int64_t most = g.one_launch ? 8 : resident * static_cast<int64_t>(num_sms);
  // Rows to a warp's step, not a block's (20000 x 128 bf16: 18 us, else 20),
  // but a step for every warp (5000 x 256 fp32: 15 us, else 18)
  int64_t per = std::max((N + most - 1) / most, kWarps * step);
  per = (per + step - 1) / step * step;
  g.rows_per_block = per;
  g.blocks = static_cast<int>((N + g.rows_per_block - 1) / g.rows_per_block);
  if (g.one_launch)
    while (g.blocks & (g.blocks - 1)) ++g.blocks;  // a power of two
  g.chunks = documents >= num_sms ? 1 : static_cast<int>((E + 31) / 32);
  return g;
}

cudaError_t launch_route_forward(int dtype, const RouteGeometry& g, const RouteArgs& a, cudaStream_t s) {
  auto run = [&](auto t) {
    using T = decltype(t);
    return for_geometry<T>(g, [&](auto G, auto NPL) { return forward_t<T, G.value, NPL.value>(a, s); });
  };
  return dtype == 0 ? run(__nv_bfloat16()) : dtype == 1 ? run(float()) : run(__half());
}

cudaError_t launch_route_finish(const RouteGeometry& g, const RouteArgs& a, cudaStream_t s) {
  const int chunk_size = g.chunks == 1 ? a.E : 32;
  // a document spread over many blocks has many units to add: more warps
  const bool many = a.blocks >= 64 * static_cast<int64_t>(a.documents);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.documents * g.chunks);
  cfg.blockDim = dim3(many ? 1024 : 256);
  cfg.stream = s;
  cudaLaunchAttribute attr;  // may start while the forward drains
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return many ? cudaLaunchKernelEx(&cfg, route_finish_kernel<32>, a, g.chunks, chunk_size)
              : cudaLaunchKernelEx(&cfg, route_finish_kernel<8>, a, g.chunks, chunk_size);
}

cudaError_t launch_route_backward(int dtype, const RouteGeometry& g, const RouteArgs& a, const float* d_weights,
                                  const float* d_balance, const float* d_z, void* d_logits, int64_t ldd,
                                  cudaStream_t s) {
  auto run = [&](auto t) {
    using T = decltype(t);
    return for_geometry<T>(g, [&](auto G, auto NPL) {
      return backward_t<T, G.value, NPL.value>(a, d_weights, d_balance, d_z, d_logits, ldd, s);
    });
  };
  return dtype == 0 ? run(__nv_bfloat16()) : dtype == 1 ? run(float()) : run(__half());
}

}  // namespace flce
