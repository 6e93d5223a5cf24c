// Row kernels of the LM-head operators (flce_score.h): what the product's
// per-group statistics become per token (log probability, entropy, the top
// alternatives), the gradient's rows, and distillation's rows.
//
// A row's softmax over all columns from its groups' (largest m, sum l of 2^y, sum
// s of y 2^y), y = (z - m) c, c = log2(e) / temperature: with M the largest m and
// w = 2^((m - M) c),  L = sum w l,  logprob = (z_t - M) / temperature - log L,
// entropy = log L - (1 / L) sum w (ln2 s + (m - M) / temperature l).
// M and log L are kept apart: one fp32 sum of both would lose log L's last bits
// where logits are large.
//
// A single logit (the given token's or an alternative's) is summed again, in twice the
// bits of fp32: products of bf16 are exact in fp32 and
// every addition's rounding error is carried along. So equal logits stay equal and
// the order of near-equal ones does not depend on how the product was tiled.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "flce_score.cuh"

namespace flce {
namespace {

constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2e = 1.4426950408889634f;

// ----------------------------------------------------- rows that count

// The call's row that is a chunk's i-th
__device__ __forceinline__ int64_t row_of(const ScoreChunk& q, int64_t i) { return q.order ? q.order[q.off + i] : q.off + i; }

// Where the zeros behind a chunk's rows end: a multiple of the products' 256 rows. A
// chunk without rows needs none, but the first one's product runs whatever there is.
__device__ __forceinline__ int tail_end(const ScoreChunk& q, int rows) {
  if (rows == 0 && q.off > 0) return 0;
  return min(q.rows, (max(rows, 1) + 255) / 256 * 256);
}

// Fills 16-byte pieces, or 4-byte ones
__device__ __forceinline__ void zero_row(uint8_t* to, int64_t bytes, int thread, int threads) {
  if ((reinterpret_cast<uint64_t>(to) | static_cast<uint64_t>(bytes)) % 16 == 0) {
    for (int64_t i = thread * 16; i < bytes; i += threads * 16) *reinterpret_cast<uint4*>(to + i) = make_uint4(0, 0, 0, 0);
  } else {
    for (int64_t i = thread * 4; i < bytes; i += threads * 4) *reinterpret_cast<uint32_t*>(to + i) = 0u;
  }
}

// What a row gets that does not count: by a warp
__device__ __forceinline__ void skip_row(const ScoreOrderArgs& a, int64_t r, int lane) {
  if (r >= a.N || (a.t ? a.t[r] != a.ignore_index : a.live[r] != 0)) return;
  if (a.dx) zero_row(static_cast<uint8_t*>(a.dx) + r * a.row_bytes, a.row_bytes, lane, 32);
  if (lane == 0) {
    if (a.logprobs) a.logprobs[r] = 0.f;
    if (a.entropy) a.entropy[r] = 0.f;
    if (a.stats) a.stats[r] = make_float2(0.f, 0.f);
  }
  for (int i = lane; i < a.top; i += 32) {
    a.top_logprobs[r * a.top + i] = 0.f;
    a.top_ids[r * a.top + i] = -1;
  }
}

// The first block puts the rows in order, 1024 at a time, each warp's and then each
// thread's place by counts: a few microseconds for a batch, which the products of the
// rows left out repay from the first 256 on. The others see to the rows left out.
__global__ void __launch_bounds__(1024) score_order_kernel(const ScoreOrderArgs a) {
  __shared__ int s_count[2][32];
  if (blockIdx.x > 0) {
    skip_row(a, (static_cast<int64_t>(blockIdx.x) - 1) * 32 + (threadIdx.x >> 5), threadIdx.x & 31);
    return;
  }
  const int64_t* t = a.t;
  const uint8_t* live = a.live;
  const int64_t N = a.N, ignore_index = a.ignore_index;
  int32_t* order = a.order;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int done = 0, turn = 0;
  auto counts = [&](int64_t i) { return i < N && (t ? t[i] != ignore_index : live[i] != 0); };
  bool next = counts(threadIdx.x);
  for (int64_t base = 0; base < N; base += 1024, turn ^= 1) {
    const bool in = next;
    next = counts(base + 1024 + threadIdx.x);
    const uint32_t mask = __ballot_sync(0xffffffffu, in);
    if (lane == 0) s_count[turn][warp] = __popc(mask);
    __syncthreads();  // the other turn's counts are read by now
    int own = s_count[turn][lane], upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const int before = __shfl_sync(0xffffffffu, upto - own, warp);
    if (in) order[done + before + __popc(mask & ((1u << lane) - 1u))] = static_cast<int32_t>(base + threadIdx.x);
    done += __shfl_sync(0xffffffffu, upto, 31);
  }
  if (threadIdx.x == 0) *a.count = static_cast<uint32_t>(done);
}

// --------------------------------------------------------- shared pieces

template <int THREADS>
__device__ __forceinline__ float block_max(float v, float* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s[0];
#pragma unroll
  for (int w = 1; w < THREADS / 32; ++w) v = max_nan(v, s[w]);
  __syncthreads();
  return v;
}

template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s[0];
#pragma unroll
  for (int w = 1; w < THREADS / 32; ++w) v += s[w];
  __syncthreads();
  return v;
}

// Two fp32 at once (the packed forms issue as one)
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// a - b (the product with -1 is exact)
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %2, %3, %1;" : "=l"(r) : "l"(a), "l"(b), "l"(0xBF800000BF800000ull));
  return r;
}
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}

// A sum in twice the bits of fp32: hi is it rounded, lo what that leaves. fp64 would
// do, at a sixty-fourth of fp32's rate: with it the sums over lanes and the ordering
// took four fifths of a row's time.
struct Pair {
  float hi, lo;
};

// a + b, and what rounding it leaves
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  const float u = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, u)), __fsub_rn(b, u))};
}

// hi + lo; an infinite hi leaves no rest
__device__ __forceinline__ Pair settled(float hi, float lo) {
  const Pair s = two_sum(hi, lo);
  return fabsf(hi) < INFINITY ? s : Pair{hi, 0.f};
}

__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  return settled(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}

// the same in all lanes: each step adds the same two numbers on both sides
__device__ __forceinline__ Pair warp_sum(Pair v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Pair w = {__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)};
    const bool first = (threadIdx.x & o) == 0;
    v = add(first ? v : w, first ? w : v);
  }
  return v;
}

// (hi, lo) += x w: the products of bf16 are exact, and lo collects what each addition
// to hi rounds away
__device__ __forceinline__ void add_product(uint64_t& hi, uint64_t& lo, uint64_t x, uint32_t w) {
  const uint64_t p = mul2(x, pack2(w << 16, w & 0xFFFF0000u));
  const uint64_t s = add2(hi, p), u = sub2(s, hi);
  lo = add2(lo, add2(sub2(hi, sub2(s, u)), sub2(p, u)));
  hi = s;
}

__device__ __forceinline__ Pair joined(const uint64_t (&hi)[2], const uint64_t (&lo)[2]) {
  Pair v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = settled(__uint_as_float(static_cast<uint32_t>(hi[i >> 1] >> (32 * (i & 1)))),
                   __uint_as_float(static_cast<uint32_t>(lo[i >> 1] >> (32 * (i & 1)))));
  return add(add(v[0], v[1]), add(v[2], v[3]));
}

// x . w0 and x . w1 of a row each, by a warp
__device__ __forceinline__ void warp_dot2(const __nv_bfloat16* x, const __nv_bfloat16* w0, const __nv_bfloat16* w1, int64_t H,
                                          int lane, Pair (&out)[2]) {
  uint64_t hi[2][2] = {{0, 0}, {0, 0}}, lo[2][2] = {{0, 0}, {0, 0}};
#pragma unroll 2
  for (int64_t h = lane * 8; h < H; h += 256) {
    const uint4 a = *reinterpret_cast<const uint4*>(x + h);
    const uint4 b[2] = {*reinterpret_cast<const uint4*>(w0 + h), *reinterpret_cast<const uint4*>(w1 + h)};
    const uint32_t av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t xv = pack2(av[i] << 16, av[i] & 0xFFFF0000u);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        add_product(hi[q][i & 1], lo[q][i & 1], xv, i == 0 ? b[q].x : i == 1 ? b[q].y : i == 2 ? b[q].z : b[q].w);
      }
    }
  }
  out[0] = joined(hi[0], lo[0]);
  out[1] = joined(hi[1], lo[1]);
  out[0] = warp_sum(out[0]);
  out[1] = warp_sum(out[1]);
}

// x . w
__device__ __forceinline__ Pair warp_dot(const __nv_bfloat16* x, const __nv_bfloat16* w, int64_t H, int lane) {
  uint64_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll 4
  for (int64_t h = lane * 8; h < H; h += 256) {
    const uint4 a = *reinterpret_cast<const uint4*>(x + h);
    const uint4 b = *reinterpret_cast<const uint4*>(w + h);
    const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      add_product(hi[i & 1], lo[i & 1], pack2(av[i] << 16, av[i] & 0xFFFF0000u), bv[i]);
  }
  return warp_sum(joined(hi, lo));
}

__device__ __forceinline__ Pair warp_dot(const float* x, const float* w, int64_t H, int lane) {
  Pair v = {0.f, 0.f};
  for (int64_t h = lane; h < H; h += 32) {
    const float p = __fmul_rn(x[h], w[h]), rest = __fmaf_rn(x[h], w[h], -p);
    const Pair s = two_sum(v.hi, p);
    v = {s.hi, __fadd_rn(v.lo, __fadd_rn(s.lo, rest))};
  }
  return warp_sum(settled(v.hi, v.lo));
}

__device__ __forceinline__ void warp_dot2(const float* x, const float* w0, const float* w1, int64_t H, int lane,
                                          Pair (&out)[2]) {
  const float* w[2] = {w0, w1};
  out[0] = out[1] = {0.f, 0.f};
  for (int64_t h = lane; h < H; h += 32) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float p = __fmul_rn(x[h], w[q][h]), rest = __fmaf_rn(x[h], w[q][h], -p);
      const Pair s = two_sum(out[q].hi, p);
      out[q] = {s.hi, __fadd_rn(out[q].lo, __fadd_rn(s.lo, rest))};
    }
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) out[q] = warp_sum(settled(out[q].hi, out[q].lo));
}

// A key that orders floats (NaN above all, 0 below every value's)
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Pairs likewise (one zero, in either part)
__device__ __forceinline__ uint64_t order_key(Pair v) {
  return (static_cast<uint64_t>(order_key(v.hi + 0.f)) << 32) | order_key(v.lo + 0.f);
}

constexpr int kMaxCandidates = 128;
constexpr int kMaxGroups = 256;
constexpr int kMaxima = 128;
static_assert(kScoreMaxTop <= kMaxCandidates, "room for the result");

template <int THREADS>
struct SelectSmem {
  int hist[256];
  int digit, above;
  int warp_cnt[THREADS / 32];
};

// The k-th largest of n keys (k <= n) by its bytes from the top; `above` gets how
// many are larger.
template <int THREADS, class Key>
__device__ __noinline__ uint32_t block_select(int64_t n, int k, SelectSmem<THREADS>& s, int& above, Key key) {
  uint32_t prefix = 0;
  int rest = k;  // rank among the keys with the prefix
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += THREADS) s.hist[i] = 0;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n; i += THREADS) {
      const uint32_t v = key(i);
      if (shift == 24 || (v >> (shift + 8)) == prefix) atomicAdd(&s.hist[(v >> shift) & 255u], 1);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      // lane i holds digits 255 - 8 i down to 248 - 8 i
      const int lane = threadIdx.x;
      int own = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) own += s.hist[255 - 8 * lane - j];
      int upto = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      int before = upto - own;
      if (before < rest && rest <= upto) {
        int d = 255 - 8 * lane;
        while (before + s.hist[d] < rest) before += s.hist[d--];
        s.digit = d;
        s.above = before;
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | static_cast<uint32_t>(s.digit);
    rest -= s.above;
    __syncthreads();
  }
  above = k - rest;
  return prefix;
}

// Positions 0 .. n - 1, in order, that `take` wants (2: always, 1: the first
// `quota` of them), at most `room`; put(slot, position). Returns how many.
template <int THREADS, class Take, class Put>
__device__ __noinline__ int block_collect(int64_t n, int quota, int room, SelectSmem<THREADS>& s, Take take, Put put) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t below = (1u << lane) - 1u;
  int done = 0, tied = 0;
  for (int64_t base = 0; base < n; base += THREADS) {
    const int64_t i = base + threadIdx.x;
    const int want = i < n ? take(i) : 0;
    const uint32_t tie = __ballot_sync(0xffffffffu, want == 1);
    if (__syncthreads_or(want) == 0) continue;
    if (lane == 0) s.warp_cnt[warp] = __popc(tie);
    __syncthreads();
    int rank = tied;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) rank += s.warp_cnt[w];
      tied += s.warp_cnt[w];
    }
    rank += __popc(tie & below);
    const bool in = want == 2 || (want == 1 && rank < quota);
    const uint32_t chosen = __ballot_sync(0xffffffffu, in);
    __syncthreads();
    if (lane == 0) s.warp_cnt[warp] = __popc(chosen);
    __syncthreads();
    int slot = done;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) slot += s.warp_cnt[w];
      done += s.warp_cnt[w];
    }
    slot += __popc(chosen & below);
    if (in && slot < room) put(slot, i);
    __syncthreads();
  }
  return min(done, room);
}

// ------------------------------------------------- log probabilities

// What a block finds the alternatives in
template <int THREADS>
struct TopSmem {
  SelectSmem<THREADS> sel;
  uint32_t key[kMaxima];
  int group[kMaxGroups];
  float lower[kMaxCandidates], upper[kMaxCandidates];
  float gmax[kScoreMaxTop];
  float border;
  int groups, found, kept;
};

// A stored value's bounds: half a step of fp16 (with the fp32 steps around it) and
// the product's own sum; -inf lies below fp16's range.
template <class Z>
__device__ __forceinline__ float stored_bound(float v, float gm, float M, float sign) {
  if (sizeof(Z) == 2 && v == -INFINITY) return sign < 0.f ? v : gm - 65500.f;
  float reach = fmaxf(fabsf(M), fabsf(v)) * 6.1e-5f;
  if (sizeof(Z) == 2) reach = fmaf(gm - v, 5.5e-4f, reach + 6e-8f);
  return reach < INFINITY ? fmaf(sign, reach, v) : v;
}

// The ids of whatever may be among the row's `top` largest logits, to id, and how
// many. m: the thread's largest group maximum.
//
// The quick way: the top-th largest of 128 maxima (each of some groups), cut to 20
// bits by halving the range with counts, is a border that at least `top` logits reach.
// Groups whose maximum reaches it, then their columns whose upper bound does, then of
// those (a few more than `top`) the ones that reach the top-th largest lower bound. Lists are filled in any order: what they hold
// does not depend on it, and the order of the result comes from the exact logits.
// Returns -1 where lists overflow (many equal or nearly equal logits) or the row
// has fewer maxima, or fewer finite ones, than `top`, or no finite largest logit.
template <class Z, int THREADS>
__device__ __forceinline__ int quick_candidates(const ScoreRowsArgs& a, const float2* part, const Z* z, float m, float M,
                                                TopSmem<THREADS>& s, int64_t* id) {
  if (!(fabsf(M) < INFINITY) || a.top > min(a.groups, kMaxima)) return -1;  // uniform
  if (threadIdx.x < kMaxima) s.key[threadIdx.x] = 0u;
  if (threadIdx.x == 0) s.groups = s.found = s.kept = 0;
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < a.groups) atomicMax(&s.key[threadIdx.x % kMaxima], order_key(m));
  __syncthreads();
  if (threadIdx.x < 32) {
    uint32_t own[kMaxima / 32];
#pragma unroll
    for (int i = 0; i < kMaxima / 32; ++i) own[i] = s.key[32 * i + threadIdx.x];
    // to 20 bits of the key, from below
    uint32_t reached = 0;
#pragma unroll 1
    for (uint32_t bit = 1u << 31; bit >= 1u << 12; bit >>= 1) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < kMaxima / 32; ++i) n += __popc(__ballot_sync(0xffffffffu, own[i] >= (reached | bit)));
      if (n >= a.top) reached |= bit;
    }
    if (threadIdx.x == 0) s.border = __uint_as_float((reached & 0x80000000u) ? reached & 0x7FFFFFFFu : ~reached);
  }
  __syncthreads();
  const float key_value = s.border;
  if (!(fabsf(key_value) < INFINITY)) return -1;  // uniform: fewer logits than `top` are finite
  const float border = key_value - fmaxf(fabsf(M), fabsf(key_value)) * 6.1e-5f;
  const float gborder = border - fmaxf(fabsf(M), fabsf(key_value)) * 6.1e-5f;
  if (m >= gborder)
    for (int g = threadIdx.x; g < a.groups; g += 8 * THREADS) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = g + i * THREADS < a.groups ? part[g + i * THREADS].x : -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (v[i] >= gborder && g + i * THREADS < a.groups) {
          const int at = atomicAdd(&s.groups, 1);
          if (at < kMaxGroups) s.group[at] = g + i * THREADS;
        }
    }
  __syncthreads();
  const int ng = s.groups;
  if (ng > kMaxGroups) return -1;
  // eight lanes to a group, eight columns to a lane
  for (int i = threadIdx.x >> 3; i < ng; i += THREADS / 8) {
    const int64_t j = static_cast<int64_t>(s.group[i]) * kScoreGroup + 8 * (threadIdx.x & 7);
    const float gm = part[s.group[i]].x;
    float v[8];
    if constexpr (sizeof(Z) == 2) {
      const uint4 y = *reinterpret_cast<const uint4*>(z + j);
      const uint32_t yv[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&yv[u]));
        v[2 * u] = gm + f.x;
        v[2 * u + 1] = gm + f.y;
      }
    } else {
      const float4 f = *reinterpret_cast<const float4*>(z + j), h = *reinterpret_cast<const float4*>(z + j + 4);
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w, v[4] = h.x, v[5] = h.y, v[6] = h.z, v[7] = h.w;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (j + u >= a.V) continue;
      const float upper = stored_bound<Z>(v[u], gm, M, 1.f);
      if (upper < border) continue;
      const int at = atomicAdd(&s.found, 1);
      if (at < kMaxCandidates) {
        id[at] = j + u;
        s.upper[at] = upper;
        s.lower[at] = stored_bound<Z>(v[u], gm, M, -1.f);
      }
    }
  }
  __syncthreads();
  const int n = s.found;
  if (n > kMaxCandidates) return -1;
  const int i = threadIdx.x;
  float lower = 0.f, upper = 0.f;
  int64_t own_id = 0;
  if (i < n) {
    lower = s.lower[i];
    upper = s.upper[i];
    own_id = id[i];
    int place = 0;
    for (int j = 0; j < n; ++j) place += s.lower[j] > lower || (s.lower[j] == lower && j < i);
    if (place == a.top - 1) s.border = lower;
  }
  __syncthreads();
  if (i < n && upper >= s.border) id[atomicAdd(&s.kept, 1)] = own_id;
  __syncthreads();
  return s.kept;
}

// The careful way: the `top` groups with the largest maxima (ties to the lower
// group: each holds an element that comes before any of another group), in order,
// and of their columns those whose upper bound reaches the top-th largest lower
// bound; where those are more than can be summed again, the largest stored values,
// ties to the lowest id.
template <class Z, int THREADS>
__device__ __noinline__ int careful_candidates(const ScoreRowsArgs& a, const float2* part, const Z* z, float M,
                                               TopSmem<THREADS>& s, int64_t* id) {
  const int kg = min(a.top, a.groups);
  int above;
  const uint32_t gkey = block_select<THREADS>(a.groups, kg, s.sel, above, [&](int64_t g) { return order_key(part[g].x); });
  block_collect<THREADS>(a.groups, kg - above, kg, s.sel,
                         [&](int64_t g) {
                           const uint32_t v = order_key(part[g].x);
                           return v > gkey ? 2 : (v == gkey ? 1 : 0);
                         },
                         [&](int slot, int64_t g) {
                           s.group[slot] = static_cast<int>(g);
                           s.gmax[slot] = part[g].x;
                         });
  __syncthreads();
  const int nv = kg * kScoreGroup;
  auto column = [&](int64_t i) { return static_cast<int64_t>(s.group[i >> 6]) * kScoreGroup + (i & 63); };
  auto value = [&](int64_t i) {  // read again each time: keeping them took room from other rows' blocks
    const int64_t j = column(i);
    if constexpr (sizeof(Z) == 2)
      return s.gmax[i >> 6] + __half2float(z[j]);
    else
      return z[j];
  };
  if (threadIdx.x == 0) s.found = 0;
  __syncthreads();
  auto bound = [&](int64_t i, float sign) { return order_key(stored_bound<Z>(value(i), s.gmax[i >> 6], M, sign)); };
  const uint32_t least =
      block_select<THREADS>(nv, a.top, s.sel, above, [&](int64_t i) { return column(i) < a.V ? bound(i, -1.f) : 0u; });
  auto maybe = [&](int64_t i) { return column(i) < a.V && bound(i, 1.f) >= least ? 2 : 0; };
  auto put = [&](int slot, int64_t i) { id[slot] = column(i); };
  int many = 0;
  for (int i = threadIdx.x; i < nv; i += THREADS) many += maybe(i) != 0;
  if (many) atomicAdd(&s.found, many);
  __syncthreads();
  if (s.found <= kMaxCandidates) return block_collect<THREADS>(nv, 0, kMaxCandidates, s.sel, maybe, put);
  const uint32_t key = block_select<THREADS>(nv, kMaxCandidates, s.sel, above,
                                             [&](int64_t i) { return column(i) < a.V ? order_key(value(i)) : 0u; });
  return block_collect<THREADS>(nv, kMaxCandidates - above, kMaxCandidates, s.sel,
                                [&](int64_t i) {
                                  if (column(i) >= a.V) return 0;
                                  const uint32_t v = order_key(value(i));
                                  return v > key ? 2 : (v == key ? 1 : 0);
                                },
                                put);
}

// log p of an exact logit: M is short of what the product lost. A column that has more
// than half of the row's probability (only one can) is the 1 in L; with its exact logit
// there too, 1 - p keeps its bits where the product's error of M is more than that.
__device__ __forceinline__ float score_log_p(const ScoreRowsArgs& a, Pair z, float M, float L, float log_L) {
  const float above = (z.hi - M) + (z.lo - M * a.loss), d = above * a.inv_temperature;
  if (L < 1.9f && d > -0.05f) return -log1pf(fmaxf(L - 1.f, 0.f) * expf(-d));
  return fmaf(above, a.inv_temperature, -log_L);
}

__device__ __forceinline__ void report(const uint32_t* ctrl, uint32_t* host_error) {
  uint32_t code = ld_volatile_u32(ctrl + kCtrlError);
  if (code == 0) code = ld_volatile_u32(ctrl + kCtrlBadId);
  if (code != 0) *reinterpret_cast<volatile uint32_t*>(host_error) = code;
}

// Without alternatives: a warp per row, its partials read once for the maximum and
// again, from L1 or L2, for the sums.
constexpr int kWarpRows = 4;

template <class E>
__global__ void __launch_bounds__(32 * kWarpRows) score_warp_rows_kernel(const ScoreRowsArgs a) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0) report(a.ctrl, a.host_error);
  if (i >= chunk_rows(a.chunk.live, a.chunk.off, a.chunk.rows)) return;
  const int64_t r = row_of(a.chunk, i);
  const int64_t t = a.t ? a.t[r] : -1;
  if (a.t && t == a.ignore_index) {
    if (lane == 0) {
      a.logprobs[r] = 0.f;
      a.entropy[r] = 0.f;
      a.stats[r] = make_float2(0.f, 0.f);
    }
    return;
  }
  const bool bad = a.t && (t < 0 || t >= a.V);
  const float2* part = a.partials + i * a.groups;
  const float* part_s = a.part_s + i * a.groups;
  const float scale = a.scale;
  float m = -INFINITY;
#pragma unroll 8
  for (int g = lane; g < a.groups; g += 32) m = max_nan(m, part[g].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float M = m;
  float L = 0.f, S = 0.f;
#pragma unroll 8
  for (int g = lane; g < a.groups; g += 32) {
    const float2 p = part[g];
    const float d = p.x - M, w = expf(max_nan(d * scale, -700.f));
    L = fmaf(w, p.y, L);
    S = fmaf(w, fmaf(max_nan(d * a.c, -1000.f), p.y, part_s[g]), S);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    L += __shfl_xor_sync(0xffffffffu, L, o);
    S += __shfl_xor_sync(0xffffffffu, S, o);
  }
  const float log_L = logf(L);
  Pair z = {0.f, 0.f};
  if (a.t && !bad)
    z = warp_dot(static_cast<const E*>(a.x) + r * a.H, static_cast<const E*>(a.W) + t * a.H, a.H, lane);
  if (lane != 0) return;
  if (a.t) a.logprobs[r] = bad ? NAN : score_log_p(a, z, M, L, log_L);
  a.entropy[r] = log_L - kLn2 * S / L;
  a.stats[r] = make_float2(M, log_L);
  if (bad) *reinterpret_cast<volatile uint32_t*>(a.host_error) = kErrBadTarget;
}

// A block per row. Whatever may be among the row's largest logits is summed again
// exactly, with the given token, and ordered by (logit, lowest id).
//
// Bound by latency: the statistics' sums, the search's steps, and the candidates'
// rows of W (top + 1 of them and a few), beside a product that reads V of them.
template <class E, class Z, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) score_rows_kernel(const ScoreRowsArgs a) {
  __shared__ float s_red[THREADS / 32];
  __shared__ int64_t s_id[kMaxCandidates];
  __shared__ Pair s_dot[kMaxCandidates + 1];
  __shared__ uint64_t s_order[kMaxCandidates + 1];
  __shared__ TopSmem<THREADS> s_top;
  const int64_t i = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (i == 0 && threadIdx.x == 0) report(a.ctrl, a.host_error);
  if (i >= chunk_rows(a.chunk.live, a.chunk.off, a.chunk.rows)) return;
  const int64_t r = row_of(a.chunk, i);
  const int64_t t = a.t ? a.t[r] : -1;
  if (a.t && t == a.ignore_index) {
    if (threadIdx.x == 0) {
      a.logprobs[r] = 0.f;
      a.entropy[r] = 0.f;
      a.stats[r] = make_float2(0.f, 0.f);
    }
    if (threadIdx.x < a.top) {
      a.top_logprobs[r * a.top + threadIdx.x] = 0.f;
      a.top_ids[r * a.top + threadIdx.x] = -1;
    }
    return;
  }
  const bool bad = a.t && (t < 0 || t >= a.V);
  const float2* part = a.partials + i * a.groups;
  const float* part_s = a.part_s + i * a.groups;
  float m = -INFINITY;
#pragma unroll 8
  for (int g = threadIdx.x; g < a.groups; g += THREADS) m = max_nan(m, part[g].x);
  const float M = block_max<THREADS>(m, s_red);
  const float scale = a.scale;
  float L = 0.f, S = 0.f;
#pragma unroll 4
  for (int g = threadIdx.x; g < a.groups; g += THREADS) {
    const float2 p = part[g];
    const float d = p.x - M, w = expf(max_nan(d * scale, -700.f));
    L = fmaf(w, p.y, L);
    S = fmaf(w, fmaf(max_nan(d * a.c, -1000.f), p.y, part_s[g]), S);
  }
  L = block_sum<THREADS>(L, s_red);
  S = block_sum<THREADS>(S, s_red);
  const float log_L = logf(L);
  const E* x = static_cast<const E*>(a.x) + r * a.H;
  const E* W = static_cast<const E*>(a.W);

  const Z* z = static_cast<const Z*>(a.z) + i * a.ldv;
  int n = quick_candidates<Z, THREADS>(a, part, z, m, M, s_top, s_id);
  if (n < 0) {
    __syncthreads();
    n = careful_candidates<Z, THREADS>(a, part, z, M, s_top, s_id);
  }
  __syncthreads();
  // the given token's logit behind the candidates'
  const int dots = n + (a.t && !bad ? 1 : 0);
  // two at a time, which share x and hide each other's latency
  for (int d = warp; d < dots; d += 2 * (THREADS / 32)) {
    const int e = d + THREADS / 32;
    const E* w0 = W + (d < n ? s_id[d] : t) * a.H;
    Pair v[2];
    if (e < dots)
      warp_dot2(x, w0, W + (e < n ? s_id[e] : t) * a.H, a.H, lane, v);
    else
      v[0] = warp_dot(x, w0, a.H, lane);
    if (lane == 0) {
      s_dot[d] = v[0];
      s_order[d] = order_key(v[0]);
      if (e < dots) {
        s_dot[e] = v[1];
        s_order[e] = order_key(v[1]);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < n) {
    const uint64_t own = s_order[threadIdx.x];
    const int64_t id = s_id[threadIdx.x];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) rank += s_order[j] > own || (s_order[j] == own && s_id[j] < id);
    if (rank < a.top) {
      a.top_logprobs[r * a.top + rank] = score_log_p(a, s_dot[threadIdx.x], M, L, log_L);
      a.top_ids[r * a.top + rank] = id;
    }
  }
  if (threadIdx.x == 0) {
    if (a.t) a.logprobs[r] = bad ? NAN : score_log_p(a, s_dot[n], M, L, log_L);
    a.entropy[r] = log_L - kLn2 * S / L;
    a.stats[r] = make_float2(M, log_L);
    if (bad) *reinterpret_cast<volatile uint32_t*>(a.host_error) = kErrBadTarget;
  }
}

// ------------------------------------------------------------ gradients

// Copies 16-byte pieces, or 4-byte ones where rows are not made of those (fp32 x may
// start at any element)
__device__ __forceinline__ void copy_row(const uint8_t* from, uint8_t* to, int64_t bytes) {
  if ((reinterpret_cast<uint64_t>(from) | reinterpret_cast<uint64_t>(to) | static_cast<uint64_t>(bytes)) % 16 == 0) {
    for (int64_t i = threadIdx.x * 16; i < bytes; i += blockDim.x * 16)
      *reinterpret_cast<uint4*>(to + i) = *reinterpret_cast<const uint4*>(from + i);
  } else {
    for (int64_t i = threadIdx.x * 4; i < bytes; i += blockDim.x * 4)
      *reinterpret_cast<uint32_t*>(to + i) = *reinterpret_cast<const uint32_t*>(from + i);
  }
}

// d_j = (1 / temperature) (g [j = t] - p_j (g + h (log p_j + H))), as a + b log2 p, and
// whole at the target.
// Rows that do not count get zeros, and a zero row of x, so that nothing that
// stands there (it may be NaN) reaches dW.
__global__ void __launch_bounds__(128) score_prepare_kernel(const ScorePrepareArgs a) {
  const int64_t i = blockIdx.x;
  const int rows = chunk_rows(a.chunk.live, a.chunk.off, a.chunk.rows);
  if (i >= rows && (!a.tail || i >= tail_end(a.chunk, rows))) return;
  const int64_t r = i < rows ? row_of(a.chunk, i) : 0;
  bool live = i < rows && (!a.alive || a.alive[r] != 0);
  if (a.t) {
    const int64_t t = live ? a.t[r] : 0;
    const bool ignored = live && t == a.ignore_index, bad = live && !ignored && (t < 0 || t >= a.V);
    live = live && !ignored && !bad;
    if (threadIdx.x == 0) {
      if (bad) a.ctrl[kCtrlBadId] = kErrBadTarget;
      ScoreRow q{0.f, 0.f, 0.f, 0.f, 0.f, -1, 0.f};
      if (live) {
        const float2 st = a.stats[r];
        const float inv = a.inv_temperature;
        const float g = a.d_logprobs ? a.d_logprobs[r] : 0.f;
        const float h = a.d_entropy ? a.d_entropy[r] : 0.f;
        q.largest = st.x * a.largest_scale;
        q.log2_total = st.y * kLog2e;
        q.inv_total = expf(-st.y);
        q.a = -inv * (a.d_entropy ? fmaf(h, a.entropy[r], g) : g);
        q.b = -inv * h * kLn2;
        q.target = static_cast<int32_t>(t);
        // the target's entry, from its exact logit: g (1 - p) without cancellation
        const float lp = max_nan(a.logprobs[r], -1000.f);  // of probability 0 either way
        q.at = -inv * (g * expm1f(lp) + (a.d_entropy ? h * expf(lp) * (lp + a.entropy[r]) : 0.f));
        // what the exponentials' lower limit would hide
        if (!(fabsf(q.log2_total) < INFINITY) || !(fabsf(q.largest) < INFINITY)) q.a = q.at = NAN;
      }
      a.row[i] = q;
      // what bf16 leaves of it goes to dx
      a.dcorr[i] = q.at - __bfloat162float(__float2bfloat16_rn(q.at));
    }
  }
  uint8_t* to = static_cast<uint8_t*>(a.xm) + i * a.row_bytes;
  if (live)
    copy_row(static_cast<const uint8_t*>(a.x) + r * a.row_bytes, to, a.row_bytes);
  else
    zero_row(to, a.row_bytes, threadIdx.x, blockDim.x);
}

// Eight columns of a row's gradient from the stored logits. The padding behind the
// last column (ldv is a multiple of 64) becomes zero.
__device__ __forceinline__ void dlogits8(uint4 in, __nv_bfloat16* d, int64_t j, int64_t V, float gmax, float c,
                                         const ScoreRow& q) {
  const uint32_t iv[4] = {in.x, in.y, in.z, in.w};
  const float shift = fmaf(gmax - q.largest, c, -q.log2_total);
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&iv[i]));
    const float t0 = max_nan(fmaf(y.x, c, shift), -1000.f), t1 = max_nan(fmaf(y.y, c, shift), -1000.f);
    v[2 * i] = ex2(t0) * fmaf(q.b, t0, q.a);
    v[2 * i + 1] = ex2(t1) * fmaf(q.b, t1, q.a);
  }
  if (j + 8 > V) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j + i >= V) v[i] = 0.f;
  }
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 o = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&o);
  }
  *reinterpret_cast<uint4*>(d + j) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The same of several pieces, `step` columns apart: their loads are all under way
// before the first is used (HBM wants some 64 bytes in flight a thread).
constexpr int kPieces = 4;

__device__ __forceinline__ void dlogits_pieces(const __half* z, __nv_bfloat16* d, int64_t j, int64_t step, int64_t ldv,
                                               int64_t V, const float2* part, float c, const ScoreRow& q) {
  uint4 in[kPieces];
  float gmax[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    if (j + i * step < ldv) {
      in[i] = __ldcs(reinterpret_cast<const uint4*>(z + j + i * step));
      gmax[i] = part[(j + i * step) / kScoreGroup].x;
    }
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    if (j + i * step < ldv) dlogits8(in[i], d, j + i * step, V, gmax[i], c, q);
}

__device__ __forceinline__ void dlogits4(const float* z, float* d, int64_t j, int64_t V, float c, float inv_t,
                                         const ScoreRow& q) {
  const float4 in = *reinterpret_cast<const float4*>(z + j);
  float v[4] = {in.x, in.y, in.z, in.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = j + i < V ? dlogit_f32(v[i], j + i, c, inv_t, q) : 0.f;
  *reinterpret_cast<float4*>(d + j) = make_float4(v[0], v[1], v[2], v[3]);
}

// Reads 2 and writes 2 bytes a logit (fp32: 4 and 4): HBM bounds it.
constexpr int kDlogitsThreads = 256;

__global__ void __launch_bounds__(kDlogitsThreads) score_dlogits_bf16_kernel(
    const ScoreChunk chunk, const __half* z, const float2* __restrict__ partials, int groups, __nv_bfloat16* d, int64_t ldv, int64_t V, float c,
    const ScoreRow* __restrict__ row) {
  const int64_t r = blockIdx.x;
  if (r >= tail_end(chunk, chunk_rows(chunk.live, chunk.off, chunk.rows))) return;
  const ScoreRow q = row[r];
  const int64_t j = (static_cast<int64_t>(blockIdx.y) * kPieces * kDlogitsThreads + threadIdx.x) * 8;
  if (q.a == 0.f && q.b == 0.f) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (j + i * kDlogitsThreads * 8 < ldv)
        *reinterpret_cast<uint4*>(d + r * ldv + j + i * kDlogitsThreads * 8) = make_uint4(0, 0, 0, 0);
    return;
  }
  dlogits_pieces(z + r * ldv, d + r * ldv, j, kDlogitsThreads * 8, ldv, V, partials + r * groups, c, q);
}

__global__ void __launch_bounds__(kDlogitsThreads) score_dlogits_f32_kernel(const ScoreChunk chunk, const float* z, float* d, int64_t ldv, int64_t V,
                                                                           float c, float inv_t, const ScoreRow* __restrict__ row) {
  const int64_t r = blockIdx.x;
  if (r >= tail_end(chunk, chunk_rows(chunk.live, chunk.off, chunk.rows))) return;
  const ScoreRow q = row[r];
  const int64_t j = (static_cast<int64_t>(blockIdx.y) * kDlogitsThreads + threadIdx.x) * 4;
  if (j >= ldv) return;
  if (q.a == 0.f && q.b == 0.f) {
    *reinterpret_cast<float4*>(d + r * ldv + j) = make_float4(0.f, 0.f, 0.f, 0.f);
    return;
  }
  dlogits4(z + r * ldv, d + r * ldv, j, V, c, inv_t, q);
}

// The targets' entries, a thread a row
__global__ void __launch_bounds__(256) score_target_kernel(const ScoreChunk chunk, __nv_bfloat16* d, int64_t ldv,
                                                           const ScoreRow* __restrict__ row) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= chunk_rows(chunk.live, chunk.off, chunk.rows)) return;
  const ScoreRow q = row[i];
  if (q.target >= 0) d[i * ldv + q.target] = __float2bfloat16_rn(q.at);
}

// dx: the sum of the splits in their order, with the target's entry put right,
// rounded once. H % 8 == 0.
__global__ void __launch_bounds__(128) score_dx_kernel(const ScoreChunk chunk, const float* __restrict__ part, int splits, int64_t split_stride,
                                                       int64_t H, const __nv_bfloat16* __restrict__ W,
                                                       const ScoreRow* __restrict__ row, const float* __restrict__ dcorr,
                                                       __nv_bfloat16* __restrict__ dx, const uint32_t* ctrl,
                                                       uint32_t* host_error) {
  const int64_t r = blockIdx.x;
  if (host_error && r == 0 && blockIdx.y == 0 && threadIdx.x == 0) report(ctrl, host_error);
  const int64_t h = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * 4;
  if (h >= H || r >= chunk_rows(chunk.live, chunk.off, chunk.rows)) return;
  const int64_t i = r * H + h;
  float4 acc = *reinterpret_cast<const float4*>(part + i);
  for (int s = 1; s < splits; ++s) {
    const float4 v = *reinterpret_cast<const float4*>(part + s * split_stride + i);
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
  }
  const int32_t t = row ? row[r].target : -1;
  if (t >= 0) {
    const float c = dcorr[r];
    const uint2 wv = *reinterpret_cast<const uint2*>(W + t * H + h);
    acc.x = fmaf(__uint_as_float(wv.x << 16), c, acc.x);
    acc.y = fmaf(__uint_as_float(wv.x & 0xFFFF0000u), c, acc.y);
    acc.z = fmaf(__uint_as_float(wv.y << 16), c, acc.z);
    acc.w = fmaf(__uint_as_float(wv.y & 0xFFFF0000u), c, acc.w);
  }
  __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y), hi = __floats2bfloat162_rn(acc.z, acc.w);
  *reinterpret_cast<uint2*>(dx + row_of(chunk, r) * H + h) = make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
}

__global__ void score_report_kernel(const uint32_t* ctrl, uint32_t* host_error) { report(ctrl, host_error); }

// --------------------------------------------------------- distillation

__device__ __forceinline__ float teacher_logit(const void* p, int64_t i, int dtype) {
  if (dtype == FLCE_DTYPE_FP32) return static_cast<const float*>(p)[i];
  if (dtype == FLCE_DTYPE_FP16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// An entry counts if its id is not -1 and its logit is above -inf (a NaN does).
__device__ __forceinline__ bool teacher_there(int64_t id, float logit) { return id != -1 && !(logit == -INFINITY); }

// A warp per row
__global__ void __launch_bounds__(256) distill_live_kernel(const int64_t* __restrict__ ids, int64_t ld_ids,
                                                           const void* __restrict__ logits, int64_t ld_logits, int dtype,
                                                           int64_t N, int k, int64_t V, uint8_t* __restrict__ live,
                                                           float* __restrict__ token_loss, uint32_t* ctrl, bool count) {
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  bool any = false, bad = false;
  if (r < N)
    for (int e = lane; e < k; e += 32) {
      const int64_t id = ids[r * ld_ids + e];
      if (!teacher_there(id, teacher_logit(logits, r * ld_logits + e, dtype))) continue;
      any = true;
      bad = bad || id < 0 || id >= V;
    }
  any = __any_sync(0xffffffffu, any);
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0 && r < N) {
    live[r] = any && !bad;
    if (!any || bad) token_loss[r] = 0.f;
    if (bad) ctrl[kCtrlBadId] = kErrBadTarget;
    if (count && any && !bad) atomicAdd(ctrl + kCtrlNValid, 1u);
  }
}

// A block per row. The entries that count are put in order of their ids (those that
// share one, of their slots) by counting the ones before each.
constexpr int kPickThreads = 128;

__global__ void __launch_bounds__(kPickThreads) distill_pick_kernel(const DistillPickArgs a) {
  __shared__ int s_id[kScoreMaxTeacher], s_sorted[kScoreMaxTeacher];
  const int64_t r = blockIdx.x;
  if (r >= chunk_rows(a.chunk.live, a.chunk.off, a.chunk.rows)) return;
  const int64_t from_row = row_of(a.chunk, r);
  uint2* parts = a.parts + r * a.num_tiles;
  constexpr int kNone = 0x7FFFFFFF;
  for (int e = threadIdx.x; e < a.k; e += kPickThreads) {
    const int64_t id = a.ids[from_row * a.ld_ids + e];
    s_id[e] = teacher_there(id, teacher_logit(a.logits, from_row * a.ld_logits + e, a.dtype)) ? static_cast<int>(id) : kNone;
    s_sorted[e] = kNone;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.k; e += kPickThreads) {
    const int id = s_id[e];
    if (id == kNone) continue;
    int place = 0;
    for (int i = 0; i < a.k; ++i) place += s_id[i] < id || (s_id[i] == id && i < e);
    s_sorted[place] = id;
    a.entries[r * a.k + place] = make_int2(id, e);
  }
  __syncthreads();
  for (int w = threadIdx.x; w < a.num_tiles; w += kPickThreads) {
    uint64_t at = 0;
    int lo = 0;
#pragma unroll 1
    for (int j = 0; j <= 4; ++j) {
      // the first entry that is not before the part
      const int64_t from = static_cast<int64_t>(w) * kScoreTileColumns + j * kScorePart;
      int hi = a.k;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (s_sorted[mid] < from)
          lo = mid + 1;
        else
          hi = mid;
      }
      at |= static_cast<uint64_t>(lo) << (9 * j);
    }
    parts[w] = make_uint2(static_cast<uint32_t>(at), static_cast<uint32_t>(at >> 32));
  }
}

constexpr int kDistillThreads = 256;

// A block per row: the row's log-sum-exp from its groups, the entries' logits, the
// loss T^2 sum_e q_e (log q_e - log p_e), and with the gradient the row of stored
// logits overwritten by d = (T / n) (p - q), first everywhere, then at the entries
// (from their unrounded logits; entries that share an id add up). The entries'
// logits are the product's fp32 sums, which its epilogue picked: summing them again
// took a row of W each, 1.2 ms of a 4096-token chunk at 64 entries instead of 0.4.
// Bound by the stored logits' way through HBM (2 bytes read, 2 written a logit).
template <class E, bool GRADIENT>
__global__ void __launch_bounds__(kDistillThreads) distill_rows_kernel(const DistillArgs a) {
  __shared__ float s_red[kDistillThreads / 32];
  __shared__ int64_t s_id[kScoreMaxTeacher];
  __shared__ float s_q[kScoreMaxTeacher];
  const int64_t i = blockIdx.x;
  constexpr bool bf16 = sizeof(E) == 2;
  uint8_t* zrow = static_cast<uint8_t*>(a.z) + i * a.ldv * sizeof(E);
  const int rows = chunk_rows(a.chunk.live, a.chunk.off, a.chunk.rows);
  if (i >= rows) {
    if (GRADIENT && i < tail_end(a.chunk, rows)) zero_row(zrow, a.ldv * sizeof(E), threadIdx.x, kDistillThreads);
    return;
  }
  const int64_t r = row_of(a.chunk, i);
  if (a.alive && !a.alive[r]) {
    if (GRADIENT) zero_row(zrow, a.ldv * sizeof(E), threadIdx.x, kDistillThreads);
    return;
  }
  // entries that do not count have id -1 from here on
  float top = -INFINITY;
  for (int e = threadIdx.x; e < a.k; e += kDistillThreads) {
    const int64_t id = a.ids[r * a.ld_ids + e];
    const float v = teacher_logit(a.logits, r * a.ld_logits + e, a.dtype);
    const bool there = teacher_there(id, v);
    s_id[e] = there ? id : -1;
    s_q[e] = v;
    if (there) top = max_nan(top, v);
  }
  top = block_max<kDistillThreads>(top, s_red);
  const float2* part = a.partials + i * a.groups;
  float m = -INFINITY;
  for (int g = threadIdx.x; g < a.groups; g += kDistillThreads) m = max_nan(m, part[g].x);
  const float M = block_max<kDistillThreads>(m, s_red);
  const float scale = a.scale;
  float L = 0.f;
  for (int g = threadIdx.x; g < a.groups; g += kDistillThreads) {
    const float2 p = part[g];
    L = fmaf(expf(max_nan((p.x - M) * scale, -700.f)), p.y, L);
  }
  L = block_sum<kDistillThreads>(L, s_red);
  const float log_L = logf(L);
  const float inv = a.inv_temperature;
  float q = 0.f;
  const int e = threadIdx.x;  // k <= kScoreMaxTeacher <= kDistillThreads
  const bool there = e < a.k && s_id[e] >= 0;
  const float rel = there ? (s_q[e] - top) * inv : 0.f;
  if (there) q = expf(rel);
  const float total = block_sum<kDistillThreads>(q, s_red);
  q /= total;
  float log_p = 0.f, term = 0.f;
  if (there) {
    const float z = bf16 ? a.picked[i * a.k + e] : reinterpret_cast<const float*>(zrow)[s_id[e]];
    log_p = fmaf(z - M, scale, -log_L);
    term = q > 0.f || q != q ? q * (rel - logf(total) - log_p) : 0.f;
    s_q[e] = q;
  }
  term = block_sum<kDistillThreads>(term, s_red);
  if (threadIdx.x == 0) a.token_loss[r] = a.temperature * (a.temperature * term);
  if constexpr (GRADIENT) {
    const float factor = a.temperature / static_cast<float>(a.ctrl[kCtrlNValid]);
    ScoreRow row{M, log_L * kLog2e, factor, 0.f, 0.f, -1, expf(-log_L)};
    if (!(fabsf(row.log2_total) < INFINITY) || !(fabsf(M) < INFINITY)) row.a = NAN;
    if constexpr (bf16) {
      for (int64_t j = threadIdx.x * 8; j < a.ldv; j += kPieces * kDistillThreads * 8)
        dlogits_pieces(reinterpret_cast<const __half*>(zrow), reinterpret_cast<__nv_bfloat16*>(zrow), j, kDistillThreads * 8,
                       a.ldv, a.V, part, a.c, row);
    } else {
      for (int64_t j = threadIdx.x * 4; j < a.ldv; j += kDistillThreads * 4)
        dlogits4(reinterpret_cast<const float*>(zrow), reinterpret_cast<float*>(zrow), j, a.V, a.c, inv, row);
    }
    __syncthreads();
    if (there) {
      float all = 0.f;
      for (int j = 0; j < a.k; ++j)
        if (s_id[j] == s_id[e]) all += s_q[j];
      const float d = factor * (expf(log_p) - all);
      if constexpr (bf16)
        reinterpret_cast<__nv_bfloat16*>(zrow)[s_id[e]] = __float2bfloat16_rn(d);
      else
        reinterpret_cast<float*>(zrow)[s_id[e]] = d;
    }
  }
}

__global__ void __launch_bounds__(1024) distill_finish_kernel(const float* __restrict__ token_loss, int64_t N,
                                                              const uint32_t* ctrl, float* loss, uint32_t* host_error) {
  __shared__ Pair s_sum[32];
  Pair v = {0.f, 0.f};
  for (int64_t i = threadIdx.x; i < N; i += 1024) v = add(v, {token_loss[i], 0.f});
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = warp_sum(s_sum[threadIdx.x]);
    if (threadIdx.x == 0) {
      const uint32_t n = ctrl[kCtrlNValid], code = ctrl[kCtrlError] | ctrl[kCtrlBadId];
      *loss = code != 0 ? NAN : (n > 0 ? v.hi / static_cast<float>(n) : 0.f);
      report(ctrl, host_error);
    }
  }
}

// With few rows a row's latency counts, and large blocks take its candidates at
// once; with many, eight blocks of 128 threads share an SM. Scoring with 20 alternatives
// at 4096 x 128256, 1024 / 128 threads: 212 / 247 us for 48 rows, 358 / 372 for 304, 568 /
// 530 for 700 (1024 x 32000: 42 / 46, 78 / 69, 138 / 89).
constexpr int kFewRows = 304;

unsigned blocks_of(int64_t n, int64_t per) { return static_cast<unsigned>((n + per - 1) / per); }

template <class E, class Z>
cudaError_t launch_rows(const ScoreRowsArgs& a, cudaStream_t s) {
  if (a.top == 0)
    score_warp_rows_kernel<E><<<blocks_of(a.chunk.rows, kWarpRows), 32 * kWarpRows, 0, s>>>(a);
  else if (a.chunk.rows <= kFewRows)
    score_rows_kernel<E, Z, 1024><<<a.chunk.rows, 1024, 0, s>>>(a);
  else
    score_rows_kernel<E, Z, 128><<<a.chunk.rows, 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_score_order(const ScoreOrderArgs& a, cudaStream_t s) {
  const bool skip = a.dx || a.logprobs || a.entropy;
  score_order_kernel<<<1 + (skip ? blocks_of(a.N, 32) : 0), 1024, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_score_rows(const ScoreRowsArgs& a, cudaStream_t s) {
  return a.bf16 ? launch_rows<__nv_bfloat16, __half>(a, s) : launch_rows<float, float>(a, s);
}

cudaError_t launch_score_prepare(const ScorePrepareArgs& a, cudaStream_t s) {
  score_prepare_kernel<<<a.chunk.rows, 128, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_score_dlogits(int bf16, const ScoreChunk& chunk, const void* z, const float2* partials, int groups, void* d,
                                 int64_t ldv, int64_t V, float c, float inv_temperature, const ScoreRow* row,
                                 cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(chunk.rows), blocks_of(ldv, kDlogitsThreads * (bf16 ? 8 * kPieces : 4)));
  if (bf16)
    score_dlogits_bf16_kernel<<<grid, kDlogitsThreads, 0, s>>>(chunk, static_cast<const __half*>(z), partials, groups,
                                                              static_cast<__nv_bfloat16*>(d), ldv, V, c, row);
  else
    score_dlogits_f32_kernel<<<grid, kDlogitsThreads, 0, s>>>(chunk, static_cast<const float*>(z), static_cast<float*>(d), ldv,
                                                             V, c, inv_temperature, row);
  return cudaGetLastError();
}

cudaError_t launch_score_target(const ScoreChunk& chunk, void* d, int64_t ldv, const ScoreRow* row, cudaStream_t s) {
  score_target_kernel<<<blocks_of(chunk.rows, 256), 256, 0, s>>>(chunk, static_cast<__nv_bfloat16*>(d), ldv, row);
  return cudaGetLastError();
}

cudaError_t launch_score_dx(const ScoreChunk& chunk, const float* part, int splits, int64_t split_stride, int64_t H,
                            const void* W, const ScoreRow* row, const float* dcorr, void* dx, const uint32_t* ctrl,
                            uint32_t* host_error, cudaStream_t s) {
  score_dx_kernel<<<dim3(static_cast<unsigned>(chunk.rows), blocks_of(H, 512)), 128, 0, s>>>(
      chunk, part, splits, split_stride, H, static_cast<const __nv_bfloat16*>(W), row, dcorr, static_cast<__nv_bfloat16*>(dx), ctrl,
      host_error);
  return cudaGetLastError();
}

cudaError_t launch_score_report(const uint32_t* ctrl, uint32_t* host_error, cudaStream_t s) {
  score_report_kernel<<<1, 1, 0, s>>>(ctrl, host_error);
  return cudaGetLastError();
}

cudaError_t launch_distill_rows(const DistillArgs& a, cudaStream_t s) {
  const int rows = a.chunk.rows;
  if (a.bf16) {
    if (a.gradient)
      distill_rows_kernel<__nv_bfloat16, true><<<rows, kDistillThreads, 0, s>>>(a);
    else
      distill_rows_kernel<__nv_bfloat16, false><<<rows, kDistillThreads, 0, s>>>(a);
  } else {
    if (a.gradient)
      distill_rows_kernel<float, true><<<rows, kDistillThreads, 0, s>>>(a);
    else
      distill_rows_kernel<float, false><<<rows, kDistillThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_distill_live(const int64_t* ids, int64_t ld_ids, const void* logits, int64_t ld_logits, int dtype,
                                int64_t N, int k, int64_t V, uint8_t* live, float* token_loss, uint32_t* ctrl,
                                bool count, cudaStream_t s) {
  distill_live_kernel<<<blocks_of(N, 8), 256, 0, s>>>(ids, ld_ids, logits, ld_logits, dtype, N, k, V, live, token_loss, ctrl,
                                                      count);
  return cudaGetLastError();
}

cudaError_t launch_distill_pick(const DistillPickArgs& a, cudaStream_t s) {
  distill_pick_kernel<<<a.chunk.rows, kPickThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_distill_finish(const float* token_loss, int64_t N, const uint32_t* ctrl, float* loss, uint32_t* host_error,
                                  cudaStream_t s) {
  distill_finish_kernel<<<1, 1024, 0, s>>>(token_loss, N, ctrl, loss, host_error);
  return cudaGetLastError();
}

}  // namespace flce
