// Host side of the training-step operators' entry points: argument checks,
// workspace layout, TMA descriptors, launches.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "flce_handle.h"
#include "flce_train.h"

using namespace flce;

namespace {

uint64_t addr(const void* p) { return reinterpret_cast<uint64_t>(p); }

uint64_t element_bytes(int dtype) { return dtype == FLCE_DTYPE_FP32 ? 4 : 2; }

// ------------------------------------------------------------------ routing

struct RouteLayout {
  uint64_t unit_p = 0, unit_c = 0, unit_live = 0, unit_z = 0, terms = 0, doc_live = 0, doc_z = 0, ticket = 0,
           total = 0;
};

RouteLayout route_layout(const RouteGeometry& g, int64_t E, int64_t documents) {
  RouteLayout l;
  const uint64_t units = static_cast<uint64_t>(g.blocks) + documents;
  uint64_t off = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  l.unit_p = take(units * E * 4);
  l.unit_c = take(units * E * 4);
  l.unit_live = take(units * 4);
  l.unit_z = take(units * 4);
  l.terms = take(static_cast<uint64_t>(documents) * g.chunks * 4);
  l.doc_live = take(static_cast<uint64_t>(documents) * 4);
  l.doc_z = take(static_cast<uint64_t>(documents) * 4);
  l.ticket = take(4);
  l.total = off;
  return l;
}

// Sizes, pointers and alignment shared by the forward and the backward.
flce_status route_check(flce_handle_t h, const flce_route_args* r) {
  if (!r) return fail(h, FLCE_ERR_INVALID_ARG, "null pointer argument");
  if (r->dtype != FLCE_DTYPE_BF16 && r->dtype != FLCE_DTYPE_FP32 && r->dtype != FLCE_DTYPE_FP16)
    return fail(h, FLCE_ERR_UNSUPPORTED, "logits must be bf16, fp32 or fp16");
  if (r->N < 0 || r->N > kMaxDim || r->E < 1 || r->E > kRouteMaxExperts)
    return fail(h, FLCE_ERR_INVALID_ARG, "need 0 <= N < 2^31 and 1 <= E <= %d", kRouteMaxExperts);
  if (r->k < 1 || r->k > std::min<int64_t>(r->E, kRouteMaxK))
    return fail(h, FLCE_ERR_INVALID_ARG, "need 1 <= k <= min(E, %d)", kRouteMaxK);
  if (r->ld < r->E) return fail(h, FLCE_ERR_INVALID_ARG, "the row stride is below E");
  if (r->documents < 1 || r->documents > (1 << 24) || (r->documents > 1 && !r->offsets))
    return fail(h, FLCE_ERR_INVALID_ARG, "need 1 <= documents <= 2^24, and offsets for more than one");
  if ((r->N > 0 && (!r->logits || !r->weights || !r->experts || !r->stats)) || !r->counts || !r->slope || !r->result)
    return fail(h, FLCE_ERR_INVALID_ARG, "null pointer argument");
  if (addr(r->logits) % element_bytes(r->dtype) ||
      (addr(r->weights) | addr(r->experts) | addr(r->slope) | addr(r->result)) % 4 ||
      (addr(r->counts) | addr(r->offsets) | addr(r->stats)) % 8)
    return fail(h, FLCE_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  return FLCE_OK;
}

RouteArgs route_args(const flce_route_args* r, const RouteGeometry& g) {
  RouteArgs a{};
  a.logits = r->logits;
  a.N = r->N;
  a.ld = r->ld;
  a.E = static_cast<int32_t>(r->E);
  a.k = r->k;
  a.renormalize = r->renormalize != 0;
  a.documents = static_cast<int32_t>(r->documents);
  a.valid = r->valid;
  a.offsets = r->offsets;
  a.weights = r->weights;
  a.experts = r->experts;
  a.counts = r->counts;
  a.stats = reinterpret_cast<float2*>(r->stats);
  a.slope = r->slope;
  a.result = r->result;
  a.rows_per_block = g.rows_per_block;
  a.blocks = g.blocks;
  a.one_launch = g.one_launch;
  return a;
}

// --------------------------------------------------------------------- muon

constexpr int64_t kMuonMaxDim = 65536;
// matrices per group of launches: as many as fit this much workspace (one at
// least); a larger group only saves launches once the GPU is full
constexpr uint64_t kMuonGroupBytes = 2ull << 30;
constexpr uint64_t kMuonSumsBytes = 40ull << 20;

struct MuonLayout {
  uint64_t ctrl = 0, done = 0, sums = 0, sums_bytes = 0, norm = 0, diag = 0, hi[2] = {0, 0}, lo = 0, gram = 0, poly = 0, gram_lo = 0,
           poly_lo = 0, total = 0;
};

struct MuonSizes {
  int64_t m, n, ldx, lda;
};

MuonSizes muon_sizes(int64_t rows, int64_t cols) {
  MuonSizes z;
  z.m = std::min(rows, cols);
  z.n = std::max(rows, cols);
  z.ldx = static_cast<int64_t>(align_up(z.n, 64));
  z.lda = static_cast<int64_t>(align_up(z.m, 64));
  return z;
}

MuonLayout muon_layout(int64_t rows, int64_t cols, int64_t count) {
  const MuonSizes z = muon_sizes(rows, cols);
  MuonLayout l;
  uint64_t off = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t at = off;
    off = align_up(off + bytes, kAlign);
    return at;
  };
  l.ctrl = take(kCtrlWords * 4);
  l.done = take(2 * kMuonMaxMats * 4);
  l.norm = take(static_cast<uint64_t>(count) * kMuonNormBlocks * 8);
  l.diag = take(static_cast<uint64_t>(count) * z.m * 4);
  const uint64_t x = static_cast<uint64_t>(count) * z.m * z.ldx * 2;
  const uint64_t g = static_cast<uint64_t>(count) * z.m * z.lda * 2;
  l.hi[0] = take(x);
  l.hi[1] = take(x);
  l.lo = take(x);
  l.gram = take(g);
  l.poly = take(g);
  if (z.m <= kMuonPairSide) {
    l.gram_lo = take(g);
    l.poly_lo = take(g);
  }
  // Splits of X Xt: their tiles' fp32 sums, at most a tile for every slot of
  // the GPU (bounded here without knowing it)
  const int64_t blocks = cdiv(z.n, 64);
  const int64_t splits = std::min<int64_t>(kMuonMaxSplits, blocks / kMuonMinSplitBlocks);
  if (splits > 1) {
    const uint64_t area = align_up(z.m, 256) * align_up(z.m, 512);
    l.sums_bytes = std::min<uint64_t>(4 * area * count * (splits - 1), kMuonSumsBytes);
  }
  // or, in the one-launch kernel, a cluster's partial products of X Xt and A (16
  // CTAs at most: the device is not known here)
  if (muon_small_cluster(z.m, z.n) > 1)
    l.sums_bytes = std::max<uint64_t>(l.sums_bytes, static_cast<uint64_t>(count) * (16 * 65536 + 32768));
  l.sums = take(l.sums_bytes);
  l.total = off;
  return l;
}

int64_t muon_group(int64_t rows, int64_t cols, int64_t count) {
  const uint64_t one = muon_layout(rows, cols, 1).total;
  const int64_t fit = std::max<int64_t>(1, static_cast<int64_t>(kMuonGroupBytes / one));
  return std::min<int64_t>({count, fit, static_cast<int64_t>(kMuonMaxMats)});
}

bool muon_size_ok(int64_t rows, int64_t cols, int64_t count) {
  return rows >= 1 && cols >= 1 && rows <= kMuonMaxDim && cols <= kMuonMaxDim && count >= 0 && count <= (1 << 20);
}

// The largest |b t + c t^2| over t in [0, r^2] and |a x + b x^3 + c x^5| over
// x in [0, r]: extrema at the ends and where the derivative vanishes.
void muon_map_bounds(double a, double b, double c, double r, double* poly, double* next) {
  auto p2 = [&](double t) { return std::fabs(b * t + c * t * t); };
  auto p5 = [&](double x) { return std::fabs(x * (a + x * x * (b + x * x * c))); };
  *poly = p2(r * r);
  if (c != 0.0) {
    const double t = -b / (2.0 * c);
    if (t > 0.0 && t < r * r) *poly = std::max(*poly, p2(t));
  }
  *next = p5(r);
  // a + 3 b t + 5 c t^2 = 0 with t = x^2
  auto visit = [&](double t) {
    if (t > 0.0 && t < r * r) *next = std::max(*next, p5(std::sqrt(t)));
  };
  if (c != 0.0) {
    const double disc = 9.0 * b * b - 20.0 * a * c;
    if (disc >= 0.0) {
      visit((-3.0 * b + std::sqrt(disc)) / (10.0 * c));
      visit((-3.0 * b - std::sqrt(disc)) / (10.0 * c));
    }
  } else if (b != 0.0) {
    visit(-a / (3.0 * b));
  }
}

bool map_half_3d(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t mats, uint64_t ld,
                 uint32_t box_cols, uint32_t box_rows, std::string* why, CUtensorMapSwizzle swizzle) {
  const uint64_t dims[3] = {cols, rows, mats};
  const uint64_t strides[2] = {ld * 2, ld * 2 * rows};
  const uint32_t box[3] = {box_cols, box_rows, 1};
  return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, base, 3, dims, strides, box, why, swizzle);
}

// One group of matrices: momentum, X, the Newton-Schulz steps, the result.
flce_status muon_group_run(flce_handle_t h, const flce_muon_args* q, const flce_muon_matrix* mats, int count,
                           const float* coefficients, uint8_t* ws, uint32_t hold, uint64_t timeout_ns, cudaStream_t s) {
  const MuonSizes z = muon_sizes(q->rows, q->cols);
  const MuonLayout L = muon_layout(q->rows, q->cols, count);
  MuonArgs a{};
  bool vec = q->cols % 4 == 0, flat = true, pairs = true;
  for (int i = 0; i < count; ++i) {
    MuonMat& t = a.mat[i];
    t.grad = mats[i].grad;
    t.momentum = mats[i].momentum;
    t.weight = mats[i].weight;
    t.update = mats[i].update;
    t.ld_grad = mats[i].ld_grad;
    t.ld_momentum = mats[i].ld_momentum;
    t.ld_weight = mats[i].ld_weight;
    t.ld_update = mats[i].ld_update;
    const uint64_t gb = 4 * element_bytes(q->grad_dtype);
    vec = vec && addr(t.grad) % gb == 0 && t.ld_grad % 4 == 0;
    flat = flat && t.ld_grad == q->cols;
    if (t.momentum) {
      vec = vec && addr(t.momentum) % 16 == 0 && t.ld_momentum % 4 == 0;
      flat = flat && t.ld_momentum == q->cols;
    }
    pairs = pairs && (t.weight ? addr(t.weight) % (2 * element_bytes(q->weight_dtype)) == 0 && t.ld_weight % 2 == 0
                               : addr(t.update) % (2 * element_bytes(q->update_dtype)) == 0 && t.ld_update % 2 == 0);
  }
  a.count = count;
  a.rows = static_cast<int32_t>(q->rows);
  a.cols = static_cast<int32_t>(q->cols);
  a.m = static_cast<int32_t>(z.m);
  a.n = static_cast<int32_t>(z.n);
  a.transposed = q->rows > q->cols;
  a.grad_dtype = q->grad_dtype;
  a.weight_dtype = q->weight_dtype;
  a.update_dtype = q->update_dtype;
  a.vec = vec;
  a.flat = flat;
  a.pairs = pairs;
  a.nesterov = q->nesterov != 0;
  // a block per 4096 elements (four vectors of four per thread), at most kMuonNormBlocks
  a.norm_blocks = static_cast<int32_t>(std::min<int64_t>(kMuonNormBlocks, cdiv(q->rows * q->cols, 4096)));
  a.beta = static_cast<float>(q->beta);
  a.one_minus_beta = static_cast<float>(1.0 - q->beta);
  a.eps = q->eps;
  a.decay = static_cast<float>(1.0 - q->lr * q->weight_decay);
  a.lr = static_cast<float>(q->lr);
  a.scale = static_cast<float>(q->scale);
  a.ctrl = reinterpret_cast<uint32_t*>(ws + L.ctrl);
  a.done = reinterpret_cast<uint32_t*>(ws + L.done);
  a.partial = a.done + kMuonMaxMats;
  a.sums = reinterpret_cast<float*>(ws + L.sums);
  a.sums_bytes = static_cast<int64_t>(L.sums_bytes);
  a.host_error = h->host_ctrl + kCtrlSticky;
  a.norm = reinterpret_cast<float2*>(ws + L.norm);
  a.diag = reinterpret_cast<float*>(ws + L.diag);
  a.hi[0] = reinterpret_cast<uint16_t*>(ws + L.hi[0]);
  a.hi[1] = reinterpret_cast<uint16_t*>(ws + L.hi[1]);
  a.lo = reinterpret_cast<uint16_t*>(ws + L.lo);
  a.gram = reinterpret_cast<uint16_t*>(ws + L.gram);
  a.poly = reinterpret_cast<uint16_t*>(ws + L.poly);
  const bool both = z.m <= kMuonPairSide;
  a.gram_lo = both ? reinterpret_cast<uint16_t*>(ws + L.gram_lo) : nullptr;
  a.poly_lo = both ? reinterpret_cast<uint16_t*>(ws + L.poly_lo) : nullptr;
  a.ldx = z.ldx;
  a.lda = z.lda;
  a.timeout_ns = timeout_ns;
  a.hold = hold;

  const double el = static_cast<double>(q->rows) * q->cols * count;
  const double dm = static_cast<double>(z.m), dn = static_cast<double>(z.n);
  const double gb = static_cast<double>(element_bytes(q->grad_dtype)), mb = mats[0].momentum ? 8.0 : 0.0;
  const double ob = mats[0].weight ? 2.0 * element_bytes(q->weight_dtype) : 1.0 * element_bytes(q->update_dtype);
  const double flops = q->steps * count * (dm * (dm + 1) * dn + dm * dm * (dm + 1) + 2 * dm * dm * dn);
  MuonSteps steps{};
  steps.count = q->steps;
  std::memcpy(steps.c, coefficients, sizeof(float) * 3 * q->steps);
  // CTAs per matrix of the one-launch kernel: one up to 256 columns (no sum over
  // slabs), else slabs of at most 256 and down to 64 while all matrices still
  // run at once: a slab's epilogues and an element's share of the sum shrink
  // with it (128 x 512: 41 us on eight CTAs, 51 on four)
  int cluster = h->muon_shape < 0 ? muon_small_cluster(z.m, z.n) : 0;
  if (cluster > 0) {
    auto at_once = [&](int c) {
      const std::array<int, 3> key{c, muon_small_chunks(z.n, c), both};
      const auto known = h->muon_small.find(key);
      if (known != h->muon_small.end()) return known->second;
      return h->muon_small.emplace(key, muon_small_clusters(c, key[1], both)).first->second;
    };
    while (cluster > 1 && cluster < 16 && cluster * 64 < z.n && count <= at_once(2 * cluster)) cluster *= 2;
    if (at_once(cluster) > 0) {
      const int chunks = muon_small_chunks(z.n, cluster);
      a.cluster = cluster;
      FLCE_LAUNCH(FLCE_K_MUON_SMALL, flops, el * (gb + mb + ob), launch_muon_small(a, steps, chunks, s));
      return FLCE_OK;
    }
  }

  MuonPairMaps maps;
  std::string why;
  bool ok = true;
  auto operand = [&](CUtensorMap* m, const void* base, uint64_t cols, uint64_t ld, uint32_t box_rows) {
    ok = ok && map_half_3d(m, base, cols, z.m, count, ld, 64, box_rows, &why, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  auto block = [&](CUtensorMap* m, const void* base, uint64_t cols, uint64_t ld, CUtensorMapSwizzle swizzle) {
    ok = ok && map_half_3d(m, base, cols, z.m, count, ld, 32, 32, &why, swizzle);
  };
  for (int i = 0; i < 2; ++i) {
    operand(&maps.xk[i], a.hi[i], z.n, z.ldx, 128);
    operand(&maps.xn[i], a.hi[i], z.n, z.ldx, 64);
    block(&maps.xe[i], a.hi[i], z.n, z.ldx, CU_TENSOR_MAP_SWIZZLE_64B);
  }
  block(&maps.lo, a.lo, z.n, z.ldx, CU_TENSOR_MAP_SWIZZLE_64B);
  operand(&maps.gk, a.gram, z.m, z.lda, 128);
  block(&maps.ge, a.gram, z.m, z.lda, CU_TENSOR_MAP_SWIZZLE_64B);
  block(&maps.gm, a.gram, z.m, z.lda, CU_TENSOR_MAP_SWIZZLE_NONE);
  operand(&maps.pk, a.poly, z.m, z.lda, 128);
  block(&maps.pe, a.poly, z.m, z.lda, CU_TENSOR_MAP_SWIZZLE_64B);
  block(&maps.pm, a.poly, z.m, z.lda, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (both) {
    operand(&maps.lk, a.lo, z.n, z.ldx, 128);
    operand(&maps.ln, a.lo, z.n, z.ldx, 64);
    operand(&maps.glk, a.gram_lo, z.m, z.lda, 128);
    block(&maps.gle, a.gram_lo, z.m, z.lda, CU_TENSOR_MAP_SWIZZLE_64B);
    operand(&maps.plk, a.poly_lo, z.m, z.lda, 128);
    block(&maps.ple, a.poly_lo, z.m, z.lda, CU_TENSOR_MAP_SWIZZLE_64B);
  }
  if (!ok) return fail(h, FLCE_ERR_CUDA, "%s", why.c_str());

  FLCE_LAUNCH(FLCE_K_MUON_MOMENTUM, 0.0, el * (gb + mb), launch_muon_momentum(a, s));
  FLCE_LAUNCH(FLCE_K_MUON_PREPARE, 0.0, el * ((mats[0].momentum ? 4.0 + (q->nesterov ? gb : 0.0) : gb) + 4.0),
              launch_muon_prepare(a, h->num_sms, s));
  // on the handle's tile shape where it was given one, but for the products on both parts
  const MuonPlan plan = muon_plan(a, both ? kMuonSingle : h->muon_shape, h->muon_clusters, h->num_sms);
  a.splits = plan.splits;
  FLCE_LAUNCH(FLCE_K_MUON_STEPS, flops, q->steps * count * (12.0 * dm * dn + 6.0 * dm * dm),
              both ? launch_muon_steps_pairs(maps, a, steps, h->num_sms, s)
                   : launch_muon_steps(plan.shape, maps, a, steps,
                                       plan.shape == kMuonSingle ? h->num_sms : h->muon_clusters, s));
  return FLCE_OK;
}

// flce_muon_update, its waits limited to timeout_ns, for `hold` finished parts more than there are
flce_status muon_run(flce_handle_t h, const flce_muon_args* q, const flce_muon_matrix* mats, int32_t count,
                     void* workspace, uint64_t workspace_bytes, uint32_t hold, uint64_t timeout_ns, void* stream) {
  if (!h) return FLCE_ERR_INVALID_ARG;
  h->err.clear();
  if (!q || count < 0 || (count > 0 && !mats)) return fail(h, FLCE_ERR_INVALID_ARG, "null pointer or bad count");
  if (!muon_size_ok(q->rows, q->cols, count))
    return fail(h, FLCE_ERR_INVALID_ARG, "need 1 <= rows, cols <= %lld", (long long)kMuonMaxDim);
  auto is_type = [](int d) { return d == FLCE_DTYPE_BF16 || d == FLCE_DTYPE_FP32; };
  if (!is_type(q->grad_dtype) || !is_type(q->weight_dtype) || !is_type(q->update_dtype))
    return fail(h, FLCE_ERR_UNSUPPORTED, "gradients, weights and updates must be bf16 or fp32");
  if (q->steps < 1 || q->steps > FLCE_MUON_MAX_STEPS)
    return fail(h, FLCE_ERR_INVALID_ARG, "need 1 <= steps <= %d", FLCE_MUON_MAX_STEPS);
  const double numbers[] = {q->beta, q->eps, q->scale, q->lr, q->weight_decay};
  for (double v : numbers)
    if (!std::isfinite(v)) return fail(h, FLCE_ERR_INVALID_ARG, "beta, eps, scale, lr and weight_decay must be finite");
  if (q->beta < 0.0 || q->beta > 1.0 || q->eps < 0.0)
    return fail(h, FLCE_ERR_INVALID_ARG, "need 0 <= beta <= 1 and eps >= 0");
  float coefficients[3 * FLCE_MUON_MAX_STEPS];
  double reach = 1.0;  // bound of X's singular values before the step
  for (int k = 0; k < q->steps; ++k) {
    static const float standard[3] = {3.4445f, -4.7750f, 2.0315f};
    const float* c = q->coefficients ? q->coefficients + 3 * k : standard;
    for (int i = 0; i < 3; ++i) {
      coefficients[3 * k + i] = c[i];
      if (!std::isfinite(c[i])) return fail(h, FLCE_ERR_INVALID_ARG, "coefficients must be finite");
    }
    double poly, next;
    muon_map_bounds(c[0], c[1], c[2], reach, &poly, &next);
    // 2^12 X, 2^12 A and 2^11 B are held in fp16 (65504)
    if (reach > 3.9 || poly > 30.0)
      return fail(h, FLCE_ERR_INVALID_ARG, "the coefficients of step %d take X out of the products' range", k);
    reach = next;
  }
  for (int i = 0; i < count; ++i) {
    const flce_muon_matrix& t = mats[i];
    if (!t.grad || (!t.weight && !t.update))
      return fail(h, FLCE_ERR_INVALID_ARG, "matrix %d: a gradient, and a weight or an update, are needed", i);
    if ((t.momentum != nullptr) != (mats[0].momentum != nullptr) ||
        (t.weight != nullptr) != (mats[0].weight != nullptr))
      return fail(h, FLCE_ERR_INVALID_ARG, "either all matrices have momentum (weights) or none");
    if (t.ld_grad < q->cols || (t.momentum && t.ld_momentum < q->cols) || (t.weight && t.ld_weight < q->cols) ||
        (!t.weight && t.ld_update < q->cols))
      return fail(h, FLCE_ERR_INVALID_ARG, "matrix %d: a row stride is below cols", i);
    if (addr(t.grad) % element_bytes(q->grad_dtype) || addr(t.momentum) % 4 ||
        (t.weight && addr(t.weight) % element_bytes(q->weight_dtype)) ||
        (!t.weight && addr(t.update) % element_bytes(q->update_dtype)))
      return fail(h, FLCE_ERR_INVALID_ARG, "matrix %d: a pointer is not aligned to its elements", i);
  }
  if (count == 0) return FLCE_OK;
  const int64_t group = muon_group(q->rows, q->cols, count);
  const uint64_t need = muon_layout(q->rows, q->cols, group).total;
  if (!workspace || addr(workspace) % kAlign || workspace_bytes < need)
    return fail(h, FLCE_ERR_BUDGET, "the workspace must hold %llu bytes, %llu-byte aligned",
                static_cast<unsigned long long>(need), static_cast<unsigned long long>(kAlign));
  // the matrices of an update whose wait ran out are unspecified, and most likely
  // this one's too: told once, here or by flce_async_status
  volatile uint32_t* earlier = h->host_ctrl + kCtrlSticky;
  if (*earlier != 0) {
    *earlier = 0;
    return fail(h, FLCE_ERR_TIMEOUT, "a device-side wait of an earlier update ran out: its results are unspecified");
  }
  DeviceGuard guard(h->device);
  if (h->muon_clusters == 0) h->muon_clusters = muon_max_clusters();
  if (h->muon_clusters <= 0) return fail(h, FLCE_ERR_UNSUPPORTED, "no CTA pair fits the device");
  for (int64_t i = 0; i < count; i += group) {
    const flce_status st = muon_group_run(h, q, mats + i, static_cast<int>(std::min<int64_t>(group, count - i)),
                                          coefficients, static_cast<uint8_t*>(workspace), hold, timeout_ns,
                                          static_cast<cudaStream_t>(stream));
    if (st != FLCE_OK) return st;
  }
  return FLCE_OK;
}

}  // namespace

// No exception leaves a C entry: what can throw here is a host allocation (a
// message, the table of cluster sizes).
extern "C" {

uint64_t flce_route_workspace_bytes(flce_handle_t h, int64_t N, int64_t E, int64_t documents) {
  if (!h || N < 0 || N > kMaxDim || E < 1 || E > kRouteMaxExperts || documents < 1 || documents > (1 << 24)) return 0;
  // without offsets a short batch needs less: one size for both
  return route_layout(route_geometry(N, E, 2, documents, true, false, h->num_sms), E, documents).total;
}

flce_status flce_route_forward(flce_handle_t h, const flce_route_args* r, void* workspace, uint64_t workspace_bytes,
                               void* stream) try {
  if (!h) return FLCE_ERR_INVALID_ARG;
  h->err.clear();
  flce_status st = route_check(h, r);
  if (st != FLCE_OK) return st;
  const RouteGeometry g =
      route_geometry(r->N, r->E, element_bytes(r->dtype), r->documents, r->offsets != nullptr, false, h->num_sms);
  const RouteLayout L =
      route_layout(route_geometry(r->N, r->E, 2, r->documents, true, false, h->num_sms), r->E, r->documents);
  if (!workspace || addr(workspace) % 256 || workspace_bytes < L.total)
    return fail(h, FLCE_ERR_BUDGET, "the workspace must hold %llu bytes, 256-byte aligned",
                static_cast<unsigned long long>(L.total));
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RouteArgs a = route_args(r, g);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.unit_p = reinterpret_cast<float*>(ws + L.unit_p);
  a.unit_c = reinterpret_cast<int32_t*>(ws + L.unit_c);
  a.unit_live = reinterpret_cast<int32_t*>(ws + L.unit_live);
  a.unit_z = reinterpret_cast<float*>(ws + L.unit_z);
  a.terms = reinterpret_cast<float*>(ws + L.terms);
  a.doc_live = reinterpret_cast<int32_t*>(ws + L.doc_live);
  a.doc_z = reinterpret_cast<float*>(ws + L.doc_z);
  a.ticket = reinterpret_cast<uint32_t*>(ws + L.ticket);
  const double n = static_cast<double>(r->N), e = static_cast<double>(r->E);
  if (r->N > 0) {
    FLCE_LAUNCH(FLCE_K_ROUTE, 5.0 * n * e, n * (e * element_bytes(r->dtype) + 8.0 * r->k + 8.0),
                launch_route_forward(r->dtype, g, a, s));
  } else {
    const cudaError_t ce = cudaMemsetAsync(a.ticket, 0, 4, s);
    if (ce != cudaSuccess) return fail(h, FLCE_ERR_CUDA, "memset: %s", cudaGetErrorString(ce));
  }
  if (!g.one_launch)
    FLCE_LAUNCH(FLCE_K_ROUTE_FINISH, 0.0, 8.0 * e * (static_cast<double>(g.blocks) + 2.0 * r->documents),
                launch_route_finish(g, a, s));
  return FLCE_OK;
} catch (...) {
  return FLCE_ERR_BUDGET;
}

flce_status flce_route_backward(flce_handle_t h, const flce_route_args* r, const float* d_weights,
                                const float* d_balance, const float* d_z, void* d_logits, int64_t ld_d,
                                void* stream) try {
  if (!h) return FLCE_ERR_INVALID_ARG;
  h->err.clear();
  flce_status st = route_check(h, r);
  if (st != FLCE_OK) return st;
  if (r->N > 0 && !d_logits) return fail(h, FLCE_ERR_INVALID_ARG, "null pointer argument");
  if (ld_d < r->E) return fail(h, FLCE_ERR_INVALID_ARG, "the row stride of d_logits is below E");
  if (addr(d_logits) % element_bytes(r->dtype) || (addr(d_weights) | addr(d_balance) | addr(d_z)) % 4)
    return fail(h, FLCE_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  if (r->N == 0) return FLCE_OK;
  const RouteGeometry g = route_geometry(r->N, r->E, element_bytes(r->dtype), r->documents, true, true, h->num_sms);
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const double n = static_cast<double>(r->N), e = static_cast<double>(r->E);
  FLCE_LAUNCH(FLCE_K_ROUTE_BACKWARD, 6.0 * n * e,
              n * (2.0 * e * element_bytes(r->dtype) + 8.0 + (d_weights ? 12.0 * r->k : 0.0)),
              launch_route_backward(r->dtype, g, route_args(r, g), d_weights, d_balance, d_z, d_logits, ld_d, s));
  return FLCE_OK;
} catch (...) {
  return FLCE_ERR_BUDGET;
}

uint64_t flce_muon_workspace_bytes(int64_t rows, int64_t cols, int64_t count) {
  if (!muon_size_ok(rows, cols, count) || count == 0) return 0;
  return muon_layout(rows, cols, muon_group(rows, cols, count)).total;
}

flce_status flce_muon_update(flce_handle_t h, const flce_muon_args* q, const flce_muon_matrix* mats, int32_t count,
                             void* workspace, uint64_t workspace_bytes, void* stream) try {
  return muon_run(h, q, mats, count, workspace, workspace_bytes, 0, h ? h->timeout_ns : 0, stream);
} catch (...) {
  return FLCE_ERR_BUDGET;
}

flce_status flce_check_muon_timeout(flce_handle_t h, const flce_muon_args* q, const flce_muon_matrix* mats,
                                    int32_t count, void* workspace, uint64_t workspace_bytes, uint32_t timeout_us,
                                    void* stream) try {
  // a CTA whose wait ran out waits as long for its own copies in flight
  if (timeout_us < 1000) return h ? fail(h, FLCE_ERR_INVALID_ARG, "need timeout_us >= 1000") : FLCE_ERR_INVALID_ARG;
  return muon_run(h, q, mats, count, workspace, workspace_bytes, 1, timeout_us * 1000ull, stream);
} catch (...) {
  return FLCE_ERR_BUDGET;
}

}  // extern "C"
