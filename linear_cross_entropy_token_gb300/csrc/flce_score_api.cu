// Host side of the LM-head operators' entry points: argument checks, chunks of
// tokens, workspace layout, TMA descriptors, launches.
#include <algorithm>
#include <cmath>

#include "flce_handle.h"
#include "flce_score.h"

using namespace flce;

namespace {

constexpr double kLog2e = 1.4426950408889634;
constexpr uint64_t kDefaultBudget = 5ull << 28;  // as the loss's planner
constexpr int64_t kMaxChunk = 32768;
constexpr uint64_t kPointerAlign = 256;          // of the workspace and of kept logits
constexpr int64_t kTileRows = 2 * kBM;

uint64_t addr(const void* p) { return reinterpret_cast<uint64_t>(p); }

bool is_bf16(flce_handle_t h) { return h->cfg.dtype == FLCE_DTYPE_BF16; }

// The logits of a row in memory, in elements (fp16 / fp32)
int64_t row_elements(int64_t V) { return static_cast<int64_t>(align_up(static_cast<uint64_t>(V), 64)); }

struct Kept {
  uint64_t partials = 0, total = 0;  // the logits lead
};

Kept kept_layout(bool bf16, int64_t N, int64_t V) {
  Kept k;
  k.partials = align_up(static_cast<uint64_t>(N) * row_elements(V) * (bf16 ? 2 : 4), kAlign);
  k.total = k.partials + align_up(static_cast<uint64_t>(N) * cdiv(V, kScoreGroup) * 8, kAlign);
  return k;
}

// What a call needs: tokens per chunk, splits of dx's sum over V, and the
// workspace's parts.
struct Plan {
  int64_t chunk = 0, ldv = 0, groups = 0, splits = 1;
  bool compact = false;  // chunks are of the rows that count
  int few_parts = 0;     // above 0: the statistics' product is flce_score_few.cu's
  uint64_t ctrl = 0, claims = 0, lead = 0, z = 0, partials = 0, part_s = 0, row = 0, dcorr = 0, xm = 0, order = 0, live = 0,
           parts = 0, entries = 0, picked = 0, dw = 0, total = 0;
};

struct Needs {
  bool z, stats, gradient, dx, dw_sum;
  bool masked;      // some rows may not count
  int64_t teacher;  // entries a row
};

// Rows that do not count are left out of the products where that can spare a tile of
// 256 rows (bf16; fp32 inputs are small models', whose products know no row count of
// the device's). Scoring 4096 x 128256, left out / computed all the same: 241 / 239 us for
// 256 rows half of which count, 244 / 343 for 512 of which 205 do, 637 / 627 for 1024
// that all do (1024 x 32000: 44 / 40, 45 / 50, 77 / 71).
constexpr int64_t kCompactRows = 256;

// Gradients: chunks, tile shapes and splits are the loss's plan with both
// products in one launch. Forward alone: as many tokens as the budget holds, in
// whole tiles, the chunks evened out.
flce_status make_plan(flce_handle_t h, int64_t N, int64_t H, int64_t V, const Needs& q, Plan* out) {
  const bool bf16 = is_bf16(h);
  const uint64_t es = bf16 ? 2 : 4;
  Plan p;
  p.ldv = row_elements(V);
  p.groups = cdiv(V, kScoreGroup);
  if (q.gradient) {
    flce_config cfg = h->cfg;
    cfg.dlogits_mode = FLCE_DLOGITS_INPLACE;
    cfg.cta_pair = FLCE_CTA_AUTO;
    cfg.backward_launch = FLCE_BACKWARD_ONE_LAUNCH;
    flce_plan lp;
    const flce_status st = flce_make_plan(&cfg, N, H, V, 0, h->num_sms, &lp);
    if (st != FLCE_OK) return fail(h, st, "no chunk of these sizes fits the HBM budget");
    p.chunk = lp.chunk;
    p.splits = lp.dx_splits;
    if (!bf16 && p.chunk > 0) {  // the partial sums take at most an eighth of the budget
      const uint64_t budget = h->cfg.hbm_budget_bytes ? h->cfg.hbm_budget_bytes : kDefaultBudget;
      p.splits = score_f32_splits(p.chunk, H, V, h->num_sms,
                                  static_cast<int64_t>(budget / 8 / (static_cast<uint64_t>(p.chunk) * H * 4)));
    }
  } else {
    const uint64_t budget = h->cfg.hbm_budget_bytes ? h->cfg.hbm_budget_bytes : kDefaultBudget;
    const uint64_t a_row = (q.z ? p.ldv * es : 0) + (q.stats ? p.groups * 12ull : 0);
    int64_t most = std::min<int64_t>(kMaxChunk, static_cast<int64_t>(budget / std::max<uint64_t>(a_row, 1)));
    if (most < std::min<int64_t>(N, kBM)) return fail(h, FLCE_ERR_BUDGET, "not even one %d-token chunk fits the HBM budget", kBM);
    if (N > most) {
      const int64_t unit = most >= kTileRows ? kTileRows : kBM;
      most = most / unit * unit;
      most = std::min(most, static_cast<int64_t>(align_up(static_cast<uint64_t>(cdiv(N, cdiv(N, most))), unit)));
    }
    p.chunk = std::min(N, most);
  }
  uint64_t off = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t at = off;
    off = align_up(off + bytes, kAlign);
    return at;
  };
  const uint64_t c = static_cast<uint64_t>(p.chunk);
  if (bf16 && q.stats && !q.teacher && N <= kScoreFew) p.few_parts = score_few_parts(N, H);
  p.compact = bf16 && q.masked && (N > kCompactRows || q.teacher > 0);
  // the control block and the chunks' counters of units, cleared together
  p.claims = kCtrlWords * 4;
  p.lead = p.claims + (q.gradient && c > 0 ? static_cast<uint64_t>(cdiv(N, p.chunk)) * 4 : 0);
  p.ctrl = take(p.lead);
  if (q.z) p.z = take(c * p.ldv * es);
  // the statistics' partials are last read before dx's partial sums are written
  const bool dx_parts = q.dx && (bf16 || p.splits > 1);
  p.partials = take(std::max<uint64_t>(q.stats ? c * p.groups * 8 : 0,
                                       dx_parts ? static_cast<uint64_t>(p.splits) * c * H * 4 : 0));
  if (q.stats) p.part_s = take(c * p.groups * 4);
  if (q.gradient) {
    p.row = take(c * sizeof(ScoreRow));
    p.dcorr = take(c * 4);
    if (q.dw_sum) p.dw = take(static_cast<uint64_t>(V) * H * 4);
  }
  if (q.gradient || p.compact) p.xm = take(c * H * es);
  if (q.masked) p.order = take(static_cast<uint64_t>(std::max<int64_t>(N, 1)) * 4);
  if (q.teacher) {
    p.live = take(static_cast<uint64_t>(std::max<int64_t>(N, 1)));
    if (bf16) {
      p.parts = take(c * cdiv(V, kScoreTileColumns) * sizeof(uint2));
      p.entries = take(c * q.teacher * sizeof(int2));
      p.picked = take(c * q.teacher * 4);
    }
  }
  p.total = off;
  *out = p;
  return FLCE_OK;
}

// Sizes, pointers and alignment of x and W
flce_status check_product(flce_handle_t h, const void* x, const void* W, int64_t N, int64_t H, int64_t V, double temperature) {
  if (N < 0 || H < 1 || V < 1 || N > kMaxDim || H > kMaxDim || V > kMaxDim)
    return fail(h, FLCE_ERR_INVALID_ARG, "sizes must satisfy 0 <= N, 1 <= H, 1 <= V, all below 2^31");
  if (!(temperature > 0.0) || !std::isfinite(temperature) || !(1.0 / temperature < 1e30) || !(temperature < 1e30))
    return fail(h, FLCE_ERR_INVALID_ARG, "the temperature must be positive and finite");
  if (!W || (N > 0 && !x)) return fail(h, FLCE_ERR_INVALID_ARG, "null pointer argument");
  if (is_bf16(h)) {
    if (H % 8 != 0) return fail(h, FLCE_ERR_INVALID_ARG, "bf16 needs H %% 8 == 0 (H = %lld)", static_cast<long long>(H));
    if ((addr(x) | addr(W)) % 16) return fail(h, FLCE_ERR_INVALID_ARG, "x and W must be 16-byte aligned");
  } else if ((addr(x) | addr(W)) % 4) {
    return fail(h, FLCE_ERR_INVALID_ARG, "x and W must be 4-byte aligned");
  }
  return FLCE_OK;
}

flce_status check_gradients(flce_handle_t h, const void* dx, const void* dW, int32_t dw_dtype) {
  if (dW && dw_dtype != FLCE_DTYPE_FP32 && !(dw_dtype == FLCE_DTYPE_BF16 && is_bf16(h)))
    return fail(h, FLCE_ERR_UNSUPPORTED, "dW must be fp32, or bf16 on a bf16 handle");
  if ((addr(dx) | addr(dW)) % (is_bf16(h) ? 16 : 4))
    return fail(h, FLCE_ERR_INVALID_ARG, "dx and dW are not aligned (16 bytes on a bf16 handle, else 4)");
  return FLCE_OK;
}

flce_status check_workspace(flce_handle_t h, const void* ws, uint64_t bytes, uint64_t need) {
  if (!ws || addr(ws) % kPointerAlign || bytes < need)
    return fail(h, FLCE_ERR_BUDGET, "the workspace must hold %llu bytes, %llu-byte aligned",
                static_cast<unsigned long long>(need), static_cast<unsigned long long>(kPointerAlign));
  return FLCE_OK;
}

// The pairs that run at once (whatever tile shape the handle's loss was created with)
flce_status ensure_clusters(flce_handle_t h) {
  if (!is_bf16(h)) return FLCE_OK;
  if (h->score_clusters == 0) h->score_clusters = score_gemm_max_clusters();
  if (h->score_clusters <= 0)
    return fail(h, FLCE_ERR_UNSUPPORTED, "no CTA pair fits the device");
  return FLCE_OK;
}

flce_status clear_ctrl(flce_handle_t h, uint32_t* ctrl, uint64_t bytes, cudaStream_t s) {
  const cudaError_t e = cudaMemsetAsync(ctrl, 0, bytes, s);
  return e == cudaSuccess ? FLCE_OK : fail(h, FLCE_ERR_CUDA, "memset: %s", cudaGetErrorString(e));
}

struct Product {
  const void* x;   // the chunk's rows
  const void* W;
  ScoreChunk chunk;
  int64_t H, V;
  const Plan* p;
  float c;                 // times the product's gain
  float inv_temperature;
  uint32_t* ctrl;
  // columns to pick
  const uint2* parts = nullptr;
  const int2* entries = nullptr;
  float* picked = nullptr;
  int k = 0;
};

ScoreF32Args f32_logits(const Product& q, void* z) {
  ScoreF32Args a{};
  a.A = static_cast<const float*>(q.x);
  a.B = static_cast<const float*>(q.W);
  a.C = static_cast<float*>(z);
  a.sam = a.sbn = q.H;
  a.sak = a.sbk = 1;
  a.ldc = q.p->ldv;
  a.M = q.chunk.rows;
  a.N = q.V;
  a.K = q.H;
  a.c = q.c;
  a.inv_temperature = q.inv_temperature;
  return a;
}

// z of a chunk and its statistics: stored to z where given
flce_status run_stats(flce_handle_t h, const Product& q, void* z, float2* partials, float* part_s, cudaStream_t s) {
  const double dr = q.chunk.rows, dH = static_cast<double>(q.H), dV = static_cast<double>(q.V);
  const int groups = static_cast<int>(q.p->groups);
  if (!is_bf16(h)) {
    ScoreF32Args a = f32_logits(q, z);
    a.partials = partials;
    a.part_s = part_s;
    a.groups = groups;
    FLCE_LAUNCH(FLCE_K_SCORE_STATS, 2 * dr * dH * dV, 4 * (dr * dH + dV * dH + dr * dV) + 12 * dr * groups,
                launch_score_f32(a, s));
    return FLCE_OK;
  }
  CUtensorMap mx, mw, mz;
  std::string why;
  if (!map_bf16_2d(&mx, q.x, q.H, q.chunk.rows, q.H * 2, 64, 128, &why) || !map_bf16_2d(&mw, q.W, q.H, q.V, q.H * 2, 64, 128, &why))
    return fail(h, FLCE_ERR_INVALID_ARG, "%s", why.c_str());
  if (q.p->few_parts > 0) {
    ScoreFewArgs f{};
    f.rows = q.chunk.rows;
    f.padded = (q.chunk.rows + 15) / 16 * 16;
    f.cols = static_cast<int>(q.V);
    f.groups = groups;
    f.kb_total = static_cast<int>(cdiv(q.H, kBK));
    f.parts = q.p->few_parts;
    f.c = q.c;
    f.ldv = q.p->ldv;
    f.z = static_cast<__half*>(z);
    f.partials = partials;
    f.part_s = part_s;
    f.ctrl = q.ctrl;
    f.timeout_ns = h->timeout_ns;
    if (!map_bf16_2d(&mx, q.x, q.H, q.chunk.rows, q.H * 2, 64, f.padded, &why))
      return fail(h, FLCE_ERR_INVALID_ARG, "%s", why.c_str());
    FLCE_LAUNCH(FLCE_K_SCORE_STATS, 2 * dr * dH * dV, 2 * (dr + dV) * dH + (z ? 2 * dr * dV : 0) + 12 * dr * groups,
                launch_score_few(mw, mx, f, h->num_sms, s));
    return FLCE_OK;
  }
  mz = mx;  // not used without a store
  if (z && !map_bf16_2d(&mz, z, q.V, q.chunk.rows, q.p->ldv * 2, 64, 32, &why))
    return fail(h, FLCE_ERR_INVALID_ARG, "%s", why.c_str());
  ScoreGemmArgs a{};
  const int num_m = static_cast<int>(cdiv(q.chunk.rows, kTileRows));
  a.num_n = static_cast<int>(cdiv(q.V, 2 * kBN));
  a.kb_total = static_cast<int>(cdiv(q.H, kBK));
  a.rows = q.chunk.rows;
  a.live = q.chunk.live;
  a.off = q.chunk.off;
  a.cols = static_cast<int>(q.V);
  a.groups = groups;
  a.store = z != nullptr;
  a.c = q.c;
  a.partials = partials;
  a.part_s = part_s;
  a.parts = q.parts;
  a.entries = q.entries;
  a.picked = q.picked;
  a.k = q.k;
  a.ctrl = q.ctrl;
  a.timeout_ns = h->timeout_ns;
  FLCE_LAUNCH(FLCE_K_SCORE_STATS, 2 * dr * dH * dV, 2 * (dr + dV) * dH + (z ? 2 * dr * dV : 0) + 12 * dr * groups,
              launch_score_gemm(q.parts ? kScorePick : kScoreStats, mx, mw, mz, a, std::min(num_m * a.num_n, h->score_clusters), s));
  return FLCE_OK;
}

// d of a chunk straight from the product
flce_status run_gradient(flce_handle_t h, const Product& q, void* d, const ScoreRow* row, cudaStream_t s) {
  const double dr = q.chunk.rows, dH = static_cast<double>(q.H), dV = static_cast<double>(q.V);
  if (!is_bf16(h)) {
    ScoreF32Args a = f32_logits(q, d);
    a.row = row;
    FLCE_LAUNCH(FLCE_K_SCORE_GRADIENT, 2 * dr * dH * dV, 4 * (dr * dH + dV * dH + dr * dV), launch_score_f32(a, s));
    return FLCE_OK;
  }
  CUtensorMap mx, mw, md;
  std::string why;
  if (!map_bf16_2d(&mx, q.x, q.H, q.chunk.rows, q.H * 2, 64, 128, &why) ||
      !map_bf16_2d(&mw, q.W, q.H, q.V, q.H * 2, 64, 128, &why) ||
      !map_bf16_2d(&md, d, q.V, q.chunk.rows, q.p->ldv * 2, 64, 32, &why))
    return fail(h, FLCE_ERR_INVALID_ARG, "%s", why.c_str());
  ScoreGemmArgs a{};
  const int num_m = static_cast<int>(cdiv(q.chunk.rows, kTileRows));
  a.num_n = static_cast<int>(cdiv(q.V, 2 * kBN));
  a.kb_total = static_cast<int>(cdiv(q.H, kBK));
  a.rows = q.chunk.rows;
  a.live = q.chunk.live;
  a.off = q.chunk.off;
  a.cols = static_cast<int>(q.V);
  a.groups = static_cast<int>(q.p->groups);
  a.c = q.c;
  a.least = q.chunk.off == 0;  // zeros, where no row of the call counts
  a.row = row;
  a.ctrl = q.ctrl;
  a.timeout_ns = h->timeout_ns;
  FLCE_LAUNCH(FLCE_K_SCORE_GRADIENT, 2 * dr * dH * dV, 2 * (dr + dV) * dH + 2 * dr * dV,
              launch_score_gemm(kScoreGradient, mx, mw, md, a, std::min(num_m * a.num_n, h->score_clusters), s));
  return FLCE_OK;
}

// dx = d W and dW (+)= dt x of a chunk, whichever is asked for. row null: no entry to
// put right.
struct Backward {
  const void* d;
  float* part;         // dx's partial sums
  void* dx;            // the call's, or null
  void* dW;            // or null
  int32_t dw_dtype;
  float* dw_sum;       // bf16 dW: the chunks' sum so far
  const ScoreRow* row;
  const float* dcorr;
  bool last;
  int32_t* claims;     // the chunk's counter of units
};

flce_status run_backward(flce_handle_t h, const Product& q, const Backward& b, cudaStream_t s) {
  const double dr = q.chunk.rows, dH = static_cast<double>(q.H), dV = static_cast<double>(q.V);
  const int64_t H = q.H, V = q.V, ldv = q.p->ldv;
  const int rows = q.chunk.rows;
  const bool first = q.chunk.off == 0, to16 = b.dW && b.dw_dtype == FLCE_DTYPE_BF16;
  const double dx_bytes = b.dx ? 2 * dr * dV + 2 * dV * dH + 4.0 * q.p->splits * dr * dH : 0.0;
  const double dw_bytes = b.dW ? 2 * dr * dV + 2 * dr * dH + ((first ? 4.0 : 8.0) - (to16 && b.last ? 2.0 : 0.0)) * dV * dH : 0.0;
  if (!is_bf16(h)) {
    const float* d = static_cast<const float*>(b.d);
    ScoreF32Args dx{}, dw{};
    dx.A = dw.A = d;
    dx.N = dx.ldc = dx.sbk = dw.N = dw.ldc = dw.sbk = H;
    dx.sbn = dw.sbn = 1;
    dx.sam = dw.sak = ldv;
    dx.sak = dw.sam = 1;
    dx.B = static_cast<const float*>(q.W);
    dx.C = static_cast<float*>(b.dx) + q.chunk.off * H;
    dx.M = dw.K = rows;
    dx.K = dw.M = V;
    dx.part = b.part;
    dw.B = static_cast<const float*>(q.x);
    dw.C = static_cast<float*>(b.dW);
    dw.accumulate = !first;
    FLCE_LAUNCH(FLCE_K_SCORE_BACKWARD, 2 * dr * dV * dH * ((b.dx != nullptr) + (b.dW != nullptr)), 2 * (dx_bytes + dw_bytes),
                launch_score_f32_backward(b.dx ? &dx : nullptr, static_cast<int>(q.p->splits), b.dW ? &dw : nullptr, s));
    return FLCE_OK;
  }
  std::string why;
  ScoreBackwardArgs a{};
  a.kb_v = static_cast<int>(cdiv(V, kBK));
  a.kb_per_split = static_cast<int>(cdiv(a.kb_v, q.p->splits));
  a.splits = static_cast<int>(cdiv(a.kb_v, a.kb_per_split));
  ScoreBackwardMaps m{};
  float* dw32 = to16 ? b.dw_sum : static_cast<float*>(b.dW);
  if (!map_bf16_2d(&m.d, b.d, V, rows, ldv * 2, 64, 128, &why) || !map_bf16_2d(&m.w, q.W, H, V, H * 2, 64, 64, &why) ||
      (b.dx &&
       !map_f32_3d(&m.part, b.part, H, rows, a.splits, H * 4, static_cast<uint64_t>(q.p->chunk) * H * 4, &why)) ||
      !map_bf16_2d(&m.dt, b.d, V, rows, ldv * 2, 64, 64, &why) || !map_bf16_2d(&m.x, q.x, H, rows, H * 2, 64, 64, &why) ||
      (dw32 && !map_f32_3d(&m.dw32, dw32, H, V, 1, H * 4, static_cast<uint64_t>(V) * H * 4, &why)) ||
      (to16 && !map_bf16_2d(&m.dw16, b.dW, H, V, H * 2, 64, 128, &why)))
    return fail(h, FLCE_ERR_INVALID_ARG, "%s", why.c_str());
  a.rows = rows;
  a.H = static_cast<int>(H);
  a.V = static_cast<int>(V);
  a.dx = b.dx != nullptr;
  a.dw = b.dW != nullptr;
  const int num_m = static_cast<int>(cdiv(rows, kTileRows)), num_n = static_cast<int>(cdiv(H, 2 * kBN));
  const int units0 = a.dx ? num_m * num_n * a.splits : 0;
  const int units = units0 + (a.dw ? static_cast<int>(cdiv(V, kTileRows)) * num_n : 0);
  a.group_m = a.dx ? group_for(h, kShapeWide, num_m, num_n, a.splits, std::min(units0, h->score_clusters)) : 1;
  a.dw_bf16 = to16;
  a.last = b.last;
  a.live = q.chunk.live;
  a.off = q.chunk.off;
  a.dw_sum = dw32;
  a.claims = b.claims;
  a.ctrl = q.ctrl;
  a.timeout_ns = h->timeout_ns;
  FLCE_LAUNCH(FLCE_K_SCORE_BACKWARD, 2 * dr * dV * dH * (a.dx + a.dw), dx_bytes + dw_bytes,
              launch_score_backward(m, a, std::min(units, h->score_clusters), s));
  if (b.dx)
    FLCE_LAUNCH(FLCE_K_DX_REDUCE, 0.0, 4.0 * a.splits * dr * dH + 4 * dr * dH,
                launch_score_dx(q.chunk, b.part, a.splits, q.p->chunk * H, H, q.W, b.row, b.dcorr, b.dx, q.ctrl,
                                b.last && b.row ? h->host_ctrl + kHostScoreError : nullptr, s));
  return FLCE_OK;
}

// dW where no token is: zeros
flce_status zero_dw(flce_handle_t h, void* dW, int32_t dtype, int64_t V, int64_t H, cudaStream_t s) {
  if (!dW) return FLCE_OK;
  const cudaError_t e = cudaMemsetAsync(dW, 0, static_cast<size_t>(V) * H * (dtype == FLCE_DTYPE_FP32 ? 4 : 2), s);
  return e == cudaSuccess ? FLCE_OK : fail(h, FLCE_ERR_CUDA, "memset: %s", cudaGetErrorString(e));
}

// ------------------------------------------------------- log probabilities

flce_status logprobs_check(flce_handle_t h, const flce_logprobs_args* r, bool backward) {
  if (!r) return fail(h, FLCE_ERR_INVALID_ARG, "null pointer argument");
  flce_status st = check_product(h, r->x, r->W, r->N, r->H, r->V, r->temperature);
  if (st != FLCE_OK) return st;
  if (r->top < 0 || r->top > std::min<int64_t>(r->V, kScoreMaxTop))
    return fail(h, FLCE_ERR_INVALID_ARG, "need 0 <= top <= min(V, %d)", kScoreMaxTop);
  if (r->N > 0 && (!r->entropy || !r->stats || (r->t && !r->logprobs) || (backward && !r->t) ||
                   (r->top > 0 && !backward && (!r->top_logprobs || !r->top_ids))))
    return fail(h, FLCE_ERR_INVALID_ARG, "null pointer argument");
  if ((addr(r->t) | addr(r->stats) | addr(r->top_ids)) % 8 ||
      (addr(r->logprobs) | addr(r->entropy) | addr(r->top_logprobs)) % 4 || addr(r->kept) % kPointerAlign)
    return fail(h, FLCE_ERR_INVALID_ARG, "a pointer is not aligned to its elements (kept: to %d bytes)", static_cast<int>(kPointerAlign));
  return FLCE_OK;
}

flce_status logprobs_plan(flce_handle_t h, const flce_logprobs_args* r, bool backward, int32_t dw_dtype, bool dx, Plan* p) {
  Needs q{};
  q.masked = r->t != nullptr;
  if (backward) {
    q.z = q.gradient = true;
    q.dx = dx;
    q.dw_sum = dw_dtype == FLCE_DTYPE_BF16;
  } else {
    q.z = !r->kept && (r->top > 0 || !is_bf16(h));
    q.stats = true;
  }
  return make_plan(h, r->N, r->H, r->V, q, p);
}

// What the forward's product of z lacks
double logprobs_gain(flce_handle_t h, const flce_logprobs_args* r) {
  return !is_bf16(h) ? 1.0 : score_gain(r->H, r->N <= kScoreFew ? score_few_parts(r->N, r->H) : 1);
}

// The rows that count in order, what the others get, and the chunks of the former
flce_status logprobs_rows(flce_handle_t h, const flce_logprobs_args* r, const Plan& p, uint8_t* ws, void* dx, bool backward,
                          cudaStream_t s) {
  if (!p.compact) return FLCE_OK;
  const double n = static_cast<double>(r->N);
  ScoreOrderArgs a{};
  a.N = r->N;
  a.ignore_index = r->ignore_index;
  a.t = r->t;
  a.order = reinterpret_cast<int32_t*>(ws + p.order);
  a.count = reinterpret_cast<uint32_t*>(ws + p.ctrl) + kCtrlNValid;
  if (backward) {
    a.dx = dx;
    a.row_bytes = r->H * 2;
  } else {
    a.top = r->top;
    a.logprobs = r->logprobs;
    a.entropy = r->entropy;
    a.stats = reinterpret_cast<float2*>(r->stats);
    a.top_logprobs = r->top_logprobs;
    a.top_ids = r->top_ids;
  }
  FLCE_LAUNCH(FLCE_K_SCORE_OTHER, 0.0, 20.0 * n, launch_score_order(a, s));
  return FLCE_OK;
}

ScoreChunk chunk_of(const Plan& p, uint8_t* ws, int64_t off, int64_t N) {
  ScoreChunk q{};
  q.rows = static_cast<int32_t>(std::min(p.chunk, N - off));
  q.off = off;
  if (p.compact) {
    q.order = reinterpret_cast<const int32_t*>(ws + p.order);
    q.live = reinterpret_cast<const uint32_t*>(ws + p.ctrl) + kCtrlNValid;
  }
  return q;
}

}  // namespace

// No exception leaves a C entry: what can throw here is a host allocation (a
// message, the table of tile orders).
extern "C" {

uint64_t flce_logprobs_kept_bytes(flce_handle_t h, int64_t N, int64_t V) {
  if (!h || N < 0 || V < 1 || N > kMaxDim || V > kMaxDim) return 0;
  return kept_layout(is_bf16(h), N, V).total;
}

uint64_t flce_logprobs_workspace_bytes(flce_handle_t h, const flce_logprobs_args* r, int32_t backward, int32_t dw_dtype) try {
  if (!h) return 0;
  h->err.clear();
  Plan p;
  if (!r || r->N < 0 || r->H < 1 || r->V < 1 || r->N > kMaxDim || r->H > kMaxDim || r->V > kMaxDim) {
    fail(h, FLCE_ERR_INVALID_ARG, "null argument or bad size");
    return 0;
  }
  return logprobs_plan(h, r, backward != 0, dw_dtype, true, &p) == FLCE_OK ? p.total : 0;
} catch (...) {
  return 0;
}

flce_status flce_logprobs_forward(flce_handle_t h, const flce_logprobs_args* r, void* workspace, uint64_t workspace_bytes,
                                  void* stream) try {
  if (!h) return FLCE_ERR_INVALID_ARG;
  h->err.clear();
  NvtxRange nvtx("flce_logprobs_forward");
  flce_status st = logprobs_check(h, r, false);
  if (st != FLCE_OK) return st;
  Plan p;
  st = logprobs_plan(h, r, false, -1, false, &p);
  if (st == FLCE_OK) st = check_workspace(h, workspace, workspace_bytes, p.total);
  if (st != FLCE_OK) return st;
  if (r->N == 0) return FLCE_OK;
  DeviceGuard guard(h->device);
  st = ensure_clusters(h);
  if (st != FLCE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = is_bf16(h);
  const uint64_t es = bf16 ? 2 : 4;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t* kept = static_cast<uint8_t*>(r->kept);
  uint32_t* ctrl = reinterpret_cast<uint32_t*>(ws + p.ctrl);
  st = clear_ctrl(h, ctrl, p.lead, s);
  if (st != FLCE_OK) return st;
  st = logprobs_rows(h, r, p, ws, nullptr, false, s);
  if (st != FLCE_OK) return st;
  const Kept K = kept_layout(bf16, r->N, r->V);
  const double gain = logprobs_gain(h, r), c = gain * kLog2e / r->temperature;
  const float inv_t = static_cast<float>(1.0 / r->temperature);
  for (int64_t off = 0; off < r->N; off += p.chunk) {
    const ScoreChunk chunk = chunk_of(p, ws, off, r->N);
    const void* x = static_cast<const uint8_t*>(r->x) + off * r->H * es;
    if (p.compact) {
      x = ws + p.xm;
      ScorePrepareArgs a{};
      a.chunk = chunk;
      a.row_bytes = r->H * static_cast<int64_t>(es);
      a.x = r->x;
      a.xm = ws + p.xm;
      FLCE_LAUNCH(FLCE_K_SCORE_OTHER, 0.0, 2.0 * chunk.rows * r->H * es, launch_score_prepare(a, s));
    }
    const Product q{x, r->W, chunk, r->H, r->V, &p, static_cast<float>(c), inv_t, ctrl};
    void* z = kept ? kept + off * p.ldv * es : (r->top > 0 || !bf16) ? ws + p.z : nullptr;
    float2* partials = reinterpret_cast<float2*>(kept ? kept + K.partials + off * p.groups * 8 : ws + p.partials);
    float* part_s = reinterpret_cast<float*>(ws + p.part_s);
    st = run_stats(h, q, z, partials, part_s, s);
    if (st != FLCE_OK) return st;
    ScoreRowsArgs a{};
    a.chunk = chunk;
    a.top = r->top;
    a.groups = static_cast<int>(p.groups);
    a.bf16 = bf16;
    a.H = r->H;
    a.V = r->V;
    a.ldv = p.ldv;
    a.ignore_index = r->ignore_index;
    a.c = static_cast<float>(c);
    a.inv_temperature = inv_t;
    a.scale = static_cast<float>(gain / r->temperature);
    a.loss = static_cast<float>(gain - 1.0);
    a.x = r->x;
    a.W = r->W;
    a.t = r->t;
    a.partials = partials;
    a.part_s = part_s;
    a.z = z;
    a.logprobs = r->logprobs;
    a.entropy = r->entropy;
    a.stats = reinterpret_cast<float2*>(r->stats);
    a.top_logprobs = r->top_logprobs;
    a.top_ids = r->top_ids;
    a.ctrl = ctrl;
    a.host_error = h->host_ctrl + kHostScoreError;
    FLCE_LAUNCH(FLCE_K_SCORE_ROWS, 0.0, chunk.rows * (12.0 * p.groups + (r->top + 1.0) * r->H * es + 12.0 * r->top + 28.0),
                launch_score_rows(a, s));
  }
  return FLCE_OK;
} catch (...) {
  return FLCE_ERR_BUDGET;
}

flce_status flce_logprobs_backward(flce_handle_t h, const flce_logprobs_args* r, const float* d_logprobs,
                                   const float* d_entropy, void* dx, void* dW, int32_t dw_dtype, void* workspace,
                                   uint64_t workspace_bytes, void* stream) try {
  if (!h) return FLCE_ERR_INVALID_ARG;
  h->err.clear();
  NvtxRange nvtx("flce_logprobs_backward");
  flce_status st = logprobs_check(h, r, true);
  if (st == FLCE_OK) st = check_gradients(h, dx, dW, dw_dtype);
  if (st != FLCE_OK) return st;
  if ((addr(d_logprobs) | addr(d_entropy)) % 4) return fail(h, FLCE_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  if (!dx && !dW) return FLCE_OK;
  Plan p;
  st = logprobs_plan(h, r, true, dW ? dw_dtype : -1, dx != nullptr, &p);
  if (st == FLCE_OK) st = check_workspace(h, workspace, workspace_bytes, p.total);
  if (st != FLCE_OK) return st;
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (r->N == 0) return zero_dw(h, dW, dw_dtype, r->V, r->H, s);
  st = ensure_clusters(h);
  if (st != FLCE_OK) return st;
  const bool bf16 = is_bf16(h);
  const uint64_t es = bf16 ? 2 : 4;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const uint8_t* kept = static_cast<const uint8_t*>(r->kept);
  uint32_t* ctrl = reinterpret_cast<uint32_t*>(ws + p.ctrl);
  st = clear_ctrl(h, ctrl, p.lead, s);
  if (st != FLCE_OK) return st;
  st = logprobs_rows(h, r, p, ws, dx, true, s);
  if (st != FLCE_OK) return st;
  const Kept K = kept_layout(bf16, r->N, r->V);
  // kept logits are the forward's; the product of those computed again is its own
  const double kept_gain = logprobs_gain(h, r), gain = kept || !bf16 ? kept_gain : score_gain(r->H);
  const float c = static_cast<float>(gain * kLog2e / r->temperature);
  const float inv_t = static_cast<float>(1.0 / r->temperature);
  ScoreRow* row = reinterpret_cast<ScoreRow*>(ws + p.row);
  float* dcorr = reinterpret_cast<float*>(ws + p.dcorr);
  void* d = ws + p.z;
  int32_t* claims = reinterpret_cast<int32_t*>(ws + p.claims);
  for (int64_t off = 0; off < r->N; off += p.chunk, ++claims) {
    const ScoreChunk chunk = chunk_of(p, ws, off, r->N);
    const double dr = chunk.rows, dV = static_cast<double>(r->V);
    ScorePrepareArgs a{};
    a.chunk = chunk;
    a.tail = 1;
    a.row_bytes = r->H * static_cast<int64_t>(es);
    a.x = r->x;
    a.xm = ws + p.xm;
    a.V = r->V;
    a.ignore_index = r->ignore_index;
    a.inv_temperature = inv_t;
    a.largest_scale = static_cast<float>(kept_gain / gain);
    a.t = r->t;
    a.stats = reinterpret_cast<const float2*>(r->stats);
    a.logprobs = r->logprobs;
    a.entropy = r->entropy;
    a.d_logprobs = d_logprobs;
    a.d_entropy = d_entropy;
    a.row = row;
    a.dcorr = dcorr;
    a.ctrl = ctrl;
    FLCE_LAUNCH(FLCE_K_SCORE_OTHER, 0.0, 2.0 * dr * r->H * es + 50.0 * dr, launch_score_prepare(a, s));
    const Product q{ws + p.xm, r->W, chunk, r->H, r->V, &p, c, inv_t, ctrl};
    if (kept) {
      FLCE_LAUNCH(FLCE_K_SCORE_DLOGITS, 0.0, 2.0 * es * dr * dV,
                  launch_score_dlogits(bf16, chunk, kept + off * p.ldv * es,
                                       reinterpret_cast<const float2*>(kept + K.partials) + off * p.groups,
                                       static_cast<int>(p.groups), d, p.ldv, r->V, c, inv_t, row, s));
    } else {
      st = run_gradient(h, q, d, row, s);
      if (st != FLCE_OK) return st;
    }
    if (bf16) FLCE_LAUNCH(FLCE_K_SCORE_OTHER, 0.0, 34.0 * dr, launch_score_target(chunk, d, p.ldv, row, s));
    const Backward b{d,   reinterpret_cast<float*>(ws + p.partials), dx, dW, dw_dtype, reinterpret_cast<float*>(ws + p.dw), row,
                     dcorr, off + p.chunk >= r->N, claims};
    st = run_backward(h, q, b, s);
    if (st != FLCE_OK) return st;
  }
  if (!dx || !bf16)  // else dx's last launch has
    FLCE_LAUNCH(FLCE_K_SCORE_OTHER, 0.0, 4.0, launch_score_report(ctrl, h->host_ctrl + kHostScoreError, s));
  return FLCE_OK;
} catch (...) {
  return FLCE_ERR_BUDGET;
}

// ------------------------------------------------------------ distillation

static flce_status distill_check(flce_handle_t h, const flce_distill_args* r) {
  if (!r) return fail(h, FLCE_ERR_INVALID_ARG, "null pointer argument");
  flce_status st = check_product(h, r->x, r->W, r->N, r->H, r->V, r->temperature);
  if (st == FLCE_OK) st = check_gradients(h, r->dx, r->dW, r->dw_dtype);
  if (st != FLCE_OK) return st;
  if (r->logits_dtype != FLCE_DTYPE_BF16 && r->logits_dtype != FLCE_DTYPE_FP32 && r->logits_dtype != FLCE_DTYPE_FP16)
    return fail(h, FLCE_ERR_UNSUPPORTED, "the teacher's logits must be bf16, fp32 or fp16");
  if (r->K < 1 || r->K > kScoreMaxTeacher) return fail(h, FLCE_ERR_INVALID_ARG, "need 1 <= K <= %d", kScoreMaxTeacher);
  if (r->ld_ids < r->K || r->ld_logits < r->K) return fail(h, FLCE_ERR_INVALID_ARG, "a row stride is below K");
  if (!r->loss || (r->N > 0 && (!r->ids || !r->logits || !r->token_loss)))
    return fail(h, FLCE_ERR_INVALID_ARG, "null pointer argument");
  if (addr(r->ids) % 8 || addr(r->logits) % (r->logits_dtype == FLCE_DTYPE_FP32 ? 4 : 2) ||
      (addr(r->loss) | addr(r->token_loss)) % 4)
    return fail(h, FLCE_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  return FLCE_OK;
}

static flce_status distill_plan(flce_handle_t h, const flce_distill_args* r, Plan* p) {
  Needs q{};
  q.stats = true;
  q.teacher = r->K;
  q.gradient = r->dx || r->dW;
  q.z = q.gradient || !is_bf16(h);
  q.dx = r->dx != nullptr;
  q.dw_sum = r->dW && r->dw_dtype == FLCE_DTYPE_BF16;
  q.masked = true;
  return make_plan(h, r->N, r->H, r->V, q, p);
}

uint64_t flce_distill_workspace_bytes(flce_handle_t h, const flce_distill_args* r) try {
  if (!h) return 0;
  h->err.clear();
  Plan p;
  if (!r || r->N < 0 || r->H < 1 || r->V < 1 || r->N > kMaxDim || r->H > kMaxDim || r->V > kMaxDim) {
    fail(h, FLCE_ERR_INVALID_ARG, "null argument or bad size");
    return 0;
  }
  return distill_plan(h, r, &p) == FLCE_OK ? p.total : 0;
} catch (...) {
  return 0;
}

flce_status flce_distill(flce_handle_t h, const flce_distill_args* r, void* workspace, uint64_t workspace_bytes,
                         void* stream) try {
  if (!h) return FLCE_ERR_INVALID_ARG;
  h->err.clear();
  NvtxRange nvtx("flce_distill");
  flce_status st = distill_check(h, r);
  if (st != FLCE_OK) return st;
  Plan p;
  st = distill_plan(h, r, &p);
  if (st == FLCE_OK) st = check_workspace(h, workspace, workspace_bytes, p.total);
  if (st != FLCE_OK) return st;
  DeviceGuard guard(h->device);
  st = ensure_clusters(h);
  if (st != FLCE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = is_bf16(h);
  const uint64_t es = bf16 ? 2 : 4, ls = r->logits_dtype == FLCE_DTYPE_FP32 ? 4 : 2;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint32_t* ctrl = reinterpret_cast<uint32_t*>(ws + p.ctrl);
  uint8_t* live = ws + p.live;
  st = clear_ctrl(h, ctrl, p.lead, s);
  if (st != FLCE_OK) return st;
  const bool gradient = r->dx || r->dW;
  const double gain = bf16 ? score_gain(r->H) : 1.0;
  const float c = static_cast<float>(gain * kLog2e / r->temperature);
  const float inv_t = static_cast<float>(1.0 / r->temperature);
  const double n = static_cast<double>(r->N);
  int32_t* claims = reinterpret_cast<int32_t*>(ws + p.claims);
  if (r->N == 0) {
    st = zero_dw(h, r->dW, r->dw_dtype, r->V, r->H, s);
    if (st != FLCE_OK) return st;
  } else {
    FLCE_LAUNCH(FLCE_K_SCORE_OTHER, 0.0, n * r->K * (8 + ls),
                launch_distill_live(r->ids, r->ld_ids, r->logits, r->ld_logits, r->logits_dtype, r->N, static_cast<int>(r->K),
                                    r->V, live, r->token_loss, ctrl, !p.compact, s));
    if (p.compact) {
      ScoreOrderArgs a{};
      a.N = r->N;
      a.live = live;
      a.order = reinterpret_cast<int32_t*>(ws + p.order);
      a.count = ctrl + kCtrlNValid;
      a.dx = r->dx;
      a.row_bytes = r->H * 2;
      FLCE_LAUNCH(FLCE_K_SCORE_OTHER, 0.0, 6.0 * n, launch_score_order(a, s));
    }
  }
  for (int64_t off = 0; off < r->N; off += p.chunk, ++claims) {
    const ScoreChunk chunk = chunk_of(p, ws, off, r->N);
    const double dr = chunk.rows, dV = static_cast<double>(r->V);
    const void* x = static_cast<const uint8_t*>(r->x) + off * r->H * es;
    if (bf16 || gradient) {
      ScorePrepareArgs a{};
      a.chunk = chunk;
      a.tail = gradient;
      a.row_bytes = r->H * static_cast<int64_t>(es);
      a.x = r->x;
      a.xm = ws + p.xm;
      a.alive = bf16 ? nullptr : live;
      x = ws + p.xm;
      FLCE_LAUNCH(FLCE_K_SCORE_OTHER, 0.0, 2.0 * dr * r->H * es, launch_score_prepare(a, s));
    }
    Product q{x, r->W, chunk, r->H, r->V, &p, c, inv_t, ctrl};
    if (bf16) {
      DistillPickArgs a{};
      a.chunk = chunk;
      a.k = static_cast<int>(r->K);
      a.dtype = r->logits_dtype;
      a.num_tiles = static_cast<int>(cdiv(r->V, kScoreTileColumns));
      a.ld_ids = r->ld_ids;
      a.ld_logits = r->ld_logits;
      a.ids = r->ids;
      a.logits = r->logits;
      a.parts = reinterpret_cast<uint2*>(ws + p.parts);
      a.entries = reinterpret_cast<int2*>(ws + p.entries);
      FLCE_LAUNCH(FLCE_K_SCORE_OTHER, 0.0, dr * (r->K * (16.0 + ls) + 8.0 * a.num_tiles), launch_distill_pick(a, s));
      q.parts = a.parts;
      q.entries = a.entries;
      q.picked = reinterpret_cast<float*>(ws + p.picked);
      q.k = a.k;
    }
    void* z = gradient || !bf16 ? ws + p.z : nullptr;
    float2* partials = reinterpret_cast<float2*>(ws + p.partials);
    st = run_stats(h, q, z, partials, reinterpret_cast<float*>(ws + p.part_s), s);
    if (st != FLCE_OK) return st;
    DistillArgs a{};
    a.chunk = chunk;
    a.k = static_cast<int>(r->K);
    a.groups = static_cast<int>(p.groups);
    a.bf16 = bf16;
    a.dtype = r->logits_dtype;
    a.gradient = gradient;
    a.V = r->V;
    a.ldv = p.ldv;
    a.ld_ids = r->ld_ids;
    a.ld_logits = r->ld_logits;
    a.c = c;
    a.temperature = static_cast<float>(r->temperature);
    a.inv_temperature = inv_t;
    a.scale = static_cast<float>(gain / r->temperature);
    a.ids = r->ids;
    a.logits = r->logits;
    a.partials = partials;
    a.picked = q.picked;
    a.z = z;
    a.token_loss = r->token_loss;
    a.alive = bf16 ? nullptr : live;
    a.ctrl = ctrl;
    FLCE_LAUNCH(FLCE_K_DISTILL_ROWS, 0.0,
                dr * (r->K * (12.0 + ls) + 8.0 * p.groups) + (gradient ? 2.0 * es * dr * dV : 0.0),
                launch_distill_rows(a, s));
    if (gradient) {
      const Backward b{z,       reinterpret_cast<float*>(ws + p.partials), r->dx, r->dW, r->dw_dtype,
                       reinterpret_cast<float*>(ws + p.dw), nullptr, nullptr, off + p.chunk >= r->N, claims};
      st = run_backward(h, q, b, s);
      if (st != FLCE_OK) return st;
    }
  }
  FLCE_LAUNCH(FLCE_K_SCORE_OTHER, 0.0, 4.0 * n,
              launch_distill_finish(r->token_loss, r->N, ctrl, r->loss, h->host_ctrl + kHostScoreError, s));
  return FLCE_OK;
} catch (...) {
  return FLCE_ERR_BUDGET;
}

}  // extern "C"
