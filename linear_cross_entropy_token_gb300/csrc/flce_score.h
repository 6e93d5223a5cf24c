// Declarations of the LM-head operators beside the mean loss: log probabilities
// of given tokens with entropy and top alternatives, and distillation from a
// teacher's top logits.
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/flce.h"

namespace flce {

constexpr int kScoreMaxTop = 64;
constexpr int kScoreMaxTeacher = 256;
constexpr int kScoreGroup = 64;          // vocabulary columns per partial

// Word of a call's control block for a token id out of range: not kCtrlError's, at
// which the products' waits give up (the other rows' results stand).
constexpr int kCtrlBadId = 8;

// What a row's gradient is made of: with t = log2 p = (z - largest) c - log2_total,
// d_j = 2^t (a + b t), and `at` at the target's column.
struct ScoreRow {
  float largest;       // of the row's logits, as the product gave them
  float log2_total;    // log2 of the sum of 2^((z - largest) c)
  float a, b;
  float at;
  int32_t target;      // column, -1: none
  float inv_total;     // fp32 logits: p = exp((z - largest) / temperature) inv_total
};

// ---------------------------------------------------- flce_score_gemm.cu

// One product z = x Wt on 256 x 512 tiles of CTA pairs, and what becomes of z.
struct ScoreGemmArgs {
  int32_t num_n;                 // tiles of columns
  int32_t kb_total;              // 64-deep k-blocks
  int32_t rows, cols;            // rows of the chunk; V
  int32_t least;                 // rows that are computed whatever `live` says (0 or 1)
  const uint32_t* live;          // how many of the call's rows count, or null: all do
  int64_t off;                   // the chunk's first row, of those
  int32_t groups;                // partials per row: ceil(V / 64)
  int32_t store;                 // statistics: also store the logits
  float c;                       // log2(e) / temperature, times score_gain(H)
  float2* partials;              // [rows][groups]: largest z, sum of 2^((z - largest) c)
  float* part_s;                 // [rows][groups]: sum of y 2^y, y = (z - largest) c
  const ScoreRow* row;           // gradient: [rows]
  // picked columns (kScorePick): a row's entries in order of column, and for each 512
  // columns (a tile) the first entry of each of its four parts of 128, and of the next
  const uint2* parts;            // [rows][num_n]: 9 bits each from bit 0
  const int2* entries;           // [rows][k]: column, slot
  float* picked;                 // [rows][k]: z of each slot
  int32_t k;
  uint32_t* ctrl;                // word 0: first error
  uint64_t timeout_ns;
};

// kScoreStats: the statistics, and with `store` z as fp16 [rows][ldv], relative to
// its group's largest (o); kScorePick:
// those and z of picked columns; kScoreGradient: d as bf16 [rows][ldv] (o).
// a: x (box 64 x 128), b: W (box 64 x 128), o: box 64 x 32
enum ScoreMode : int { kScoreStats = 0, kScoreGradient = 1, kScorePick = 2 };
constexpr int kScoreTileColumns = 512;
constexpr int kScorePart = 128;
cudaError_t launch_score_gemm(int mode, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o,
                              const ScoreGemmArgs& args, int pairs, cudaStream_t s);
int score_gemm_max_clusters();

// What the product's sums lack. The tensor cores cut a running sum toward zero at
// every 16-deep step: by half a last place on average, 2^-24 of a binade's upper
// end. A sum that ends at z has been at z k / n after k of its n steps on average
// (products come in no order), so it loses 2^-24 z (average over a binade 0.72) n / 2
// in all: 2^-23 n 0.18. Measured: 0.10 at 64 columns, 0.135 at 1024, 0.135 to 0.14 at
// 2048 to 8192 (those bits that a step's aligned products keep below the last place
// are not cut). It matters because all logits of a row shrink alike and their
// log-sum-exp with them: 3.8e-6 at 4096 columns, where rounding to nearest would
// leave a tenth of that. A sum that is taken in parts loses as much less (0.128 to
// 0.13 by the part).
inline double score_gain(int64_t H, int parts = 1) {
  return 1.0 + (parts > 1 ? 0.13 : 0.136) / 8388608.0 * (static_cast<double>(H) / 16.0) / parts;
}

// ----------------------------------------------------- flce_score_few.cu

// The statistics for at most kScoreFew rows: the two kernels meet at 128 (scoring 4096 x
// 128256 in a captured graph: 212 us here and 230 on pair tiles at 64 rows, 216 and 231
// at 96, 225 and 232 at 128; 1024 x 32000: 36 and 38, 38 and 40, 40 and 40)
constexpr int kScoreFew = 128;
// The parts that a sum is taken in, each in TMEM columns of its own (two tiles' at once)
inline int score_few_parts(int64_t rows, int64_t H) {
  const int64_t padded = (rows + 15) / 16 * 16, blocks = (H + kBK - 1) / kBK;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({4, 256 / std::max<int64_t>(padded, 1), blocks})));
}
struct ScoreFewArgs {
  int32_t rows, padded;          // tokens; rounded up to 16
  int32_t cols, groups;          // V; partials per row
  int32_t kb_total;
  int32_t parts;                 // score_few_parts()
  int32_t tiles, stages, tmem_columns;  // filled in by the launch
  float c;
  int64_t ldv;
  __half* z;                     // [rows][ldv] as ScoreGemmArgs' stored, or null
  float2* partials;
  float* part_s;
  uint32_t* ctrl;
  uint64_t timeout_ns;
};
// w: W (box 64 x 128), x: x (box 64 x padded)
cudaError_t launch_score_few(const CUtensorMap& w, const CUtensorMap& x, ScoreFewArgs args, int sms, cudaStream_t s);

// ----------------------------------------------------- flce_score_f32.cu

// C[m][n] (+)= sum over k of A(m, k) B(k, n) in fp32, operands by strides
struct ScoreF32Args {
  const float* A;
  const float* B;
  float* C;
  int64_t sam, sak, sbk, sbn, ldc, M, N, K;
  int32_t accumulate;
  float* part;                   // splits x M x N, or null
  // z = x Wt: the statistics of its 64-column groups, or with `row` their gradient
  // in z's place
  float2* partials;
  float* part_s;
  int32_t groups;
  float c, inv_temperature;
  const ScoreRow* row;
  int64_t k_per_split;           // filled in by the launches, as what follows
  int32_t vectors_a, vectors_b;
};
struct ScoreF32Pair {
  ScoreF32Args p[2];
  int64_t blocks0;               // of the first
};
int score_f32_splits(int64_t M, int64_t N, int64_t K, int sms, int64_t most);
// z with its statistics or as its gradient
cudaError_t launch_score_f32(ScoreF32Args args, cudaStream_t s);
// dx (its sum over V in splits) and dW, either may be null, in one launch
cudaError_t launch_score_f32_backward(const ScoreF32Args* dx, int splits, const ScoreF32Args* dw, cudaStream_t s);

// ------------------------------------------------ flce_score_backward.cu

struct ScoreBackwardMaps {
  CUtensorMap d, w, part;        // dx = d W: d (box 64 x 128), W (64 x 64), fp32 partial sums (32 x 128 x 1)
  CUtensorMap dt, x, dw32, dw16; // dW = dt x: d (64 x 64), x (64 x 64), fp32 (32 x 128 x 1), bf16 (64 x 128)
};
struct ScoreBackwardArgs {
  int32_t rows;                  // of the chunk; d and x hold zeros from the rows that count up to a multiple of 256
  int32_t H, V;
  int32_t dx, dw;                // which of the products
  int32_t splits, kb_v, kb_per_split;  // of dx's sum over V
  int32_t group_m;               // tile rows per group, of dx
  int32_t dw_bf16;               // the last chunk stores dW as bf16
  int32_t last;                  // without `live`: this is the last chunk
  const uint32_t* live;          // as ScoreGemmArgs
  int64_t off;
  const float* dw_sum;           // dw_bf16: what dw32 describes
  int32_t* claims;               // zero: the chunk's counter of units
  uint32_t* ctrl;
  uint64_t timeout_ns;
};
cudaError_t launch_score_backward(const ScoreBackwardMaps& maps, const ScoreBackwardArgs& args, int pairs, cudaStream_t s);

// --------------------------------------------------------- flce_score.cu

// A chunk: rows off .. off + rows - 1 of the rows that count (`live` of them), each
// the order[i]-th of the call; order null: all rows count, as they stand.
struct ScoreChunk {
  int32_t rows;
  int64_t off;
  const int32_t* order;
  const uint32_t* live;
};

// The rows that count, in order, and how many: t[i] != ignore_index, or live[i] != 0
// where t is null. The rows that do not get zeros in what is given of the outputs.
struct ScoreOrderArgs {
  int64_t N, ignore_index;
  const int64_t* t;
  const uint8_t* live;
  int32_t* order;
  uint32_t* count;
  int32_t top;
  float* logprobs;
  float* entropy;
  float2* stats;
  float* top_logprobs;
  int64_t* top_ids;
  void* dx;
  int64_t row_bytes;             // of dx
};
cudaError_t launch_score_order(const ScoreOrderArgs& a, cudaStream_t s);

struct ScoreRowsArgs {
  ScoreChunk chunk;
  int32_t top, groups;
  int32_t bf16;                  // x and W bf16 and z stored as fp16, or all fp32
  int64_t H, V, ldv, ignore_index;
  float c;                       // log2(e) / temperature, times gain
  float inv_temperature;
  float scale;                   // inv_temperature times gain
  float loss;                    // gain - 1
  const void* x;                 // the call's, by row, as are t and the outputs
  const void* W;
  const int64_t* t;              // null: no given tokens
  const float2* partials;        // by row of the chunk
  const float* part_s;
  const void* z;                 // [rows][ldv] fp16 z - its group's largest, or fp32 z; read for alternatives only
  float* logprobs;
  float* entropy;
  float2* stats;                 // largest z, log of the sum of exp((z - largest) / temperature)
  float* top_logprobs;           // [N][top]
  int64_t* top_ids;
  const uint32_t* ctrl;
  uint32_t* host_error;          // pinned host word
};
cudaError_t launch_score_rows(const ScoreRowsArgs& a, cudaStream_t s);

// A chunk's rows before a product: those of x that count side by side, with zeros
// behind them up to a multiple of 256 rows (tail), or zeros in the place of those
// that do not (order null).
// With t: what the gradient of each row is made of.
struct ScorePrepareArgs {
  ScoreChunk chunk;
  int32_t tail;
  int64_t row_bytes;
  const void* x;
  void* xm;
  const uint8_t* alive;          // order null: zero where a row does not count, or null
  // gradient
  int64_t V, ignore_index;
  float inv_temperature;
  float largest_scale;           // from the forward's product to the gradient's
  const int64_t* t;              // null: rows of x alone
  const float2* stats;
  const float* logprobs;
  const float* entropy;          // read where d_entropy is given
  const float* d_logprobs;       // may be null
  const float* d_entropy;        // may be null
  ScoreRow* row;                 // by row of the chunk
  float* dcorr;
  uint32_t* ctrl;
};
cudaError_t launch_score_prepare(const ScorePrepareArgs& a, cudaStream_t s);

// d from kept logits: fp16 relative to their groups' largest (partials), or fp32 z
cudaError_t launch_score_dlogits(int bf16, const ScoreChunk& chunk, const void* z, const float2* partials, int groups, void* d,
                                 int64_t ldv, int64_t V, float c, float inv_temperature, const ScoreRow* row,
                                 cudaStream_t s);
// bf16 d's entries at the targets
cudaError_t launch_score_target(const ScoreChunk& chunk, void* d, int64_t ldv, const ScoreRow* row, cudaStream_t s);
// host_error not null: the call's last launch, which hands ctrl's error on to it
cudaError_t launch_score_dx(const ScoreChunk& chunk, const float* part, int splits, int64_t split_stride, int64_t H,
                            const void* W, const ScoreRow* row, const float* dcorr, void* dx, const uint32_t* ctrl,
                            uint32_t* host_error, cudaStream_t s);
// hands ctrl's error on to the host's word
cudaError_t launch_score_report(const uint32_t* ctrl, uint32_t* host_error, cudaStream_t s);

struct DistillArgs {
  ScoreChunk chunk;
  int32_t k, groups;
  int32_t bf16;
  int32_t dtype;                 // of the teacher's logits
  int32_t gradient;              // 1: z becomes d, in place
  int64_t V, ldv, ld_ids, ld_logits;
  float c;                       // log2(e) / temperature, times gain
  float temperature, inv_temperature;
  float scale;                   // inv_temperature times gain
  const int64_t* ids;            // the call's, by row, as are logits and token_loss
  const void* logits;
  const float2* partials;        // by row of the chunk
  const float* picked;           // [rows][k]: z of the entries that count (fp32: taken from z)
  void* z;                       // [rows][ldv] fp16 / fp32 z in, bf16 / fp32 d out
  float* token_loss;
  const uint8_t* alive;          // as ScorePrepareArgs
  const uint32_t* ctrl;          // kCtrlNValid: rows that count
};
cudaError_t launch_distill_rows(const DistillArgs& a, cudaStream_t s);
// which of N rows have an entry; the others' losses; ids out of range (ctrl's error;
// their rows do not count). count: and how many (kCtrlNValid)
cudaError_t launch_distill_live(const int64_t* ids, int64_t ld_ids, const void* logits, int64_t ld_logits, int dtype,
                                int64_t N, int k, int64_t V, uint8_t* live, float* token_loss, uint32_t* ctrl,
                                bool count, cudaStream_t s);
// the columns to pick of a chunk's rows (ScoreGemmArgs)
struct DistillPickArgs {
  ScoreChunk chunk;
  int32_t k, dtype, num_tiles;
  int64_t ld_ids, ld_logits;
  const int64_t* ids;            // the call's
  const void* logits;
  uint2* parts;
  int2* entries;
};
cudaError_t launch_distill_pick(const DistillPickArgs& a, cudaStream_t s);
cudaError_t launch_distill_finish(const float* token_loss, int64_t N, const uint32_t* ctrl, float* loss,
                                  uint32_t* host_error, cudaStream_t s);

}  // namespace flce
