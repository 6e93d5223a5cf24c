// Declarations of the LM-head operators beside the mean loss: log probabilities
// of given tokens with entropy and top alternatives, and distillation from a
// teacher's top logits.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/flce.h"

namespace flce {

constexpr int kScoreMaxTop = 64;
constexpr int kScoreMaxTeacher = 256;
constexpr int kScoreGroup = 64;          // vocabulary columns per partial

// What a row's gradient is made of: with t = log2 p = (z - largest) c - log2_total,
// d_j = 2^t (a + b t), plus `add` at the target's column.
struct ScoreRow {
  float largest;       // of the row's logits, as the product gave them
  float log2_total;    // log2 of the sum of 2^((z - largest) c)
  float a, b;
  float add;
  int32_t target;      // column, -1: none
  float inv_total;     // fp32 logits: p = exp((z - largest) / temperature) inv_total
};

// ---------------------------------------------------- flce_score_gemm.cu

// One product z = x Wt on 256 x 512 tiles of CTA pairs, and what becomes of z.
struct ScoreGemmArgs {
  int32_t num_m, num_n;          // tiles
  int32_t kb_total;              // 64-deep k-blocks
  int32_t rows, cols;            // valid rows; V
  int32_t groups;                // partials per row: ceil(V / 64)
  int32_t store;                 // statistics: also store the scaled logits
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
  float* dcorr;                  // gradient: [rows] what rounding took from the target's entry
  uint32_t* ctrl;                // word 0: first error
  uint64_t timeout_ns;
};

// kScoreStats: the statistics, and with `store` y as fp16 [rows][ldv] (o); kScorePick:
// those and z of picked columns; kScoreGradient: d as bf16 [rows][ldv] (o).
// a: x (box 64 x 128), b: W (box 64 x 128), o: box 64 x 128
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
// in all: 2^-23 n 0.18. Measured at 64 to 8192 columns: 0.10 to 0.13, the share
// rising to 0.133 (those bits that a step's aligned products keep below the last
// place are not cut). It matters because all logits of a row shrink alike and their
// log-sum-exp with them: 3.8e-6 at 4096 columns, where rounding to nearest would
// leave a tenth of that.
inline double score_gain(int64_t H) { return 1.0 + 0.13 / 8388608.0 * (static_cast<double>(H) / 16.0); }

// --------------------------------------------------------- flce_score.cu

// The statistics of fp32 logits, as the product's epilogue takes them.
cudaError_t launch_score_stats_f32(const float* z, int64_t ldv, int rows, int64_t V, int groups, float c,
                                   float inv_temperature, float2* partials, float* part_s, cudaStream_t s);

struct ScoreRowsArgs {
  int32_t rows, top, groups;
  int32_t bf16;                  // x and W bf16 and z stored as fp16 y, or all fp32
  int64_t H, V, ldv, ignore_index;
  float c, inv_c;                // log2(e) / temperature, times gain
  float inv_temperature;
  float scale;                   // inv_temperature times gain
  float loss;                    // gain - 1
  const void* x;                 // this chunk's rows
  const void* W;
  const int64_t* t;              // null: no given tokens
  const float2* partials;
  const float* part_s;
  const void* z;                 // [rows][ldv] fp16 y, or fp32 z; read for alternatives only
  float* logprobs;
  float* entropy;
  float2* stats;                 // largest z, log of the sum of exp((z - largest) / temperature)
  float* top_logprobs;           // [rows][top]
  int64_t* top_ids;
  const uint32_t* ctrl;
  uint32_t* host_error;          // pinned host word
};
cudaError_t launch_score_rows(const ScoreRowsArgs& a, cudaStream_t s);

// rowc and, with xm, a copy of x whose rows that do not count are zero
struct ScorePrepareArgs {
  int32_t rows;
  int32_t bf16;
  int64_t H, V, ignore_index;
  float inv_temperature;
  const void* x;
  void* xm;                      // may be null
  const int64_t* t;
  const float2* stats;
  const float* entropy;          // read where d_entropy is given
  const float* d_logprobs;       // may be null
  const float* d_entropy;        // may be null
  ScoreRow* row;
  float* dcorr;
  uint32_t* ctrl;
};
cudaError_t launch_score_prepare(const ScorePrepareArgs& a, cudaStream_t s);

// d from kept logits: y as fp16 with its groups' largest (partials), or fp32 z
cudaError_t launch_score_dlogits(int bf16, const void* z, const float2* partials, int groups, void* d, int64_t ldv,
                                 int rows, int64_t V, float c, float inv_temperature, const ScoreRow* row, float* dcorr,
                                 cudaStream_t s);

cudaError_t launch_score_dx(const float* part, int splits, int64_t split_stride, int rows, int64_t H, const void* W,
                            const ScoreRow* row, const float* dcorr, void* dx, cudaStream_t s);
cudaError_t launch_score_cast(const float* in, void* out, int64_t n, cudaStream_t s);
// hands ctrl's error on to the host's word
cudaError_t launch_score_report(const uint32_t* ctrl, uint32_t* host_error, cudaStream_t s);

struct DistillArgs {
  int32_t rows, k, groups;
  int32_t bf16;
  int32_t dtype;                 // of the teacher's logits
  int32_t gradient;              // 1: z becomes d, in place
  int64_t V, ldv, ld_ids, ld_logits;
  float c;                       // log2(e) / temperature, times gain
  float temperature, inv_temperature;
  float scale;                   // inv_temperature times gain
  const int64_t* ids;            // this chunk's
  const void* logits;
  const float2* partials;
  const float* picked;           // [rows][k]: z of the entries that count (fp32: taken from z)
  void* z;                       // [rows][ldv] fp16 y / fp32 z in, bf16 / fp32 d out
  const uint8_t* live;           // [rows]
  float* token_loss;             // [rows]
  uint32_t* ctrl;                // kCtrlNValid: rows that count
};
cudaError_t launch_distill_rows(const DistillArgs& a, cudaStream_t s);
// which of N rows have an entry, how many (ctrl), and ids out of range (ctrl's error)
cudaError_t launch_distill_live(const int64_t* ids, int64_t ld_ids, const void* logits, int64_t ld_logits, int dtype,
                                int64_t N, int k, int64_t V, uint8_t* live, uint32_t* ctrl, cudaStream_t s);

// A chunk's rows before their product: a copy of x whose rows that do not count are
// zero (xm not null), and the columns to pick (parts not null; ScoreGemmArgs)
struct DistillPrepareArgs {
  int32_t rows, k, dtype, num_tiles;
  int64_t row_bytes, ld_ids, ld_logits;
  const void* x;
  void* xm;
  const int64_t* ids;
  const void* logits;
  const uint8_t* live;
  uint2* parts;
  int2* entries;
};
cudaError_t launch_distill_prepare(const DistillPrepareArgs& a, cudaStream_t s);
cudaError_t launch_distill_finish(const float* token_loss, int64_t N, const uint32_t* ctrl, float* loss,
                                  uint32_t* host_error, cudaStream_t s);

}  // namespace flce
