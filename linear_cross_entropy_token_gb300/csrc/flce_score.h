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
};

// ---------------------------------------------------- flce_score_gemm.cu

// One product z = x Wt on 256 x 512 tiles of CTA pairs, and what becomes of z.
struct ScoreGemmArgs {
  int32_t num_m, num_n;          // tiles
  int32_t kb_total;              // 64-deep k-blocks
  int32_t rows, cols;            // valid rows; V
  int32_t groups;                // partials per row: ceil(V / 64)
  int32_t store;                 // statistics: also store the scaled logits
  float c;                       // log2(e) / temperature
  float2* partials;              // [rows][groups]: largest z, sum of 2^((z - largest) c)
  float* part_s;                 // [rows][groups]: sum of y 2^y, y = (z - largest) c
  const ScoreRow* row;           // gradient: [rows]
  float* dcorr;                  // gradient: [rows] what rounding took from the target's entry
  uint32_t* ctrl;                // word 0: first error
  uint64_t timeout_ns;
};

// gradient == 0: the statistics, and with `store` y as fp16 [rows][ldv] (o);
// 1: d as bf16 [rows][ldv] (o). a: x (box 64 x 128), b: W (box 64 x 128), o: box 64 x 128
cudaError_t launch_score_gemm(int gradient, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o,
                              const ScoreGemmArgs& args, int pairs, cudaStream_t s);
int score_gemm_max_clusters();

// --------------------------------------------------------- flce_score.cu

// The statistics of fp32 logits, as the product's epilogue takes them.
cudaError_t launch_score_stats_f32(const float* z, int64_t ldv, int rows, int64_t V, int groups, float c,
                                   float2* partials, float* part_s, cudaStream_t s);

struct ScoreRowsArgs {
  int32_t rows, top, groups;
  int32_t bf16;                  // x and W bf16 and z stored as fp16 y, or all fp32
  int64_t H, V, ldv, ignore_index;
  float c, inv_c;                // log2(e) / temperature
  double inv_temperature;
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
  double temperature;
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
                                 int rows, int64_t V, float c, const ScoreRow* row, float* dcorr, cudaStream_t s);

// the gradient at the target's column of fp32 logits that were recomputed: in
// place of launch_score_dlogits with z == d

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
  int64_t H, V, ldv, ld_ids, ld_logits;
  float c;
  double temperature;
  const void* x;                 // this chunk's
  const void* W;
  const int64_t* ids;
  const void* logits;
  const float2* partials;
  void* z;                       // [rows][ldv] fp16 y / fp32 z in, bf16 / fp32 d out
  const uint8_t* live;           // [rows]
  float* token_loss;             // [rows]
  uint32_t* ctrl;                // kCtrlNValid: rows that count
};
cudaError_t launch_distill_rows(const DistillArgs& a, cudaStream_t s);
// which of N rows have an entry, how many (ctrl), and ids out of range (ctrl's error)
cudaError_t launch_distill_live(const int64_t* ids, int64_t ld_ids, const void* logits, int64_t ld_logits, int dtype,
                                int64_t N, int k, int64_t V, uint8_t* live, uint32_t* ctrl, cudaStream_t s);
cudaError_t launch_distill_mask(const void* x, void* xm, const uint8_t* live, int rows, int64_t row_bytes, cudaStream_t s);
cudaError_t launch_distill_finish(const float* token_loss, int64_t N, const uint32_t* ctrl, float* loss,
                                  uint32_t* host_error, cudaStream_t s);

}  // namespace flce
