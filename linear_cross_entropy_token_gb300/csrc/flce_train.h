// Declarations of the training-step operators beside the fused loss: expert
// routing with its balance loss, and the orthogonalised momentum update.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/flce.h"

namespace flce {

// ------------------------------------------------------- flce_route.cu

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxK = 32;
constexpr int kRouteThreads = 256;

// Unit u = b + d of the workspace holds what block b saw of document d: since
// consecutive pieces of the token axis move to the next block, the next
// document or both, the sum names a piece uniquely.
struct RouteArgs {
  const void* logits;
  int64_t N, ld;
  int32_t E, k;
  int32_t renormalize;
  int32_t documents;        // >= 1
  const uint8_t* valid;     // [N] or null
  const int64_t* offsets;   // [documents + 1] or null (one document)
  float* weights;           // [N][k]
  int32_t* experts;         // [N][k]
  int64_t* counts;          // [documents][E]
  float2* stats;            // [N]: largest logit m (-inf for a token that routes nowhere), log sum exp(z - m)
  float* slope;             // [documents][E]: E c / (k n_d)
  float* result;            // balance, z, 1 / n, n (int32 bits)
  int64_t rows_per_block;
  int32_t blocks;
  int32_t one_launch;
  // workspace
  float* unit_p;            // [units][E] sums of probabilities
  int32_t* unit_c;          // [units][E] chosen slots
  int32_t* unit_live;       // [units]
  float* unit_z;            // [units] sums of lse^2
  float* terms;             // [documents * chunks] balance terms
  int32_t* doc_live;        // [documents]
  float* doc_z;             // [documents]
  uint32_t* ticket;
};

struct RouteGeometry {
  int lanes;                // lanes per token row
  int per_lane;             // experts per lane
  int64_t rows_per_block;
  int blocks;
  int chunks;               // expert chunks per document in the closing launch
  bool one_launch;          // the forward is one cluster that closes the call itself
};
// with 2-byte elements the most blocks: what the workspace is sized for
RouteGeometry route_geometry(int64_t N, int64_t E, int element_bytes, int64_t documents, bool offsets, bool backward,
                             int num_sms);

cudaError_t launch_route_forward(int dtype, const RouteGeometry& g, const RouteArgs& a, cudaStream_t s);
cudaError_t launch_route_finish(const RouteGeometry& g, const RouteArgs& a, cudaStream_t s);
cudaError_t launch_route_backward(int dtype, const RouteGeometry& g, const RouteArgs& a, const float* d_weights,
                                  const float* d_balance, const float* d_z, void* d_logits, int64_t ldd,
                                  cudaStream_t s);

// -------------------------------------------------------- flce_muon.cu

constexpr int kMuonMaxMats = 32;     // matrices of one launch
constexpr int kMuonNormBlocks = 1024; // partial sums of squares per matrix
// Short sides up to this run their products on both parts of X, A and B: what
// the roundings to fp16 leave falls with the rows over which it spreads, and on few
// rows comes to 1.2e-3 to 3.4e-3 of O (8 x 8 to 32 x 32; with both parts 1e-6). A
// warp's 32 rows, which are then A and B whole; with 128, 128 x 128 took 37 us
// instead of 25 for an error of 1e-3.
constexpr int kMuonPairSide = 32;
static_assert(kMuonPairSide == 32, "A and B are one warp's block");

struct MuonMat {
  const void* grad;
  float* momentum;                   // or null
  void* weight;                      // or null: then `update` is written
  void* update;
  int64_t ld_grad, ld_momentum, ld_weight, ld_update;
};

struct MuonArgs {
  MuonMat mat[kMuonMaxMats];
  int32_t count, rows, cols;         // rows x cols matrices, as the caller holds them
  int32_t m, n;                      // the short and the long side
  int32_t transposed;                // rows > cols: X is the transpose of the update
  int32_t grad_dtype, weight_dtype, update_dtype;
  int32_t vec;                       // 16-byte (bf16: 8-byte) accesses of four elements are aligned
  int32_t flat;                      // and the matrices' rows follow one another without gaps
  int32_t pairs;                     // the results' rows are aligned to two elements
  int32_t nesterov, norm_blocks;
  float beta, one_minus_beta;
  double eps;
  float decay, lr;                   // W = decay W - lr scale O
  float scale;
  // workspace
  uint32_t* ctrl;
  uint32_t* done;                    // [count] finished tile parts of the products so far
  uint32_t* partial;                 // [count] finished parts of the splits of X Xt but the last
  float* sums;                       // fp32 sums of those splits
  int64_t sums_bytes;
  int32_t splits;                    // units per tile of X Xt
  uint32_t* host_error;              // pinned host word: first device-side error
  float2* norm;                      // [count][kMuonNormBlocks]: mantissa, exponent
  float* diag;                       // [count][m]: diagonal of B
  uint16_t* hi[2];                   // [count][m][ldx] fp16, X scaled by 2^12, two buffers
  uint16_t* lo;                      // [count][m][ldx] fp16 remainder of X
  uint16_t* gram;                    // [count][m][lda] fp16, A scaled by 2^12
  uint16_t* poly;                    // [count][m][lda] fp16, B scaled by 2^11, zero diagonal
  uint16_t* gram_lo;                 // [count][m][lda] fp16 remainders of A and B (short sides up to kMuonPairSide)
  uint16_t* poly_lo;
  int64_t ldx, lda;
  uint64_t timeout_ns;
  uint32_t hold;                     // finished parts waited for beyond those there are: 0, but where waits are to run out
  int32_t cluster;                   // small matrices: CTAs per matrix
};

enum MuonTileShape : int { kMuonSingle = 0, kMuonPair = 1, kMuonWide = 2 };

enum MuonPhase : int { kMuonGram = 0, kMuonPoly = 1, kMuonApply = 2, kMuonLast = 3 };

// All steps' coefficients, for the kernel that runs them in one launch
struct MuonSteps {
  int32_t count;
  float c[FLCE_MUON_MAX_STEPS][3];
};

struct MuonStep {
  float a, b, c;                     // X = aX + (bA + cA^2) X
};

// TMA descriptors of the products: X (either buffer) as K-major operand and as
// right operand of B X, A and B as K-major operands, and what the epilogues
// read and write in boxes of 32 x 32: X hi, X lo, A, B and the mirror images
// of A and B. Step k reads X from buffer k % 2 and writes it to the other.
struct MuonMaps {
  CUtensorMap xk[2], xn[2], xe[2], lo, gk, ge, gm, pk, pe, pm;
};
// and, where the products run on both parts, X lo as either operand, and the
// remainders of A and B as operand and as block
struct MuonPairMaps : MuonMaps {
  CUtensorMap lk, ln, glk, gle, plk, ple;
};

cudaError_t launch_muon_momentum(const MuonArgs& a, cudaStream_t s);
cudaError_t launch_muon_prepare(const MuonArgs& a, int sms, cudaStream_t s);
// All steps on tiles of one shape (slots: CTA pairs that fit at once, or SMs
// for single tiles); muon_plan picks it and a.splits.
cudaError_t launch_muon_steps(int shape, const MuonMaps& maps, const MuonArgs& a, const MuonSteps& steps, int slots,
                              cudaStream_t s);
// on single tiles, for short sides up to kMuonPairSide
cudaError_t launch_muon_steps_pairs(const MuonPairMaps& maps, const MuonArgs& a, const MuonSteps& steps, int slots,
                                    cudaStream_t s);
constexpr int kMuonMaxSplits = 8, kMuonMinSplitBlocks = 8;   // and the k-blocks of a split at least
struct MuonPlan {
  int shape = -1, splits = 1;
};
MuonPlan muon_plan(const MuonArgs& a, int fixed_shape, int pairs, int sms);
int muon_max_clusters();

// flce_muon_small.cu: matrices whose short side is at most 128, one launch
// (long side at most 4096). The least CTAs per matrix (0: not such a shape),
// 64-column chunks of a CTA's slab, clusters that fit the device at once
// (pairs: of the kernel for short sides up to kMuonPairSide).
int muon_small_cluster(int64_t m, int64_t n);
int muon_small_chunks(int64_t n, int cluster);
int muon_small_clusters(int cluster, int chunks, bool pairs);
cudaError_t launch_muon_small(const MuonArgs& a, const MuonSteps& steps, int chunks, cudaStream_t s);

}  // namespace flce
