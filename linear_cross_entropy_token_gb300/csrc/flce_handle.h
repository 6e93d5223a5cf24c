// The library handle and the host helpers that every entry point uses: error
// text, per-kernel timing, the launch macro and TMA descriptor encoding.
#pragma once
#include <cudaTypedefs.h>

#include <array>
#include <cstdarg>
#include <cstdio>
#include <map>
#include <mutex>
#include <string>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "../../include/flce.h"
#include "flce_internal.h"

namespace flce {

constexpr int64_t kMaxDim = (1ll << 31) - 1;
constexpr uint64_t kAlign = 1024;
inline uint64_t align_up(uint64_t v, uint64_t a) { return (v + a - 1) / a * a; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tile shapes of one GEMM launch
enum Shape : int { kShapeSingle = 0, kShapePair = 1, kShapeWide = 2 };

// ------------------------------------------------------------ driver entry

inline PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
inline std::once_flag g_encode_once;

inline bool get_encode() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode != nullptr;
}

// --------------------------------------------------------------- profiling

struct EventPair {
  cudaEvent_t start = nullptr, stop = nullptr;
  int kind = 0;
  double flops = 0, bytes = 0;
};

struct Profiler {
  bool enabled = false;
  std::vector<EventPair> pool;
  size_t used = 0;
  flce_kernel_profile totals[FLCE_K_NUM_KINDS] = {};
};

}  // namespace flce

// ------------------------------------------------------------------ handle

struct flce_handle_s {
  flce_config cfg{};
  int device = 0;
  int num_sms = 0;
  int pair_clusters = 0;  // clusters of two the pair kernels fit at once
  int wide_clusters = 0;  // clusters of two the wide kernels fit at once
  std::map<std::array<int, 3>, int> muon_small;  // clusters (size, chunks, kernel) that fit at once
  int muon_shape = -1;    // tile shape of the muon products (created with FLCE_CTA_AUTO: picked by size)
  int score_clusters = 0; // pairs of the head's operators that fit at once (0: not asked yet)
  int muon_clusters = 0;  // clusters of two the muon kernels fit at once (0: not asked yet)
  // tile shape of the handle's GEMMs; an AUTO handle (cfg.cta_pair stays
  // FLCE_CTA_AUTO) runs each GEMM on the shape its plan names, wide or pair
  int shape = flce::kShapeSingle;
  uint64_t timeout_ns = 0;
  std::string err;
  // workspace
  void* ws = nullptr;
  uint64_t ws_bytes = 0;
  bool ws_external = false;
  bool ws_fresh = true;  // the control block, sticky word included, needs zeroing
  // staging for the host-buffer entry point
  void* stage = nullptr;
  uint64_t stage_bytes = 0;
  uint32_t* host_ctrl = nullptr;  // pinned
  // pipelined host-buffer entry: two staging slots, copies on their own stream
  struct Slot {
    void* stage = nullptr;
    uint64_t bytes = 0;
    cudaEvent_t copied = nullptr;  // the slot's inputs have landed (copy stream)
    cudaEvent_t freed = nullptr;   // the call that read the slot has finished with it
    cudaEvent_t done = nullptr;    // the call's control words are in host memory
    uint32_t* host = nullptr;      // pinned copy of the control words
    uint64_t ticket = 0;
    bool pending = false;
  };
  Slot slots[2];
  cudaStream_t copy_stream = nullptr;
  // SLABS: the dW GEMM of a slab runs on a second stream beside the dx GEMM
  // of the same slab, so each fills the other's last wave
  cudaStream_t side_stream = nullptr;
  cudaEvent_t slab_ready = nullptr;  // the slab's dlogits are in the buffer
  cudaEvent_t slab_freed = nullptr;  // the slab's dW GEMM has read the buffer
  uint64_t next_ticket = 1;
  flce_plan last_plan{};
  int64_t last_N = -1;
  uint64_t token_loss_off = 0;
  bool has_plan = false;
  int64_t launches = 0;
  flce::Profiler prof;
  std::map<std::array<int, 5>, int> group_cache;  // pick_group_m by (shape, num_m, num_n, num_s, slots)
  // the plan of the last sizes planned (a training loop repeats them)
  std::array<int64_t, 4> plan_key{-1, -1, -1, -1};
  flce_plan plan_cached{};
};

namespace flce {

inline flce_status fail(flce_handle_t h, flce_status st, const char* fmt, ...) {
  if (h) {
    char b[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(b, sizeof b, fmt, ap);
    va_end(ap);
    h->err = b;
  }
  return st;
}

// Word of the handle's pinned memory where the head's operators record a
// device-side error (kCtrlSticky is the training-step operators').
constexpr int kHostScoreError = 14;

// flce_api.cu: what other operators' launches need too
bool map_bf16_2d(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t row_bytes, uint32_t box_inner,
                 uint32_t box_outer, std::string* why);
bool map_f32_3d(CUtensorMap* m, void* base, uint64_t cols, uint64_t rows, uint64_t planes, uint64_t row_bytes,
                uint64_t plane_bytes, std::string* why);
int group_for(flce_handle_t h, int shape, int num_m, int num_n, int num_s, int slots);

struct DeviceGuard {
  int prev = -1;
  explicit DeviceGuard(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != dev) cudaSetDevice(dev);
  }
  ~DeviceGuard() {
    int cur = -1;
    if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
  }
};

inline void prof_begin(flce_handle_t h, int kind, cudaStream_t s) {
  if (!h->prof.enabled) return;
  Profiler& p = h->prof;
  if (p.used == p.pool.size()) {
    EventPair e;
    cudaEventCreate(&e.start);
    cudaEventCreate(&e.stop);
    p.pool.push_back(e);
  }
  EventPair& e = p.pool[p.used];
  e.kind = kind;
  cudaEventRecord(e.start, s);
}

inline void prof_end(flce_handle_t h, cudaStream_t s, double flops, double bytes) {
  if (!h->prof.enabled) return;
  Profiler& p = h->prof;
  EventPair& e = p.pool[p.used];
  e.flops = flops;
  e.bytes = bytes;
  cudaEventRecord(e.stop, s);
  ++p.used;
}

// NVTX range over the host-side enqueue of a call, a chunk or a launch, so a
// timeline profiler can attribute the GPU work to the path's steps. Costs a
// few nanoseconds when no profiler is attached.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

#define FLCE_LAUNCH(kind, flops, bytes, expr)                                                \
  do {                                                                                      \
    NvtxRange nvtx_(flce_kernel_name(kind));                                                \
    prof_begin(h, (kind), s);                                                               \
    cudaError_t e_ = (expr);                                                                \
    prof_end(h, s, (flops), (bytes));                                                       \
    ++h->launches;                                                                          \
    if (e_ != cudaSuccess)                                                                  \
      return fail(h, FLCE_ERR_CUDA, "%s: %s", flce_kernel_name(kind), cudaGetErrorString(e_)); \
  } while (0)

inline bool encode_map(CUtensorMap* m, CUtensorMapDataType dt, int esize, const void* base, int rank,
                const uint64_t* dims, const uint64_t* strides_bytes, const uint32_t* box,
                std::string* why, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  if (!get_encode()) {
    *why = "cuTensorMapEncodeTiled is not available from the driver";
    return false;
  }
  cuuint64_t gd[3], gs[2];
  cuuint32_t bx[3], es[3] = {1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    gd[i] = dims[i];
    bx[i] = box[i];
  }
  for (int i = 0; i < rank - 1; ++i) gs[i] = strides_bytes[i];
  (void)esize;
  CUresult r = g_encode(m, dt, static_cast<cuuint32_t>(rank), const_cast<void*>(base), gd, gs, bx, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    char b[160];
    std::snprintf(b, sizeof b, "cuTensorMapEncodeTiled failed (%d), rank %d, dims %llu x %llu", int(r),
                  rank, static_cast<unsigned long long>(dims[0]),
                  static_cast<unsigned long long>(dims[1]));
    *why = b;
    return false;
  }
  return true;
}

}  // namespace flce
