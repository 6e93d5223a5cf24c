// The training-step operators' launchers against a stand-in for the CUDA
// runtime with two devices, on the host alone: a kernel's attributes belong to
// one device, and a launch that needs more dynamic shared memory, or a larger
// cluster, than was opted into on the current device is refused. Each launcher
// runs on device 0, then on device 1; prints what was refused.
#include <cstdio>
#include <map>
#include <utility>

#include "flce_train.h"

namespace {
int current = 0;
std::map<std::pair<int, const void*>, int> dynamic_bytes;
std::map<std::pair<int, const void*>, bool> large_clusters;
int launches = 0;

// static shared memory counts towards the default 48 KB: 8 KB is more than any kernel here has
constexpr size_t kDefaultDynamic = (48 - 8) * 1024;

cudaError_t admit(const void* f, size_t smem, unsigned cluster) {
  const auto at = dynamic_bytes.find({current, f});
  const size_t most = at == dynamic_bytes.end() ? kDefaultDynamic : static_cast<size_t>(at->second);
  if (smem > most) return cudaErrorInvalidValue;
  if (cluster > 8 && !large_clusters[{current, f}]) return cudaErrorInvalidClusterSize;
  return cudaSuccess;
}

unsigned cluster_of(const cudaLaunchConfig_t* c) {
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) return c->attrs[i].val.clusterDim.x;
  return 1;
}
}  // namespace

extern "C" {
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute attr, int value) {
  if (attr == cudaFuncAttributeMaxDynamicSharedMemorySize)
    dynamic_bytes[{current, f}] = value;
  else if (attr == cudaFuncAttributeNonPortableClusterSizeAllowed)
    large_clusters[{current, f}] = value != 0;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  ++launches;
  return admit(f, c->dynamicSmemBytes, cluster_of(c));
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* c) {
  const cudaError_t e = admit(f, c->dynamicSmemBytes, cluster_of(c));
  *n = e == cudaSuccess ? 8 : 0;
  return e;
}
// launches with <<<>>>: their error is the next cudaGetLastError's
static cudaError_t last = cudaSuccess;
cudaError_t cudaGetLastError() {
  const cudaError_t e = last;
  last = cudaSuccess;
  return e;
}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* f) {
  *k = reinterpret_cast<cudaKernel_t>(const_cast<void*>(f));
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3, dim3, void**, size_t smem, cudaStream_t) {
  ++launches;
  const cudaError_t e = admit(reinterpret_cast<const void*>(k), smem, 1);
  if (e != cudaSuccess) last = e;
  return e;
}
static dim3 pushed_grid, pushed_block;
static size_t pushed_smem;
static cudaStream_t pushed_stream;
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, cudaStream_t s) {
  pushed_grid = grid, pushed_block = block, pushed_smem = smem, pushed_stream = s;
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* grid, dim3* block, size_t* smem, void* s) {
  *grid = pushed_grid, *block = pushed_block, *smem = pushed_smem;
  *static_cast<cudaStream_t*>(s) = pushed_stream;
  return cudaSuccess;
}
// what the objects register at start-up
void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
}

int main() {
  using namespace flce;
  int refused = 0;
  auto expect = [&](cudaError_t e, const char* what, int i) {
    if (e == cudaSuccess) return;
    std::printf("device %d: %s %d: error %d\n", current, what, i, static_cast<int>(e));
    ++refused;
  };
  for (current = 0; current < 2; ++current) {
    MuonArgs a{};
    a.count = 1;
    a.rows = a.m = 300;
    a.cols = a.n = 600;
    a.norm_blocks = 44;
    a.splits = 1;
    static MuonMaps maps;
    MuonSteps steps{};
    steps.count = 1;
    for (int shape = 0; shape < 3; ++shape) expect(launch_muon_steps(shape, maps, a, steps, 4, nullptr), "muon_steps shape", shape);
    static MuonPairMaps pair_maps;
    expect(launch_muon_steps_pairs(pair_maps, a, steps, 4, nullptr), "muon_steps_pairs", 0);
    expect(launch_muon_momentum(a, nullptr), "muon_momentum", 0);
    expect(launch_muon_prepare(a, 152, nullptr), "muon_prepare", 0);
    if (muon_max_clusters() <= 0) expect(cudaErrorUnknown, "muon_max_clusters", 0);
    for (int chunks = 1; chunks <= 4; ++chunks) {
      a.cluster = 16;
      for (int side : {20, 100}) {   // the products on both parts, and on the high ones
        a.m = side;
        expect(launch_muon_small(a, steps, chunks, nullptr), "muon_small chunks", chunks);
      }
      for (bool pairs : {false, true})
        if (muon_small_clusters(16, chunks, pairs) <= 0) expect(cudaErrorUnknown, "muon_small_clusters", chunks);
    }
    for (int E : {8, 40, 128, 256, 512, 1024})
      for (int64_t N : {100, 100000})
        for (int dtype = 0; dtype < 3; ++dtype) {
          RouteArgs r{};
          const RouteGeometry g = route_geometry(N, E, dtype == 1 ? 4 : 2, 1, false, false, 152);
          r.N = N;
          r.E = E;
          r.k = E < 32 ? E : 32;
          r.documents = 1;
          r.blocks = g.blocks;
          r.rows_per_block = g.rows_per_block;
          r.one_launch = g.one_launch;
          expect(launch_route_forward(dtype, g, r, nullptr), "route_forward", E);
          if (!g.one_launch) expect(launch_route_finish(g, r, nullptr), "route_finish", E);
          const RouteGeometry b = route_geometry(N, E, dtype == 1 ? 4 : 2, 1, true, true, 152);
          r.blocks = b.blocks;
          expect(launch_route_backward(dtype, b, r, nullptr, nullptr, nullptr, nullptr, E, nullptr), "route_backward", E);
        }
  }
  std::printf("%d launches, %d refused\n", launches, refused);
  return refused != 0;
}
