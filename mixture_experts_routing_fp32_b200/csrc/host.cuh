// Host side shared by the library's translation units: launch counting,
// per-launch timing and error codes.  The state behind
// these (thread-local) is defined in moe.cu.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <utility>

#include "common.cuh"

namespace moe {
namespace host {

int fail(cudaError_t e);                               // records e, returns MOE_ERR_CUDA
void before_launch(cudaStream_t s);                    // timing event, if enabled
int after_launch(cudaStream_t s, const char* name);    // counts, checks, timing event
bool use_pdl();
int sm_count();                                        // of the current device

#define MOE_HCK(expr)                                          \
  do {                                                         \
    cudaError_t e__ = (expr);                                  \
    if (e__ != cudaSuccess) return moe::host::fail(e__);       \
  } while (0)
#define MOE_HTRY(expr)               \
  do {                               \
    int r__ = (expr);                \
    if (r__ != MOE_OK) return r__;   \
  } while (0)

// One launch with programmatic stream serialisation (the kernel waits for
// its predecessor itself), counted and timed as the other units' launches.
template <typename... KP, typename... A>
int launch(const char* name, void (*kern)(KP...), dim3 grid, dim3 block, size_t smem,
           cudaStream_t s, int cluster, A&&... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = block;
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (use_pdl()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  lc.attrs = attr;
  lc.numAttrs = n;
  before_launch(s);
  MOE_HCK(cudaLaunchKernelEx(&lc, kern, std::forward<A>(args)...));
  return after_launch(s, name);
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool misaligned(const void* p, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0;
}

}  // namespace host
}  // namespace moe
