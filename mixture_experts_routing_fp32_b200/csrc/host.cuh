// Host side shared by the library's translation units: launch counting,
// per-launch timing, error codes and tensor maps.  The state behind
// these (thread-local) is defined in moe.cu.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <algorithm>
#include <cstdint>
#include <utility>

#include "common.cuh"

namespace moe {
namespace host {

int fail(cudaError_t e);                               // records e, returns MOE_ERR_CUDA
void before_launch(cudaStream_t s);                    // timing event, if enabled
int after_launch(cudaStream_t s, const char* name);    // counts, checks, timing event
bool use_pdl();
int sm_count();                                        // of the current device

// 8-bit matrices [n][halves][rows][K] for loads of several 128-byte k blocks
// at once: seen as [n][K / 128][halves][rows][128], 128-byte swizzle, box
// {128, box_rows, box_halves, kb, 1}, which lands in shared memory k block by
// k block, each as its rows of 128 swizzled bytes.  k blocks past K / 128
// read zeros.
int make_map_k(CUtensorMap* m, const void* ptr, int64_t n, int64_t halves, int64_t rows, int64_t K,
               uint32_t box_rows, uint32_t box_halves, uint32_t kb);
// TMA-store targets [rows][cols]: bf16 (64-byte swizzle) or fp32 (128-byte
// swizzle), 32 x 32 boxes.
int make_out_map(CUtensorMap* m, const void* ptr, int64_t rows, int64_t cols, bool fp32);

// Layout facts of a layer configuration (moe_get_sizes's) for the units that
// work on permuted rows.
struct LayerView {
  int64_t rows_max, tiles_max;
  int align, local_experts;
  bool tensor_cores;
};
int layer_view(const moe_config_t* c, LayerView* out);   // MOE_ERR_ARG for an invalid cfg

// The error words of the other units (each has its own copy of the device
// error word): read and cleared by moe_check_status.
int take_i8_error(unsigned* bits);

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

// Raises a kernel's dynamic shared-memory limit, once per device and kernel
// (the call costs as much as a fifth of a launch).
template <typename K>
int allow_smem(K k, int bytes) {
  struct Seen {
    const void* fn;
    uint64_t devices;
  };
  static thread_local Seen seen[64];
  int dev = 0;
  MOE_HCK(cudaGetDevice(&dev));
  const void* fn = reinterpret_cast<const void*>(k);
  Seen& at = seen[(reinterpret_cast<uintptr_t>(fn) >> 4) % 64];
  if (at.fn != fn) at = Seen{fn, 0};
  if (dev < 64 && (at.devices >> dev) & 1) return MOE_OK;
  MOE_HCK(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  if (dev < 64) at.devices |= 1ull << dev;
  return MOE_OK;
}

// Clusters of `size` CTAs of kernel k that the current device holds at once.
template <typename K>
int resident_clusters(K k, int size, int threads, size_t smem, int64_t* out) {
  cudaLaunchConfig_t lc = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.gridDim = dim3(size * (sm_count() / size));
  lc.blockDim = dim3(threads);
  lc.dynamicSmemBytes = smem;
  lc.attrs = attr;
  lc.numAttrs = 1;
  int n = 0;
  MOE_HCK(cudaOccupancyMaxActiveClusters(&n, k, &lc));
  *out = n > 0 ? n : sm_count() / size;
  return MOE_OK;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool misaligned(const void* p, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0;
}

}  // namespace host
}  // namespace moe
