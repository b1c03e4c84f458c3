// AdamW over a list of tensors in one launch, states in 32 bits or in 8.
//
//   m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2,
//   p' = p - lr (m'/c1 / (sqrt(v'/c2) + eps) + wd p),  c_i = 1 - b_i^t
//
// Every element is independent, so the step is bound by DRAM: parameter,
// gradient and states are read and written once.  A chunk of 2048 elements
// goes to a block of 8 warps, 8 consecutive elements to a thread; a warp
// then holds exactly one 256-element block of the 8-bit states, whose new
// scale is one warp-wide maximum (redux.sync on the bits of the magnitudes,
// which order as the values do, NaN on top), and no value leaves registers.
// The tensors' descriptors are kernel arguments: nothing is copied to the
// device, and a chunk finds its tensor by bisection in constant memory.
//
// 8-bit states are e4m3 (4 exponent bits, half a step is 2^-4 of the value)
// with the largest of a block at 448.  The second moment is kept as its
// root: e4m3 spans a factor of 2.3e5 below the block's largest, which for
// the root is 5e10 of v; a positive v that would round to zero takes the
// smallest positive value instead, or m / sqrt(v) would have nothing to
// divide by.
#include <cuda_fp8.h>
#include <cmath>

#include "host.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = kThreads * 8;
constexpr float kE4m3Max = 448.0f;
constexpr float kE4m3Least = 0.001953125f;        // 2^-9, the smallest positive e4m3
constexpr unsigned kStateMinBits = 0x0d800000u;   // 2^-100: blocks below hold zeros

struct Tensor {
  void* p;
  const void* g;
  float* master;
  void *m, *v;
  float *ms, *vs;
  int64_t n;
  float lr_mult;
  uint8_t p_bf16, g_bf16, fp8, decay;
  uint8_t wide;            // pointers allow 16-byte accesses
};
struct Args {
  Tensor t[MOE_ADAMW_MAX];
  int64_t first[MOE_ADAMW_MAX + 1];      // first chunk of each tensor; [n] = their number
  int n, last;                           // last: this launch ends the step
  float lr, b1, omb1, b2, omb2, lb1, lb2, eps, wd;
  int32_t* step;
  const float *lr_dev, *grad_scale;
};

__device__ __forceinline__ void load_any(const void* base, int64_t i, int64_t n, bool bf16,
                                         bool whole, float* f) {
  if (bf16) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + i;
    if (whole) { load8(p, f); return; }
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = i + k < n ? __bfloat162float(p[k]) : 0.f;
  } else {
    const float* p = static_cast<const float*>(base) + i;
    if (whole) { load8(p, f); return; }
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = i + k < n ? p[k] : 0.f;
  }
}
__device__ __forceinline__ void store_any(void* base, int64_t i, int64_t n, bool bf16, bool whole,
                                          const float* f) {
  if (bf16) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + i;
    if (whole) { store8(p, f); return; }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < n) p[k] = __float2bfloat16_rn(f[k]);
  } else {
    float* p = static_cast<float*>(base) + i;
    if (whole) { store8(p, f); return; }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < n) p[k] = f[k];
  }
}
__device__ __forceinline__ void load_fp8(const void* base, int64_t i, int64_t n, bool whole,
                                         float scale, float* f) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + i;
  union { uint2 u; __nv_fp8x2_storage_t q[4]; uint8_t b[8]; } w;
  if (whole) {
    w.u = *reinterpret_cast<const uint2*>(p);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) w.b[k] = i + k < n ? p[k] : 0;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(w.q[k], __NV_E4M3)));
    f[2 * k] = v.x * scale;
    f[2 * k + 1] = v.y * scale;
  }
}
__device__ __forceinline__ void store_fp8(void* base, int64_t i, int64_t n, bool whole,
                                          const float* f) {
  uint8_t* p = static_cast<uint8_t*>(base) + i;
  union { uint2 u; __nv_fp8x2_storage_t q[4]; uint8_t b[8]; } w;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w.q[k] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * k], f[2 * k + 1]), __NV_SATFINITE,
                                      __NV_E4M3);
  if (whole) {
    *reinterpret_cast<uint2*>(p) = w.u;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < n) p[k] = w.b[k];
  }
}
// Scale of a block from its largest magnitude's bits, and what its values
// are multiplied by before rounding.  Not finite: everything becomes NaN.
__device__ __forceinline__ float2 block_scale(unsigned bits) {
  if (bits >= 0x7f800000u) return make_float2(__int_as_float(0x7fffffff), 0.f);
  if (bits < kStateMinBits) return make_float2(0.f, 0.f);
  const float big = __uint_as_float(bits);
  return make_float2(big / kE4m3Max, kE4m3Max / big);
}

__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Args a) {
  pdl_begin();
  const int step = a.step[0] + 1;
  // 1 - b^t without cancellation
  const float ic1 = 1.0f / -expm1f((float)step * a.lb1);
  const float ic2 = rsqrtf(-expm1f((float)step * a.lb2));
  const float gs = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
  const float lr0 = a.lr_dev != nullptr ? *a.lr_dev : a.lr;
  const int64_t total = a.first[a.n];
  for (int64_t chunk = blockIdx.x; chunk < total; chunk += gridDim.x) {
    int lo = 0, hi = a.n;                  // the last tensor with first <= chunk
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.first[mid] <= chunk) lo = mid; else hi = mid;
    }
    const Tensor& t = a.t[lo];
    const int64_t n = t.n;
    const int64_t i = (chunk - a.first[lo]) * kChunk + threadIdx.x * 8;
    const bool whole = t.wide && i + 8 <= n;
    const float lr = lr0 * t.lr_mult, wd = t.decay ? a.wd : 0.f;
    float p[8], g[8], m[8], v[8];
    const int64_t blk = i / MOE_ADAMW_BLOCK;
    const bool some = i < n;
    load_any(t.g, i, n, t.g_bf16, whole, g);
    if (t.master != nullptr) load_any(t.master, i, n, false, whole, p);
    else load_any(t.p, i, n, t.p_bf16, whole, p);
    if (t.fp8) {
      load_fp8(t.m, i, n, whole, some ? t.ms[blk] : 0.f, m);
      load_fp8(t.v, i, n, whole, some ? t.vs[blk] : 0.f, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= v[k];
    } else {
      load_any(t.m, i, n, false, whole, m);
      load_any(t.v, i, n, false, whole, v);
    }
    float root[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float gk = g[k] * gs;
      m[k] = fmaf(a.b1, m[k], a.omb1 * gk);
      v[k] = fmaf(a.b2, v[k], a.omb2 * gk * gk);
      root[k] = sqrtf(v[k]);
      const float up = (m[k] * ic1) / fmaf(root[k], ic2, a.eps);
      p[k] = fmaf(-lr, fmaf(wd, p[k], up), p[k]);
    }
    store_any(t.p, i, n, t.p_bf16, whole, p);
    if (t.master != nullptr) store_any(t.master, i, n, false, whole, p);
    if (t.fp8) {
      unsigned bm = 0, bv = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (!whole && i + k >= n) continue;
        bm = max(bm, __float_as_uint(m[k]) & 0x7fffffffu);
        bv = max(bv, __float_as_uint(root[k]) & 0x7fffffffu);
      }
      const float2 sm = block_scale(__reduce_max_sync(0xffffffffu, bm));
      const float2 sv = block_scale(__reduce_max_sync(0xffffffffu, bv));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        m[k] *= sm.y;
        const float s = root[k] * sv.y;
        root[k] = s > 0.f && s < kE4m3Least ? kE4m3Least : s;
      }
      store_fp8(t.m, i, n, whole, m);
      store_fp8(t.v, i, n, whole, root);
      if ((threadIdx.x & 31) == 0 && some) {
        t.ms[blk] = sm.x;
        t.vs[blk] = sv.x;
      }
    } else {
      store_any(t.m, i, n, false, whole, m);
      store_any(t.v, i, n, false, whole, v);
    }
  }
  // the block that comes last counts the step: all have read the old count
  if (a.last) {
    __syncthreads();
    if (threadIdx.x == 0 && atomicAdd(a.step + 1, 1) == (int)gridDim.x - 1) {
      a.step[0] = step;
      a.step[1] = 0;
    }
  }
}

int describe(const moe_adamw_tensor_t& t, Tensor* o) {
  if (t.n < 0 || t.n > (1ll << 40) || t.reserved != 0) return MOE_ERR_ARG;
  if (t.dtype != MOE_FP32 && t.dtype != MOE_BF16) return MOE_ERR_ARG;
  if (t.grad_dtype != MOE_FP32 && t.grad_dtype != MOE_BF16) return MOE_ERR_ARG;
  if (t.state != MOE_STATE_FP32 && t.state != MOE_STATE_FP8) return MOE_ERR_ARG;
  if ((t.decay != 0 && t.decay != 1) || !(t.lr_mult == t.lr_mult)) return MOE_ERR_ARG;
  const bool fp8 = t.state == MOE_STATE_FP8;
  const uintptr_t pb = t.dtype == MOE_BF16 ? 2 : 4, gb = t.grad_dtype == MOE_BF16 ? 2 : 4;
  const uintptr_t sb = fp8 ? 1 : 4;
  if (t.n > 0) {
    if (!t.param || !t.grad || !t.m || !t.v) return MOE_ERR_ARG;
    if (fp8 != (t.m_scale != nullptr) || fp8 != (t.v_scale != nullptr)) return MOE_ERR_ARG;
    if (t.master != nullptr && t.dtype != MOE_BF16) return MOE_ERR_ARG;
    if (host::misaligned(t.param, pb) || host::misaligned(t.grad, gb) ||
        host::misaligned(t.m, sb) || host::misaligned(t.v, sb) || host::misaligned(t.master, 4) ||
        host::misaligned(t.m_scale, 4) || host::misaligned(t.v_scale, 4))
      return MOE_ERR_ARG;
  }
  o->p = t.param; o->g = t.grad; o->master = t.master; o->m = t.m; o->v = t.v;
  o->ms = t.m_scale; o->vs = t.v_scale; o->n = t.n; o->lr_mult = t.lr_mult;
  o->p_bf16 = t.dtype == MOE_BF16; o->g_bf16 = t.grad_dtype == MOE_BF16; o->fp8 = fp8;
  o->decay = (uint8_t)t.decay;
  const uintptr_t st = fp8 ? 8 : 16;
  o->wide = !host::misaligned(t.param, 16) && !host::misaligned(t.grad, 16) &&
            !host::misaligned(t.master, 16) && !host::misaligned(t.m, st) &&
            !host::misaligned(t.v, st);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_adamw(const moe_adamw_config_t* c, const moe_adamw_tensor_t* tensors,
                         int32_t n_tensors, int32_t* step, const float* lr,
                         const float* grad_scale, cudaStream_t s) {
  if (c == nullptr || n_tensors < 0 || (n_tensors > 0 && tensors == nullptr) || step == nullptr)
    return MOE_ERR_ARG;
  if (!(c->beta1 >= 0.0 && c->beta1 < 1.0) || !(c->beta2 >= 0.0 && c->beta2 < 1.0) ||
      !(c->eps > 0.0) || !std::isfinite(c->lr) || !std::isfinite(c->weight_decay))
    return MOE_ERR_ARG;
  if (host::misaligned(step, 4) || host::misaligned(lr, 4) || host::misaligned(grad_scale, 4))
    return MOE_ERR_ARG;
  Args a{};
  // every descriptor is checked before the first launch
  for (int i = 0; i < n_tensors; ++i) MOE_HTRY(describe(tensors[i], &a.t[0]));
  a.lr = (float)c->lr;
  a.b1 = (float)c->beta1; a.omb1 = (float)(1.0 - c->beta1); a.lb1 = (float)std::log(c->beta1);
  a.b2 = (float)c->beta2; a.omb2 = (float)(1.0 - c->beta2); a.lb2 = (float)std::log(c->beta2);
  a.eps = (float)c->eps; a.wd = (float)c->weight_decay;
  a.step = step; a.lr_dev = lr; a.grad_scale = grad_scale;
  int i = 0;
  do {
    a.n = 0;
    int64_t chunks = 0;
    for (; i < n_tensors && a.n < MOE_ADAMW_MAX; ++i) {
      if (tensors[i].n == 0) continue;
      describe(tensors[i], &a.t[a.n]);
      a.first[a.n++] = chunks;
      chunks += host::ceil_div(tensors[i].n, kChunk);
    }
    a.first[a.n] = chunks;
    while (i < n_tensors && tensors[i].n == 0) ++i;
    a.last = i == n_tensors;
    const int grid = (int)std::max<int64_t>(
        1, std::min<int64_t>(chunks, (int64_t)host::sm_count() * (2048 / kThreads)));
    MOE_HTRY(host::launch("adamw", adamw_kernel, grid, kThreads, 0, s, 1, a));
  } while (i < n_tensors);
  return MOE_OK;
}
