// AdamW over a list of tensors in one launch, states in 32 bits or in 8.
//
//   m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2,
//   p' = p - lr (m'/c1 / (sqrt(v'/c2) + eps) + wd p),  c_i = 1 - b_i^t
//
// Every element is independent, so the step is bound by DRAM: parameter,
// gradient and states are read and written once (10 bytes an element with
// bf16 weights and 8-bit states, 22 with 32-bit ones).  At that rate an
// element may take about 55 instructions, so the arithmetic runs on packed
// pairs, with the hardware's approximate reciprocal and, for 32-bit states,
// root (2^-22 relative, far inside the update's own rounding).  The root
// takes subnormal v: flushed to zero they would leave m' / eps, an update of
// any size where eps is small.  A chunk of 2048 elements goes to a block of 8 warps, 8 consecutive
// elements to a thread; a warp then holds exactly one 256-element block of
// the 8-bit states, whose new scales are warp-wide maxima, and no value
// leaves registers.  The tensors' descriptors
// are kernel arguments: nothing is copied to the device, and a chunk finds
// its tensor by bisection in constant memory.  Tensors of one state kind
// share a launch; parameter, gradient and master types select straight-line
// code per chunk.
//
// 8-bit states are e4m3 (4 exponent bits, half a step is 2^-4 of the value)
// with the largest of a block at 448.  The second moment is kept as its
// root: e4m3 spans a factor of 2.3e5 below the block's largest, which for
// the root is 5e10 of v; a positive v that would round to zero takes the
// smallest positive value instead, or m / sqrt(v) would have nothing to
// divide by.
#include <cuda_fp8.h>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "f32x2.cuh"
#include "host.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = kThreads * 8;
// Blocks that an SM holds (48 and 62 registers a thread), and grids that
// the launch asks for at most: with 32 the hardware evens out what faster
// and slower SMs take (one grid of resident blocks measured 105.8 us on the
// MiniMind-shaped layer's 32-bit states against 90.3, and 834 against 780 us
// on the OLMoE-shaped layer's 8-bit ones; a block per chunk 91 and 960, its
// own start then costs as much as the chunk).
template <bool FP8> constexpr int kPerSm = FP8 ? 5 : 4;
constexpr int kGrids = 32;
constexpr float kE4m3Max = 448.0f;
constexpr float kE4m3Least = 0.001953125f;        // 2^-9, the smallest positive e4m3
constexpr float kStateMin = 7.8886091e-31f;       // 2^-100: blocks below hold zeros

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

// The root: where it is kept in 8 bits the rounded one, else the hardware's
// approximation.
template <bool FP8>
__device__ __forceinline__ float root_of(float v) {
  float d;
  if constexpr (FP8) asm("sqrt.rn.f32 %0, %1;" : "=f"(d) : "f"(v));
  else asm("sqrt.approx.f32 %0, %1;" : "=f"(d) : "f"(v));
  return d;
}
__device__ __forceinline__ float recip(float v) {
  float d;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
  return d;
}
__device__ __forceinline__ F8 widen_fp8(const uint2& u) {
  auto two = [](uint32_t w) {
    const float2 f = __half22float2(__half2(
        __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3)));
    return pack2(f.x, f.y);
  };
  return F8{{two(u.x), two(u.x >> 16), two(u.y), two(u.y >> 16)}};
}
__device__ __forceinline__ uint2 narrow_fp8(const F8& a) {
  auto two = [](uint64_t v) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(unpack2(v), __NV_SATFINITE, __NV_E4M3);
  };
  return make_uint2(two(a.p[0]) | (two(a.p[1]) << 16), two(a.p[2]) | (two(a.p[3]) << 16));
}

// Eight elements of a tensor as they lie in memory.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int64_t n) {
    uint16_t b[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) b[k] = k < n ? __bfloat16_as_ushort(p[k]) : 0;
    u = make_uint4(b[0] | (uint32_t)b[1] << 16, b[2] | (uint32_t)b[3] << 16,
                   b[4] | (uint32_t)b[5] << 16, b[6] | (uint32_t)b[7] << 16);
  }
  __device__ __forceinline__ F8 wide() const { return widen8(u); }
};
template <> struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void load(const float* p, int64_t n) {
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = k < n ? p[k] : 0.f;
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ F8 wide() const { return f8_of(a, b); }
};
template <> struct Raw<uint8_t> {      // e4m3
  uint2 u;
  __device__ __forceinline__ void load(const uint8_t* p) { u = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void load(const uint8_t* p, int64_t n) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) w[k >> 2] |= (uint32_t)p[k] << (8 * (k & 3));
    u = make_uint2(w[0], w[1]);
  }
  __device__ __forceinline__ F8 wide() const { return widen_fp8(u); }
};
// The first n of eight values.
__device__ __forceinline__ void store_part(float* p, const F8& a, int64_t n) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = unpack2(a.p[k]);
    if (2 * k < n) p[2 * k] = f.x;
    if (2 * k + 1 < n) p[2 * k + 1] = f.y;
  }
}
__device__ __forceinline__ void store_part(__nv_bfloat16* p, const F8& a, int64_t n) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = unpack2(a.p[k]);
    if (2 * k < n) p[2 * k] = __float2bfloat16_rn(f.x);
    if (2 * k + 1 < n) p[2 * k + 1] = __float2bfloat16_rn(f.y);
  }
}
__device__ __forceinline__ void store_fp8(uint8_t* p, const uint2& u, bool whole, int64_t n) {
  if (whole) {
    *reinterpret_cast<uint2*>(p) = u;
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) p[k] = (uint8_t)((k < 4 ? u.x : u.y) >> (8 * (k & 3)));
}
// Scale of a block from its largest magnitude, and what its values are
// multiplied by before rounding: fl(448 fl(1 / big)) and fl(big fl(1 / 448)),
// two roundings each, where quotients would take one.  A code is that of the
// quotient 448 v / big unless that lies within 2^-22 (relative) of a border
// between two.  Not finite: everything becomes NaN.
__device__ __forceinline__ float2 block_scale(float big) {
  // (magnitudes order as their bits do, NaN on top)
  big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
  if (!(big < __int_as_float(0x7f800000))) return make_float2(__int_as_float(0x7fffffff), 0.f);
  if (big < kStateMin) return make_float2(0.f, 0.f);
  return make_float2(big * (1.0f / kE4m3Max), __frcp_rn(big) * kE4m3Max);
}
__device__ __forceinline__ float biggest(const F8& a) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = unpack2(a.p[k]);
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(f.x), "f"(f.y));
  }
  return m;
}
__device__ __forceinline__ uint64_t both(float v) { return pack2(v, v); }

__device__ __forceinline__ bool has_zero_byte(uint32_t w) {
  return ((w - 0x01010101u) & ~w & 0x80808080u) != 0u;
}
// a + b, by scalar sums: packed ones are contracted with the products before
// them.
__device__ __forceinline__ F8 add_apart(const F8& a, const F8& b) {
  F8 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = unpack2(a.p[j]), y = unpack2(b.p[j]);
    r.p[j] = pack2(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
  }
  return r;
}

struct Step {           // one step's values, the same for all elements
  float gs, lr;
  // m'/c1 / (sqrt(v'/c2) + eps) = m' / (sqrt(v') root_mul + root_add)
  float root_mul, root_add;
};

// One chunk of tensor t: TP, TG the types of parameter and gradient; MASTER:
// the parameter is rounded from an fp32 copy.
template <bool FP8, typename TP, typename TG, bool MASTER>
__device__ __forceinline__ void run_chunk(const Args& a, const Tensor& t, int64_t i,
                                          const Step& st) {
  using TS = typename std::conditional<FP8, uint8_t, float>::type;
  using TW = typename std::conditional<MASTER, float, TP>::type;
  const TG* gp = static_cast<const TG*>(t.g);
  TW* wp = MASTER ? reinterpret_cast<TW*>(t.master) : static_cast<TW*>(t.p);
  TS *mp = static_cast<TS*>(t.m), *vp = static_cast<TS*>(t.v);
  Raw<TG> rg;
  Raw<TW> rw;
  Raw<TS> rm, rv;
  float ms, vs;
  const uint64_t block = (uint64_t)i / MOE_ADAMW_BLOCK;
  const int64_t left = t.n - i;       // elements from this thread's first on (may be negative)
  const bool whole = t.wide && left >= 8;
  if (whole) {
    rg.load(gp + i);
    rw.load(wp + i);
    rm.load(mp + i);
    rv.load(vp + i);
  } else {
    rg.load(gp + i, left);
    rw.load(wp + i, left);
    rm.load(mp + i, left);
    rv.load(vp + i, left);
  }
  if constexpr (FP8) {
    ms = left > 0 ? t.ms[block] : 0.f;
    vs = left > 0 ? t.vs[block] : 0.f;
  }
  const uint64_t lr = both(-st.lr * t.lr_mult), wd = both(t.decay ? a.wd : 0.f);
  const F8 g = mul8(rg.wide(), both(st.gs));
  F8 m = rm.wide(), v = rv.wide();
  if constexpr (FP8) {
    m = mul8(m, both(ms));
    v = mul8(v, both(vs));
    v = mul8(v, v);
  }
  // For 8-bit states products and sums are rounded apart, as single fp32
  // operations in the formulas' order round them, so that m' and the root
  // that are rounded to 8 bits below (on which later steps depend) do not
  // depend on how they were computed.
  const F8 gm = mul8(g, both(a.omb1)), gv = mul8(mul8(g, both(a.omb2)), g);
  if constexpr (FP8) {
    m = add_apart(mul8(m, both(a.b1)), gm);
    v = add_apart(mul8(v, both(a.b2)), gv);
  } else {
    m = fma8(m, both(a.b1), gm);
    v = fma8(v, both(a.b2), gv);
  }
  F8 root, den;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack2(v.p[j]);
    root.p[j] = pack2(root_of<FP8>(f.x), root_of<FP8>(f.y));
  }
  den = fma8(root, both(st.root_mul), both(st.root_add));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack2(den.p[j]);
    den.p[j] = pack2(recip(f.x), recip(f.y));
  }
  const F8 p = rw.wide();
  const F8 up = fma8(p, wd, mul8(m, den));
  const F8 w = fma8(up, lr, p);
  TP* pp = static_cast<TP*>(t.p);
  if (whole) {
    store_f8(pp + i, w);
    if (MASTER) store_f8(wp + i, w);
  } else {
    store_part(pp + i, w, left);
    if (MASTER) store_part(wp + i, w, left);
  }
  if constexpr (FP8) {
    // elements behind the tensor's end were loaded as zeros and stay zeros
    const float2 sm = block_scale(biggest(m)), sv = block_scale(biggest(root));
    m = mul8(m, both(sm.y));
    root = mul8(root, both(sv.y));
    uint2 qv = narrow_fp8(root);
    // a positive root is never stored as zero (bytes that came out zero, or
    // could have: looked at one by one only where there are such)
    if (has_zero_byte(qv.x) || has_zero_byte(qv.y)) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack2(root.p[j]);
        root.p[j] = pack2(f.x > 0.f ? fmaxf(f.x, kE4m3Least) : f.x,
                          f.y > 0.f ? fmaxf(f.y, kE4m3Least) : f.y);
      }
      qv = narrow_fp8(root);
    }
    store_fp8(mp + i, narrow_fp8(m), whole, left);
    store_fp8(vp + i, qv, whole, left);
    if ((threadIdx.x & 31) == 0 && left > 0) {
      t.ms[block] = sm.x;
      t.vs[block] = sv.x;
    }
  } else if (whole) {
    store_f8(mp + i, m);
    store_f8(vp + i, v);
  } else {
    store_part(mp + i, m, left);
    store_part(vp + i, v, left);
  }
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads, kPerSm<FP8>) adamw_kernel(const __grid_constant__ Args a) {
  __shared__ Step st_s;
  __shared__ int step_s;
  pdl_begin();
  if (threadIdx.x == 0) {
    const int t = a.step[0] + 1;
    step_s = t;
    // 1 - b^t without cancellation
    const float c1 = -expm1f((float)t * a.lb1);
    st_s.root_mul = c1 * rsqrtf(-expm1f((float)t * a.lb2));
    st_s.root_add = c1 * a.eps;
    st_s.gs = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
    st_s.lr = a.lr_dev != nullptr ? *a.lr_dev : a.lr;
  }
  __syncthreads();
  const Step st = st_s;
  const int step = step_s;
  const int64_t total = a.first[a.n];
  int lo = 0;                              // the last tensor with first <= chunk
  for (int64_t chunk = blockIdx.x; chunk < total; chunk += gridDim.x) {
    if (chunk >= a.first[lo + 1]) {
      int hi = a.n;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.first[mid] <= chunk) lo = mid; else hi = mid;
      }
    }
    const Tensor& t = a.t[lo];
    const int64_t i = (chunk - a.first[lo]) * kChunk + threadIdx.x * 8;
    using bf16 = __nv_bfloat16;
    if (t.master != nullptr) {
      if (t.g_bf16) run_chunk<FP8, bf16, bf16, true>(a, t, i, st);
      else run_chunk<FP8, bf16, float, true>(a, t, i, st);
    } else if (t.p_bf16) {
      if (t.g_bf16) run_chunk<FP8, bf16, bf16, false>(a, t, i, st);
      else run_chunk<FP8, bf16, float, false>(a, t, i, st);
    } else {
      if (t.g_bf16) run_chunk<FP8, float, bf16, false>(a, t, i, st);
      else run_chunk<FP8, float, float, false>(a, t, i, st);
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
      !((float)(c->eps * (1.0 - c->beta1)) >= FLT_MIN) || !std::isfinite(c->lr) || !std::isfinite(c->weight_decay))
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
  // launches of up to MOE_ADAMW_MAX tensors of one state kind; the last one
  // counts the step (a list without elements still is a step)
  auto fill = [&](int from, bool fp8) {    // next tensors of a kind; where to go on
    a.n = 0;
    int64_t chunks = 0;
    int i = from;
    for (; i < n_tensors && a.n < MOE_ADAMW_MAX; ++i) {
      if (tensors[i].n == 0 || (tensors[i].state == MOE_STATE_FP8) != fp8) continue;
      describe(tensors[i], &a.t[a.n]);
      a.first[a.n++] = chunks;
      chunks += host::ceil_div(tensors[i].n, kChunk);
    }
    a.first[a.n] = chunks;
    return i;
  };
  auto more = [&](int from, bool fp8) {
    for (int i = from; i < n_tensors; ++i)
      if (tensors[i].n != 0 && (tensors[i].state == MOE_STATE_FP8) == fp8) return true;
    return false;
  };
  for (int kind = 0; kind < 2; ++kind) {
    const bool fp8 = kind == 1;
    int i = 0;
    // the 8-bit kind comes last and ends the step, with nothing to do if
    // there is none of either
    while (more(i, fp8) || (fp8 && i == 0 && !more(0, false))) {
      i = fill(i, fp8);
      a.last = !more(i, fp8) && (fp8 || !more(0, true));
      const int grid = (int)std::max<int64_t>(
          1, std::min<int64_t>(a.first[a.n], (int64_t)host::sm_count() * (fp8 ? kPerSm<true> : kPerSm<false>) * kGrids));
      MOE_HTRY(host::launch("adamw", fp8 ? adamw_kernel<true> : adamw_kernel<false>, grid, kThreads,
                            0, s, 1, a));
      if (a.last) return MOE_OK;
    }
  }
  return MOE_OK;
}
