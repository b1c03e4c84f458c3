// Eight fp32 values at a time in packed pairs.
#pragma once
#include "common.cuh"

namespace moe {

// 8 fp32 values as four register pairs: fma.rn.f32x2 and its like work on a
// pair in one instruction, each half rounded as the scalar form (kernels that
// stream rows through fp32 arithmetic issue close to an instruction per cycle,
// so halving these is what brings them near DRAM's rate).
struct F8 {
  uint64_t p[4];
};
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ F8 zero8f() { return F8{{0ull, 0ull, 0ull, 0ull}}; }
// a * b + c, with b and c one value for all (or a pair of them)
__device__ __forceinline__ F8 fma8(const F8& a, uint64_t b, uint64_t c) {
  return F8{{fma2(a.p[0], b, c), fma2(a.p[1], b, c), fma2(a.p[2], b, c), fma2(a.p[3], b, c)}};
}
__device__ __forceinline__ F8 fma8(const F8& a, uint64_t b, const F8& c) {
  return F8{{fma2(a.p[0], b, c.p[0]), fma2(a.p[1], b, c.p[1]), fma2(a.p[2], b, c.p[2]),
             fma2(a.p[3], b, c.p[3])}};
}
__device__ __forceinline__ F8 fma8(const F8& a, const F8& b, const F8& c) {
  return F8{{fma2(a.p[0], b.p[0], c.p[0]), fma2(a.p[1], b.p[1], c.p[1]),
             fma2(a.p[2], b.p[2], c.p[2]), fma2(a.p[3], b.p[3], c.p[3])}};
}
__device__ __forceinline__ F8 mul8(const F8& a, const F8& b) {
  return F8{{mul2(a.p[0], b.p[0]), mul2(a.p[1], b.p[1]), mul2(a.p[2], b.p[2]),
             mul2(a.p[3], b.p[3])}};
}
__device__ __forceinline__ F8 mul8(const F8& a, uint64_t b) {
  return F8{{mul2(a.p[0], b), mul2(a.p[1], b), mul2(a.p[2], b), mul2(a.p[3], b)}};
}
__device__ __forceinline__ F8 add8(const F8& a, const F8& b) {
  return F8{{add2(a.p[0], b.p[0]), add2(a.p[1], b.p[1]), add2(a.p[2], b.p[2]),
             add2(a.p[3], b.p[3])}};
}
__device__ __forceinline__ F8 add8(const F8& a, uint64_t b) {
  return F8{{add2(a.p[0], b), add2(a.p[1], b), add2(a.p[2], b), add2(a.p[3], b)}};
}
__device__ __forceinline__ float dot8(const F8& a, const F8& b) {
  const float2 f = unpack2(fma2(a.p[3], b.p[3], fma2(a.p[2], b.p[2],
                                fma2(a.p[1], b.p[1], mul2(a.p[0], b.p[0])))));
  return f.x + f.y;
}
__device__ __forceinline__ float sum8(const F8& a) {
  const float2 f = unpack2(add2(add2(a.p[0], a.p[1]), add2(a.p[2], a.p[3])));
  return f.x + f.y;
}
__device__ __forceinline__ F8 widen8(const uint4& u) {
  auto two = [](uint32_t w) {
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  };
  return F8{{two(u.x), two(u.y), two(u.z), two(u.w)}};
}
__device__ __forceinline__ F8 f8_of(const float4& a, const float4& b) {
  return F8{{pack2(a.x, a.y), pack2(a.z, a.w), pack2(b.x, b.y), pack2(b.z, b.w)}};
}
__device__ __forceinline__ F8 load_f8(const __nv_bfloat16* p) {
  return widen8(*reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ F8 load_f8(const float* p) {
  return f8_of(*reinterpret_cast<const float4*>(p), *reinterpret_cast<const float4*>(p + 4));
}
__device__ __forceinline__ void store_f8(float* p, const F8& a) {
  const float2 q0 = unpack2(a.p[0]), q1 = unpack2(a.p[1]), q2 = unpack2(a.p[2]), q3 = unpack2(a.p[3]);
  *reinterpret_cast<float4*>(p) = make_float4(q0.x, q0.y, q1.x, q1.y);
  *reinterpret_cast<float4*>(p + 4) = make_float4(q2.x, q2.y, q3.x, q3.y);
}
__device__ __forceinline__ void store_f8_split(float4* lo, float4* hi, const F8& a) {
  const float2 q0 = unpack2(a.p[0]), q1 = unpack2(a.p[1]), q2 = unpack2(a.p[2]), q3 = unpack2(a.p[3]);
  *lo = make_float4(q0.x, q0.y, q1.x, q1.y);
  *hi = make_float4(q2.x, q2.y, q3.x, q3.y);
}
__device__ __forceinline__ uint4 narrow8(const F8& a) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(a.p[i]);
    h[i] = __floats2bfloat162_rn(f.x, f.y);
  }
  return u;
}
__device__ __forceinline__ void store_f8(__nv_bfloat16* p, const F8& a) {
  *reinterpret_cast<uint4*>(p) = narrow8(a);
}

}  // namespace moe
