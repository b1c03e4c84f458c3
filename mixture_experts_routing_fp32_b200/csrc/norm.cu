// The norms around a block, fused with its gate and residual scale: forward
// and backward.  With N(v) = (v - mean) * rstd (mean = 0 for RMSNorm),
//
//   z = N(y) w_post + b_post,  r' = r + alpha gate z,  x = N(r') w_pre + b_pre
//
// and, with yh = N(y), rh = N(r'), <.> the mean over the row, L = 1 for
// LayerNorm and 0 for RMSNorm,
//
//   u  = dx w_pre;   d  = dr' + rstd_r (u - L<u> - rh <u rh>)    (= dr)
//   e  = alpha gate d w_post;   dy = rstd_y (e - L<e> - yh <e yh>)
//   dw_pre = sum_t dx rh,  db_pre = sum_t dx,
//   dw_post = alpha sum_t gate d yh,  db_post = alpha sum_t gate d,
//   dgate_g = alpha (w_post sum_{t in g} d yh + b_post sum_{t in g} d).
//
// Both directions are bound by DRAM: every tensor of T rows is read or
// written once (2 reads and 2 writes forward, 4 and 2 backward), so the
// kernels keep one row in registers (8 columns per thread, a row per group
// of D/8 threads) and stream the next rows into shared memory with cp.async.
// Each thread copies exactly the 16-byte pieces that it reads back itself,
// so the ring needs no barrier; the only ones are those of the row sums.
#include <type_traits>

#include "host.cuh"

namespace moe {
namespace {

constexpr int kMaxD = 8192;          // 1024 threads of 8 columns
constexpr int kMaxThreads = 1024;
constexpr int kSms = 148;            // the backward's partial sums are sized for this grid
constexpr size_t kSmemLimit = 227 * 1024;

struct NormArgs {
  int T, D, nv, tpr, R, stages;      // nv = D / 8; tpr threads a row, R rows at once in a CTA
  int layer, gate_len;
  float eps, alpha, inv_d;
  const void* r;                     // forward: r; backward: r_out
  const void* y;
  const float *w_post, *b_post, *gate, *w_pre, *b_pre;
  void *r_out, *x;
  float* stats;
  const float* stats_in;             // backward from here on
  const void *dx, *dr_out;
  void *dy, *dr;
  float* dgate;
  float* part;                       // partial column sums, kSlots arrays of [P][D]
  int several;                       // gate rows change inside the batch
};

// Partial column sums a CTA leaves (arrays of [P][D] floats in this order).
// One gate row or none: S1, S2, P1, P2 alone.
enum { S1H = 0, S2H = 1, P1 = 2, P2 = 3, S1T = 4, S2T = 5, W1 = 6, W2 = 7 };

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits until at most n (0..3) of this thread's newest groups are in flight.
__device__ __forceinline__ void cp_wait(int n) {
  if (n >= 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// A thread's 8 columns of one tensor: 16 bytes (bf16) or 32 (fp32).
template <typename T> constexpr int kPiece = 8 * (int)sizeof(T);

// Copies the piece to this thread's slot: 16-byte chunk c of thread t sits
// at (c * threads + t) * 16, so neighbouring threads use neighbouring banks.
template <typename T>
__device__ __forceinline__ void fetch(uint32_t slot, int pitch, const T* p) {
  cp16(slot, p);
  if constexpr (sizeof(T) == 4) cp16(slot + pitch, p + 4);
}
template <typename T>
__device__ __forceinline__ void take(const uint8_t* slot, int pitch, float* f);
template <>
__device__ __forceinline__ void take<__nv_bfloat16>(const uint8_t* slot, int, float* f) {
  bf16x8_to_f32(*reinterpret_cast<const uint4*>(slot), f);
}
template <>
__device__ __forceinline__ void take<float>(const uint8_t* slot, int pitch, float* f) {
  const float4 a = *reinterpret_cast<const float4*>(slot);
  const float4 b = *reinterpret_cast<const float4*>(slot + pitch);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// The rounded values of 8 columns (what a reader of the stored row sees).
__device__ __forceinline__ void round8(const __nv_bfloat16*, float* f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __bfloat162float(__float2bfloat16_rn(f[i]));
}
__device__ __forceinline__ void round8(const float*, float*) {}

// Sums of a and b over the tpr threads of a row group (all get them, in the
// same order).  `buf` alternates, so one barrier per sum is enough: a warp
// still reading one buffer is behind the barrier of the next sum, which
// writes the other.
struct RowSum {
  float2* red;      // [2][32] of this row group
  int warps, warp, lane, bar, tpr, buf;
  __device__ __forceinline__ float2 operator()(float a, float b) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (warps == 1) return make_float2(a, b);
    if (lane == 0) red[buf * 32 + warp] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(tpr) : "memory");
    const float2 v = lane < warps ? red[buf * 32 + lane] : make_float2(0.f, 0.f);
    buf ^= 1;
    return make_float2(warp_sum(v.x), warp_sum(v.y));
  }
  __device__ __forceinline__ float operator()(float a) {
    a = warp_sum(a);
    if (warps == 1) return a;
    if (lane == 0) red[buf * 32 + warp] = make_float2(a, 0.f);
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(tpr) : "memory");
    const float v = lane < warps ? red[buf * 32 + lane].x : 0.f;
    buf ^= 1;
    return warp_sum(v);
  }
};

// mean and rstd of a row held 8 values a thread (zeros in idle threads).
// The variance is that of the centred values (a second sum), so a mean that
// is large against the spread costs no digits.
__device__ __forceinline__ float2 moments(const float* v, bool active, const NormArgs& a,
                                          RowSum& sum) {
  float mean = 0.f;
  if (a.layer) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
    mean = sum(s) * a.inv_d;
  }
  float q = 0.f;
  if (active) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = v[i] - mean;
      q = fmaf(d, d, q);
    }
  }
  return make_float2(mean, rsqrtf(sum(q) * a.inv_d + a.eps));
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <typename TA, typename TR>
__global__ void __launch_bounds__(kMaxThreads) block_norm_kernel(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 red_s[16 * 64];
  const int tid = threadIdx.x;
  const int g = tid / a.tpr, vec = tid - g * a.tpr;
  const bool active = vec < a.nv;
  const int c0 = active ? vec * 8 : 0;
  RowSum sum{red_s + g * 64, a.tpr >> 5, vec >> 5, tid & 31, 1 + g, a.tpr, 0};
  const int pitch = blockDim.x * 16;
  constexpr int kChunks = (kPiece<TA> + kPiece<TR>) / 16;
  const int stage_bytes = kChunks * pitch;
  const int r_off = (kPiece<TA> / 16) * pitch;
  uint8_t* mine = ring + tid * 16;
  const uint32_t mine_a = smem_addr(mine);
  const TA* y = static_cast<const TA*>(a.y);
  const TR* r = static_cast<const TR*>(a.r);
  const int step = gridDim.x * a.R;
  pdl_begin();

  int ahead = blockIdx.x * a.R + g, slot_in = 0;
  auto issue = [&] {
    if (ahead < a.T && active) {
      const uint32_t s = mine_a + slot_in * stage_bytes;
      const int64_t at = (int64_t)ahead * a.D + c0;
      if (y != nullptr) fetch<TA>(s, pitch, y + at);
      fetch<TR>(s + r_off, pitch, r + at);
    }
    cp_commit();
    ahead += step;
    if (++slot_in == a.stages) slot_in = 0;
  };
  for (int i = 0; i < a.stages - 1; ++i) issue();
  int slot = 0;
  for (int t = blockIdx.x * a.R + g; t < a.T; t += step) {
    issue();
    cp_wait(a.stages - 1);
    float v[8], z[8];
    const uint8_t* from = mine + slot * stage_bytes;
    if (++slot == a.stages) slot = 0;
    if (active) {
      take<TR>(from + r_off, pitch, v);
      if (y != nullptr) take<TA>(from, pitch, z);
    }
    if (!active || y == nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = 0.f;
    }
    if (!active) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
    const int64_t at = (int64_t)t * a.D + c0;
    float2 my = make_float2(0.f, 1.f), mr = make_float2(0.f, 1.f);
    if (y != nullptr) {
      if (a.w_post != nullptr) {
        my = moments(z, active, a, sum);
        float w[8];
        load8(a.w_post + c0, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = (z[i] - my.x) * my.y * w[i];
        if (a.b_post != nullptr) {
          load8(a.b_post + c0, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] += w[i];
        }
      }
      if (a.gate_len > 0) {
        float w[8];
        load8(a.gate + (int64_t)(t / a.gate_len) * a.D + c0, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] *= w[i];
      }
      if (active) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fmaf(a.alpha, z[i], v[i]);
        TR* out = static_cast<TR*>(a.r_out) + at;
        store8(out, v);
        // the second norm reads the stream as it is stored: the backward
        // then sees the same values
        round8(out, v);
      }
    }
    if (a.w_pre != nullptr) {
      mr = moments(v, active, a, sum);
      if (active) {
        float w[8];
        load8(a.w_pre + c0, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (v[i] - mr.x) * mr.y * w[i];
        if (a.b_pre != nullptr) {
          load8(a.b_pre + c0, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += w[i];
        }
        store8(static_cast<TA*>(a.x) + at, v);
      }
    }
    if (a.stats != nullptr && vec == 0)
      *reinterpret_cast<float4*>(a.stats + 4 * (int64_t)t) = make_float4(my.x, my.y, mr.x, mr.y);
  }
  cp_wait(0);
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// First row of CTA p of P (even split).
__device__ __forceinline__ int first_row(int T, int p, int P) {
  return (int)((int64_t)T * p / P);
}

// The column sums over tokens stay in registers while a CTA walks its rows
// (8 columns a thread: sums of d yh and dx rh, with BIAS also of d and dx)
// and leave as one partial per CTA, which block_norm_sum_kernel adds up in
// CTA order.  When gate rows change inside the batch (`several`), the rows
// run in segments of one gate row: at a segment's end its sums of d yh and d
// give dgate (complete segments are written here, those cut by a CTA's ends
// go out as partials) and, times the gate, add to the CTA's sums for w_post,
// which live in shared memory.  R row groups of a CTA add up through shared
// memory at a segment's end, in group order.
//
// A row of 7168 columns leaves one CTA of 28 warps per SM, so what a row
// waits for is not hidden by other rows: the vectors (w_pre, and alpha gate
// w_post as one) sit in shared memory in the ring's layout, the row's
// statistics are loaded a row ahead, and a tensor's values are taken from
// the ring only where they are used (64 registers hold 16 sums and 24
// values).
template <typename TA, typename TR, bool BIAS>
__global__ void __launch_bounds__(kMaxThreads) block_norm_bwd_kernel(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 red_s[16 * 64];
  const int tid = threadIdx.x;
  const int g = tid / a.tpr, vec = tid - g * a.tpr;
  const bool active = vec < a.nv;
  const int c0 = active ? vec * 8 : 0;
  RowSum sum{red_s + g * 64, a.tpr >> 5, vec >> 5, tid & 31, 1 + g, a.tpr, 0};
  const int pitch = blockDim.x * 16;
  constexpr int kA = kPiece<TA> / 16, kR = kPiece<TR> / 16;
  const int stage_bytes = 2 * (kA + kR) * pitch;
  const int o_dx = kA * pitch, o_r = 2 * kA * pitch, o_g = (2 * kA + kR) * pitch;
  uint8_t* mine = ring + tid * 16;
  const uint32_t mine_a = smem_addr(mine);
  // after the ring: this thread's 8 columns of w_pre and of alpha gate w_post,
  // [2][D] running sums for w_post, b_post (several), and one [R][8 tpr]
  // exchange buffer (R > 1)
  uint8_t* v_pre = mine + a.stages * stage_bytes;
  uint8_t* v_post = v_pre + 2 * pitch;
  constexpr int kW = BIAS ? 2 : 1;
  float* w_sum = reinterpret_cast<float*>(ring + a.stages * stage_bytes + 4 * pitch);
  float* swap = w_sum + (a.several ? kW * a.D : 0);
  const TA* y = static_cast<const TA*>(a.y);
  const TA* dx = static_cast<const TA*>(a.dx);
  const TR* r = static_cast<const TR*>(a.r);
  const TR* gin = static_cast<const TR*>(a.dr_out);
  const int P = gridDim.x, p = blockIdx.x;
  const int row0 = first_row(a.T, p, P), row1 = first_row(a.T, p + 1, P);
  const int64_t arr = (int64_t)P * a.D;             // floats of one partial array
  float* part = a.part + (int64_t)p * a.D + c0;

  if (a.several && active && g == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      for (int k = 0; k < kW; ++k) w_sum[k * a.D + c0 + i] = 0.f;
  }
  pdl_begin();

  // idle threads of a row's last warp hold zeros in both vectors and in
  // every tensor they weight, so they add nothing to the row's sums
  auto keep = [&](uint8_t* at, const float* f) {
    *reinterpret_cast<float4*>(at) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(at + pitch) = make_float4(f[4], f[5], f[6], f[7]);
  };
  {
    float w[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (active && a.w_pre != nullptr) load8(a.w_pre + c0, w);
    keep(v_pre, w);
  }

  // rows of a segment: [seg0, seg1), row group g takes seg0 + g, + R, ...
  const int L = a.several ? a.gate_len : a.T;
  auto seg_end = [&](int row) {
    return a.several ? (int)min((int64_t)row1, (int64_t)(row / L + 1) * L) : row1;
  };
  // this row group's first row in the segments from s0 on (row1: none)
  auto first_in = [&](int s0) {
    while (s0 < row1) {
      const int e = seg_end(s0);
      if (s0 + g < e) return s0 + g;
      s0 = e;
    }
    return row1;
  };
  auto next_row = [&](int t) {
    const int e = seg_end(t);
    return t + a.R < e ? t + a.R : first_in(e);
  };
  int ahead = first_in(row0), slot_in = 0;
  auto issue = [&] {
    if (a.stages == 0) return;
    if (ahead < row1) {
      if (active) {
        const uint32_t s = mine_a + slot_in * stage_bytes;
        const int64_t at = (int64_t)ahead * a.D + c0;
        if (y != nullptr) fetch<TA>(s, pitch, y + at);
        if (dx != nullptr) {
          fetch<TA>(s + o_dx, pitch, dx + at);
          fetch<TR>(s + o_r, pitch, r + at);
        }
        if (gin != nullptr) fetch<TR>(s + o_g, pitch, gin + at);
      }
      ahead = next_row(ahead);
    }
    cp_commit();
    if (++slot_in == a.stages) slot_in = 0;
  };
  float s1[8], p1[8], s2[BIAS ? 8 : 1], p2[BIAS ? 8 : 1];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s1[i] = p1[i] = 0.f;
    if constexpr (BIAS) s2[i] = p2[i] = 0.f;
  }
  // sum of v over the row groups, in group order (in group 0's threads)
  auto join = [&](float* v) {
    if (a.R == 1) return;
    __syncthreads();
    float* at = swap + (g * a.tpr + vec) * 8;
    store8(at, v);
    __syncthreads();
    if (g == 0) {
      for (int k = 1; k < a.R; ++k) {
        float o[8];
        load8(swap + (k * a.tpr + vec) * 8, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += o[i];
      }
    }
  };

  const float4* stats = reinterpret_cast<const float4*>(a.stats_in);
  float4 st_next = make_float4(0.f, 0.f, 0.f, 0.f);
  if (ahead < row1) st_next = stats[ahead];
  for (int i = 0; i < a.stages - 1; ++i) issue();
  int slot = 0;
  for (int seg0 = row0; seg0 < row1;) {
    const int seg1 = seg_end(seg0);
    const float* gate = a.gate_len > 0 ? a.gate + (int64_t)(seg0 / a.gate_len) * a.D + c0 : nullptr;
    if (y != nullptr) {
      float w[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (active) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = a.alpha;
        float o[8];
        if (gate != nullptr) {
          load8(gate, o);
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] *= o[i];
        }
        if (a.w_post != nullptr) {
          load8(a.w_post + c0, o);
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] *= o[i];
        }
      }
      keep(v_post, w);
    }
    for (int t = seg0 + g; t < seg1; t += a.R) {
      issue();
      const float4 st = st_next;
      const int tn = next_row(t);
      if (tn < row1) st_next = stats[tn];
      const int64_t at = (int64_t)t * a.D + c0;
      const uint8_t* from = mine + slot * stage_bytes;
      if (a.stages > 0) {
        cp_wait(a.stages - 1);
        if (++slot == a.stages) slot = 0;
      }
      // this thread's columns of one tensor (rows that fit no ring: from
      // global memory)
      auto get = [&](auto* base, int off, float* f) {
        using T = std::remove_cv_t<std::remove_pointer_t<decltype(base)>>;
        if (a.stages > 0) take<T>(from + off, pitch, f);
        else load8(base + at, f);
      };
      float d[8];
      if (dx != nullptr) {
        float u[8], h[8], w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = h[i] = 0.f;
        if (active) {
          get(dx, o_dx, u);
          get(r, o_r, h);
        }
        take<float>(v_pre, pitch, w);
        float q1 = 0.f, q2 = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[i] = (h[i] - st.z) * st.w;
          p1[i] = fmaf(u[i], h[i], p1[i]);
          if constexpr (BIAS) p2[i] += u[i];
          u[i] *= w[i];
          q1 = fmaf(u[i], h[i], q1);
        }
        float m2 = 0.f;
        if (a.layer) {
#pragma unroll
          for (int i = 0; i < 8; ++i) q2 += u[i];
          const float2 q = sum(q1, q2);
          q1 = q.x;
          m2 = q.y * a.inv_d;
        } else {
          q1 = sum(q1);
        }
        const float m1 = -q1 * a.inv_d;
        // rstd (u - m2 - h m1) + dr_out
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = fmaf(h[i], m1, u[i] - m2);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = 0.f;
        if (gin != nullptr && active) get(gin, o_g, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = fmaf(st.w, u[i], d[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = 0.f;
        if (gin != nullptr && active) get(gin, o_g, d);
      }
      if (active) store8(static_cast<TR*>(a.dr) + at, d);
      if (y != nullptr) {
        float yv[8], e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) yv[i] = 0.f;
        if (active) get(y, 0, yv);
        take<float>(v_post, pitch, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          yv[i] = (yv[i] - st.x) * st.y;
          s1[i] = fmaf(d[i], yv[i], s1[i]);
          if constexpr (BIAS) s2[i] += d[i];
          e[i] *= d[i];
        }
        if (a.w_post != nullptr) {
          float q1 = 0.f, q2 = 0.f, m2 = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) q1 = fmaf(e[i], yv[i], q1);
          if (a.layer) {
#pragma unroll
            for (int i = 0; i < 8; ++i) q2 += e[i];
            const float2 q = sum(q1, q2);
            q1 = q.x;
            m2 = q.y * a.inv_d;
          } else {
            q1 = sum(q1);
          }
          const float m1 = -q1 * a.inv_d;
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] = st.y * fmaf(yv[i], m1, e[i] - m2);
        }
        if (active) store8(static_cast<TA*>(a.dy) + at, e);
      }
    }
    if (a.several) {
      join(s1);
      if constexpr (BIAS) join(s2);
      if (g == 0 && active) {
        float wg[8];
        load8(gate, wg);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          w_sum[c0 + i] = fmaf(wg[i], s1[i], w_sum[c0 + i]);
          if constexpr (BIAS) w_sum[a.D + c0 + i] = fmaf(wg[i], s2[i], w_sum[a.D + c0 + i]);
        }
        const int gr = seg0 / L;
        const int64_t gs = (int64_t)gr * L, ge = min((int64_t)a.T, gs + L);
        if (gs >= row0 && ge <= row1) {
          if (a.dgate != nullptr) {
            float w[8], o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = s1[i];
            if (a.w_post != nullptr) {
              load8(a.w_post + c0, w);
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] *= w[i];
            }
            if constexpr (BIAS) {
              if (a.b_post != nullptr) {
                load8(a.b_post + c0, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = fmaf(w[i], s2[i], o[i]);
              }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] *= a.alpha;
            store8(a.dgate + (int64_t)gr * a.D + c0, o);
          }
        } else {
          const bool head = gs < row0;
          store8(part + (head ? S1H : S1T) * arr, s1);
          if constexpr (BIAS) store8(part + (head ? S2H : S2T) * arr, s2);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s1[i] = 0.f;
        if constexpr (BIAS) s2[i] = 0.f;
      }
    }
    seg0 = seg1;
  }
  cp_wait(0);
  if (!a.several && a.y != nullptr) {
    join(s1);
    if (g == 0 && active) store8(part + S1H * arr, s1);
    if constexpr (BIAS) {
      join(s2);
      if (g == 0 && active) store8(part + S2H * arr, s2);
    }
  }
  if (a.dx != nullptr) {
    join(p1);
    if (g == 0 && active) store8(part + P1 * arr, p1);
    if constexpr (BIAS) {
      join(p2);
      if (g == 0 && active) store8(part + P2 * arr, p2);
    }
  }
  if (a.several && g == 0 && active) {
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = w_sum[c0 + i];
    store8(part + W1 * arr, o);
    if constexpr (BIAS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = w_sum[a.D + c0 + i];
      store8(part + W2 * arr, o);
    }
  }
}

// Adds the partials up: 32 columns a block, 32 strands of partials joined by
// a warp.  blockIdx.y = 0: the weights' and biases' gradients (and the
// gate's, when it has one row); blockIdx.y > 0: a gate row that CTAs cut.
// With fewer gate rows than CTAs, y - 1 is the gate row; else y is a CTA, and
// the gate row is the one cut at its start.
struct SumArgs {
  NormArgs n;
  int P, by_row;
  float *dw_post, *db_post, *dw_pre, *db_pre;
};

__global__ void __launch_bounds__(1024) block_norm_sum_kernel(const SumArgs s) {
  __shared__ float tile[32][33];
  const NormArgs& a = s.n;
  const int cx = threadIdx.x & 31, strand = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + cx;
  const bool in = col < a.D;
  const int64_t arr = (int64_t)s.P * a.D;
  pdl_begin();
  // over CTAs [p0, p1) of array `which` (the same in every thread of a column)
  auto add = [&](int which, int p0, int p1) {
    const float* at = a.part + which * arr + col;
    float v = 0.f;
    if (in) {
#pragma unroll 4
      for (int p = p0 + strand; p < p1; p += 32) v += at[(int64_t)p * a.D];
    }
    __syncthreads();
    tile[strand][cx] = v;
    __syncthreads();
    float t = tile[cx][strand];     // the warp's 32 strands of column `strand`
    t = warp_sum(t);
    __syncthreads();
    if (cx == 0) tile[0][strand] = t;
    __syncthreads();
    return tile[0][cx];
  };
  auto gate_grad = [&](float s1, float s2) {
    float o = a.w_post != nullptr ? a.w_post[col] * s1 : s1;
    if (a.b_post != nullptr) o = fmaf(a.b_post[col], s2, o);
    return a.alpha * o;
  };
  if (blockIdx.y == 0) {
    const bool bias_y = s.db_post != nullptr || (a.dgate != nullptr && a.b_post != nullptr);
    if (a.y != nullptr && (s.dw_post != nullptr || s.db_post != nullptr || !a.several)) {
      const float s1 = add(a.several ? W1 : S1H, 0, s.P);
      const float s2 = bias_y ? add(a.several ? W2 : S2H, 0, s.P) : 0.f;
      if (in && strand == 0) {
        // several gate rows: the sums already hold the gate
        const float gate = (a.gate_len > 0 && !a.several) ? a.gate[col] : 1.f;
        if (s.dw_post != nullptr) s.dw_post[col] = a.alpha * gate * s1;
        if (s.db_post != nullptr) s.db_post[col] = a.alpha * gate * s2;
        if (a.dgate != nullptr && !a.several) a.dgate[col] = gate_grad(s1, s2);
      }
    }
    if (s.dw_pre != nullptr) {
      const float v = add(P1, 0, s.P);
      if (in && strand == 0) s.dw_pre[col] = v;
    }
    if (s.db_pre != nullptr) {
      const float b = add(P2, 0, s.P);
      if (in && strand == 0) s.db_pre[col] = b;
    }
    return;
  }
  // The CTA that starts the gate row left its share as its tail, those that
  // go on with it as their heads.
  int64_t gs;
  if (s.by_row) {
    gs = (int64_t)(blockIdx.y - 1) * a.gate_len;
  } else {
    const int cut = first_row(a.T, blockIdx.y, s.P);
    gs = (int64_t)(cut / a.gate_len) * a.gate_len;
    if (gs == cut || first_row(a.T, blockIdx.y - 1, s.P) > gs) return;   // not its first cut
  }
  const int64_t ge = min((int64_t)a.T, gs + a.gate_len);
  auto holder = [&](int64_t row) { return (int)(((row + 1) * s.P - 1) / a.T); };
  const int pa = holder(gs), pb = holder(ge - 1);
  if (pa == pb) return;                        // whole in one CTA: written there
  // (a row that ends where its last CTA does is cut all the same)
  float s1 = add(S1H, pa + 1, pb + 1);
  float s2 = a.b_post != nullptr ? add(S2H, pa + 1, pb + 1) : 0.f;
  if (!in || strand != 0) return;
  const float* at = a.part + (int64_t)pa * a.D + col;
  s1 += at[S1T * arr];
  if (a.b_post != nullptr) s2 += at[S2T * arr];
  a.dgate[gs / a.gate_len * a.D + col] = gate_grad(s1, s2);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
int check(const moe_norm_config_t* c) {
  if (c == nullptr) return MOE_ERR_ARG;
  if (c->T < 1 || c->D < 8 || c->D > kMaxD || (c->D % 8)) return MOE_ERR_ARG;
  if (c->norm != MOE_RMSNORM && c->norm != MOE_LAYERNORM) return MOE_ERR_ARG;
  if (c->dtype != MOE_FP32 && c->dtype != MOE_BF16) return MOE_ERR_ARG;
  if (c->resid != MOE_FP32 && c->resid != MOE_BF16) return MOE_ERR_ARG;
  if (c->resid == MOE_BF16 && c->dtype != MOE_BF16) return MOE_ERR_ARG;
  if (c->gate_len < 0 || !(c->eps > 0.f) || !(c->alpha == c->alpha)) return MOE_ERR_ARG;
  return MOE_OK;
}

bool several_rows(const moe_norm_config_t* c) { return c->gate_len > 0 && c->gate_len < c->T; }
int threads_per_row(int D) { return (int)(host::ceil_div(D / 8, 32) * 32); }
// Row groups of a CTA of about `threads` threads (at most 15: a named
// barrier each; single-warp groups need none, up to 16).
int row_groups(int tpr, int threads) {
  return std::max(1, std::min(threads / tpr, tpr == 32 ? 16 : 15));
}
// The backward's CTAs and their row groups.  An SM holds one CTA when a row
// takes more than half of its threads (the column sums fill the register
// file), else two of up to 512 threads.  Row groups share a CTA's partial
// sums, so short batches run fewer CTAs rather than CTAs of one group; with
// short gate segments, which a CTA's groups share, each needs four rows.
void bwd_shape(const moe_norm_config_t* c, int* ctas, int* groups) {
  const int tpr = threads_per_row(c->D);
  const int64_t most = (int64_t)kSms * (tpr > 512 ? 1 : 2);
  int64_t R = row_groups(tpr, 512);
  if (several_rows(c)) R = std::max<int64_t>(1, std::min<int64_t>(R, c->gate_len / 4));
  *ctas = (int)std::max<int64_t>(1, std::min<int64_t>(most, host::ceil_div(c->T, R)));
  *groups = (int)std::min<int64_t>(R, host::ceil_div(c->T, *ctas));
}

NormArgs args_of(const moe_norm_config_t* c) {
  NormArgs a{};
  a.T = c->T; a.D = c->D; a.nv = c->D / 8; a.tpr = threads_per_row(c->D);
  a.layer = c->norm == MOE_LAYERNORM;
  a.gate_len = c->gate_len; a.eps = c->eps; a.alpha = c->alpha;
  a.inv_d = 1.0f / (float)c->D;
  return a;
}
template <typename... P>
bool any_misaligned(P... p) {
  return (host::misaligned(p, 16) || ...);
}

template <typename TA, typename TR>
int forward(NormArgs a, cudaStream_t s) {
  auto k = block_norm_kernel<TA, TR>;
  a.R = row_groups(a.tpr, 256);
  const int sms = host::sm_count();
  a.R = (int)std::max<int64_t>(1, std::min<int64_t>(a.R, host::ceil_div(a.T, sms)));
  const int threads = a.R * a.tpr;
  const size_t stage = (size_t)(kPiece<TA> + kPiece<TR>) * threads;
  const int per_sm = std::max(1, 2048 / threads);
  // the ring holds what a CTA's share of shared memory takes, 3 stages at most
  a.stages = (int)std::max<size_t>(1, std::min<size_t>(3, kSmemLimit / per_sm / stage));
  const size_t smem = a.stages * stage;
  MOE_HCK(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemLimit - 9 * 1024));
  const int64_t want = host::ceil_div(a.T, a.R);
  const int grid = (int)std::min<int64_t>(want, (int64_t)sms * per_sm);
  return host::launch("block_norm", k, grid, threads, smem, s, 1, a);
}

template <typename TA, typename TR, bool BIAS>
int backward(NormArgs a, int P, SumArgs& sum, cudaStream_t s) {
  auto k = block_norm_bwd_kernel<TA, TR, BIAS>;
  const int threads = a.R * a.tpr;
  const size_t stage = 2 * (size_t)(kPiece<TA> + kPiece<TR>) * threads;
  const size_t fixed = (size_t)threads * 64 + (a.several ? (BIAS ? 2 : 1) * (size_t)a.D * 4 : 0) +
                       (a.R > 1 ? (size_t)threads * 32 : 0);
  // two CTAs an SM share its shared memory (8 KB static and 1 KB of the
  // system's each)
  const size_t room = (threads > 512 ? kSmemLimit : kSmemLimit / 2) - 9 * 1024 - fixed;
  // a ring of one stage would overlap nothing: rows too long for two (wide
  // fp32 rows) are read where they are used
  a.stages = (int)std::min<size_t>(3, room / stage);
  if (a.stages < 2) a.stages = 0;
  const size_t smem = a.stages * stage + fixed;
  MOE_HCK(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemLimit - 9 * 1024));
  MOE_HTRY(host::launch("block_norm_bwd", k, P, threads, smem, s, 1, a));
  sum.n = a;
  sum.P = P;
  // dgate of the gate rows that CTAs cut: by gate row where there are fewer
  // of those than CTAs, else by CTA
  int cuts = 0;
  if (a.several && a.dgate != nullptr) {
    const int64_t rows = host::ceil_div(a.T, a.gate_len);
    sum.by_row = rows < P;
    cuts = (int)std::min<int64_t>(rows, P - 1);
  }
  const dim3 grid((unsigned)host::ceil_div(a.D, 32), 1 + cuts);
  return host::launch("block_norm_sum", block_norm_sum_kernel, grid, 1024, 0, s, 1, sum);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_block_norm(const moe_norm_config_t* c, const void* r, const void* y,
                   const float* w_post, const float* b_post, const float* gate,
                   const float* w_pre, const float* b_pre, void* r_out, void* x, float* stats,
                   cudaStream_t s) {
  MOE_HTRY(check(c));
  if (r == nullptr || (y == nullptr && w_pre == nullptr)) return MOE_ERR_ARG;
  if (y == nullptr ? (w_post || b_post || gate || r_out)
                   : (r_out == nullptr || (gate != nullptr) != (c->gate_len > 0)))
    return MOE_ERR_ARG;
  if ((b_post && !w_post) || (b_pre && !w_pre) || (w_pre != nullptr) != (x != nullptr))
    return MOE_ERR_ARG;
  if (any_misaligned(r, y, w_post, b_post, gate, w_pre, b_pre, r_out, x, stats)) return MOE_ERR_ARG;
  NormArgs a = args_of(c);
  if (y == nullptr) a.gate_len = 0;
  a.r = r; a.y = y; a.w_post = w_post; a.b_post = b_post; a.gate = gate; a.w_pre = w_pre;
  a.b_pre = b_pre; a.r_out = r_out; a.x = x; a.stats = stats;
  if (c->dtype == MOE_FP32) return forward<float, float>(a, s);
  if (c->resid == MOE_FP32) return forward<__nv_bfloat16, float>(a, s);
  return forward<__nv_bfloat16, __nv_bfloat16>(a, s);
}

int64_t moe_block_norm_ws_bytes(const moe_norm_config_t* c) {
  if (check(c) != MOE_OK) return 0;
  int ctas = 0, groups = 0;
  bwd_shape(c, &ctas, &groups);
  return (int64_t)ctas * c->D * 4 * (several_rows(c) ? 8 : 4);
}

int moe_block_norm_backward(const moe_norm_config_t* c, const void* r_out, const void* y,
                            const float* w_post, const float* b_post, const float* gate,
                            const float* w_pre, const float* stats, const void* dx,
                            const void* dr_out, void* dy, void* dr, float* dw_post,
                            float* db_post, float* dgate, float* dw_pre, float* db_pre, void* ws,
                            cudaStream_t s) {
  MOE_HTRY(check(c));
  if (r_out == nullptr || stats == nullptr || dr == nullptr || ws == nullptr) return MOE_ERR_ARG;
  if ((y != nullptr) != (dy != nullptr) || (w_pre != nullptr) != (dx != nullptr)) return MOE_ERR_ARG;
  if (y == nullptr ? (w_pre == nullptr || w_post || b_post || gate)
                   : (gate != nullptr) != (c->gate_len > 0))
    return MOE_ERR_ARG;
  if ((b_post && !w_post) || (dw_post && !w_post) || (db_post && !w_post) || (dgate && !gate) ||
      ((dw_pre || db_pre) && !w_pre))
    return MOE_ERR_ARG;
  if (any_misaligned(r_out, y, w_post, b_post, gate, w_pre, stats, dx, dr_out, dy, dr, dgate, ws))
    return MOE_ERR_ARG;
  NormArgs a = args_of(c);
  if (y == nullptr) a.gate_len = 0;
  a.r = r_out; a.y = y; a.w_post = w_post; a.b_post = b_post; a.gate = gate; a.w_pre = w_pre;
  a.stats_in = stats; a.dx = dx; a.dr_out = dr_out; a.dy = dy; a.dr = dr; a.dgate = dgate;
  a.part = static_cast<float*>(ws);
  a.several = y != nullptr && several_rows(c);
  SumArgs sum{};
  sum.dw_post = dw_post; sum.db_post = db_post; sum.dw_pre = dw_pre; sum.db_pre = db_pre;
  int P = 0;
  bwd_shape(c, &P, &a.R);
  const bool bias = db_post != nullptr || db_pre != nullptr || (dgate != nullptr && b_post != nullptr);
  auto go = [&](auto ta, auto tr) {
    using TA = decltype(ta);
    using TR = decltype(tr);
    return bias ? backward<TA, TR, true>(a, P, sum, s) : backward<TA, TR, false>(a, P, sum, s);
  };
  if (c->dtype == MOE_FP32) return go(float{}, float{});
  if (c->resid == MOE_FP32) return go(__nv_bfloat16{}, float{});
  return go(__nv_bfloat16{}, __nv_bfloat16{});
}

}  // extern "C"
