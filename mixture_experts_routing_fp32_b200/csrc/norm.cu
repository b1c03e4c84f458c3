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
// Of the copy rate of 6.46 TB/s the bf16 RMSNorm forms reach 91% (forward,
// 16384 x 4096: 91 us in a replayed graph) and 82% (backward, 8192 x 7168: 134
// us); LayerNorm with biases, which has twice the row sums, 57% and 55%;
// RMSNorm of fp32 rows (half as many) 64% and 73%, of bf16 rows beside an fp32
// stream 73% and 61%.  Gate rows of a few tokens are the slowest form (65536 x
// 256 backward: 42 us without a gate, 71 with 16 tokens a gate row, 183 with 4,
// 292 with one): their CTAs run one row group and meet at every gate row's end.
#include <type_traits>

#include "f32x2.cuh"
#include "host.cuh"
#include "norm_shape.h"

namespace moe {
namespace {

using norm_shape::kMaxThreads;
using norm_shape::kSmallBlock;
using norm_shape::row_groups;
using norm_shape::threads_per_row;

constexpr int kMaxD = 8192;          // 1024 threads of 8 columns
constexpr int kSms = 148;            // the backward's partial sums are sized for this grid
constexpr size_t kSmemLimit = 227 * 1024;
constexpr int kDynSmem = (int)kSmemLimit - 8 * 1024;   // beside the row sums' static 8 KB

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
  float *dw_post, *db_post, *dw_pre, *db_pre;
  int several;                       // gate rows change inside the batch
  int wide;                          // r_out and x (dr and dy): aligned to 32 bytes
  int finish;                        // backward: one CTA, which writes the gradients itself
  int bias_smem;                     // forward: the biases sit in shared memory too
  int w_smem;                        // backward: the running sums for w_post do
  int swap_ring;                     // backward: the groups' exchange takes the ring's place
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
// This thread's piece back from its slot (bf16 rows use one 16-byte chunk,
// fp32 rows two), and a piece of its own put there.  The backward, short of
// registers, addresses its slots in 32 bits (16384 rows of 4096 bf16: 142 us
// against 172); the forward is the faster with plain loads, which the
// compiler moves (91 us against 102).
__device__ __forceinline__ float4 lds(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
template <typename T>
__device__ __forceinline__ F8 take(uint32_t slot, int pitch) {
  const float4 a = lds(slot);
  if constexpr (sizeof(T) == 2)
    return widen8(make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(a.z),
                             __float_as_uint(a.w)));
  else return f8_of(a, lds(slot + pitch));
}
template <typename T>
__device__ __forceinline__ F8 take(const uint8_t* slot, int pitch) {
  if constexpr (sizeof(T) == 2) return widen8(*reinterpret_cast<const uint4*>(slot));
  else return f8_of(*reinterpret_cast<const float4*>(slot),
                    *reinterpret_cast<const float4*>(slot + pitch));
}
__device__ __forceinline__ void keep(uint8_t* slot, int pitch, const F8& a) {
  store_f8_split(reinterpret_cast<float4*>(slot), reinterpret_cast<float4*>(slot + pitch), a);
}
__device__ __forceinline__ void keep(uint32_t slot, int pitch, const F8& a) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 p = unpack2(a.p[2 * i]), q = unpack2(a.p[2 * i + 1]);
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(slot + i * pitch), "f"(p.x),
                 "f"(p.y), "f"(q.x), "f"(q.y)
                 : "memory");
  }
}

// 8 columns to global memory: fp32 in one 32-byte store where the tensors are
// aligned to that, so that every store fills whole sectors (4096 rows of 7168
// fp32, forward: 124 -> 104 us).
__device__ __forceinline__ void put8(__nv_bfloat16* p, const F8& a, int) { store_f8(p, a); }
__device__ __forceinline__ void put8(float* p, const F8& a, int wide) {
  if (!wide) return store_f8(p, a);
  asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p), "l"(a.p[0]), "l"(a.p[1]),
               "l"(a.p[2]), "l"(a.p[3])
               : "memory");
}

// Sums over the tpr threads of a row group (all get them, in the same order).
// `buf` alternates, so one barrier per sum is enough: a warp still reading
// one buffer is behind the barrier of the next sum, which writes the other.
struct RowSum {
  float2* red;      // [2][32] of this row group
  int warps, warp, lane, bar, tpr, buf;
  __device__ __forceinline__ void sync() const {
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(tpr) : "memory");
  }
  // Two values in the shuffles of one: the halves of the warp exchange what
  // the other half goes on to sum.  a's sum is left in lanes 0-15, b's in
  // 16-31.
  __device__ __forceinline__ float halves(float a, float b) const {
    const bool hi = (lane & 16) != 0;
    float v = (hi ? b : a) + __shfl_xor_sync(0xffffffffu, hi ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  __device__ __forceinline__ float2 spread(float v) const {
    return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
  }
  __device__ __forceinline__ float2 operator()(float a, float b) {
    float v = halves(a, b);
    if (warps == 1) return spread(v);
    if ((lane & 15) == 0) reinterpret_cast<float*>(red + buf * 32 + warp)[lane >> 4] = v;
    sync();
    const float2 w = lane < warps ? red[buf * 32 + lane] : make_float2(0.f, 0.f);
    buf ^= 1;
    return spread(halves(w.x, w.y));
  }
  __device__ __forceinline__ float operator()(float a) {
    a = warp_sum(a);
    if (warps == 1) return a;
    if (lane == 0) red[buf * 32 + warp].x = a;
    sync();
    const float v = lane < warps ? red[buf * 32 + lane].x : 0.f;
    buf ^= 1;
    return warp_sum(v);
  }
};

// First row of CTA p of P (even split).
__device__ __forceinline__ int first_row(int T, int p, int P) {
  return (int)((int64_t)T * p / P);
}

// mean and rstd of a row held 8 values a thread; v is left without its mean.
// Idle threads (those of a row's last warp behind its end) hold the row's
// last 8 values again: they load and compute like the others, so that nothing
// but sums and stores has to ask which they are.
// The variance is that of the centred values (a second sum), and these are
// what rstd multiplies: v rstd - mean rstd in one step would round the
// second term, 2^-24 of the mean in units of the spread.  The mean is a
// quotient, not a product with 1 / D, so that rows whose sum and mean are
// fp32 values are centred exactly.  (Joining each warp's own centred sums
// instead, with one exchange, measured 166 against 142 us for 16384 rows of
// 4096 bf16: its chain of shuffles is as long.)
__device__ __forceinline__ float2 centre(F8& v, bool active, const NormArgs& a, RowSum& sum) {
  float mean = 0.f;
  if (a.layer) {
    mean = __fdiv_rn(sum(active ? sum8(v) : 0.f), (float)a.D);
    v = add8(v, pack2(-mean, -mean));
  }
  return make_float2(mean, rsqrtf(fmaf(sum(active ? dot8(v, v) : 0.f), a.inv_d, a.eps)));
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// A CTA walks a run of consecutive rows, R at a time.  The vectors stay in
// shared memory, each thread's own 8 columns: w_pre, alpha gate w_post and,
// with BIAS, b_pre and alpha gate b_post; those with the gate are formed
// again when the gate row changes.  FULL: D is a multiple of 256, every
// thread of a row holds columns.
// SMALL: blocks of up to 576 threads in at most 56 registers, so that an SM
// holds 1168 threads of them (two rows of 4104 columns, not one; three of
// 2568); norm_shape.h says which run so.
template <typename TA, typename TR, bool BIAS, bool FULL, bool SMALL>
__global__ void __launch_bounds__(SMALL ? kSmallBlock : kMaxThreads, SMALL ? 2 : 1)
block_norm_kernel(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 red_s[16 * 64];
  const int tid = threadIdx.x;
  const int g = a.R == 1 ? 0 : tid / a.tpr, vec = tid - g * a.tpr;
  const bool active = FULL || vec < a.nv;
  const int c0 = (FULL ? vec : min(vec, a.nv - 1)) * 8;
  RowSum sum{red_s + g * 64, a.tpr >> 5, vec >> 5, tid & 31, 1 + g, a.tpr, 0};
  const int pitch = blockDim.x * 16;
  constexpr int kChunks = (kPiece<TA> + kPiece<TR>) / 16;
  const int stage_bytes = kChunks * pitch;
  const int r_off = (kPiece<TA> / 16) * pitch;
  uint8_t* mine = ring + tid * 16;
  const uint32_t mine_a = smem_addr(mine);
  uint8_t* v_pre = mine + a.stages * stage_bytes;
  uint8_t *v_post = v_pre + 2 * pitch, *v_bpre = v_pre + 4 * pitch, *v_bpost = v_pre + 6 * pitch;
  const TA* y = static_cast<const TA*>(a.y);
  const TR* r = static_cast<const TR*>(a.r);
  const int row0 = first_row(a.T, blockIdx.x, gridDim.x) + g;
  const int row1 = first_row(a.T, blockIdx.x + 1, gridDim.x);
  pdl_begin();

  int ahead = row0;
  uint32_t slot_in = mine_a;
  const uint32_t ring_end = mine_a + a.stages * stage_bytes;
  auto issue = [&] {
    if (ahead < row1) {
      const int64_t at = (int64_t)ahead * a.D + c0;
      if (y != nullptr) fetch<TA>(slot_in, pitch, y + at);
      fetch<TR>(slot_in + r_off, pitch, r + at);
    }
    cp_commit();
    ahead += a.R;
    slot_in += stage_bytes;
    if (slot_in == ring_end) slot_in = mine_a;
  };
  for (int i = 0; i < a.stages; ++i) issue();
  if (a.w_pre != nullptr) keep(v_pre, pitch, load_f8(a.w_pre + c0));
  if (BIAS && a.bias_smem && a.w_pre != nullptr)
    keep(v_bpre, pitch, a.b_pre != nullptr ? load_f8(a.b_pre + c0) : zero8f());
  // alpha gate w_post and alpha gate b_post of gate row gr
  auto post_vectors = [&](int gr) {
    F8 e = fma8(zero8f(), 0ull, pack2(a.alpha, a.alpha)), eb = zero8f();
    if (a.gate_len > 0) e = mul8(e, load_f8(a.gate + (int64_t)gr * a.D + c0));
    if (BIAS && a.b_post != nullptr) eb = mul8(e, load_f8(a.b_post + c0));
    if (a.w_post != nullptr) e = mul8(e, load_f8(a.w_post + c0));
    keep(v_post, pitch, e);
    if (BIAS && a.bias_smem) keep(v_bpost, pitch, eb);
  };
  // alpha gate b_post and b_pre where the ring leaves no room for them
  auto post_bias = [&](int gr) {
    if (a.b_post == nullptr) return zero8f();
    F8 eb = mul8(load_f8(a.b_post + c0), pack2(a.alpha, a.alpha));
    return a.gate_len > 0 ? mul8(eb, load_f8(a.gate + (int64_t)gr * a.D + c0)) : eb;
  };
  int gate_row = -1;
  const uint8_t* slot = mine;
  for (int t = row0; t < row1; t += a.R) {
    if (y != nullptr) {
      const int gr = a.gate_len > 0 ? t / a.gate_len : 0;
      if (gr != gate_row) post_vectors(gate_row = gr);
    }
    cp_wait(a.stages - 1);
    const int64_t at = (int64_t)t * a.D + c0;
    float2 my = make_float2(0.f, 1.f), mr = make_float2(0.f, 1.f);
    // the row leaves the ring at once, so that all of the ring is in flight
    // while it is worked on
    F8 v = take<TR>(slot + r_off, pitch), z = zero8f();
    if (y != nullptr) z = take<TA>(slot, pitch);
    __syncwarp();
    issue();
    if (y != nullptr) {
      if (a.w_post != nullptr) {
        my = centre(z, active, a, sum);
        z = mul8(z, pack2(my.y, my.y));
      }
      if (BIAS) v = add8(v, a.bias_smem ? take<float>(v_bpost, pitch) : post_bias(gate_row));
      v = fma8(z, take<float>(v_post, pitch), v);
      TR* out = static_cast<TR*>(a.r_out) + at;
      // the second norm reads the stream as it is stored: the backward then
      // sees the same values
      if constexpr (sizeof(TR) == 2) {
        const uint4 u = narrow8(v);
        if (active) *reinterpret_cast<uint4*>(out) = u;
        v = widen8(u);
      } else {
        if (active) put8(out, v, a.wide);
      }
    }
    if (a.w_pre != nullptr) {
      mr = centre(v, active, a, sum);
      v = mul8(v, pack2(mr.y, mr.y));
      if (BIAS)
        v = fma8(v, take<float>(v_pre, pitch),
                 a.bias_smem ? take<float>(v_bpre, pitch)
                 : a.b_pre != nullptr ? load_f8(a.b_pre + c0) : zero8f());
      else v = mul8(v, take<float>(v_pre, pitch));
      if (active) put8(static_cast<TA*>(a.x) + at, v, a.wide);
    }
    if (a.stats != nullptr && vec == 0)
      *reinterpret_cast<float4*>(a.stats + 4 * (int64_t)t) = make_float4(my.x, my.y, mr.x, mr.y);
    slot += stage_bytes;
    if (smem_addr(slot) == ring_end) slot = mine;
  }
  cp_wait(0);
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// The column sums over tokens stay in registers while a CTA walks its rows
// (8 columns a thread: sums of d yh and dx rh, in the general form also of
// d and dx)
// and leave as one partial per CTA, which block_norm_sum_kernel adds up in
// CTA order.  When gate rows change inside the batch (SEVERAL), the rows
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
// GENERAL: LayerNorm, or sums for biases; else RMSNorm without them.
// THREADS: the most that an SM's CTAs have together.
template <typename TA, typename TR, bool GENERAL, bool SEVERAL, bool FULL, int THREADS>
__global__ void __launch_bounds__(THREADS) block_norm_bwd_kernel(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 red_s[16 * 64];
  const int tid = threadIdx.x;
  const int g = a.R == 1 ? 0 : tid / a.tpr, vec = tid - g * a.tpr;
  const bool active = FULL || vec < a.nv;
  const int c0 = (FULL ? vec : min(vec, a.nv - 1)) * 8;
  RowSum sum{red_s + g * 64, a.tpr >> 5, vec >> 5, tid & 31, 1 + g, a.tpr, 0};
  const int pitch = blockDim.x * 16;
  constexpr int kA = kPiece<TA> / 16, kR = kPiece<TR> / 16, kW = GENERAL ? 2 : 1;
  const int stage_bytes = 2 * (kA + kR) * pitch;
  const int o_dx = kA * pitch, o_r = 2 * kA * pitch, o_g = (2 * kA + kR) * pitch;
  const uint32_t mine = smem_addr(ring) + tid * 16;
  // after the ring: w_pre and alpha gate w_post (each thread its 8 columns,
  // the row groups the same ones), [kW][D] running sums for w_post, b_post
  // (SEVERAL, where they fit; else the CTA's partial in global memory), and
  // for R > 1 one [R][8 tpr] exchange buffer (in the ring's place where the
  // groups meet only after their last rows)
  const int vpitch = a.tpr * 16;
  const uint32_t v_pre = smem_addr(ring) + a.stages * stage_bytes + vec * 16,
                 v_post = v_pre + 2 * vpitch;
  float* w_smem = reinterpret_cast<float*>(ring + a.stages * stage_bytes + 4 * vpitch);
  float* swap = a.swap_ring ? reinterpret_cast<float*>(ring)
                            : w_smem + (SEVERAL && a.w_smem ? kW * a.D : 0);
  const TA* y = static_cast<const TA*>(a.y);
  const TA* dx = static_cast<const TA*>(a.dx);
  const TR* r = static_cast<const TR*>(a.r);
  const TR* gin = static_cast<const TR*>(a.dr_out);
  const int P = gridDim.x, p = blockIdx.x;
  const int row0 = first_row(a.T, p, P), row1 = first_row(a.T, p + 1, P);
  const int64_t arr = (int64_t)P * a.D;             // floats of one partial array
  float* part = a.part + (int64_t)p * a.D + c0;

  pdl_begin();
  float* w_sum[2] = {a.w_smem ? w_smem + c0 : part + W1 * arr,
                     a.w_smem ? w_smem + a.D + c0 : part + W2 * arr};
  if (SEVERAL && active && g == 0) {
    for (int k = 0; k < kW; ++k) store_f8(w_sum[k], zero8f());
  }

  // Row group g takes rows row0 + g, + R, ...; segments are runs of rows of
  // one gate row, at whose ends the groups meet.
  const int L = SEVERAL ? a.gate_len : a.T;
  auto seg_end = [&](int row) {
    return SEVERAL ? (int)min((int64_t)row1, (int64_t)(row / L + 1) * L) : row1;
  };
  int ahead = row0 + g;
  uint32_t slot_in = mine;
  const uint32_t ring_end = mine + a.stages * stage_bytes;
  auto issue = [&] {
    if (a.stages == 0) return;
    if (ahead < row1) {
      const int64_t at = (int64_t)ahead * a.D + c0;
      if (y != nullptr) fetch<TA>(slot_in, pitch, y + at);
      if (dx != nullptr) {
        fetch<TA>(slot_in + o_dx, pitch, dx + at);
        fetch<TR>(slot_in + o_r, pitch, r + at);
      }
      if (gin != nullptr) fetch<TR>(slot_in + o_g, pitch, gin + at);
      ahead += a.R;
    }
    cp_commit();
    slot_in += stage_bytes;
    if (slot_in == ring_end) slot_in = mine;
  };
  F8 s1 = zero8f(), p1 = zero8f(), s2 = zero8f(), p2 = zero8f();
  // sum of v over the row groups, in group order (in group 0's threads)
  auto join = [&](F8& v) {
    if (a.R == 1) return;
    __syncthreads();
    store_f8(swap + (g * a.tpr + vec) * 8, v);
    __syncthreads();
    if (g == 0)
      for (int k = 1; k < a.R; ++k) v = add8(v, load_f8(swap + (k * a.tpr + vec) * 8));
  };

  // (v - mean) rstd, as the forward forms it; RMSNorm's mean is 0
  auto normal = [&](F8 v, float mean, float rstd) {
    if (GENERAL) v = add8(v, pack2(-mean, -mean));
    return mul8(v, pack2(rstd, rstd));
  };
  const float4* stats = reinterpret_cast<const float4*>(a.stats_in);
  float4 st_next = make_float4(0.f, 0.f, 0.f, 0.f);
  int t = row0 + g;
  if (t < row1) st_next = stats[t];
  for (int i = 0; i < a.stages - 1; ++i) issue();
  keep(v_pre, vpitch, a.w_pre != nullptr ? load_f8(a.w_pre + c0) : zero8f());
  uint32_t slot = mine;
  for (int seg0 = row0; seg0 < row1;) {
    const int seg1 = seg_end(seg0);
    const float* gate = a.gate_len > 0 ? a.gate + (int64_t)(seg0 / a.gate_len) * a.D + c0 : nullptr;
    if (y != nullptr) {
      F8 w = add8(zero8f(), pack2(a.alpha, a.alpha));
      if (gate != nullptr) w = mul8(w, load_f8(gate));
      if (a.w_post != nullptr) w = mul8(w, load_f8(a.w_post + c0));
      keep(v_post, vpitch, w);
    }
    for (; t < seg1; t += a.R) {
      issue();
      const float4 st = st_next;
      if (t + a.R < row1) st_next = stats[t + a.R];
      const int64_t at = (int64_t)t * a.D + c0;
      if (a.stages > 0) cp_wait(a.stages - 1);
      // this thread's columns of one tensor (rows that fit no ring: from
      // global memory)
      auto get = [&](auto* base, int off) -> F8 {
        using T = std::remove_cv_t<std::remove_pointer_t<decltype(base)>>;
        return a.stages > 0 ? take<T>(slot + off, pitch) : load_f8(base + at);
      };
      F8 d;
      if (dx != nullptr) {
        F8 u = get(dx, o_dx);
        const F8 h = normal(get(r, o_r), st.z, st.w);
        p1 = fma8(u, h, p1);
        if (GENERAL) p2 = add8(p2, u);
        u = mul8(u, take<float>(v_pre, vpitch));
        float m1;
        if (GENERAL && a.layer) {
          const float2 q = sum(active ? dot8(u, h) : 0.f, active ? sum8(u) : 0.f);
          m1 = -q.x * a.inv_d;
          const float m2 = -q.y * a.inv_d;
          u = add8(u, pack2(m2, m2));
        } else {
          m1 = -sum(active ? dot8(u, h) : 0.f) * a.inv_d;
        }
        // rstd (u - m2 - h m1) + dr_out
        u = fma8(h, pack2(m1, m1), u);
        d = gin != nullptr ? get(gin, o_g) : zero8f();
        d = fma8(u, pack2(st.w, st.w), d);
      } else {
        d = gin != nullptr ? get(gin, o_g) : zero8f();
      }
      if (active) put8(static_cast<TR*>(a.dr) + at, d, a.wide);
      if (y != nullptr) {
        const F8 yh = normal(get(y, 0), st.x, st.y);
        s1 = fma8(d, yh, s1);
        if (GENERAL) s2 = add8(s2, d);
        F8 e = mul8(d, take<float>(v_post, vpitch));
        if (a.w_post != nullptr) {
          float m1;
          if (GENERAL && a.layer) {
            const float2 q = sum(active ? dot8(e, yh) : 0.f, active ? sum8(e) : 0.f);
            m1 = -q.x * a.inv_d;
            const float m2 = -q.y * a.inv_d;
            e = add8(e, pack2(m2, m2));
          } else {
            m1 = -sum(active ? dot8(e, yh) : 0.f) * a.inv_d;
          }
          e = mul8(fma8(yh, pack2(m1, m1), e), pack2(st.y, st.y));
        }
        if (active) put8(static_cast<TA*>(a.dy) + at, e, a.wide);
      }
      slot += stage_bytes;
      if (slot == ring_end) slot = mine;
    }
    if constexpr (SEVERAL) {
      join(s1);
      if (GENERAL) join(s2);
      if (g == 0 && active) {
        const F8 wg = load_f8(gate);
        store_f8(w_sum[0], fma8(wg, s1, load_f8(w_sum[0])));
        if (GENERAL) store_f8(w_sum[1], fma8(wg, s2, load_f8(w_sum[1])));
        const int gr = seg0 / L;
        const int64_t gs = (int64_t)gr * L, ge = min((int64_t)a.T, gs + L);
        if (gs >= row0 && ge <= row1) {
          if (a.dgate != nullptr) {
            F8 o = s1;
            if (a.w_post != nullptr) o = mul8(o, load_f8(a.w_post + c0));
            if (GENERAL && a.b_post != nullptr) o = fma8(load_f8(a.b_post + c0), s2, o);
            store_f8(a.dgate + (int64_t)gr * a.D + c0, mul8(o, pack2(a.alpha, a.alpha)));
          }
        } else {
          const bool head = gs < row0;
          store_f8(part + (head ? S1H : S1T) * arr, s1);
          if (GENERAL) store_f8(part + (head ? S2H : S2T) * arr, s2);
        }
      }
      s1 = s2 = zero8f();
    }
    seg0 = seg1;
  }
  cp_wait(0);
  if (!SEVERAL && a.finish) {
    // one CTA held all rows: its sums are the gradients
    auto put = [&](float* out, const F8& v) {
      if (out == nullptr) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(v.p[i]);
        out[c0 + 2 * i] = f.x;
        out[c0 + 2 * i + 1] = f.y;
      }
    };
    join(s1);
    join(p1);
    if (GENERAL) {
      join(s2);
      join(p2);
    }
    if (g != 0 || !active) return;
    if (a.y != nullptr) {
      F8 dg = s1;
      if (a.w_post != nullptr) dg = mul8(dg, load_f8(a.w_post + c0));
      if (GENERAL && a.b_post != nullptr) dg = fma8(load_f8(a.b_post + c0), s2, dg);
      put(a.dgate, mul8(dg, pack2(a.alpha, a.alpha)));
      F8 w = add8(zero8f(), pack2(a.alpha, a.alpha));
      if (a.gate_len > 0) w = mul8(w, load_f8(a.gate + c0));
      put(a.dw_post, mul8(w, s1));
      if (GENERAL) put(a.db_post, mul8(w, s2));
    }
    if (a.dx != nullptr) {
      put(a.dw_pre, p1);
      if (GENERAL) put(a.db_pre, p2);
    }
    return;
  }
  if (!SEVERAL && a.y != nullptr) {
    join(s1);
    if (g == 0 && active) store_f8(part + S1H * arr, s1);
    if (GENERAL) {
      join(s2);
      if (g == 0 && active) store_f8(part + S2H * arr, s2);
    }
  }
  if (a.dx != nullptr) {
    join(p1);
    if (g == 0 && active) store_f8(part + P1 * arr, p1);
    if (GENERAL) {
      join(p2);
      if (g == 0 && active) store_f8(part + P2 * arr, p2);
    }
  }
  if (SEVERAL && a.w_smem && g == 0 && active) {
    store_f8(part + W1 * arr, load_f8(w_sum[0]));
    if (GENERAL) store_f8(part + W2 * arr, load_f8(w_sum[1]));
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
};

__global__ void __launch_bounds__(1024) block_norm_sum_kernel(const SumArgs s) {
  __shared__ float tile[4][32][33];
  const NormArgs& a = s.n;
  const int cx = threadIdx.x & 31, strand = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + cx;
  const bool in = col < a.D;
  const int64_t arr = (int64_t)s.P * a.D;
  pdl_begin();
  // Sums over CTAs [p0, p1) of up to four arrays (which[i] < 0: none), all
  // loads before the first exchange; the sums of column cx end in every
  // thread of it.
  auto add = [&](const int (&which)[4], int p0, int p1, float (&out)[4]) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (in) {
#pragma unroll 2
      for (int p = p0 + strand; p < p1; p += 32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (which[i] >= 0) v[i] += a.part[which[i] * arr + (int64_t)p * a.D + col];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) tile[i][strand][cx] = v[i];
    __syncthreads();
    // the warp's lanes take the 32 strands of column `strand`
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = which[i] >= 0 ? warp_sum(tile[i][cx][strand]) : 0.f;
    __syncthreads();
    if (cx == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) tile[i][0][strand] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = tile[i][0][cx];
  };
  auto gate_grad = [&](float s1, float s2, int c) {
    float o = a.w_post != nullptr ? a.w_post[c] * s1 : s1;
    if (a.b_post != nullptr) o = fmaf(a.b_post[c], s2, o);
    return a.alpha * o;
  };
  if (blockIdx.y == 0) {
    float v[4];
    const bool gate1 = a.dgate != nullptr && !a.several;
    const bool s1 = a.y != nullptr && (a.dw_post != nullptr || gate1);
    const bool s2 = a.y != nullptr && (a.db_post != nullptr || (gate1 && a.b_post != nullptr));
    // several gate rows: the sums already hold the gate
    const int which[4] = {s1 ? (a.several ? W1 : S1H) : -1, s2 ? (a.several ? W2 : S2H) : -1,
                          a.dw_pre != nullptr ? P1 : -1, a.db_pre != nullptr ? P2 : -1};
    add(which, 0, s.P, v);
    if (!in || strand != 0) return;
    const float gate = (a.gate_len > 0 && !a.several) ? a.gate[col] : 1.f;
    if (a.dw_post != nullptr) a.dw_post[col] = a.alpha * gate * v[0];
    if (a.db_post != nullptr) a.db_post[col] = a.alpha * gate * v[1];
    if (gate1) a.dgate[col] = gate_grad(v[0], v[1], col);
    if (a.dw_pre != nullptr) a.dw_pre[col] = v[2];
    if (a.db_pre != nullptr) a.db_pre[col] = v[3];
    return;
  }
  // The CTA that starts the gate row left its share as its tail, those that
  // go on with it as their heads.  A thread takes a column (few CTAs hold a
  // gate row), a block 1024 of them.
  if (blockIdx.x * 1024 >= a.D) return;
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
  const int gc = blockIdx.x * 1024 + threadIdx.x;
  if (gc >= a.D) return;
  const float* at = a.part + gc;
  float s1 = at[S1T * arr + (int64_t)pa * a.D];
  float s2 = a.b_post != nullptr ? at[S2T * arr + (int64_t)pa * a.D] : 0.f;
#pragma unroll 4
  for (int p = pa + 1; p <= pb; ++p) {
    s1 += at[S1H * arr + (int64_t)p * a.D];
    if (a.b_post != nullptr) s2 += at[S2H * arr + (int64_t)p * a.D];
  }
  a.dgate[gs / a.gate_len * a.D + gc] = gate_grad(s1, s2, gc);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
int check(const moe_norm_config_t* c) {
  if (c == nullptr) return MOE_ERR_ARG;
  if (c->T < 1 || c->T > (1 << 30) || c->D < 8 || c->D > kMaxD || (c->D % 8)) return MOE_ERR_ARG;
  if (c->norm != MOE_RMSNORM && c->norm != MOE_LAYERNORM) return MOE_ERR_ARG;
  if (c->dtype != MOE_FP32 && c->dtype != MOE_BF16) return MOE_ERR_ARG;
  if (c->resid != MOE_FP32 && c->resid != MOE_BF16) return MOE_ERR_ARG;
  if (c->resid == MOE_BF16 && c->dtype != MOE_BF16) return MOE_ERR_ARG;
  if (c->gate_len < 0 || !(c->eps > 0.f) || !(c->alpha == c->alpha)) return MOE_ERR_ARG;
  return MOE_OK;
}

bool several_rows(const moe_norm_config_t* c) { return c->gate_len > 0 && c->gate_len < c->T; }
// Threads of the backward that share an SM.  LayerNorm's 32 column sums a
// thread want 80 registers (with 64 they spill: 16384 rows of 4104 bf16 349
// -> 249 us, of 768 (twice as many) 89 -> 70); fp32 rows, whose rings are
// short, want the threads (4096 fp32: 191 us against 251), and get the
// registers only where a row's threads leave them.
int sm_threads(bool layer, bool bf16) { return layer && bf16 ? 768 : 1024; }
// CTAs an SM holds: more than three leave more partial sums than they gain
// (65536 rows of 256, gate rows of 16: 73 us with up to three, 88 with two,
// 127 with eight).
int bwd_ctas(int sm_threads, int threads) {
  return std::max(1, std::min(3, sm_threads / threads));
}
// The backward's CTAs and their row groups: up to half of an SM's threads a
// CTA, or one row where that takes more.  Row groups share a CTA's partial
// sums, so short batches run fewer CTAs rather than CTAs of one group; with
// short gate segments, which a CTA's groups share, each needs four rows.
// Up to two rows per group of one gate row go to one CTA, which then writes
// the gradients itself: a second launch costs more than a second row.
void bwd_shape(const moe_norm_config_t* c, int* ctas, int* groups) {
  const int tpr = threads_per_row(c->D);
  const int on_sm = sm_threads(c->norm == MOE_LAYERNORM, c->dtype == MOE_BF16);
  int64_t R = row_groups(tpr, on_sm / 2);
  if (several_rows(c)) R = std::max<int64_t>(1, std::min<int64_t>(R, c->gate_len / 4));
  const int64_t most = (int64_t)kSms * bwd_ctas(on_sm, (int)R * tpr);
  *ctas = (int)std::max<int64_t>(1, std::min<int64_t>(most, host::ceil_div(c->T, R)));
  if (!several_rows(c) && c->T <= 2 * R) *ctas = 1;
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
bool any_misaligned(uintptr_t to, P... p) {
  return (host::misaligned(p, to) || ...);
}

// Calls f with the template's truth values for two run-time ones.
template <typename F>
int with_flags(bool p, bool q, F f) {
  if (p) return q ? f(std::true_type{}, std::true_type{}) : f(std::true_type{}, std::false_type{});
  return q ? f(std::false_type{}, std::true_type{}) : f(std::false_type{}, std::false_type{});
}

template <typename TA, typename TR>
int forward(NormArgs a, cudaStream_t s) {
  const bool bias = a.b_post != nullptr || a.b_pre != nullptr;
  const norm_shape::Forward f =
      norm_shape::forward(a.T, a.D, host::sm_count(), kPiece<TA> + kPiece<TR>, bias);
  a.R = f.R;
  a.stages = f.stages;
  a.bias_smem = f.bias_smem;
  auto go = [&](auto k) {
    MOE_HTRY(host::allow_smem(k, kDynSmem));
    return host::launch("block_norm", k, f.grid, f.threads, (size_t)f.smem, s, 1, a);
  };
  return with_flags(bias, a.D % 256 == 0, [&](auto b, auto full) {
    constexpr bool B = decltype(b)::value, F = decltype(full)::value;
    if (f.small) return go(block_norm_kernel<TA, TR, B, F, true>);
    return go(block_norm_kernel<TA, TR, B, F, false>);
  });
}

template <typename TA, typename TR>
int backward(NormArgs a, int P, bool bias, cudaStream_t s) {
  const int threads = a.R * a.tpr;
  const bool general = bias || a.layer;
  const size_t stage = 2 * (size_t)(kPiece<TA> + kPiece<TR>) * threads;
  const size_t swap = a.R > 1 ? (size_t)threads * 32 : 0;
  size_t fixed = (size_t)a.tpr * 64 + (a.several ? swap : 0);
  // two CTAs an SM share its shared memory (8 KB static and 1 KB of the
  // system's each)
  const int ctas = bwd_ctas(sm_threads(a.layer, sizeof(TA) == 2), threads);
  const int on_sm = ctas * threads;
  const size_t room = (kSmemLimit + 1024) / ctas - 9 * 1024;
  // the running sums for w_post where a ring of two rows still fits
  const size_t w_bytes = (general ? 2 : 1) * (size_t)a.D * 4;
  a.w_smem = a.several && fixed + w_bytes + 2 * stage <= room;
  if (a.w_smem) fixed += w_bytes;
  // a ring of one stage would overlap nothing: where two do not fit, rows are
  // read where they are used.  That is so for fp32 rows of most widths (at 768
  // and 2048 columns two CTAs of about 500 threads have 105 KB each and a stage
  // takes 60 to 64; at 7168 one CTA has 219 KB and a stage takes 112), and for
  // an fp32 stream beside bf16 rows of 4096
  a.stages = (int)std::min<size_t>(3, (room - fixed) / stage);
  if (a.stages < 2) a.stages = 0;
  a.swap_ring = !a.several && a.stages > 0;      // (a stage is at least the buffer's size)
  if (!a.several && !a.swap_ring) fixed += swap;
  const size_t smem = a.stages * stage + fixed;
  auto go = [&](auto k) {
    MOE_HTRY(host::allow_smem(k, kDynSmem));
    return host::launch("block_norm_bwd", k, P, threads, smem, s, 1, a);
  };
  a.finish = P == 1 && !a.several;
  MOE_HTRY(with_flags(general, a.several != 0, [&](auto ge, auto se) {
    constexpr bool G = decltype(ge)::value, S = decltype(se)::value;
    auto full = [&](auto n) {
      constexpr int N = G ? decltype(n)::value : kMaxThreads;
      return a.D % 256 == 0 ? go(block_norm_bwd_kernel<TA, TR, G, S, true, N>)
                            : go(block_norm_bwd_kernel<TA, TR, G, S, false, N>);
    };
    if (on_sm <= 768) return full(std::integral_constant<int, 768>{});
    if (on_sm <= 896) return full(std::integral_constant<int, 896>{});
    return full(std::integral_constant<int, kMaxThreads>{});
  }));
  if (a.finish) return MOE_OK;
  SumArgs sum{};
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
  if (any_misaligned(16, r, y, w_post, b_post, gate, w_pre, b_pre, r_out, x, stats)) return MOE_ERR_ARG;
  NormArgs a = args_of(c);
  if (y == nullptr) a.gate_len = 0;
  a.r = r; a.y = y; a.w_post = w_post; a.b_post = b_post; a.gate = gate; a.w_pre = w_pre;
  a.b_pre = b_pre; a.r_out = r_out; a.x = x; a.stats = stats;
  a.wide = !any_misaligned(32, r_out, x);
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
  if (any_misaligned(16, r_out, y, w_post, b_post, gate, w_pre, stats, dx, dr_out, dy, dr, dgate, ws))
    return MOE_ERR_ARG;
  NormArgs a = args_of(c);
  if (y == nullptr) a.gate_len = 0;
  a.r = r_out; a.y = y; a.w_post = w_post; a.b_post = b_post; a.gate = gate; a.w_pre = w_pre;
  a.stats_in = stats; a.dx = dx; a.dr_out = dr_out; a.dy = dy; a.dr = dr; a.dgate = dgate;
  a.part = static_cast<float*>(ws);
  a.wide = !any_misaligned(32, dy, dr);
  a.several = y != nullptr && several_rows(c);
  a.dw_post = dw_post; a.db_post = db_post; a.dw_pre = dw_pre; a.db_pre = db_pre;
  int P = 0;
  bwd_shape(c, &P, &a.R);
  const bool bias = db_post != nullptr || db_pre != nullptr || (dgate != nullptr && b_post != nullptr);
  if (c->dtype == MOE_FP32) return backward<float, float>(a, P, bias, s);
  if (c->resid == MOE_FP32) return backward<__nv_bfloat16, float>(a, P, bias, s);
  return backward<__nv_bfloat16, __nv_bfloat16>(a, P, bias, s);
}

}  // extern "C"
