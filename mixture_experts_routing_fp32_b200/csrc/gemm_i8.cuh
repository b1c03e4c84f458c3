// Grouped tensor-core products in 8-bit integers (tcgen05 kind::i8) with a
// scale for each row (token) and each column (output channel):
//
//   C[r, n] = s_r t_{e,n} sum_k A[r, k] B_e[n, k]       (sums in int32, exact)
//
// over the permuted rows of the dispatch, for the two products of the SwiGLU
// experts: gate/up (the epilogue forms h = silu(a) b in fp32, writes it and
// keeps each row's largest |h|) and down (bf16 out).
//
// The down product's rows are rounded to bf16 here and their weighted sum once
// more in the combine, as the bf16 layer's are (moe_combine reads bf16 rows):
// y is 0.0023-0.0025 off in the 2-norm, 0.0017 with one rounding; fp32 rows
// would move 537 MB more on OLMoE-shaped prompts (83 us at the copy rate,
// beside 573).
//
// The kernel is the bf16 grouped product's in outline: persistent CTAs (or
// CTA pairs sharing 256-row MMAs), a TMA producer warp filling a ring of
// 128-byte-swizzled stages, one thread issuing MMAs (K = 32) into a ring of
// accumulators in tensor memory, eight epilogue warps.  In bytes a stage is
// the bf16 kernel's (128 bytes of k per row, now 128 elements), and every
// MMA does twice the products on them, so the operands' way into the SM
// bounds it sooner.  Experts of few rows (decoding) run in a second
// kernel, at the end of this file.
#pragma once
#include "f32x2.cuh"
#include "gemm_tc.cuh"

namespace moe {
namespace i8 {

using namespace tc;

constexpr int kBK = 128;          // k per stage: one 128-byte swizzle row
constexpr int kUmmaK = 32;        // k of one 8-bit MMA
enum { I8_SWIGLU = 0, I8_STORE = 1 };

struct Params {
  int E, F, nk, nN, group_m;
  const int32_t* tile_expert;
  const int32_t* tile_rows;       // rows in use of each 128-row tile
  const int32_t* stats;           // stats[3]: 128-row tiles in use
  const float* row_scale;         // I8_SWIGLU: s_r
  unsigned* row_max;              // I8_SWIGLU out / I8_STORE in: bits of max |h| of each row
  const float* col_scale;         // [E, cols]
  const float* col_scale_s;       // shared expert
  int cols;                       // 2F or D
};

__device__ __forceinline__ void umma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
__device__ __forceinline__ void umma_i8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
// Instruction descriptor: kind::i8, s8 x s8 -> s32, both operands K-major.
__host__ __device__ constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
// Loads of host::make_map_k boxes: k block kb, rows from r, half h, matrix e.
__device__ __forceinline__ void tma_k(uint32_t dst, const CUtensorMap* map, uint32_t bar, int kb,
                                      int r, int h, int e, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(r), "r"(h), "r"(kb), "r"(e), "r"(bar),
      "l"(pol)
      : "memory");
}
__device__ __forceinline__ void tma_k_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                           int kb, int r, int h, int e, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(r), "r"(h), "r"(kb), "r"(e), "r"(bar),
      "l"(pol)
      : "memory");
}
__device__ __forceinline__ uint64_t policy_normal() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// Scale of a row from the bits of its largest |h|; NaN when that is not
// finite (its 8-bit values are zeros then).
__device__ __forceinline__ float scale_of(unsigned bits) {
  return bits >= 0x7f800000u ? __int_as_float(0x7fffffff) : __uint_as_float(bits) / 127.0f;
}

// KB k blocks to a stage, each operand's by one copy: the producer thread
// needs about 350 ns for a stage's wait, arming and copies, whatever they
// move.  Pair tiles and 128-wide ones take two (64 KB and 48-64 KB stages);
// two 96 KB stages of the 256-wide single tile would be too few.
template <int BN, bool PAIR>
constexpr int kKb = (PAIR || BN == 128) ? 2 : 1;

template <int BN, int STAGES, bool PAIR>
struct Smem {
  static constexpr int KB = kKb<BN, PAIR>;
  static constexpr int BNC = PAIR ? BN / 2 : BN;      // columns of B this CTA holds
  static constexpr int NACC = BN <= 128 ? 4 : 2;
  static constexpr int kA = BM * kBK;
  static constexpr int kB = BNC * kBK;
  static constexpr int kStage = KB * (kA + kB);       // [A of each k block | B of each]
  static constexpr int kBars = (2 * STAGES + 2 * NACC + 1) * 8;
  static constexpr int kEpiOff = (STAGES * kStage + kBars + 16 + 1023) / 1024 * 1024;
  static constexpr int kStgW = 4096;                  // one 32 x 32 fp32 box, or two bf16 boxes
  static constexpr int kBytes = 1024 + kEpiOff + kEpiWarps * kStgW;
  static_assert(kBytes <= 232448 - 64, "shared memory per CTA");
};

struct Tile8 {
  int e, m0, n0, rows;
};

template <int EPI, int BN, bool PAIR>
__device__ __forceinline__ Tile8 decode8(int t, const Params& p, int rank, int n_mt) {
  constexpr int MU = PAIR ? 2 * BM : BM;
  const int group = t / (p.group_m * p.nN);
  const int first = group * p.group_m;
  const int gm = min(p.group_m, n_mt - first);
  const int local = t - group * p.group_m * p.nN;
  const int mt = first + local % gm, nt = local / gm;
  Tile8 d;
  d.e = p.tile_expert[mt * (MU / BM)];
  d.m0 = mt * MU + rank * BM;
  d.n0 = nt * (EPI == I8_SWIGLU ? BN / 2 : BN);
  d.rows = p.tile_rows[mt * (MU / BM) + rank];
  return d;
}

// mapA: [rows_max][K]; mapB / mapBs: [E][halves][cols][K] (the shared expert's own); mapO: h [rows_max][F]
// fp32, or o [rows_max][D] bf16, for the epilogue's TMA stores.
template <int BN, int STAGES, int EPI, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
gemm_i8_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB, const __grid_constant__ CUtensorMap mapBs,
               const __grid_constant__ CUtensorMap mapO, const Params p) {
  using S = Smem<BN, STAGES, PAIR>;
  constexpr int NACC = S::NACC, KB = S::KB;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int abort_flag_s;
  volatile int* abort_flag = &abort_flag_s;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + STAGES * S::kStage;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (STAGES + s); };
  auto accf_bar = [&](int b) { return bars + 8u * (2 * STAGES + b); };
  auto acce_bar = [&](int b) { return bars + 8u * (2 * STAGES + NACC + b); };
  const uint32_t done_bar = bars + 8u * (2 * STAGES + 2 * NACC);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + STAGES * S::kStage + S::kBars);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? (int)cluster_rank() : 0;
  const bool leader = rank == 0;
  const int unit = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  const int n_units = PAIR ? gridDim.x >> 1 : gridDim.x;
  constexpr uint32_t kCols = 512;
  static_assert(NACC * BN == kCols, "tensor-memory columns");

  if (threadIdx.x == 0) {
    abort_flag_s = 0;
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < NACC; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), kEpiWarps * (PAIR ? 2 : 1));
    }
    mbar_init(done_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0) {
    __syncwarp();
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(tmem_slot)),
                   "r"(kCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(tmem_slot)),
                   "r"(kCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_begin();

  const int n_mt = p.stats[3] / (PAIR ? 2 : 1);
  const int total = n_mt * p.nN;
  auto decode_at = [&](int t) {
    return t < total ? decode8<EPI, BN, PAIR>(t, p, rank, n_mt) : Tile8{0, 0, 0, 0};
  };

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer (both CTAs of a pair) ----------------
      const uint64_t pol_a = policy_evict_last(), pol_b = policy_normal();
      int stage = 0;
      uint32_t phase = 0;
      int issued_parity[STAGES];
#pragma unroll
      for (int s = 0; s < STAGES; ++s) issued_parity[s] = -1;
      bool ok = true;
      Tile8 nxt = decode_at(unit);
      for (int t = unit; t < total && ok; t += n_units) {
        const Tile8 d = nxt;
        nxt = decode_at(t + n_units);
        const CUtensorMap* mb = d.e >= p.E ? &mapBs : &mapB;
        const int eb = d.e >= p.E ? 0 : d.e;
        for (int kb = 0; kb < p.nk; kb += KB) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag)) { ok = false; break; }
          const uint32_t sa = base + stage * S::kStage;
          const uint32_t sb = sa + KB * S::kA;
          const uint32_t fb = full_bar(stage);
          if (!PAIR || leader) mbar_expect_tx(fb, (PAIR ? 2 : 1) * S::kStage);
          issued_parity[stage] = (int)phase;
          if constexpr (PAIR) {
            const uint32_t lfb = mapa(fb, 0);
            tma_k_pair(sa, &mapA, lfb, kb, d.m0, 0, 0, pol_a);
            // SwiGLU: this CTA holds the gate (rank 0) or the up (rank 1) rows
            tma_k_pair(sb, mb, lfb, kb, EPI == I8_SWIGLU ? d.n0 : d.n0 + rank * (BN / 2),
                       EPI == I8_SWIGLU ? rank : 0, eb, pol_b);
          } else {
            tma_k(sa, &mapA, fb, kb, d.m0, 0, 0, pol_a);
            tma_k(sb, mb, fb, kb, d.n0, 0, eb, pol_b);   // (SwiGLU: gate and up rows)
          }
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // the copies this CTA's barriers track have landed before teardown
      if (!PAIR || leader)
        for (int s = 0; s < STAGES; ++s)
          if (issued_parity[s] >= 0) mbar_wait(full_bar(s), (uint32_t)issued_parity[s], abort_flag);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (the pair leader only) ----------------
    if (lane == 0 && leader) {
      constexpr uint32_t idesc = idesc_i8(PAIR ? 2 * BM : BM, BN);
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += n_units) {
        if (!mbar_wait(acce_bar(acc), acc_phase ^ 1u, abort_flag)) break;
        tc_fence_after();
        const uint32_t dt = tmem + acc * BN;
        for (int kb = 0; kb < p.nk; kb += KB) {
          if (!mbar_wait(full_bar(stage), phase, abort_flag)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < KB; ++j) {      // (a block past the last holds zeros)
            const uint32_t sa = base + stage * S::kStage + j * S::kA;
            const uint32_t sb = base + stage * S::kStage + KB * S::kA + j * S::kB;
#pragma unroll
            for (int ks = 0; ks < kBK / kUmmaK; ++ks) {
              const uint64_t ad = sw128_desc(sa + ks * kUmmaK, 16, 1024);
              const uint64_t bd = sw128_desc(sb + ks * kUmmaK, 16, 1024);
              if constexpr (PAIR) umma_i8_pair(dt, ad, bd, idesc, (kb | j | ks) != 0 ? 1u : 0u);
              else umma_i8(dt, ad, bd, idesc, (kb | j | ks) != 0 ? 1u : 0u);
            }
          }
          if constexpr (PAIR) umma_commit_pair_both(empty_bar(stage));
          else umma_commit(empty_bar(stage));
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        if (!ok) break;
        if constexpr (PAIR) umma_commit_pair_both(accf_bar(acc));
        else umma_commit(accf_bar(acc));
        if (++acc == NACC) { acc = 0; acc_phase ^= 1u; }
      }
      if constexpr (PAIR) umma_commit_pair_local(done_bar);
      else umma_commit(done_bar);
      mbar_wait(done_bar, 0, abort_flag);
    }
  } else {
    // ---------------- epilogue (warps 2..9) ----------------
    // Two warps per TMEM lane quarter; warp half hh takes half of the columns.
    const int q = warp & 3;
    const int hh = (warp - 2) >> 2;
    const uint32_t stg = base + S::kEpiOff + (warp - 2) * S::kStgW;
    int acc = 0, box = 0;
    uint32_t acc_phase = 0;
    Tile8 nxt = decode_at(unit);
    for (int t = unit; t < total; t += n_units) {
      const Tile8 d = nxt;
      nxt = decode_at(t + n_units);
      const int row0 = d.m0 + q * 32;
      const bool any = d.rows > q * 32;                 // some row of this warp holds a token
      const bool valid = d.rows > q * 32 + lane;
      float rs = 0.f;
      if (valid) rs = EPI == I8_SWIGLU ? p.row_scale[row0 + lane] : scale_of(p.row_max[row0 + lane]);
      const float* cs = d.e >= p.E ? p.col_scale_s : p.col_scale + (int64_t)d.e * p.cols;
      bool ok = (lane == 0) ? mbar_wait(accf_bar(acc), acc_phase, abort_flag) : true;
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      tc_fence_after();
      const uint32_t trow = tmem + acc * BN + ((uint32_t)(q * 32) << 16);
      if (any) {
        if constexpr (EPI == I8_SWIGLU) {
          // gate columns [0, HB) and up columns behind them, for F columns
          // n0 ..
          constexpr int HB = BN / 2, HJ = HB / 2;       // HJ: this warp's share
          unsigned big = 0;
#pragma unroll 1
          for (int c = 0; c < HJ; c += 32) {
            const int j = hh * HJ + c;
            uint32_t ra[32], rb[32];
            tmem_ld32(trow + j, ra);
            tmem_ld32(trow + HB + j, rb);
            const int f0 = d.n0 + j;
            const float4* ca = reinterpret_cast<const float4*>(cs + f0);
            const float4* cb = reinterpret_cast<const float4*>(cs + p.F + f0);
            tmem_wait();
            float h[32];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 sa = __ldg(ca + i), sb = __ldg(cb + i);
              const float wa[4] = {sa.x, sa.y, sa.z, sa.w}, wb[4] = {sb.x, sb.y, sb.z, sb.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float a = __int2float_rn((int)ra[4 * i + k]) * (rs * wa[k]);
                const float b = __int2float_rn((int)rb[4 * i + k]) * (rs * wb[k]);
                const float v = a * fast_sigmoid(a) * b;
                h[4 * i + k] = v;
                big = max(big, __float_as_uint(v) & 0x7fffffffu);
              }
            }
            if (lane == 0) bulk_wait_read_0();
            __syncwarp();
            stage_box_f32_sw128(stg, h);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&mapO, stg, f0, row0);
              bulk_commit();
            }
          }
          if (valid) atomicMax(p.row_max + row0 + lane, big);
        } else {
          // 32 columns at a time; the next ones' accumulators and scales are
          // on their way while these are scaled and stored (a chunk that
          // waits for its own took 1400 cycles, four of them longer than a
          // short tile's products)
          constexpr int NC = BN / 2 / 32;
          const int n = d.n0 + hh * (BN / 2);
          const uint32_t at = trow + hh * (BN / 2);
          const float4* cn = reinterpret_cast<const float4*>(cs + n);
          uint32_t r[2][32];
          float4 sc[2][8];
          tmem_ld32(at, r[0]);
#pragma unroll
          for (int i = 0; i < 8; ++i) sc[0][i] = __ldg(cn + i);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            tmem_wait();
            if (c + 1 < NC) {
              tmem_ld32(at + 32 * (c + 1), r[(c + 1) & 1]);
#pragma unroll
              for (int i = 0; i < 8; ++i) sc[(c + 1) & 1][i] = __ldg(cn + 8 * (c + 1) + i);
            }
            const uint32_t(&a)[32] = r[c & 1];
            const uint64_t rs2 = pack2(rs, rs);
            uint4 u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              F8 v;
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float4 w = sc[c & 1][2 * j + i];
                const uint32_t* q4 = a + 8 * j + 4 * i;
                v.p[2 * i] = mul2(pack2(__int2float_rn((int)q4[0]), __int2float_rn((int)q4[1])),
                                  mul2(rs2, pack2(w.x, w.y)));
                v.p[2 * i + 1] = mul2(pack2(__int2float_rn((int)q4[2]), __int2float_rn((int)q4[3])),
                                      mul2(rs2, pack2(w.z, w.w)));
              }
              u[j] = narrow8(v);
            }
            const uint32_t buf = stg + box * kTmaBox;
            box ^= 1;
            if (lane == 0) bulk_wait_read_1();
            __syncwarp();
            stage_box_sw64(buf, u);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&mapO, buf, n + 32 * c, row0);
              bulk_commit();
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (!PAIR || leader) mbar_arrive(acce_bar(acc));
        else mbar_arrive_remote(mapa(acce_bar(acc), 0));
      }
      if (++acc == NACC) { acc = 0; acc_phase ^= 1u; }
    }
    if (lane == 0) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();
  tc_fence_after();
  if (warp == 0) {
    __syncwarp();
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols)
                   : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols)
                   : "memory");
  }
}

// ---------------------------------------------------------------------------
// Experts of few rows
// ---------------------------------------------------------------------------
// With a handful of tokens per expert a product is bound by reading its
// weights once, so the operands change places: 128 weight rows are the MMA's
// M side and NT = 16, 32 or 64 tokens its N side, and of a stage's bytes all
// but the tokens' few are weights.  A stage holds two k blocks, each
// operand's brought by one copy, and the stages together 128 to 192 KB of
// weights per SM: under full load a copy takes about 3 us from issue to
// arrival here, so DRAM's rate needs some 20 MB in flight over the 148 SMs
// (the general kernel's narrow tiles held 8 MB and read the Mixtral-shaped
// down projection at 2.7 TB/s), and the producer thread needs about 350 ns
// for a stage, which held stages of 16 KB to 45 GB/s per SM.
//
// Accumulators are [channel][token]: a lane owns a channel, so a token's
// outputs leave as coalesced 32-lane rows.  A gate/up tile holds 64 gate
// rows (lanes 0-63) and the 64 up rows of the same channels (lanes 64-127);
// the up warps pass their values through shared memory.  More than NT tokens
// in a 128-row tile run in turns over the same weights (the second turn
// reads them from L2).
constexpr int kThinKb = 2;
template <int NT>
struct ThinSmem {
  static constexpr int kA = 128 * kBK;
  static constexpr int kB = NT * kBK;
  static constexpr int kStage = kThinKb * (kA + kB);
  static constexpr int kStages = NT == 16 ? 6 : NT == 32 ? 5 : 4;
  static constexpr int NACC = 4;
  static constexpr int kAccCols = NT < 32 ? 32 : NT;     // columns of an accumulator
  static constexpr int kHalves = NT > 32 ? 2 : 1;        // 32-token halves of a turn
  static constexpr int kBars = (2 * kStages + 2 * NACC + 1) * 8;
  // the gate/up form's exchange buffer, [pair of warps][token][channel] fp32
  static constexpr int kSwapOff = kStages * kStage;
  static constexpr int kBarOff = kSwapOff + 2 * kHalves * 32 * 32 * 4;
  static constexpr int kBytes = 1024 + kBarOff + kBars + 16;
  static_assert(kBytes <= 232448 - 64, "shared memory per CTA");
};
// Bytes to come on `bar`, without an arrival.
__device__ __forceinline__ void mbar_expect_only(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
// Both warps of a pair (64 threads, named barrier `bar`): whether v holds in both.
__device__ __forceinline__ bool pair_and(int bar, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(v ? 1 : 0), "r"(bar)
      : "memory");
  return r != 0;
}

// Asks for a box of a weight tensor to be brought into L2.
__device__ __forceinline__ void prefetch_k(const CUtensorMap* map, int kb, int r, int e) {
  asm volatile("cp.async.bulk.prefetch.tensor.5d.L2.global.tile [%0, {%1, %2, %3, %4, %5}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(0), "r"(r), "r"(0), "r"(kb), "r"(e)
               : "memory");
}
// A thin product that follows: what its blocks load first.  A decoded
// token's kernels are short against DRAM's latency, so a kernel that has
// issued its own loads brings the next product's first stages (at most 28 MB)
// into L2.
struct Ahead {
  int E, nN, nk, ctas, ch, stages;       // ch: channels of a tile
  __device__ __forceinline__ void bring(const CUtensorMap* w, const CUtensorMap* ws,
                                        const int32_t* tile_expert, int n_mt, int b) const {
    if (b >= min(ctas, n_mt * nN)) return;
    const int e = __ldcg(tile_expert + b / nN), r = b % nN * ch;
    for (int k = 0; k < min(nk, stages * kThinKb); k += kThinKb)
      prefetch_k(e >= E ? ws : w, k, r, e >= E ? 0 : e);
  }
};

struct ThinParams {
  Params p;
  Ahead next;                    // I8_SWIGLU: the down product
  float* h;                      // I8_SWIGLU out [rows_max, F]
  __nv_bfloat16* o;              // I8_STORE out [rows_max, cols]
};

template <int EPI, int NT>
__global__ void __launch_bounds__(kThreads, 1)
gemm_i8_thin_kernel(const __grid_constant__ CUtensorMap mapW,
                    const __grid_constant__ CUtensorMap mapWs,
                    const __grid_constant__ CUtensorMap mapT,
                    const __grid_constant__ CUtensorMap mapN,
                    const __grid_constant__ CUtensorMap mapNs, const ThinParams tp) {
  using S = ThinSmem<NT>;
  const Params& p = tp.p;
  constexpr int STAGES = S::kStages, NACC = S::NACC, KB = kThinKb;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int abort_flag_s;
  volatile int* abort_flag = &abort_flag_s;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + S::kBarOff;
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (STAGES + s); };
  auto accf_bar = [&](int b) { return bars + 8u * (2 * STAGES + b); };
  auto acce_bar = [&](int b) { return bars + 8u * (2 * STAGES + NACC + b); };
  const uint32_t done_bar = bars + 8u * (2 * STAGES + 2 * NACC);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + S::kBarOff + S::kBars);
  float* swap = reinterpret_cast<float*>(gbase + S::kSwapOff);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr uint32_t kCols = NACC * S::kAccCols;
  if (threadIdx.x == 0) {
    abort_flag_s = 0;
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < NACC; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), kEpiWarps);
    }
    mbar_init(done_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // a tile: 64 channels of F (gate and up rows), or 128 output channels
  constexpr int kCh = EPI == I8_SWIGLU ? 64 : 128;
  const int n_mt = __ldcg(p.stats + 3);
  const int total = n_mt * p.nN;
  struct T {
    int e, m0, n0, rows;
  };
  auto decode_at = [&](int t) {
    if (t >= total) return T{0, 0, 0, 0};
    const int mt = t / p.nN, nt = t - mt * p.nN;
    // (a tile in use holds a row; one without would leave requested weights
    // unused)
    return T{__ldcg(p.tile_expert + mt), mt * BM, nt * kCh, max(1, __ldcg(p.tile_rows + mt))};
  };
  const uint64_t pol = policy_normal();
  auto load_weights = [&](int s, int kb, int n0, int e) {
    tma_k(base + s * S::kStage, e >= p.E ? &mapWs : &mapW, full_bar(s), kb, n0, 0,
          e >= p.E ? 0 : e, pol);
  };
  // The first stages' weights are requested before the wait for the previous
  // kernel of the stream: they and the dispatch's tables are older than it
  // (each kernel here lets its successor start only once its own predecessor
  // is complete, and between the dispatch and either product runs another
  // kernel), so their way overlaps that kernel.  The stage's barrier is told
  // of the bytes without an arrival; that follows with the tokens' bytes.
  int early = 0;
  if (warp == 0 && lane == 0 && (int)blockIdx.x < total) {
    const int t = blockIdx.x;
    const int e = __ldcg(p.tile_expert + t / p.nN), n0 = t % p.nN * kCh;
    early = min(STAGES, (p.nk + KB - 1) / KB);
    for (int s = 0; s < early; ++s) {
      mbar_expect_only(full_bar(s), KB * S::kA);
      load_weights(s, s * KB, n0, e);
    }
  }
  pdl_begin();

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int issued_parity[STAGES];
#pragma unroll
      for (int s = 0; s < STAGES; ++s) issued_parity[s] = s < early ? 0 : -1;
      // the same stages' tokens: the tile's first turn starts at its first
      // row whatever else it holds
      for (int s = 0; s < early; ++s) {
        mbar_expect_tx(full_bar(s), KB * S::kB);
        tma_k(base + s * S::kStage + KB * S::kA, &mapT, full_bar(s), s * KB,
              (int)blockIdx.x / p.nN * BM, 0, 0, pol);
      }
      bool ok = true;
      T nxt = decode_at(blockIdx.x);
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const T d = nxt;
        nxt = decode_at(t + gridDim.x);
        for (int r0 = 0; r0 < d.rows && ok; r0 += NT) {
          for (int kb = 0; kb < p.nk; kb += KB) {
            if (early > 0) {              // on its way already
              --early;
            } else {
              if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag)) { ok = false; break; }
              const uint32_t fb = full_bar(stage);
              mbar_expect_tx(fb, S::kStage);
              load_weights(stage, kb, d.n0, d.e);
              issued_parity[stage] = (int)phase;
              tma_k(base + stage * S::kStage + KB * S::kA, &mapT, fb, kb, d.m0 + r0, 0, 0, pol);
            }
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          }
        }
      }
      if (EPI == I8_SWIGLU)
        for (int b = blockIdx.x; b < tp.next.ctas; b += gridDim.x)
          tp.next.bring(&mapN, &mapNs, p.tile_expert, n_mt, b);
      for (int s = 0; s < STAGES; ++s)
        if (issued_parity[s] >= 0) mbar_wait(full_bar(s), (uint32_t)issued_parity[s], abort_flag);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_i8(BM, NT);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      T nxt = decode_at(blockIdx.x);
      for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
        const T d = nxt;
        nxt = decode_at(t + gridDim.x);
        for (int r0 = 0; r0 < d.rows && ok; r0 += NT) {
          if (!mbar_wait(acce_bar(acc), acc_phase ^ 1u, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t dt = tmem + acc * S::kAccCols;
          for (int kb = 0; kb < p.nk; kb += KB) {
            if (!mbar_wait(full_bar(stage), phase, abort_flag)) { ok = false; break; }
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < KB; ++j) {      // (a block past the last holds zeros)
              const uint32_t sw = base + stage * S::kStage + j * S::kA;
              const uint32_t st = base + stage * S::kStage + KB * S::kA + j * S::kB;
#pragma unroll
              for (int ks = 0; ks < kBK / kUmmaK; ++ks)
                umma_i8(dt, sw128_desc(sw + ks * kUmmaK, 16, 1024),
                        sw128_desc(st + ks * kUmmaK, 16, 1024), idesc,
                        (kb | j | ks) != 0 ? 1u : 0u);
            }
            umma_commit(empty_bar(stage));
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          umma_commit(accf_bar(acc));
          if (++acc == NACC) { acc = 0; acc_phase ^= 1u; }
        }
      }
      umma_commit(done_bar);
      mbar_wait(done_bar, 0, abort_flag);
    }
  } else {
    // Warp quarter q owns channels (lanes) 32 q ..; half hh the tokens
    // 32 hh .. of the turn.
    const int q = warp & 3, hh = (warp - 2) >> 2;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    T nxt = decode_at(blockIdx.x);
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const T d = nxt;
      nxt = decode_at(t + gridDim.x);
      const float* cs = d.e >= p.E ? p.col_scale_s : p.col_scale + (int64_t)d.e * p.cols;
      // this lane's channel: of the outputs, or of F with its gate or up scale
      const int ch = EPI == I8_SWIGLU ? d.n0 + (q & 1) * 32 + lane : d.n0 + q * 32 + lane;
      const float ws = cs[EPI == I8_SWIGLU && q >= 2 ? p.F + ch : ch];
      for (int r0 = 0; r0 < d.rows; r0 += NT) {
        const int row0 = d.m0 + r0 + hh * 32;
        // tokens of this warp (may be <= 0; with one half, none of hh = 1)
        const int cnt = hh < S::kHalves ? min(min(32, NT), d.rows - r0 - hh * 32) : 0;
        float rs = 0.f;                                   // lane j: scale of token j
        if (lane < cnt)
          rs = EPI == I8_SWIGLU ? p.row_scale[row0 + lane] : scale_of(p.row_max[row0 + lane]);
        ok = (lane == 0) ? mbar_wait(accf_bar(acc), acc_phase, abort_flag) : true;
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        // a gate warp and its up warp go on or give up together; past this
        // both have also read the exchange buffer of the last turn
        if (EPI == I8_SWIGLU) ok = pair_and(1 + (q & 1) + 2 * hh, ok);
        if (!ok) break;
        tc_fence_after();
        uint32_t r[32];
        if (cnt > 0) {
          tmem_ld32(tmem + acc * S::kAccCols + hh * 32 + ((uint32_t)(q * 32) << 16), r);
          tmem_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acce_bar(acc));
        if (++acc == NACC) { acc = 0; acc_phase ^= 1u; }
        if (cnt <= 0) continue;
        if constexpr (EPI == I8_SWIGLU) {
          float* at = swap + ((q & 1) + 2 * hh) * 1024 + lane;
          const int bar = 1 + (q & 1) + 2 * hh;           // the gate warp and the up warp
          if (q >= 2) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j < cnt)
                at[j * 32] = __int2float_rn((int)r[j]) * (__shfl_sync(0xffffffffu, rs, j) * ws);
            asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");
          } else {
            asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");   // the up values are there
            float* h = tp.h + (int64_t)row0 * p.F + ch;
            unsigned mine = 0;                            // lane j: largest |h| of token j
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (j < cnt) {
                const float a = __int2float_rn((int)r[j]) * (__shfl_sync(0xffffffffu, rs, j) * ws);
                const float v = a * fast_sigmoid(a) * at[j * 32];
                h[(int64_t)j * p.F] = v;
                const unsigned big = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu);
                if (lane == j) mine = big;
              }
            }
            if (lane < cnt) atomicMax(p.row_max + row0 + lane, mine);
          }
        } else {
          __nv_bfloat16* o = tp.o + (int64_t)row0 * p.cols + ch;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j < cnt)
              o[(int64_t)j * p.cols] = __float2bfloat16_rn(
                  __int2float_rn((int)r[j]) * (__shfl_sync(0xffffffffu, rs, j) * ws));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols)
                 : "memory");
  }
}

}  // namespace i8
}  // namespace moe
