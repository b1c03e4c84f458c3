// The experts in 8-bit integers: row quantisation, the quantised dispatch of
// tokens, the two grouped products (gemm_i8.cuh) and the requantisation of h
// between them.
//
//   q(v)_j = round(127 v_j / max|v|),  s(v) = max|v| / 127   for a row v
//
// The quotient is formed as a division of 127 v_j (exact for bf16 v_j), so a
// tie of the definition is a tie here and goes to even.
#include "host.cuh"
#include "gemm_i8.cuh"

namespace moe {
namespace {

constexpr int kQThreads = 128;    // a row's threads: 16 columns each and turn
constexpr int kHThreads = 256;
constexpr int kMaxCols = 65536;

// Power of two that keeps 127 v and the quotient's parts in range whatever
// the row's magnitude (exact, so the quotient does not change).
__device__ __forceinline__ float range_shift(float big) {
  return big < 7.9e-31f ? 1.8446744e19f : big > 1e36f ? 9.765625e-4f : 1.0f;   // 2^64, 2^-10
}
__device__ __forceinline__ uint32_t pack4_i8(const int* q) {
  return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
}
__device__ __forceinline__ uint4 pack16_i8(const int* q) {
  return make_uint4(pack4_i8(q), pack4_i8(q + 4), pack4_i8(q + 8), pack4_i8(q + 12));
}
// Largest magnitude's bits over the block (NaN orders above infinity).
__device__ __forceinline__ unsigned block_max(unsigned v, unsigned* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();            // the previous row's readers are done
  if (lane == 0) red[warp] = v;
  __syncthreads();
  return max(max(red[0], red[1]), max(red[2], red[3]));
}
__device__ __forceinline__ unsigned max_bits(const float* f, unsigned m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  return m;
}

// One row per block and turn: NV pieces of 16 columns per thread (the last
// one 8 where the row ends) stay in registers between the maximum and the
// rounding; NV = 0: rows longer than that are read twice (the second time
// from L2).  out(col, u) stores 16 values, out(col, lower half, true) 8; the
// scale is returned.
template <typename TX, int NV, typename Out>
__device__ __forceinline__ float quantise_row(const TX* x, int cols, unsigned* red, Out out) {
  unsigned m = 0;
  constexpr int kStep = kQThreads * 16;
  Raw8<TX> keep[NV > 0 ? 2 * NV : 1];
  const int c0 = threadIdx.x * 16;
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < 2 * NV; ++i) {
      const int c = c0 + (i >> 1) * kStep + (i & 1) * 8;
      if (c < cols) keep[i].load(x + c);
    }
#pragma unroll
    for (int i = 0; i < 2 * NV; ++i) {
      float f[8];
      keep[i].widen(f);
      if (c0 + (i >> 1) * kStep + (i & 1) * 8 < cols) m = max_bits(f, m);
    }
  } else {
    for (int c = threadIdx.x * 8; c < cols; c += kQThreads * 8) {
      float f[8];
      load8(x + c, f);
      m = max_bits(f, m);
    }
  }
  m = block_max(m, red);
  const bool finite = m < 0x7f800000u;
  const float big = __uint_as_float(m);
  const float shift = range_shift(big), den = big > 0.f ? big * shift : 1.0f;
  auto round8 = [&](const float* f, int* q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = finite ? __float2int_rn(127.0f * (f[i] * shift) / den) : 0;
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * kStep;
      if (c < cols) {
        float f[8];
        int q[16];
        keep[2 * i].widen(f);
        round8(f, q);
        keep[2 * i + 1].widen(f);
        round8(f, q + 8);        // (unused values behind the row's end)
        out(c, pack16_i8(q), c + 16 <= cols);
      }
    }
  } else {
    for (int c = threadIdx.x * 16; c < cols; c += kStep) {
      float f[8];
      int q[16];
      load8(x + c, f);
      round8(f, q);
      if (c + 16 <= cols) load8(x + c + 8, f);
      round8(f, q + 8);
      out(c, pack16_i8(q), c + 16 <= cols);
    }
  }
  return i8::scale_of(m);
}

template <typename TX, int NV>
__global__ void __launch_bounds__(kQThreads)
quant_rows_kernel(const TX* x, int64_t rows, int cols, int64_t ld, int8_t* q, float* scale) {
  __shared__ unsigned red[kQThreads / 32];
  const bool wide = (cols & 15) == 0 && (reinterpret_cast<uintptr_t>(q) & 15) == 0;
  pdl_begin();
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    int8_t* dst = q + r * cols;
    const float s = quantise_row<TX, NV>(x + r * ld, cols, red, [&](int c, uint4 u, bool whole) {
      if (wide) {
        *reinterpret_cast<uint4*>(dst + c) = u;
      } else {
        *reinterpret_cast<uint2*>(dst + c) = make_uint2(u.x, u.y);
        if (whole) *reinterpret_cast<uint2*>(dst + c + 8) = make_uint2(u.z, u.w);
      }
    });
    if (threadIdx.x == 0) scale[r] = s;
  }
}

// Tokens: each row of x is read and quantised once and its 8-bit form goes
// to every row that holds the token (its slots' rows, the shared expert's).
// The blocks behind the last token count the rows in use of each 128-row
// tile: a routed expert's rows are a prefix of its segment, so the tile's
// count is that of its non-negative row slots.  For experts of few rows
// one more block per block of the gate/up product brings that one's first
// weights into L2 (from one SM its copy engine would take 100 us).
template <int NV>
__global__ void __launch_bounds__(kQThreads)
quant_dispatch_kernel(const __grid_constant__ CUtensorMap mapW,
                      const __grid_constant__ CUtensorMap mapWs, const i8::Ahead next,
                      const int32_t* tile_expert, const __nv_bfloat16* x, int T, int D, int K, int E, int n_shared,
                      const int32_t* offsets, const int32_t* slot_row, const int32_t* row_slot,
                      const int32_t* stats, int token_blocks, int tile_blocks, int8_t* xq, float* scale,
                      unsigned* row_max, int32_t* tile_rows) {
  __shared__ unsigned red[kQThreads / 32];
  const int lane = threadIdx.x & 31;
  pdl_begin();
  if ((int)blockIdx.x >= token_blocks + tile_blocks) {
    if (threadIdx.x == 0)
      next.bring(&mapW, &mapWs, tile_expert, stats[3], blockIdx.x - token_blocks - tile_blocks);
    return;
  }
  if ((int)blockIdx.x >= token_blocks) {
    const int warp = threadIdx.x >> 5;
    const int n_tiles = stats[3], shared0 = offsets[E] / kRowTile;
    const int step = tile_blocks * (kQThreads >> 5);
    for (int t = (blockIdx.x - token_blocks) * (kQThreads >> 5) + warp; t < n_tiles; t += step) {
      int n = 0;
      if (t >= shared0) {
        n = max(0, min(kRowTile, T - (t - shared0) * kRowTile));
      } else {
#pragma unroll
        for (int i = 0; i < kRowTile / 32; ++i)
          n += __popc(__ballot_sync(0xffffffffu, row_slot[t * kRowTile + i * 32 + lane] >= 0));
      }
      if (lane == 0) tile_rows[t] = n;
    }
    return;
  }
  // the rows that hold the token, compacted by the first warp (K is at most
  // 16); two lists take turns, so that a warp still reading one is behind a
  // barrier of the row in between
  __shared__ int held_s[2][32];
  __shared__ int n_held_s[2];
  const int shared_row = n_shared ? offsets[E] : 0;
  int turn = 0;
  for (int t = blockIdx.x; t < T; t += token_blocks, turn ^= 1) {
    int row = -1;
    if (threadIdx.x < 32) {
      if (lane < K) row = slot_row[(int64_t)t * K + lane];
      else if (lane == K && n_shared) row = shared_row + t;
      const unsigned some = __ballot_sync(0xffffffffu, row >= 0);
      if (row >= 0) held_s[turn][__popc(some & ((1u << lane) - 1u))] = row;
      if (lane == 0) n_held_s[turn] = __popc(some);
    }
    // (the barriers of the row's maximum publish the list)
    const float s = quantise_row<__nv_bfloat16, NV>(
        x + (int64_t)t * D, D, red, [&](int c, uint4 u, bool) {
          const int n = n_held_s[turn];
          for (int k = 0; k < n; ++k)
            *reinterpret_cast<uint4*>(xq + (int64_t)held_s[turn][k] * D + c) = u;
        });
    if (row >= 0) {
      scale[row] = s;
      row_max[row] = 0u;
    }
  }
}

// h (fp32, each row's largest magnitude already known from the product's
// epilogue) to 8 bits: 16 columns a thread, 512 a warp and turn.  The values
// are moe_quant_i8's.  A product with 127 / max is within 127 * 4 * 2^-24 <
// 2^-15 of that one's quotient (two roundings each), so the two round alike
// except next to a tie, where the division decides (a warp in 16; dividing
// for every value took 11 of the 582 us of OLMoE-shaped prompts).
__global__ void __launch_bounds__(kHThreads)
quant_h_kernel(const float* h, int F, int64_t rows_max, const int32_t* stats, const int32_t* tile_rows,
               const unsigned* row_max, int8_t* hq) {
  pdl_begin();
  const int lane = threadIdx.x & 31;
  const int per = (F + 511) / 512;
  const int64_t step = (int64_t)gridDim.x * (kHThreads >> 5);
  const int64_t total = (int64_t)stats[2] * per, most = rows_max * per;
  // (a row's facts are asked for whether it is in use or not: one latency
  // instead of three where there are few rows)
  for (int64_t u = (int64_t)blockIdx.x * (kHThreads >> 5) + (threadIdx.x >> 5); u < most;
       u += step) {
    const int64_t r = u / per;
    const int c = (int)(u - r * per) * 512 + lane * 16;
    const int held = tile_rows[r / kRowTile];
    const unsigned bits = row_max[r];
    if (u >= total) break;
    if (c >= F || (int)(r % kRowTile) >= held) continue;
    const float big = __uint_as_float(bits);
    const float shift = range_shift(big);
    const bool some = bits < 0x7f800000u && bits > 0u;
    const float den = some ? big * shift : 1.0f, inv = some ? 127.0f / den : 0.f;
    constexpr float kRound = 12582912.0f;      // 1.5 * 2^23: the sum's low bits are the integer
    float f[16], off = 0.f;
    load8(h + r * F + c, f);
    load8(h + r * F + c + 8, f + 8);
    int q[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float at = some ? f[i] * shift * inv : 0.f, sum = __fadd_rn(at, kRound);
      q[i] = __float_as_int(sum);
      off = fmaxf(off, fabsf(at - __fsub_rn(sum, kRound)));
    }
    if (off > 0.5f - 0x1p-14f) {
#pragma unroll
      for (int i = 0; i < 16; ++i) q[i] = __float2int_rn(127.0f * (f[i] * shift) / den);
    }
    *reinterpret_cast<uint4*>(hq + r * F + c) = pack16_i8(q);
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
struct Work {
  host::LayerView v;
  int64_t xq, xs, h, hq, row_max, tile_rows, total;
};
constexpr int64_t kAlign = 256;

int work_of(const moe_config_t* c, Work* w) {
  MOE_HTRY(host::layer_view(c, &w->v));
  // (sums of 65536 products of 8-bit values stay below 2^31)
  if (!w->v.tensor_cores || c->expert_choice || c->D > kMaxCols || c->F > kMaxCols)
    return MOE_ERR_ARG;
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    const int64_t at = off;
    off += host::ceil_div(bytes, kAlign) * kAlign;
    return at;
  };
  const int64_t R = w->v.rows_max;
  w->xq = take(R * c->D);
  w->xs = take(R * 4);
  w->h = take(R * c->F * 4);
  w->hq = take(R * c->F);
  w->row_max = take(R * 4);
  w->tile_rows = take(w->v.tiles_max * 4);
  w->total = off;
  return MOE_OK;
}

template <int BN, int ST, int EPI, bool PAIR>
int run_gemm(const char* name, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& bs,
             const CUtensorMap& o, const i8::Params& p, int64_t units, cudaStream_t s) {
  using S = i8::Smem<BN, ST, PAIR>;
  auto k = i8::gemm_i8_kernel<BN, ST, EPI, PAIR>;
  MOE_HTRY(host::allow_smem(k, S::kBytes));
  int64_t resident = host::sm_count();
  if (PAIR) MOE_HTRY(host::resident_clusters(k, 2, tc::kThreads, S::kBytes, &resident));
  const int ctas = (int)std::min<int64_t>(resident, units * p.nN) * (PAIR ? 2 : 1);
  return host::launch(name, k, ctas, tc::kThreads, S::kBytes, s, PAIR ? 2 : 1, a, b, bs, o, p);
}

// Row tiles per rasterisation group: as many of depth K bytes as fit in about
// 24 MiB of L2, so that long weights are read for many rows at a time (16384
// rows, 112 MiB of gate/up weights an expert: 1.39 ms, 1.55 with 4 MiB); 4
// MiB where an expert's weights are short enough to stay in L2 anyway (65536
// rows, 4 MiB: 214 us, 222 with 24 MiB; between 8 and 32 MiB both take the
// same time).
int group_rows(int64_t k_bytes, int64_t weight_bytes, bool pair) {
  const int64_t rows = pair ? 256 : 128, room = weight_bytes <= (8 << 20) ? 4 << 20 : 24 << 20;
  return (int)std::max<int64_t>(1, std::min<int64_t>(64, room / (rows * k_bytes)));
}

// Few rows per expert: the weights' way in bounds the product.  A layer pass,
// thin against general kernels: at 8 and 16 rows per expert 101 against 105
// and 106 against 111 us (OLMoE-shaped), at 16 rows 255 against 262
// (Mixtral-shaped), at 24 rows 116 against 113 and 259 against 266, at 64 rows
// 168 against 129.  The shared expert's T rows run in turns over its weights:
// at 64 tokens the thin form already loses (37 against 33 us, 32 experts of
// 1024 x 512).
bool few_rows(const moe_config_t* c, const Work& w) {
  return (int64_t)c->T * c->K <= 16ll * w.v.local_experts && (c->n_shared == 0 || c->T <= 32);
}

// Maps and shape of one thin product's weights.
struct ThinWeights {
  CUtensorMap w, ws;
  i8::Ahead a;
};
template <int EPI>
int thin_weights(const moe_config_t* c, const Work& w, const int8_t* b, const int8_t* b_s,
                 int stages, ThinWeights* t) {
  constexpr uint32_t box = EPI == i8::I8_SWIGLU ? 64 : 128;
  const int64_t K = EPI == i8::I8_SWIGLU ? c->D : c->F;
  t->a.E = w.v.local_experts;
  t->a.ch = (int)box;
  t->a.nN = (EPI == i8::I8_SWIGLU ? c->F : c->D) / (int)box;
  t->a.nk = (int)(K / i8::kBK);
  t->a.ctas = (int)std::min<int64_t>(host::sm_count(), w.v.tiles_max * t->a.nN);
  const int64_t halves = EPI == i8::I8_SWIGLU ? 2 : 1, rows = EPI == i8::I8_SWIGLU ? c->F : c->D;
  t->a.stages = stages;
  MOE_HTRY(host::make_map_k(&t->w, b, w.v.local_experts, halves, rows, K, box, (uint32_t)halves,
                            i8::kThinKb));
  return host::make_map_k(&t->ws, b_s != nullptr ? b_s : b, 1, halves, rows, K, box,
                          (uint32_t)halves, i8::kThinKb);
}

template <int EPI, int NT>
int thin_product(const Work& w, const char* name, const int8_t* a, const ThinWeights& t,
                 const ThinWeights& next, void* out, i8::Params p, cudaStream_t s) {
  auto k = i8::gemm_i8_thin_kernel<EPI, NT>;
  p.E = t.a.E; p.F = EPI == i8::I8_SWIGLU ? t.a.nN * t.a.ch : 0; p.nk = t.a.nk; p.nN = t.a.nN;
  p.cols = EPI == i8::I8_SWIGLU ? 2 * p.F : t.a.nN * t.a.ch;
  CUtensorMap ma;
  MOE_HTRY(host::make_map_k(&ma, a, 1, 1, w.v.rows_max, (int64_t)t.a.nk * i8::kBK, NT, 1,
                            i8::kThinKb));
  i8::ThinParams tp{p, next.a, nullptr, nullptr};
  if (EPI == i8::I8_SWIGLU) tp.h = static_cast<float*>(out);
  else tp.o = static_cast<__nv_bfloat16*>(out);
  constexpr int bytes = i8::ThinSmem<NT>::kBytes;
  MOE_HTRY(host::allow_smem(k, bytes));
  return host::launch(name, k, t.a.ctas, tc::kThreads, bytes, s, 1, t.w, t.ws, ma, next.w, next.ws,
                      tp);
}
// Tokens of an MMA: an expert holds a token once, so T tokens need no more
// than T rows.
int thin_tokens(const moe_config_t* c) { return c->T <= 16 ? 16 : c->T <= 32 ? 32 : 64; }
template <int EPI, typename... A>
int thin_product_of(int nt, A&&... args) {
  if (nt == 16) return thin_product<EPI, 16>(std::forward<A>(args)...);
  if (nt == 32) return thin_product<EPI, 32>(std::forward<A>(args)...);
  return thin_product<EPI, 64>(std::forward<A>(args)...);
}

template <int EPI>
int product(const moe_config_t* c, const Work& w, const char* name, const int8_t* a, int64_t K,
            const int8_t* b, const int8_t* b_s, int64_t cols, void* out, i8::Params p,
            cudaStream_t s) {
  const bool pair = w.v.align == 256;
  const int64_t n_out = EPI == i8::I8_SWIGLU ? c->F : c->D;
  const int64_t E = w.v.local_experts;
  p.E = (int)E; p.F = c->F; p.nk = (int)(K / i8::kBK); p.cols = (int)cols;
  // D and F are multiples of 128: a 256-wide plain tile may not divide D
  const int bn = EPI == i8::I8_STORE && n_out % 256 ? 128 : 256;
  p.nN = (int)(n_out / (EPI == i8::I8_SWIGLU ? bn / 2 : bn));
  p.group_m = group_rows(K, cols * K, pair);
  CUtensorMap ma, mb, mbs, mo;
  const bool sw = EPI == i8::I8_SWIGLU;
  const uint32_t kb = pair || bn == 128 ? 2 : 1;     // i8::kKb
  const uint32_t box = (uint32_t)(sw || pair ? bn / 2 : bn), halves = sw && !pair ? 2 : 1;
  const int64_t rows = sw ? cols / 2 : cols;
  MOE_HTRY(host::make_map_k(&ma, a, 1, 1, w.v.rows_max, K, 128, 1, kb));
  MOE_HTRY(host::make_map_k(&mb, b, E, sw ? 2 : 1, rows, K, box, halves, kb));
  MOE_HTRY(host::make_map_k(&mbs, b_s != nullptr ? b_s : b, 1, sw ? 2 : 1, rows, K, box, halves, kb));
  MOE_HTRY(host::make_out_map(&mo, out, w.v.rows_max, n_out, EPI == i8::I8_SWIGLU));
  const int64_t units = w.v.tiles_max / (pair ? 2 : 1);
  if (pair) {
    if (bn == 256) return run_gemm<256, 3, EPI, true>(name, ma, mb, mbs, mo, p, units, s);
    if constexpr (EPI == i8::I8_STORE)
      return run_gemm<128, 4, EPI, true>(name, ma, mb, mbs, mo, p, units, s);
  }
  if constexpr (EPI == i8::I8_STORE) {
    if (bn == 128) return run_gemm<128, 3, EPI, false>(name, ma, mb, mbs, mo, p, units, s);
  }
  return run_gemm<256, 4, EPI, false>(name, ma, mb, mbs, mo, p, units, s);
}

template <typename TX>
int quant_rows(const TX* x, int64_t rows, int64_t cols, int64_t ld, int8_t* q, float* scale,
               cudaStream_t s) {
  const int grid = (int)std::min<int64_t>(rows, (int64_t)host::sm_count() * 16);
  const int64_t nv = host::ceil_div(cols, kQThreads * 16);
  auto go = [&](auto k) {
    return host::launch("quant_i8", k, grid, kQThreads, 0, s, 1, x, rows, (int)cols, ld, q, scale);
  };
  if (nv <= 1) return go(quant_rows_kernel<TX, 1>);
  if (nv <= 2) return go(quant_rows_kernel<TX, 2>);
  if (nv <= 4) return go(quant_rows_kernel<TX, 4>);
  return go(quant_rows_kernel<TX, 0>);
}

}  // namespace

namespace host {
int take_i8_error(unsigned* bits) {
  unsigned zero = 0;
  MOE_HCK(cudaMemcpyFromSymbol(bits, g_dev_error, sizeof(*bits)));
  if (*bits) MOE_HCK(cudaMemcpyToSymbol(g_dev_error, &zero, sizeof(zero)));
  return MOE_OK;
}
}  // namespace host
}  // namespace moe

using namespace moe;

extern "C" {

int moe_quant_i8(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld_x,
                 int8_t* q, float* scale, cudaStream_t s) {
  if (dtype != MOE_FP32 && dtype != MOE_BF16) return MOE_ERR_ARG;
  if (rows < 0 || cols < 8 || cols > kMaxCols || cols % 8 || ld_x < cols || ld_x % 8)
    return MOE_ERR_ARG;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scale || host::misaligned(x, 16) || host::misaligned(q, 8) ||
      host::misaligned(scale, 4))
    return MOE_ERR_ARG;
  if (dtype == MOE_BF16)
    return quant_rows(static_cast<const __nv_bfloat16*>(x), rows, cols, ld_x, q, scale, s);
  return quant_rows(static_cast<const float*>(x), rows, cols, ld_x, q, scale, s);
}

int64_t moe_expert_ffn_i8_ws_bytes(const moe_config_t* c) {
  Work w;
  return work_of(c, &w) == MOE_OK ? w.total : 0;
}

int moe_expert_ffn_i8(const moe_config_t* c, const void* x, const int32_t* offsets,
                      const int32_t* slot_row, const int32_t* row_slot,
                      const int32_t* tile_expert, const int32_t* stats, const int8_t* w13,
                      const float* w13_scale, const int8_t* w_down, const float* w_down_scale,
                      const int8_t* w13_s, const float* w13_s_scale, const int8_t* w_down_s,
                      const float* w_down_s_scale, void* o, void* ws, cudaStream_t s) {
  Work w;
  MOE_HTRY(work_of(c, &w));
  if (!x || !offsets || !slot_row || !row_slot || !tile_expert || !stats || !w13 || !w13_scale ||
      !w_down || !w_down_scale || !o || !ws)
    return MOE_ERR_ARG;
  if (c->n_shared && (!w13_s || !w13_s_scale || !w_down_s || !w_down_s_scale)) return MOE_ERR_ARG;
  for (const void* p : {x, (const void*)w13, (const void*)w13_scale, (const void*)w_down,
                        (const void*)w_down_scale, (const void*)w13_s, (const void*)w13_s_scale,
                        (const void*)w_down_s, (const void*)w_down_s_scale, (const void*)o})
    if (host::misaligned(p, 16)) return MOE_ERR_ARG;
  if (host::misaligned(ws, kAlign)) return MOE_ERR_ARG;
  uint8_t* base = static_cast<uint8_t*>(ws);
  int8_t* xq = reinterpret_cast<int8_t*>(base + w.xq);
  int8_t* hq = reinterpret_cast<int8_t*>(base + w.hq);
  float* xs = reinterpret_cast<float*>(base + w.xs);
  float* h = reinterpret_cast<float*>(base + w.h);
  unsigned* row_max = reinterpret_cast<unsigned*>(base + w.row_max);
  int32_t* tile_rows = reinterpret_cast<int32_t*>(base + w.tile_rows);
  const int sms = host::sm_count();
  const bool thin = few_rows(c, w);
  const int nt = thin_tokens(c);
  ThinWeights t13{}, td{};
  if (thin) {
    const int st = nt == 16 ? i8::ThinSmem<16>::kStages
                   : nt == 32 ? i8::ThinSmem<32>::kStages : i8::ThinSmem<64>::kStages;
    MOE_HTRY((thin_weights<i8::I8_SWIGLU>(c, w, w13, w13_s, st, &t13)));
    MOE_HTRY((thin_weights<i8::I8_STORE>(c, w, w_down, w_down_s, st, &td)));
  }
  {
    const int tokens = (int)std::min<int64_t>(c->T, (int64_t)sms * 16);
    const int tiles = (int)std::min<int64_t>(host::ceil_div(w.v.tiles_max, kQThreads / 32), 64);
    auto go = [&](auto k) {
      return host::launch("quant_dispatch", k, tokens + tiles + t13.a.ctas, kQThreads, 0, s, 1, t13.w, t13.ws,
                          t13.a, tile_expert, static_cast<const __nv_bfloat16*>(x), c->T, c->D,
                          c->K, w.v.local_experts, c->n_shared, offsets, slot_row, row_slot, stats,
                          tokens, tiles, xq, xs, row_max, tile_rows);
    };
    const int64_t nv = host::ceil_div(c->D, kQThreads * 16);
    if (nv <= 1) MOE_HTRY(go(quant_dispatch_kernel<1>));
    else if (nv <= 2) MOE_HTRY(go(quant_dispatch_kernel<2>));
    else if (nv <= 4) MOE_HTRY(go(quant_dispatch_kernel<4>));
    else MOE_HTRY(go(quant_dispatch_kernel<0>));
  }
  i8::Params p{}, q{};
  p.tile_expert = tile_expert; p.tile_rows = tile_rows; p.stats = stats;
  p.row_scale = xs; p.row_max = row_max;
  q = p;
  p.col_scale = w13_scale; p.col_scale_s = w13_s_scale;
  q.col_scale = w_down_scale; q.col_scale_s = w_down_s_scale;
  if (thin)
    MOE_HTRY((thin_product_of<i8::I8_SWIGLU>(nt, w, "i8_gate_up_thin", xq, t13, td, h, p, s)));
  else
    MOE_HTRY((product<i8::I8_SWIGLU>(c, w, "i8_gate_up", xq, c->D, w13, w13_s, 2 * (int64_t)c->F,
                                     h, p, s)));
  MOE_HTRY(host::launch("quant_h", quant_h_kernel,
                        (int)std::min<int64_t>(host::ceil_div(w.v.rows_max * host::ceil_div(c->F, 512), 8),
                                               (int64_t)sms * 8),
                        kHThreads, 0, s, 1, h, c->F, w.v.rows_max, stats, tile_rows, row_max, hq));
  if (thin) return thin_product_of<i8::I8_STORE>(nt, w, "i8_down_thin", hq, td, td, o, q, s);
  return product<i8::I8_STORE>(c, w, "i8_down", hq, c->F, w_down, w_down_s, c->D, o, q, s);
}

}  // extern "C"
