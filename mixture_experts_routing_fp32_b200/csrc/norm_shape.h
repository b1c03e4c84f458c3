// Launch shape of the block norms' forward: host arithmetic alone, so that it
// can be checked without a GPU.
#pragma once
#include <algorithm>
#include <cstdint>

namespace moe {
namespace norm_shape {

constexpr int64_t kSmSmem = 228 * 1024;       // of an SM
constexpr int64_t kBlockSmem = 9 * 1024;      // of each block: row sums (8 KB), the system's 1 KB
constexpr int kMaxThreads = 1024;
// Blocks of up to 576 threads run in at most 56 registers, so that an SM
// holds 1168 threads of them.
constexpr int kSmallBlock = 576, kSmallThreads = 1168;

inline int threads_per_row(int D) { return (D / 8 + 31) / 32 * 32; }
// Row groups of a CTA of about `threads` threads (at most 15: a named
// barrier each; single-warp groups need none, up to 16).
inline int row_groups(int tpr, int threads) {
  return std::max(1, std::min(threads / tpr, tpr == 32 ? 16 : 15));
}

struct Forward {
  int R, threads, per_sm, stages, grid;
  int64_t smem;                  // dynamic
  bool small, bias_smem;
};

// piece: bytes of a thread's 8 columns of y and r together.
inline Forward forward(int T, int D, int sms, int piece, bool bias) {
  Forward f{};
  const int tpr = threads_per_row(D);
  f.R = std::max(1, std::min(row_groups(tpr, 256), (T + sms - 1) / sms));
  f.threads = f.R * tpr;
  const int64_t blocks = ((int64_t)T + f.R - 1) / f.R;
  const int64_t stage = (int64_t)piece * f.threads;
  int64_t fixed = (int64_t)f.threads * 32 * (bias ? 4 : 2);
  // with biases only where that makes room for another block (the registers
  // are short there: 16384 x 4104 bf16 228 -> 175 us, but 16384 x 4096 with
  // an fp32 stream 231 -> 281)
  f.small = f.threads <= kSmallBlock &&
            (!bias || kSmallThreads / f.threads > kMaxThreads / f.threads);
  // 64 registers a thread: 1024 threads of an SM; no more blocks than there
  // are (narrow blocks come with few rows: they share the SM with none)
  f.per_sm = (int)std::max<int64_t>(
      1, std::min<int64_t>((f.small ? kSmallThreads : kMaxThreads) / f.threads,
                           (blocks + sms - 1) / sms));
  const int64_t room = kSmSmem / f.per_sm - kBlockSmem;
  // biases in shared memory only where they leave two rows' room (16384 rows
  // of 4096 bf16: 142 us with two rows and the biases, 172 with four rows and
  // the biases read from L2)
  f.bias_smem = bias && fixed + 2 * stage <= room;
  if (!f.bias_smem) fixed = (int64_t)f.threads * 64;
  f.stages = (int)std::max<int64_t>(1, std::min<int64_t>(4, (room - fixed) / stage));
  f.smem = f.stages * stage + fixed;
  f.grid = (int)std::min<int64_t>(blocks, (int64_t)sms * f.per_sm);
  return f;
}

}  // namespace norm_shape
}  // namespace moe
