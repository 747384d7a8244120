// How kernels share an SM's memory: the host's arithmetic of blocks and stages.
// No CUDA in it, so that it compiles and can be swept over every size by itself.
#pragma once

#include <stddef.h>

#include <algorithm>

#ifdef __CUDACC__
#define BIL_LAYOUT_FN __host__ __device__ inline
#else
#define BIL_LAYOUT_FN inline
#endif

namespace bil_layout {

constexpr int kWarp = 32;
constexpr size_t kSmBytes = 228 * 1024;  // an SM's shared memory
constexpr size_t kReserved = 1024;       // of it, for each resident block

// The dynamic shared memory the kernels are launched with at most: a block's
// opt-in limit less 1 KB, which their own variables fit.  The attribute is always
// set to this one value, so that host threads do not undo each other's.
inline size_t dynamic_limit(int smem_optin) { return static_cast<size_t>(smem_optin) - 1024; }

// What a block can have where `blocks` share an SM and its variables take
// `statics` bytes.  For one block the launch limit is the smaller of the two.
inline size_t dynamic_room(int blocks, size_t statics, size_t limit) {
  return std::min(kSmBytes / static_cast<size_t>(blocks) - kReserved - statics, limit);
}

// ---- the norm's rows ----

constexpr int kVec = 8;        // elements of a group
constexpr int kMaxGroups = 4;  // groups a thread holds
constexpr int kMaxRowThreads = 512;
constexpr int kMaxStages = 4;  // of the backward's ring
constexpr size_t kNormStatics = 512;

// A row's threads and the groups each holds (rounded up to what is compiled), by
// the width alone: as few warps as hold the row in `most` groups a lane (four in
// the forward, two in the backward, whose rows past 8192 elements take four).
inline void row_shape(int width, int most, int* threads, int* per_thread) {
  const int groups = (width + kVec - 1) / kVec;
  if (groups > kMaxRowThreads * most) most = kMaxGroups;
  *threads = (groups + kWarp * most - 1) / (kWarp * most) * kWarp;
  const int need = (groups + *threads - 1) / *threads;
  *per_thread = need <= 1 ? 1 : need <= 2 ? 2 : 4;
}

// Shared memory of a row that may start anywhere in a 16-byte unit.
BIL_LAYOUT_FN unsigned slot_bytes(int row_bytes) { return static_cast<unsigned>((row_bytes + 15 + 15) & ~15); }

// The ring of the forward: as many blocks as hold 1024 threads an SM, or 640 of
// float32 (at up to 64, 96 registers a thread) with two stages each; fewer
// blocks, then one stage, for the widest rows.
inline void fwd_ring(size_t stage_bytes, int row_threads, int elem_bytes, size_t limit, int* per_sm, int* stages) {
  *per_sm = std::max(1, std::min(32, (elem_bytes == 4 ? 640 : 1024) / row_threads));
  for (;; --*per_sm) {
    *stages = static_cast<int>(std::min<size_t>(3, dynamic_room(*per_sm, kNormStatics, limit) / stage_bytes));
    if (*stages >= 2 || *per_sm == 1) return;
  }
}

// Blocks of the backward an SM: 768 threads at up to 80 registers, or 512 at 128
// with four groups a lane; 1024 where a warp takes a row.
inline int bwd_per_sm(int row_threads, int per_thread) {
  if (row_threads == kWarp) return 4;
  return std::max(1, (per_thread == 4 ? 512 : 768) / row_threads);
}

// The ring of the backward: of up to *per_sm blocks an SM the most that leave each
// three stages, or one block with two.  0 stages: the rows are too wide for that.
inline void bwd_ring(size_t stage_bytes, size_t limit, int* per_sm, int* stages) {
  for (; *per_sm >= 1; --*per_sm) {
    *stages = static_cast<int>(std::min<size_t>(kMaxStages, dynamic_room(*per_sm, kNormStatics, limit) / stage_bytes));
    if (*stages >= 3 || (*per_sm == 1 && *stages == 2)) return;
  }
  *stages = 0;
}

// ---- the pass over the logits of the forward with the alternatives ----

constexpr int kTopkMaxWarps = 8;  // of a block
constexpr size_t kTopkStatics = 128;

// Warps of a block and blocks of an SM.  One stage a warp: its copy is on the way
// while the tile before it is reduced from registers (or, past 8 KB, while the
// other warps reduce theirs), and 16 warps (at up to 128 registers a thread) have
// 128 KB of stages.  (Measured at 16384 x 151936 bf16: two stages for 14 warps
// 843 us, one for 16 warps 792 us: the reduction's latencies want the warps.)
// Two blocks an SM where that leaves them four warps each or more, else one.
inline void topk_stream(size_t stage_bytes, size_t limit, int* warps, int* blocks) {
  for (*blocks = 2; *blocks >= 1; --*blocks) {
    *warps = static_cast<int>(std::min<size_t>(kTopkMaxWarps, dynamic_room(*blocks, kTopkStatics, limit) / stage_bytes));
    if (*blocks == 1 || *warps >= 4) return;
  }
}

}  // namespace bil_layout
