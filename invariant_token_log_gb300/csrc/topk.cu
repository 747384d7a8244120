// Selected-token log-probability with the row's k largest alternatives, and the
// gradient of both.  The C ABI is declared in include/bil.h.
//
// The alternatives of a row are the first k of its columns in the order of
// (stored logit descending, column ascending), NaN last; their log-probability
// is z - LSE, as the target's.  One pass over the logits gives everything:
//
//   topk_stream_kernel  a warp takes a contiguous run of a row's tiles (a unit:
//                       the whole row where there are enough rows), streams
//                       them through two shared-memory stages of its own with
//                       bulk copies, and gives each tile's (max, sum-exp[,
//                       entropy sum]) partial, by the library's one arithmetic
//                       contract, and the unit's k best columns;
//   topk_merge_kernel   a row's partials in the one fixed order (merge_lse: so
//                       logp, lse and the entropy are bil_logp_fwd's bits) and
//                       its units' lists into one.
//
// The k best are a list sorted across the warp's lanes (slot 32 r + lane), each
// entry one 64-bit word: the logit's bits made monotone, above the column's
// complement, so that a larger word is a better column and ties are decided.
// A lane's maximum over a tile, which the partial needs anyway, is compared
// with the list's k-th: most tiles past a row's first hold nothing better and
// cost one comparison and a vote.  Otherwise the tile's groups are gone
// through in column order, so that a column equal to the k-th never enters: a
// row of one value costs k insertions.  A unit's first tile starts from a
// bound instead of an empty list: the k-th largest of the 32 lanes' maxima (k
// <= 32) has k columns at or above it.
//
// Bound: HBM, one read of the logits (16384 x 151936 bf16: 4.98 GB), with the
// issue slots of the reduction close behind.
//
//   topk_grad_sum_kernel  g + sum_j gk_j, what the softmax term is scaled by;
//   (bil_logp_bwd)        d = -(g + sum gk) p - gh p (a + H), one pass;
//   topk_grad_fix_kernel  the k + 1 columns per row that have a term of their own.

#include "../../include/bil.h"
#include "device_common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "logp_device.cuh"

#include <algorithm>

namespace {

constexpr int kTopkStages = 2;    // stages of a warp
constexpr int kTopkMaxWarps = 8;  // warps of a block
constexpr int kTopkMaxUnits = 64; // units a row is cut into at most (two lists a lane in the merge)

typedef unsigned long long u64;

// A logit's bits as a number that orders as the logit does, -0 as +0, NaN
// below everything.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
  const uint32_t k = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return x != x ? 0u : k;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  if (k == 0u) return __int_as_float(0x7fc00000);
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;

__device__ __forceinline__ u64 entry_of(uint32_t key, int64_t column) {
  return (static_cast<u64>(key) << 32) | (0xffffffffu - static_cast<uint32_t>(column));
}
__device__ __forceinline__ int64_t entry_column(u64 e) { return 0xffffffffu - static_cast<uint32_t>(e); }

// The best entries so far, slot 32 r + lane in v[r], descending; 0: none.
template <int R>
struct Best {
  u64 v[R];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = 0;
  }
  __device__ __forceinline__ void insert(u64 c, int lane) {
    int pos = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) pos += __popc(__ballot_sync(0xffffffffu, v[r] > c));
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      u64 prev = __shfl_up_sync(0xffffffffu, v[r], 1);
      if (r > 0) {
        const u64 last = __shfl_sync(0xffffffffu, v[r > 0 ? r - 1 : 0], kLanes - 1);
        if (lane == 0) prev = last;
      }
      const int slot = r * kLanes + lane;
      if (slot >= pos) v[r] = slot == pos ? c : prev;
    }
  }
  __device__ __forceinline__ u64 at(int slot) const {
    u64 e = 0;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r == slot / kLanes) e = __shfl_sync(0xffffffffu, v[r], slot % kLanes);
    return e;
  }
};

struct TopkParams {
  const unsigned char* logits;
  int64_t n_rows, vocab, ld;
  int tile_v, num_tiles;
  int chunk;  // tiles of a unit
  int units;  // units of a row
  const int64_t* targets;
  int64_t ignore_index;
  float rcp;
  int k;
  float* part_max;  // [n_rows, num_tiles]
  float* part_sum;
  float* part_ent;
  u64* cand;  // [n_rows, units, k]
  unsigned stage_bytes;
};

// Where a warp is in its units: unit u, tile within it.  Units of ignored
// rows are passed over.
struct UnitCursor {
  int64_t unit, row;
  int tile, end;

  __device__ __forceinline__ bool more(const TopkParams& p) const { return unit < p.n_rows * p.units; }
  __device__ __forceinline__ void settle(const TopkParams& p, int64_t stride) {
    for (; more(p); unit += stride) {
      row = unit / p.units;
      if (p.targets[row] == p.ignore_index) continue;
      tile = static_cast<int>(unit - row * p.units) * p.chunk;
      end = min(tile + p.chunk, p.num_tiles);
      return;
    }
  }
  __device__ __forceinline__ void next(const TopkParams& p, int64_t stride) {
    if (++tile < end) return;
    unit += stride;
    settle(p, stride);
  }
};

// The tile's columns that are better than the list's k-th, into the list.
// tk: the smallest key that enters (kept up to date).
template <int DT, int WOFF, int R>
__device__ __noinline__ void scan_tile_t(const unsigned char* tile, unsigned off, unsigned sh, int valid, int64_t col0,
                                         int lane, int k, Best<R>& best, uint32_t& tk) {
  const int groups = (valid + kGroup - 1) / kGroup;
  const int rem = valid % kGroup;
  for (int g0 = 0; g0 < groups; g0 += kLanes) {
    const int g = g0 + lane;
    uint32_t key = 0;
    if (g < groups) {
      uint32_t w[Group<DT>::kW], mx[Group<DT>::kW];
      load_group<DT, WOFF>(tile, g, sh, w);
      if (rem != 0 && g == groups - 1) Group<DT>::mask_tail(w, rem);
      Group<DT>::max_init(mx);
      Group<DT>::max_acc(mx, w);
      key = order_key(Group<DT>::max_fin(mx));
    }
    unsigned mask = __ballot_sync(0xffffffffu, g < groups && key >= tk);
    while (mask != 0u) {
      const int src = __ffs(mask) - 1;
      mask &= mask - 1;
      const int e0 = (g0 + src) * kGroup, e = e0 + lane;
      const bool in = lane < kGroup && e < valid;
      const uint32_t ek = in ? order_key(Elem<DT>::one(tile + off + static_cast<size_t>(e) * Elem<DT>::kBytes)) : 0u;
      unsigned sub = __ballot_sync(0xffffffffu, in && ek >= tk);
      while (sub != 0u) {
        const int j = __ffs(sub) - 1;
        sub &= sub - 1;
        const uint32_t kj = __shfl_sync(0xffffffffu, ek, j);
        if (kj < tk) continue;  // the bound has risen
        best.insert(entry_of(kj, col0 + e0 + j), lane);
        const u64 kth = best.at(k - 1);
        if (kth != 0) tk = static_cast<uint32_t>(kth >> 32) + 1u;
      }
    }
  }
}

template <int DT, bool SHIFTED, int R>
__device__ __forceinline__ void scan_tile(const unsigned char* tile, unsigned off, int valid, int64_t col0, int lane,
                                          int k, Best<R>& best, uint32_t& tk) {
  const unsigned sh = 8u * (off & 3u);
  if (!SHIFTED || off == 0) return scan_tile_t<DT, -1, R>(tile, 0, 0, valid, col0, lane, k, best, tk);
  switch (off >> 2) {
    case 0: return scan_tile_t<DT, 0, R>(tile, off, sh, valid, col0, lane, k, best, tk);
    case 1: return scan_tile_t<DT, 1, R>(tile, off, sh, valid, col0, lane, k, best, tk);
    case 2: return scan_tile_t<DT, 2, R>(tile, off, sh, valid, col0, lane, k, best, tk);
    default: return scan_tile_t<DT, 3, R>(tile, off, sh, valid, col0, lane, k, best, tk);
  }
}

// The k-th largest (k <= 32) of the lanes' keys, in every lane.
__device__ __forceinline__ uint32_t kth_of_lanes(uint32_t key, int k, int lane) {
  int above = 0;
#pragma unroll
  for (int j = 0; j < kLanes; ++j) {
    const uint32_t o = __shfl_sync(0xffffffffu, key, j);
    above += (o > key || (o == key && j < lane)) ? 1 : 0;
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, above == k - 1)) - 1;
  return __shfl_sync(0xffffffffu, key, src);
}

template <int DT, bool ALIGNED, bool ENT, int R>
__global__ void __launch_bounds__(kTopkMaxWarps * kLanes, 2) topk_stream_kernel(const TopkParams p) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  __shared__ uint64_t full_bars[kTopkMaxWarps][kTopkStages];
  __shared__ int abort_flag;
  constexpr int EB = Elem<DT>::kBytes;
  const int warp = threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  const int warps = blockDim.x / kLanes;
  volatile int* abort = &abort_flag;
  uint64_t* full = full_bars[warp];
  unsigned char* ring = smem_raw + static_cast<size_t>(warp) * kTopkStages * p.stage_bytes;
  if (threadIdx.x == 0) *abort = 0;
  if (lane == 0) {
    for (int s = 0; s < kTopkStages; ++s) mbar_init(&full[s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  // Consecutive units go to different blocks.
  const int64_t stride = static_cast<int64_t>(gridDim.x) * warps;
  const int64_t first = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;
  const uint64_t policy = evict_first_policy();
  UnitCursor ahead{first, 0, 0, 0}, at{first, 0, 0, 0};
  ahead.settle(p, stride);
  at = ahead;
  int64_t issued = 0, taken = 0;

  // The next tile's copy into stage issued % 2 (its last reader is done).  The
  // 16-byte aligned span that covers the tile, as in the streaming forward.
  auto issue = [&]() {
    if (!ahead.more(p)) return;
    if (lane == 0) {
      const int64_t col0 = static_cast<int64_t>(ahead.tile) * p.tile_v;
      const int valid = static_cast<int>(min(static_cast<int64_t>(p.tile_v), p.vocab - col0));
      const unsigned char* src = p.logits + (ahead.row * p.ld + col0) * EB;
      const unsigned off = ALIGNED ? 0u : static_cast<unsigned>(reinterpret_cast<uintptr_t>(src) & 15u);
      const unsigned bytes = static_cast<unsigned>(align_up(off + static_cast<size_t>(valid) * EB, 16));
      const int s = static_cast<int>(issued % kTopkStages);
      mbar_arrive_expect_tx(&full[s], bytes);
      bulk_g2s(ring + static_cast<size_t>(s) * p.stage_bytes, src - off, bytes, &full[s], policy);
    }
    ++issued;
    ahead.next(p, stride);
  };
  for (int s = 0; s < kTopkStages; ++s) issue();

  Best<R> best;
  best.clear();
  uint32_t tk = 0;
  bool start = true;
  while (at.more(p)) {
    const int s = static_cast<int>(taken % kTopkStages);
    if (!warp_wait(&full[s], static_cast<unsigned>((taken / kTopkStages) & 1), abort, kWatchFull)) break;
    ++taken;
    const int64_t col0 = static_cast<int64_t>(at.tile) * p.tile_v;
    const int valid = static_cast<int>(min(static_cast<int64_t>(p.tile_v), p.vocab - col0));
    const unsigned char* src = p.logits + (at.row * p.ld + col0) * EB;
    const unsigned off = ALIGNED ? 0u : static_cast<unsigned>(reinterpret_cast<uintptr_t>(src) & 15u);
    const unsigned char* tile = ring + static_cast<size_t>(s) * p.stage_bytes;
    const bool in_regs = p.tile_v <= TileRegs<DT>::kMaxTile;

    // candidates, given the lane's maximum over the tile
    auto offer = [&](float lane_max) {
      const uint32_t key = order_key(lane_max);
      if (start && p.k <= kLanes) {
        tk = kth_of_lanes(key, p.k, lane);
        // a lane whose columns are all NaN, or that has none, also says -inf: no bound then
        if (tk <= kKeyNegInf) tk = 0;
      }
      start = false;
      if (__any_sync(0xffffffffu, key >= tk))
        scan_tile<DT, !ALIGNED, R>(tile, off, valid, col0, lane, p.k, best, tk);
    };

    TilePartial tp;
    if (in_regs) {
      TileRegs<DT> regs;
      tile_load_regs<DT, !ALIGNED>(tile, valid, lane, regs, off);
      {
        const int ng = lane_groups(valid, lane);
        uint32_t mx[Group<DT>::kW];
        Group<DT>::max_init(mx);
#pragma unroll
        for (int i = 0; i < TileRegs<DT>::kMaxGroups; ++i)
          if (i < ng) Group<DT>::max_acc(mx, regs.w[i]);
        offer(Group<DT>::max_fin(mx));
      }
      __syncwarp();  // the stage has been read
      issue();
      tp = tile_reduce_regs<DT, ENT, false>(regs, valid, lane, p.rcp);
      if (ENT && tp.u != tp.u) {  // as in the streaming forward: u from a clamped pass
        if (ALIGNED) {
          tile_load_regs<DT>(src, valid, lane, regs);
        } else {
          tile_load_regs<DT, true, true>(src - off, valid, lane, regs, off);
        }
        tp.u = tile_reduce_regs<DT, ENT, true>(regs, valid, lane, p.rcp).u;
      }
    } else {
      float m = -INFINITY;
      for (int e = lane; e < valid; e += kLanes) m = fmaxf(m, Elem<DT>::one(tile + off + static_cast<size_t>(e) * EB));
      offer(m);
      tp = tile_reduce_smem<DT, ENT, !ALIGNED>(tile, valid, lane, p.rcp, off);
      __syncwarp();
      issue();
    }
    if (lane == 0) {
      const int64_t o = at.row * p.num_tiles + at.tile;
      p.part_max[o] = tp.m;
      p.part_sum[o] = tp.s;
      if (ENT) p.part_ent[o] = tp.u;
    }
    if (at.tile + 1 == at.end) {
      u64* out = p.cand + at.unit * p.k;
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r * kLanes + lane < p.k) out[r * kLanes + lane] = best.v[r];
      best.clear();
      tk = 0;
      start = true;
    }
    at.next(p, stride);
  }
  // A warp that gave up waits (bounded) for its own copies in flight.
  if (lane == 0) {
    for (; taken < issued; ++taken)
      if (!thread_wait_watch(&full[taken % kTopkStages], static_cast<unsigned>((taken / kTopkStages) & 1), abort,
                             kWatchDrain, &g_watchdog, false))
        break;
  }
}

// A row a block: warp 0 merges the partials, warp 1 the units' lists (each
// sorted; every round takes the best of the heads), and both write the row.
constexpr int kTopkMergeThreads = 2 * kLanes;

template <int DT, bool ENT>
__global__ void __launch_bounds__(kTopkMergeThreads) topk_merge_kernel(const TopkParams p, float* logp, float* lse,
                                                                       float* entropy, int64_t* top_ids, float* top_logp) {
  extern __shared__ u64 lists[];  // [units, k] where a row has more than one unit
  __shared__ u64 merged[BIL_MAX_TOPK];
  __shared__ float scratch[kMergeScratch];
  __shared__ float row_lse;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % kLanes;
  const int64_t row = blockIdx.x;
  const int64_t t = p.targets[row];
  int64_t* ids = top_ids + row * p.k;
  float* top = top_logp + row * p.k;
  if (t == p.ignore_index) {
    for (int j = threadIdx.x; j < p.k; j += kTopkMergeThreads) {
      ids[j] = -1;
      top[j] = 0.0f;
    }
    if (threadIdx.x == 0) {
      logp[row] = 0.0f;
      if (lse != nullptr) lse[row] = 0.0f;
      if (ENT) entropy[row] = 0.0f;
    }
    return;
  }
  if (threadIdx.x < kLanes) {
    const int64_t o = row * p.num_tiles;
    float H = 0.0f;
    const float L = merge_lse<ENT, true>(p.part_max + o, p.part_sum + o, ENT ? p.part_ent + o : nullptr, p.num_tiles,
                                         lane, &H, scratch);
    if (lane == 0) {
      row_lse = L;
      float z = __int_as_float(0x7fc00000);
      if (t >= 0 && t < p.vocab) {
        z = Elem<DT>::one(p.logits + (row * p.ld + t) * Elem<DT>::kBytes);
        if (p.rcp != 1.0f) z = __fmul_rn(z, p.rcp);
      }
      logp[row] = __fsub_rn(z, L);
      if (lse != nullptr) lse[row] = L;
      if (ENT) entropy[row] = H;
    }
  } else {
    const u64* cand = p.cand + row * p.units * p.k;
    if (p.units == 1) {
      for (int j = lane; j < p.k; j += kLanes) merged[j] = cand[j];
    } else {
      for (int j = lane; j < p.units * p.k; j += kLanes) lists[j] = cand[j];
      __syncwarp();
      int h[2] = {0, 0};
      u64 head[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int l = lane + q * kLanes;
        head[q] = l < p.units ? lists[l * p.k] : 0;
      }
      for (int j = 0; j < p.k; ++j) {
        const u64 mine = head[0] > head[1] ? head[0] : head[1];
        const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(mine >> 32));
        const uint32_t lo = __reduce_max_sync(
            0xffffffffu, static_cast<uint32_t>(mine >> 32) == hi ? static_cast<uint32_t>(mine) : 0u);
        const u64 won = (static_cast<u64>(hi) << 32) | lo;
        if (lane == 0) merged[j] = won;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (won != 0 && head[q] == won) {
            ++h[q];
            head[q] = h[q] < p.k ? lists[(lane + q * kLanes) * p.k + h[q]] : 0;
          }
        }
      }
    }
  }
  __syncthreads();
  for (int j = threadIdx.x; j < p.k; j += kTopkMergeThreads) {
    const u64 e = merged[j];
    float z = key_value(static_cast<uint32_t>(e >> 32));
    if (p.rcp != 1.0f) z = __fmul_rn(z, p.rcp);
    ids[j] = entry_column(e);
    top[j] = __fsub_rn(z, row_lse);
  }
}

// ---------------------------------------------------------------------------
// Backward.
// ---------------------------------------------------------------------------

// G[r] = g[r] + (gk[r, 0] + gk[r, 1] + ...), a warp a row: lane l adds entries
// l, l + 32, ... in order, then the butterfly.
__global__ void __launch_bounds__(256) topk_grad_sum_kernel(const float* __restrict__ grad_logp,
                                                            const float* __restrict__ grad_top, int k, int64_t n_rows,
                                                            float* __restrict__ sum) {
  const int lane = threadIdx.x % kLanes;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / kLanes) + threadIdx.x / kLanes;
  if (row >= n_rows) return;
  float s = 0.0f;
  for (int j = lane; j < k; j += kLanes) s = __fadd_rn(s, grad_top[row * k + j]);
  s = warp_sum(s);
  if (lane == 0) sum[row] = __fadd_rn(grad_logp[row], s);
}

struct TopkFixParams {
  const unsigned char* logits;
  int64_t n_rows, vocab, ld;
  const int64_t* targets;
  int64_t ignore_index;
  float rcp;
  const int64_t* top_ids;
  int k;
  const float* lse;
  const float* grad_logp;
  const float* grad_top;
  const float* grad_sum;
  const float* entropy;       // NULL: no entropy term
  const float* grad_entropy;
  unsigned char* dlogits;
  int64_t ld_out;
};

// The columns with a term of their own: with W = g [c = t] + sum_j gk_j [c =
// ids_j] and G = g + sum_j gk_j,
//     d_c = (W - G p - gh p (a + H)) * rcp
// written over what the full pass (which knows G alone) left there.  A column
// named more than once is written more than once, with the same bits.
template <int DT, int OT>
__global__ void __launch_bounds__(BIL_MAX_TOPK + kLanes) topk_grad_fix_kernel(const TopkFixParams p) {
  __shared__ int64_t ids[BIL_MAX_TOPK + 1];
  __shared__ float w[BIL_MAX_TOPK + 1];
  const int64_t row = blockIdx.x;
  const int64_t t = p.targets[row];
  // ignored rows are zero, rows with a target outside the vocabulary NaN: as the full pass left them
  if (t == p.ignore_index || t < 0 || t >= p.vocab) return;
  for (int j = threadIdx.x; j <= p.k; j += blockDim.x) {
    ids[j] = j < p.k ? p.top_ids[row * p.k + j] : t;
    w[j] = j < p.k ? p.grad_top[row * p.k + j] : p.grad_logp[row];
  }
  __syncthreads();
  for (int j = threadIdx.x; j <= p.k; j += blockDim.x) {
    const int64_t c = ids[j];
    if (c < 0 || c >= p.vocab) continue;
    float W = 0.0f;
    for (int i = 0; i <= p.k; ++i)
      if (ids[i] == c) W = __fadd_rn(W, w[i]);
    const float x = Elem<DT>::one(p.logits + (row * p.ld + c) * Elem<DT>::kBytes);
    const float a = p.rcp != 1.0f ? __fmaf_rn(x, p.rcp, -p.lse[row]) : __fsub_rn(x, p.lse[row]);
    const float e = contract_exp(a);
    float d = __fmaf_rn(-p.grad_sum[row], e, W);
    if (p.entropy != nullptr)
      d = __fsub_rn(d, __fmul_rn(p.grad_entropy[row], __fmul_rn(e, __fadd_rn(fmaxf(a, kNegMax), p.entropy[row]))));
    if (p.rcp != 1.0f) d = __fmul_rn(d, p.rcp);
    const int64_t o = row * p.ld_out + c;
    if (OT == BIL_F32)
      reinterpret_cast<float*>(p.dlogits)[o] = d;
    else if (OT == BIL_BF16)
      reinterpret_cast<__nv_bfloat16*>(p.dlogits)[o] = __float2bfloat16_rn(d);
    else
      reinterpret_cast<__half*>(p.dlogits)[o] = __float2half_rn(d);
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// How the stream kernel is laid out: warps of a block, blocks of an SM.  Two
// blocks an SM where that leaves them four warps each or more (the partials
// need up to 128 registers a thread: 16 warps), else one block.
constexpr size_t kSmSmemBytes = 228 * 1024;  // an SM's shared memory, 1 KB of it reserved for each block
void stream_layout(size_t stage_bytes, int* warps, int* blocks) {
  const size_t per_warp = kTopkStages * stage_bytes;
  for (*blocks = 2; *blocks >= 1; --*blocks) {
    const size_t room = kSmSmemBytes / *blocks - 1024 - 256;  // 256: the barriers
    *warps = static_cast<int>(std::min<size_t>(kTopkMaxWarps, room / per_warp));
    if (*blocks == 1 || *warps >= 4) return;
  }
}

// Tiles of a unit: the cut of the rows that gives the least time, a warp's time
// being its units' tiles plus three quarters of a tile a unit for the filling of
// an empty list.  By the sizes alone (not by the alignment).
int unit_tiles(int64_t n_rows, int num_tiles, int k, int64_t warps) {
  const int most = std::min<int>(kTopkMaxUnits, 40 * 1024 / (8 * k));  // the merge's lists in shared memory
  int best = num_tiles;
  double least = 0.0;
  for (int u = 1; u <= std::min(num_tiles, most); ++u) {
    const int chunk = (num_tiles + u - 1) / u;
    const int64_t units = n_rows * ((num_tiles + chunk - 1) / chunk);
    const double cost = static_cast<double>((units + warps - 1) / warps) * (chunk + 0.75);
    if (u == 1 || cost < least) {
      least = cost;
      best = chunk;
    }
  }
  return best;
}

struct TopkPlan {
  int chunk, units;
  size_t part, cand, total;  // bytes: one partial array, the lists, all
};

size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

int topk_plan(int dtype, int64_t n_rows, int num_tiles, int tile_v, int k, bool ent, TopkPlan* plan) {
  int sms = 0, smem = 0;
  if (int st = bil_internal::device_limits(&sms, &smem)) return st;
  int warps = 0, blocks = 0;
  stream_layout(static_cast<size_t>(tile_v) * bil_internal::elem_bytes(dtype), &warps, &blocks);
  plan->chunk = unit_tiles(n_rows, num_tiles, k, static_cast<int64_t>(sms) * warps * blocks);
  plan->units = (num_tiles + plan->chunk - 1) / plan->chunk;
  plan->part = round256(static_cast<size_t>(n_rows) * num_tiles * sizeof(float));
  plan->cand = round256(static_cast<size_t>(n_rows) * plan->units * k * sizeof(u64));
  plan->total = plan->part * (ent ? 3 : 2) + plan->cand;
  return BIL_OK;
}

// The sizes both the workspace query and the forward check.
int check_topk_sizes(int dtype, int64_t n_rows, int64_t vocab, int32_t tile_v, int32_t k, int64_t* num_tiles) {
  if (n_rows < 0 || vocab < 1 || k < 1 || k > vocab) return BIL_E_INVALID_ARG;
  if (int st = bil_internal::check_tile(dtype, vocab, tile_v, num_tiles)) return st;
  if (k > BIL_MAX_TOPK || vocab > INT32_MAX || *num_tiles > BIL_MAX_FUSED_TILES || n_rows > INT32_MAX)
    return BIL_E_UNSUPPORTED;
  return BIL_OK;
}

template <int DT, bool ALIGNED, bool ENT, int R>
int launch_topk_t(const TopkParams& p, cudaStream_t stream) {
  int sms = 0, smem_optin = 0;
  if (int st = bil_internal::device_limits(&sms, &smem_optin)) return st;
  int warps = 0, blocks = 0;
  stream_layout(p.stage_bytes, &warps, &blocks);
  const int64_t units = p.n_rows * p.units;
  const int64_t slots = static_cast<int64_t>(sms) * blocks;
  // few units: one warp a block, so that they spread over the SMs
  warps = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(warps, (units + slots - 1) / slots)));
  const int64_t grid = std::min<int64_t>(slots, (units + warps - 1) / warps);
  const size_t smem = static_cast<size_t>(warps) * kTopkStages * p.stage_bytes;
  if (smem > static_cast<size_t>(smem_optin)) return BIL_E_UNSUPPORTED;
  auto kernel = topk_stream_kernel<DT, ALIGNED, ENT, R>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
    return BIL_E_CUDA;
  return launch_pdl(kernel, grid, warps * kLanes, smem, stream, 1, p) == cudaSuccess ? BIL_OK : BIL_E_CUDA;
}

template <int DT>
int launch_topk(TopkParams p, bool ent, float* logp, float* lse, float* entropy, int64_t* top_ids, float* top_logp,
                cudaStream_t stream) {
  constexpr int EB = Elem<DT>::kBytes;
  const bool vec = aligned_to(p.logits, 16) && (p.n_rows <= 1 || (p.ld * EB) % 16 == 0) && (p.tile_v * EB) % 16 == 0;
  p.stage_bytes = static_cast<unsigned>(align_up(static_cast<size_t>(p.tile_v) * EB + (vec ? 0 : 16), 128));
  const bool one = p.k <= kLanes;
  int st;
  if (vec)
    st = ent ? (one ? launch_topk_t<DT, true, true, 1>(p, stream) : launch_topk_t<DT, true, true, 4>(p, stream))
             : (one ? launch_topk_t<DT, true, false, 1>(p, stream) : launch_topk_t<DT, true, false, 4>(p, stream));
  else
    st = ent ? (one ? launch_topk_t<DT, false, true, 1>(p, stream) : launch_topk_t<DT, false, true, 4>(p, stream))
             : (one ? launch_topk_t<DT, false, false, 1>(p, stream) : launch_topk_t<DT, false, false, 4>(p, stream));
  if (st) return st;
  const size_t smem = p.units > 1 ? static_cast<size_t>(p.units) * p.k * sizeof(u64) : 0;
  const cudaError_t e = ent ? launch_pdl(topk_merge_kernel<DT, true>, p.n_rows, kTopkMergeThreads, smem, stream, 1, p,
                                         logp, lse, entropy, top_ids, top_logp)
                            : launch_pdl(topk_merge_kernel<DT, false>, p.n_rows, kTopkMergeThreads, smem, stream, 1, p,
                                         logp, lse, entropy, top_ids, top_logp);
  return e == cudaSuccess ? BIL_OK : BIL_E_CUDA;
}

template <int DT>
int launch_fix(int out_dtype, const TopkFixParams& p, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(p.n_rows);
  const int threads = (p.k + 1 + kLanes - 1) / kLanes * kLanes;
  switch (out_dtype) {
    case BIL_F32: topk_grad_fix_kernel<DT, BIL_F32><<<grid, threads, 0, s>>>(p); break;
    case BIL_BF16: topk_grad_fix_kernel<DT, BIL_BF16><<<grid, threads, 0, s>>>(p); break;
    default: topk_grad_fix_kernel<DT, BIL_F16><<<grid, threads, 0, s>>>(p); break;
  }
  return cudaGetLastError() == cudaSuccess ? BIL_OK : BIL_E_CUDA;
}

}  // namespace

namespace bil_internal {

int topk_watchdog(unsigned int* flags, int clear) {
  if (cudaMemcpyFromSymbol(flags, g_watchdog, sizeof(unsigned int)) != cudaSuccess) return BIL_E_CUDA;
  if (clear) {
    const unsigned int zero = 0;
    if (cudaMemcpyToSymbol(g_watchdog, &zero, sizeof(unsigned int)) != cudaSuccess) return BIL_E_CUDA;
  }
  return BIL_OK;
}

}  // namespace bil_internal

extern "C" {

int bil_logp_topk_workspace_bytes(int dtype, int64_t n_rows, int64_t vocab, int32_t tile_v, int32_t k, int entropy,
                                  int64_t* bytes) {
  if (bytes == nullptr) return BIL_E_INVALID_ARG;
  int64_t num_tiles = 0;
  if (int st = check_topk_sizes(dtype, n_rows, vocab, tile_v, k, &num_tiles)) return st;
  TopkPlan plan;
  if (int st = topk_plan(dtype, n_rows, static_cast<int>(num_tiles), tile_v, k, entropy != 0, &plan)) return st;
  *bytes = static_cast<int64_t>(plan.total);
  return BIL_OK;
}

int bil_logp_topk_fwd(const void* logits, int dtype, int64_t n_rows, int64_t vocab, int64_t ld,
                      const int64_t* target_ids, int64_t ignore_index, int32_t tile_v, float temperature, int32_t k,
                      float* logp, float* lse, float* entropy, int64_t* top_ids, float* top_logp, void* workspace,
                      int64_t workspace_bytes, int validate, bil_stream_t stream) {
  bil_internal::NvtxRange nvtx_range("bil_logp_topk_fwd");
  const int eb = bil_internal::elem_bytes(dtype);
  if (eb == 0) return BIL_E_DTYPE;
  if (ld < vocab) return BIL_E_INVALID_ARG;
  int64_t num_tiles = 0;
  if (int st = check_topk_sizes(dtype, n_rows, vocab, tile_v, k, &num_tiles)) return st;
  if (!bil_internal::extent_ok(n_rows, ld, eb)) return BIL_E_UNSUPPORTED;
  float rcp = 1.0f;
  if (int st = bil_internal::temperature_rcp(temperature, &rcp)) return st;
  if (n_rows == 0) return BIL_OK;
  if (logits == nullptr || target_ids == nullptr || logp == nullptr || top_ids == nullptr || top_logp == nullptr ||
      workspace == nullptr)
    return BIL_E_INVALID_ARG;
  if (!aligned_to(logits, static_cast<size_t>(eb)) || !aligned_to(target_ids, 8) || !aligned_to(logp, 4) ||
      (lse && !aligned_to(lse, 4)) || (entropy && !aligned_to(entropy, 4)) || !aligned_to(top_ids, 8) ||
      !aligned_to(top_logp, 4) || !aligned_to(workspace, 256))
    return BIL_E_ALIGN;
  const bool ent = entropy != nullptr;
  TopkPlan plan;
  if (int st = topk_plan(dtype, n_rows, static_cast<int>(num_tiles), tile_v, k, ent, &plan)) return st;
  if (workspace_bytes < static_cast<int64_t>(plan.total)) return BIL_E_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (validate) {
    if (int st = bil_internal::check_targets_host(target_ids, n_rows, ignore_index, vocab, s)) return st;
  }
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  TopkParams p{};
  p.logits = static_cast<const unsigned char*>(logits);
  p.n_rows = n_rows;
  p.vocab = vocab;
  p.ld = ld;
  p.tile_v = tile_v;
  p.num_tiles = static_cast<int>(num_tiles);
  p.chunk = plan.chunk;
  p.units = plan.units;
  p.targets = target_ids;
  p.ignore_index = ignore_index;
  p.rcp = rcp;
  p.k = k;
  p.cand = reinterpret_cast<u64*>(ws);
  p.part_max = reinterpret_cast<float*>(ws + plan.cand);
  p.part_sum = reinterpret_cast<float*>(ws + plan.cand + plan.part);
  p.part_ent = ent ? reinterpret_cast<float*>(ws + plan.cand + 2 * plan.part) : nullptr;
  switch (dtype) {
    case BIL_BF16: return launch_topk<BIL_BF16>(p, ent, logp, lse, entropy, top_ids, top_logp, s);
    case BIL_F16: return launch_topk<BIL_F16>(p, ent, logp, lse, entropy, top_ids, top_logp, s);
    default: return launch_topk<BIL_F32>(p, ent, logp, lse, entropy, top_ids, top_logp, s);
  }
}

int bil_logp_topk_bwd(const void* logits, int dtype, int64_t n_rows, int64_t vocab, int64_t ld,
                      const int64_t* target_ids, int64_t ignore_index, float temperature, const int64_t* top_ids,
                      int32_t k, const float* lse, const float* grad_logp, const float* grad_top, const float* entropy,
                      const float* grad_entropy, void* dlogits, int dlogits_dtype, int64_t ld_out, int64_t out_cols,
                      float* workspace, bil_stream_t stream) {
  bil_internal::NvtxRange nvtx_range("bil_logp_topk_bwd");
  const int eb = bil_internal::elem_bytes(dtype), ob = bil_internal::elem_bytes(dlogits_dtype);
  if (eb == 0 || ob == 0) return BIL_E_DTYPE;
  if (n_rows < 0 || k < 1 || k > vocab) return BIL_E_INVALID_ARG;
  if (k > BIL_MAX_TOPK || n_rows > INT32_MAX) return BIL_E_UNSUPPORTED;
  // the sizes, as the full pass checks them for an empty batch
  if (int st = bil_logp_bwd(nullptr, dtype, 0, vocab, ld, nullptr, ignore_index, temperature, nullptr, nullptr, entropy,
                            grad_entropy, nullptr, dlogits_dtype, ld_out, out_cols, stream))
    return st;
  if (!bil_internal::extent_ok(n_rows, ld, eb) || !bil_internal::extent_ok(n_rows, ld_out, ob)) return BIL_E_UNSUPPORTED;
  if (n_rows == 0) return BIL_OK;
  if (logits == nullptr || target_ids == nullptr || top_ids == nullptr || lse == nullptr || grad_logp == nullptr ||
      grad_top == nullptr || dlogits == nullptr || workspace == nullptr)
    return BIL_E_INVALID_ARG;
  if (!aligned_to(logits, static_cast<size_t>(eb)) || !aligned_to(target_ids, 8) || !aligned_to(top_ids, 8) ||
      !aligned_to(lse, 4) || !aligned_to(grad_logp, 4) || !aligned_to(grad_top, 4) ||
      !aligned_to(dlogits, static_cast<size_t>(ob)) || !aligned_to(workspace, 4) ||
      (entropy && !aligned_to(entropy, 4)) || (grad_entropy && !aligned_to(grad_entropy, 4)))
    return BIL_E_ALIGN;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  topk_grad_sum_kernel<<<static_cast<unsigned>((n_rows + 7) / 8), 256, 0, s>>>(grad_logp, grad_top, k, n_rows,
                                                                              workspace);
  if (cudaGetLastError() != cudaSuccess) return BIL_E_CUDA;
  if (int st = bil_logp_bwd(logits, dtype, n_rows, vocab, ld, target_ids, ignore_index, temperature, lse, workspace,
                            entropy, grad_entropy, dlogits, dlogits_dtype, ld_out, out_cols, stream))
    return st;
  float rcp = 1.0f;
  if (int st = bil_internal::temperature_rcp(temperature, &rcp)) return st;
  TopkFixParams p{};
  p.logits = static_cast<const unsigned char*>(logits);
  p.n_rows = n_rows;
  p.vocab = vocab;
  p.ld = ld;
  p.targets = target_ids;
  p.ignore_index = ignore_index;
  p.rcp = rcp;
  p.top_ids = top_ids;
  p.k = k;
  p.lse = lse;
  p.grad_logp = grad_logp;
  p.grad_top = grad_top;
  p.grad_sum = workspace;
  p.entropy = entropy;
  p.grad_entropy = grad_entropy;
  p.dlogits = static_cast<unsigned char*>(dlogits);
  p.ld_out = ld_out;
  switch (dtype) {
    case BIL_BF16: return launch_fix<BIL_BF16>(dlogits_dtype, p, s);
    case BIL_F16: return launch_fix<BIL_F16>(dlogits_dtype, p, s);
    default: return launch_fix<BIL_F32>(dlogits_dtype, p, s);
  }
}

}  // extern "C"
