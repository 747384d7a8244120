// Selected-token log-probability with the row's k largest alternatives, and the
// gradient of both.  The C ABI is declared in include/bil.h.
//
// The alternatives of a row are the first k of its columns in the order of
// (stored logit descending, column ascending), NaN last; their log-probability
// is z - LSE, as the target's.  Two kernels:
//
//   topk_stream_kernel  one pass over the logits.  A warp takes a run of a
//                       row's tiles and gives each tile's (max, sum-exp[,
//                       entropy sum]) partial by the library's one arithmetic
//                       contract, and with it what it has on the way there: the
//                       maximum of each lane's columns (a chunk: up to 128
//                       columns of a 4096-column tile).
//   topk_row_kernel     a row a block.  One warp merges the partials in the one
//                       fixed order (merge_lse: logp, lse and the entropy are
//                       bil_logp_fwd's bits).  Four warps find the columns from
//                       the chunks' maxima: of 128 (k > 32: 256) groups of
//                       chunks, the k-th largest maximum has k columns at or
//                       above it, and few chunks reach it (about 22 columns in
//                       as many of 1216 chunks for k = 20 of 151936), so that
//                       only those are read again, 1.7% of the row.
//
// The choice of columns thus costs the pass over the logits one store a tile,
// whatever k is.  (Measured before, 4096 x 151936 bf16, k = 20: a list of the
// best columns kept by the streaming warp, sorted across its lanes, took 437 to
// 528 us; most of its instructions went into the columns that came in early
// and left again.)
//
// Bound: HBM, one read of the logits (16384 x 151936 bf16: 4.98 GB).
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

constexpr int kTopkMaxWarps = 8;  // warps of a block of the stream kernel

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

// An entry: the key above the column's complement, so that a larger word is a
// better column and no two are equal.
__device__ __forceinline__ u64 entry_of(uint32_t key, int column) {
  return (static_cast<u64>(key) << 32) | (0xffffffffu - static_cast<uint32_t>(column));
}
__device__ __forceinline__ int64_t entry_column(u64 e) { return 0xffffffffu - static_cast<uint32_t>(e); }

struct TopkParams {
  const unsigned char* logits;
  int64_t n_rows, vocab, ld;
  int tile_v, num_tiles;
  int unit_tiles;  // tiles of a unit: what one warp of the stream kernel takes at a time
  int units;       // units of a row
  int tile_chunks; // chunks of a tile: its lanes that hold columns (32, or fewer in narrow tiles)
  const int64_t* targets;
  int64_t ignore_index;
  float rcp;
  int k;
  float* part_max;  // [n_rows, num_tiles]
  float* part_sum;
  float* part_ent;
  unsigned char* chunk_max;  // [n_rows, num_tiles, tile_chunks] of the logits' type
  unsigned stage_bytes;
};

// ---------------------------------------------------------------------------
// The pass over the logits.
// ---------------------------------------------------------------------------

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
      tile = static_cast<int>(unit - row * p.units) * p.unit_tiles;
      end = min(tile + p.unit_tiles, p.num_tiles);
      return;
    }
  }
  __device__ __forceinline__ void next(const TopkParams& p, int64_t stride) {
    if (++tile < end) return;
    unit += stride;
    settle(p, stride);
  }
};

// A tile in registers: the lane's maximum, and the sums for the tile's maximum
// (the operations of tile_reduce_regs_t, in its order).
template <int DT, bool FULL>
__device__ __forceinline__ float regs_max(const TileRegs<DT>& r, int valid, int lane) {
  const int ng = FULL ? TileRegs<DT>::kMaxGroups : lane_groups(valid, lane);
  uint32_t mx[Group<DT>::kW];
  Group<DT>::max_init(mx);
#pragma unroll
  for (int i = 0; i < TileRegs<DT>::kMaxGroups; ++i)
    if (FULL || i < ng) Group<DT>::max_acc(mx, r.w[i]);
  return Group<DT>::max_fin(mx);
}

template <int DT, bool FULL, bool ENT>
__device__ __forceinline__ TilePartial regs_sums(const TileRegs<DT>& r, int valid, int lane, float mx_all, float rcp) {
  const int ng = FULL ? TileRegs<DT>::kMaxGroups : lane_groups(valid, lane);
  const float m = rcp == 1.0f ? mx_all : __fmul_rn(mx_all, rcp);
  const float shift = (mx_all == -INFINITY) ? 0.0f : mx_all;
  const float c = __fmul_rn(rcp, kLog2e);
  const uint64_t shift2 = pk(shift, shift), c2 = pk(c, c);
  uint64_t a[4] = {0, 0, 0, 0}, u[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < TileRegs<DT>::kMaxGroups; ++i)
    if (FULL || i < ng) Group<DT>::template sum_acc<ENT, false>(a, u, r.w[i], shift2, c2);
  return finish_tile<ENT>(m, a, u);
}

// The lane's maximum of a tile in shared memory (tiles past what registers hold).
template <int DT, int WOFF>
__device__ __forceinline__ float smem_max_t(const unsigned char* tile, int valid, int lane, unsigned sh) {
  const int groups = (valid + kGroup - 1) / kGroup;
  const int rem = valid % kGroup;
  uint32_t mx[Group<DT>::kW];
  Group<DT>::max_init(mx);
  for (int g = lane; g < groups; g += kLanes) {
    uint32_t w[Group<DT>::kW];
    load_group<DT, WOFF>(tile, g, sh, w);
    if (rem != 0 && g == groups - 1) Group<DT>::mask_tail(w, rem);
    Group<DT>::max_acc(mx, w);
  }
  return Group<DT>::max_fin(mx);
}

template <int DT, bool SHIFTED>
__device__ __forceinline__ float smem_max(const unsigned char* tile, int valid, int lane, unsigned off) {
  const unsigned sh = 8u * (off & 3u);
  if (!SHIFTED || off == 0) return smem_max_t<DT, -1>(tile, valid, lane, 0);
  switch (off >> 2) {
    case 0: return smem_max_t<DT, 0>(tile, valid, lane, sh);
    case 1: return smem_max_t<DT, 1>(tile, valid, lane, sh);
    case 2: return smem_max_t<DT, 2>(tile, valid, lane, sh);
    default: return smem_max_t<DT, 3>(tile, valid, lane, sh);
  }
}

// A maximum of stored values, in their type (exact).
template <int DT>
__device__ __forceinline__ void store_value(unsigned char* base, int64_t i, float v) {
  if (DT == BIL_F32)
    reinterpret_cast<float*>(base)[i] = v;
  else if (DT == BIL_BF16)
    reinterpret_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v);
  else
    reinterpret_cast<__half*>(base)[i] = __float2half_rn(v);
}

template <int DT, bool ALIGNED, bool ENT>
__global__ void __launch_bounds__(kTopkMaxWarps * kLanes, 2) topk_stream_kernel(const TopkParams p) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  __shared__ uint64_t full_bars[kTopkMaxWarps];
  __shared__ int abort_flag;
  constexpr int EB = Elem<DT>::kBytes;
  const int warp = threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  const int warps = blockDim.x / kLanes;
  volatile int* abort = &abort_flag;
  uint64_t* full = &full_bars[warp];
  unsigned char* stage = smem_raw + static_cast<size_t>(warp) * p.stage_bytes;
  if (threadIdx.x == 0) *abort = 0;
  if (lane == 0) {
    mbar_init(full, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  // Consecutive units go to different blocks.
  const int64_t stride = static_cast<int64_t>(gridDim.x) * warps;
  const uint64_t policy = evict_first_policy();
  UnitCursor at{static_cast<int64_t>(warp) * gridDim.x + blockIdx.x, 0, 0, 0};
  at.settle(p, stride);

  // The copy of the tile at `c` into the warp's stage (its last reader is
  // done): the 16-byte aligned span that covers the tile, as in the streaming
  // forward.
  auto issue = [&](const UnitCursor& c) {
    if (lane != 0 || !c.more(p)) return;
    const int64_t col0 = static_cast<int64_t>(c.tile) * p.tile_v;
    const int valid = static_cast<int>(min(static_cast<int64_t>(p.tile_v), p.vocab - col0));
    const unsigned char* src = p.logits + (c.row * p.ld + col0) * EB;
    const unsigned off = ALIGNED ? 0u : static_cast<unsigned>(reinterpret_cast<uintptr_t>(src) & 15u);
    const unsigned bytes = static_cast<unsigned>(align_up(off + static_cast<size_t>(valid) * EB, 16));
    mbar_arrive_expect_tx(full, bytes);
    bulk_g2s(stage, src - off, bytes, full, policy);
  };
  issue(at);

  unsigned parity = 0;
  bool ok = true;
  while (at.more(p)) {
    ok = warp_wait(full, parity, abort, kWatchFull);
    if (!ok) break;
    parity ^= 1u;
    const UnitCursor now = at;
    at.next(p, stride);
    const int64_t col0 = static_cast<int64_t>(now.tile) * p.tile_v;
    const int valid = static_cast<int>(min(static_cast<int64_t>(p.tile_v), p.vocab - col0));
    const unsigned char* src = p.logits + (now.row * p.ld + col0) * EB;
    const unsigned off = ALIGNED ? 0u : static_cast<unsigned>(reinterpret_cast<uintptr_t>(src) & 15u);
    const int64_t o = now.row * p.num_tiles + now.tile;
    TilePartial tp;
    float lane_max;
    if (p.tile_v <= TileRegs<DT>::kMaxTile) {
      const bool whole = valid == TileRegs<DT>::kMaxTile;
      TileRegs<DT> regs;
      tile_load_regs<DT, !ALIGNED>(stage, valid, lane, regs, off);
      __syncwarp();  // the stage has been read
      issue(at);
      lane_max = whole ? regs_max<DT, true>(regs, valid, lane) : regs_max<DT, false>(regs, valid, lane);
      const float mx_all = warp_max(lane_max);
      tp = whole ? regs_sums<DT, true, ENT>(regs, valid, lane, mx_all, p.rcp)
                 : regs_sums<DT, false, ENT>(regs, valid, lane, mx_all, p.rcp);
      if (ENT && tp.u != tp.u) {  // as in the streaming forward: u from a clamped pass
        if (ALIGNED) {
          tile_load_regs<DT>(src, valid, lane, regs);
        } else {
          tile_load_regs<DT, true, true>(src - off, valid, lane, regs, off);
        }
        tp.u = tile_reduce_regs<DT, ENT, true>(regs, valid, lane, p.rcp).u;
      }
    } else {
      lane_max = smem_max<DT, !ALIGNED>(stage, valid, lane, off);
      tp = tile_reduce_smem<DT, ENT, !ALIGNED>(stage, valid, lane, p.rcp, off);
      __syncwarp();
      issue(at);
    }
    if (lane < p.tile_chunks) store_value<DT>(p.chunk_max, o * p.tile_chunks + lane, lane_max);
    if (lane == 0) {
      p.part_max[o] = tp.m;
      p.part_sum[o] = tp.s;
      if (ENT) p.part_ent[o] = tp.u;
    }
  }
  // A warp that gave up waits (bounded) for its own copy in flight.
  if (!ok && lane == 0) thread_wait_watch(full, parity, abort, kWatchDrain, &g_watchdog, false);
}

// ---------------------------------------------------------------------------
// The row.
// ---------------------------------------------------------------------------

constexpr int kSelWarps = 4;                     // warps that choose the columns
constexpr int kSelThreads = kSelWarps * kLanes;
constexpr int kRowThreads = kSelThreads + kLanes;  // and one that merges the partials
constexpr int kCandidates = 1024;                // entries the selection holds
constexpr int kDigitBits = 11;                   // of a pass of the radix selection
constexpr int kBins = 1 << kDigitBits;
constexpr int kQueue = 2 * kLanes;               // chunks a warp holds between two rounds of reading

__device__ __forceinline__ void sel_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSelThreads) : "memory"); }

struct alignas(16) SelShared {
  union {
    u64 cand[kCandidates];
    uint32_t bins[kBins];
  };
  uint32_t group_max[2 * kSelThreads];
  int queue[kSelWarps][kQueue];
  u64 merged[BIL_MAX_TOPK];
  int count;
  uint32_t bound;
  int above;
};
static_assert(sizeof(uint32_t) * kBins <= sizeof(u64) * kCandidates, "the bins share the candidates' space");

// The columns of one row by way of its chunks.
template <int DT>
struct RowColumns {
  static constexpr int EB = Elem<DT>::kBytes;
  const unsigned char* row;    // column 0
  const unsigned char* chunks; // the row's chunk maxima
  int vocab, tile_v, tile_chunks, num_chunks;
  int warp, lane;
  int* queue;

  __device__ __forceinline__ uint32_t chunk_key(int c) const {
    return order_key(Elem<DT>::one(chunks + static_cast<size_t>(c) * EB));
  }
  // keys of the 8 columns of a group from column c0; `n` exist (the others count as none: key 0)
  __device__ __forceinline__ void keys8(int c0, int n, uint32_t (&key)[kGroup]) const {
    const unsigned char* p = row + static_cast<int64_t>(c0) * EB;
    float v[kGroup];
    if (n == kGroup && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
      uint32_t w[Group<DT>::kW];
      Group<DT>::load(p, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t x = Group<DT>::xpair(w, j);
        v[2 * j] = lo_of(x);
        v[2 * j + 1] = hi_of(x);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kGroup; ++j) v[j] = j < n ? Elem<DT>::one(p + j * EB) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < kGroup; ++j) key[j] = order_key(v[j]);
  }
  // fn(key, column) for the columns of the queue's first n chunks: half a warp a
  // chunk, a lane a group of 8, two chunks in flight.
  template <typename F>
  __device__ __forceinline__ void read_queue(int n, F fn) const {
    __syncwarp();
    for (int i = lane / 16; i < n; i += 4) {
      int c0[2], steps[2], cols[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const bool have = i + 2 * q < n;
        const int c = queue[have ? i + 2 * q : 0];
        const int tile = c / tile_chunks, l = c - tile * tile_chunks;
        const int valid = min(tile_v, vocab - tile * tile_v);
        c0[q] = tile * tile_v;
        cols[q] = valid;
        steps[q] = have ? l * kGroup : valid;  // first column of the chunk, in the tile
      }
      for (int s = (lane % 16) * kLanes * kGroup; s < tile_v; s += 16 * kLanes * kGroup) {
        uint32_t key[2][kGroup];
        int left[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int e = steps[q] + s;
          left[q] = min(kGroup, cols[q] - e);
          if (left[q] > 0) keys8(c0[q] + e, left[q], key[q]);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (left[q] <= 0) continue;
#pragma unroll
          for (int j = 0; j < kGroup; ++j)
            if (j < left[q]) fn(key[q][j], c0[q] + steps[q] + s + j);
        }
      }
    }
    __syncwarp();
  }
  // fn(key, column) for every column of the chunks whose maximum is `least` or
  // more (the four warps share them).
  template <typename F>
  __device__ __forceinline__ void visit(uint32_t least, F fn) const {
    int n = 0;
    for (int c0 = warp * kLanes; c0 < num_chunks; c0 += kSelThreads) {
      const int c = c0 + lane;
      const bool in = c < num_chunks && chunk_key(c) >= least;
      const unsigned vote = __ballot_sync(0xffffffffu, in);
      if (vote == 0u) continue;
      if (in) queue[n + __popc(vote & ((1u << lane) - 1u))] = c;
      n += __popc(vote);
      if (n > kQueue - kLanes) {
        read_queue(n, fn);
        n = 0;
      }
    }
    if (n != 0) read_queue(n, fn);
  }
};

// The row's k best columns, best first, into sm.merged (kSelThreads threads).
template <int DT>
__device__ void select_columns(const RowColumns<DT>& cols, int k, SelShared& sm) {
  const int tid = threadIdx.x;
  // 1. the groups' maxima: thread i has chunks i, i + 128, ...; for k > 32 in two groups, odd and even.
  {
    uint32_t m[2] = {0, 0};
    int j = 0;
    for (int c = tid; c < cols.num_chunks; c += kSelThreads, j ^= 1) m[j] = max(m[j], cols.chunk_key(c));
    if (k <= kLanes) m[0] = max(m[0], m[1]);
    sm.group_max[tid] = m[0];
    if (k > kLanes) sm.group_max[kSelThreads + tid] = m[1];
    if (tid == 0) {
      sm.count = 0;
      sm.bound = 0;
    }
  }
  sel_sync();
  // 2. the k-th largest of them: it has k columns at or above it (0 where there are fewer groups than k)
  {
    const int groups = k <= kLanes ? kSelThreads : 2 * kSelThreads;
    for (int i = tid; i < groups; i += kSelThreads) {
      const uint32_t mine = sm.group_max[i];
      int above = 0;
#pragma unroll 4
      for (int j = 0; j < groups; j += 4) {
        const uint4 o = *reinterpret_cast<const uint4*>(&sm.group_max[j]);
        above += (o.x > mine || (o.x == mine && j < i)) + (o.y > mine || (o.y == mine && j + 1 < i)) +
                 (o.z > mine || (o.z == mine && j + 2 < i)) + (o.w > mine || (o.w == mine && j + 3 < i));
      }
      if (above == k - 1) sm.bound = mine;
    }
  }
  sel_sync();
  uint32_t least = sm.bound;  // columns with this key or more are wanted
  auto append = [&](uint32_t key, int c) {
    if (key < least) return;
    const int at = atomicAdd(&sm.count, 1);
    if (at < kCandidates) sm.cand[at] = entry_of(key, c);
  };
  // 3. those columns; at and below -inf the bound says nothing (a chunk of NaN also says -inf)
  bool enough = false;  // sm.cand holds all columns >= least, k of them at least
  if (least > kKeyNegInf) {
    cols.visit(least, append);
    sel_sync();
    enough = sm.count <= kCandidates;
  } else {
    least = kKeyNegInf;
  }
  if (!enough) {
    // Too many columns reach the bound, or there is none: the columns above it.
    const uint32_t floor_key = least;
    least = floor_key + 1;
    sel_sync();
    if (tid == 0) sm.count = 0;
    sel_sync();
    cols.visit(least, append);
    sel_sync();
    int found = sm.count;
    sel_sync();  // every thread has read the count before any may change it
    if (found > kCandidates) {
      // Radix selection over the keys above floor_key, from the top digit, until few enough are left: `prefix`
      // and above, `fixed` bits of it known.
      uint32_t prefix = 0;
      int fixed = 0, taken = 0;  // taken: columns above prefix's range
      for (;;) {
        const int bits = min(kDigitBits, 32 - fixed), shift = 32 - fixed - bits;
        sel_sync();
        for (int i = tid; i < kBins; i += kSelThreads) sm.bins[i] = 0;
        sel_sync();
        const uint32_t lo = max(least, prefix);
        cols.visit(lo, [&](uint32_t key, int) {
          if (key < lo || (fixed != 0 && (key >> (32 - fixed)) != (prefix >> (32 - fixed)))) return;
          atomicAdd(&sm.bins[(key >> shift) & ((1u << bits) - 1u)], 1u);
        });
        sel_sync();
        if (cols.warp == 0) {
          // from the highest bin down: the bin that holds the k-th column
          int sum = taken, digit = -1, before = 0;
          for (int b0 = (1 << bits) - kLanes; b0 >= 0 && digit < 0; b0 -= kLanes) {
            const int n = static_cast<int>(sm.bins[b0 + kLanes - 1 - cols.lane]);  // lane 0: the highest
            int upto = n;
#pragma unroll
            for (int o = 1; o < kLanes; o *= 2) {
              const int v = __shfl_up_sync(0xffffffffu, upto, o);
              if (cols.lane >= o) upto += v;
            }
            const unsigned vote = __ballot_sync(0xffffffffu, sum + upto >= k);
            if (vote != 0u) {
              const int src = __ffs(vote) - 1;
              digit = b0 + kLanes - 1 - src;
              before = sum + __shfl_sync(0xffffffffu, upto - n, src);
              found = sum + __shfl_sync(0xffffffffu, upto, src);
            }
            sum += __shfl_sync(0xffffffffu, upto, kLanes - 1);
          }
          if (cols.lane == 0) {
            sm.bound = prefix | (static_cast<uint32_t>(max(digit, 0)) << shift);
            sm.above = before;
            sm.count = found;
          }
        }
        sel_sync();
        prefix = sm.bound;
        taken = sm.above;
        found = sm.count;  // columns >= prefix
        fixed += bits;
        if (found <= kCandidates || fixed == 32) break;
      }
      // `prefix` and above hold k columns; where even those are too many (equal logits), the ones above it
      // are fewer than k and the rest is found below
      least = found <= kCandidates ? max(least, prefix) : prefix + 1;
      sel_sync();
      if (tid == 0) sm.count = 0;
      sel_sync();
      cols.visit(least, append);
      sel_sync();
      found = sm.count;
      sel_sync();
    }
    // Equal columns just below `least`, then NaN, in column order: one warp, tile by tile.
    if (found < k) {
      if (cols.warp == 0) {
        uint32_t want = least - 1;
        for (;;) {
          for (int tile = 0; tile * cols.tile_chunks < cols.num_chunks && found < k; ++tile) {
            const bool any = cols.lane < cols.tile_chunks &&
                             cols.chunk_key(tile * cols.tile_chunks + cols.lane) >= max(want, kKeyNegInf);
            if (!__any_sync(0xffffffffu, any)) continue;
            const int valid = min(cols.tile_v, cols.vocab - tile * cols.tile_v);
            for (int e0 = 0; e0 < valid && found < k; e0 += kLanes) {
              const int c = tile * cols.tile_v + e0 + cols.lane;
              const bool in = e0 + cols.lane < valid &&
                              order_key(Elem<DT>::one(cols.row + static_cast<int64_t>(c) * Elem<DT>::kBytes)) == want;
              const unsigned vote = __ballot_sync(0xffffffffu, in);
              const int at = found + __popc(vote & ((1u << cols.lane) - 1u));
              if (in && at < k) sm.cand[at] = entry_of(want, c);
              found = min(k, found + __popc(vote));
            }
          }
          if (found >= k || want == 0) break;
          want = 0;
        }
        if (cols.lane == 0) sm.count = found;
      }
      sel_sync();
    }
  }
  // 4. in order: an entry's place is the number of entries above it
  const int n = sm.count;
  for (int i = tid; i < n; i += kSelThreads) {
    const u64 mine = sm.cand[i];
    int above = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) above += sm.cand[j] > mine ? 1 : 0;
    if (above < k) sm.merged[above] = mine;
  }
}

template <int DT, bool ENT>
__global__ void __launch_bounds__(kRowThreads) topk_row_kernel(const TopkParams p, float* logp, float* lse,
                                                               float* entropy, int64_t* top_ids, float* top_logp) {
  __shared__ SelShared sm;
  __shared__ float scratch[kMergeScratch];
  __shared__ float row_lse;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % kLanes, warp = threadIdx.x / kLanes;
  const int64_t row = blockIdx.x;
  const int64_t t = p.targets[row];
  int64_t* ids = top_ids + row * p.k;
  float* top = top_logp + row * p.k;
  if (t == p.ignore_index) {
    for (int j = threadIdx.x; j < p.k; j += kRowThreads) {
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
  const unsigned char* src = p.logits + row * p.ld * Elem<DT>::kBytes;
  if (warp == kSelWarps) {
    const int64_t o = row * p.num_tiles;
    float H = 0.0f;
    const float L = merge_lse<ENT, true>(p.part_max + o, p.part_sum + o, ENT ? p.part_ent + o : nullptr, p.num_tiles,
                                         lane, &H, scratch);
    if (lane == 0) {
      row_lse = L;
      float z = __int_as_float(0x7fc00000);
      if (t >= 0 && t < p.vocab) {
        z = Elem<DT>::one(src + t * Elem<DT>::kBytes);
        if (p.rcp != 1.0f) z = __fmul_rn(z, p.rcp);
      }
      logp[row] = __fsub_rn(z, L);
      if (lse != nullptr) lse[row] = L;
      if (ENT) entropy[row] = H;
    }
  } else {
    RowColumns<DT> cols;
    cols.row = src;
    cols.num_chunks = p.num_tiles * p.tile_chunks;
    cols.chunks = p.chunk_max + row * cols.num_chunks * Elem<DT>::kBytes;
    cols.vocab = static_cast<int>(p.vocab);
    cols.tile_v = p.tile_v;
    cols.tile_chunks = p.tile_chunks;
    cols.warp = warp;
    cols.lane = lane;
    cols.queue = sm.queue[warp];
    select_columns<DT>(cols, p.k, sm);
  }
  __syncthreads();
  for (int j = threadIdx.x; j < p.k; j += kRowThreads) {
    const u64 e = sm.merged[j];
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

// How the stream kernel is laid out: warps of a block, blocks of an SM.  One
// stage a warp: a tile is in registers (or, past 8 KB, being reduced) while the
// others' copies are in flight, and 16 warps (at up to 128 registers a thread)
// keep 128 KB of them on the way, twice what the latency needs.  Two blocks an
// SM where that leaves them four warps each or more, else one.
constexpr size_t kSmSmemBytes = 228 * 1024;  // an SM's shared memory, 1 KB of it reserved for each block
void stream_layout(size_t stage_bytes, int* warps, int* blocks) {
  for (*blocks = 2; *blocks >= 1; --*blocks) {
    const size_t room = kSmSmemBytes / *blocks - 1024 - 128;  // 128: the barriers
    *warps = static_cast<int>(std::min<size_t>(kTopkMaxWarps, room / stage_bytes));
    if (*blocks == 1 || *warps >= 4) return;
  }
}

// Tiles of a unit: the cut of the rows that gives the least time, a warp's time
// being its units' tiles and a quarter of a tile a unit for the change of row.
int unit_tiles(int64_t n_rows, int num_tiles, int64_t warps) {
  int best = num_tiles;
  double least = 0.0;
  for (int u = 1; u <= std::min(num_tiles, 64); ++u) {
    const int tiles = (num_tiles + u - 1) / u;
    const int64_t units = n_rows * ((num_tiles + tiles - 1) / tiles);
    const double cost = static_cast<double>((units + warps - 1) / warps) * (tiles + 0.25);
    if (u == 1 || cost < least) {
      least = cost;
      best = tiles;
    }
  }
  return best;
}

size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

// The workspace: chunk maxima, then the partials.
struct TopkWorkspace {
  int tile_chunks;
  size_t chunks, part, total;  // bytes: the chunk maxima, one partial array, all
};

TopkWorkspace topk_workspace(int dtype, int64_t n_rows, int64_t num_tiles, int tile_v, bool ent) {
  TopkWorkspace w;
  w.tile_chunks = std::min(kLanes, tile_v / kGroup);
  w.chunks = round256(static_cast<size_t>(n_rows) * num_tiles * w.tile_chunks * bil_internal::elem_bytes(dtype));
  w.part = round256(static_cast<size_t>(n_rows) * num_tiles * sizeof(float));
  w.total = w.chunks + w.part * (ent ? 3 : 2);
  return w;
}

// The sizes both the workspace query and the forward check.
int check_topk_sizes(int dtype, int64_t n_rows, int64_t vocab, int32_t tile_v, int32_t k, int64_t* num_tiles) {
  if (n_rows < 0 || vocab < 1 || k < 1 || k > vocab) return BIL_E_INVALID_ARG;
  if (int st = bil_internal::check_tile(dtype, vocab, tile_v, num_tiles)) return st;
  if (k > BIL_MAX_TOPK || vocab > INT32_MAX || *num_tiles > BIL_MAX_FUSED_TILES || n_rows > INT32_MAX)
    return BIL_E_UNSUPPORTED;
  return BIL_OK;
}

template <int DT, bool ALIGNED, bool ENT>
int launch_topk_t(TopkParams p, float* logp, float* lse, float* entropy, int64_t* top_ids, float* top_logp,
                  cudaStream_t stream) {
  int sms = 0, smem_optin = 0;
  if (int st = bil_internal::device_limits(&sms, &smem_optin)) return st;
  p.stage_bytes =
      static_cast<unsigned>(align_up(static_cast<size_t>(p.tile_v) * Elem<DT>::kBytes + (ALIGNED ? 0 : 16), 128));
  int warps = 0, blocks = 0;
  stream_layout(p.stage_bytes, &warps, &blocks);
  const int64_t slots = static_cast<int64_t>(sms) * blocks;
  p.unit_tiles = unit_tiles(p.n_rows, p.num_tiles, slots * warps);
  p.units = (p.num_tiles + p.unit_tiles - 1) / p.unit_tiles;
  const int64_t units = p.n_rows * p.units;
  // few units: one warp a block, so that they spread over the SMs
  warps = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(warps, (units + slots - 1) / slots)));
  const int64_t grid = std::min<int64_t>(slots, (units + warps - 1) / warps);
  const size_t smem = static_cast<size_t>(warps) * p.stage_bytes;
  if (smem > static_cast<size_t>(smem_optin)) return BIL_E_UNSUPPORTED;
  auto kernel = topk_stream_kernel<DT, ALIGNED, ENT>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
    return BIL_E_CUDA;
  if (launch_pdl(kernel, grid, warps * kLanes, smem, stream, 1, p) != cudaSuccess) return BIL_E_CUDA;
  return launch_pdl(topk_row_kernel<DT, ENT>, p.n_rows, kRowThreads, 0, stream, 1, p, logp, lse, entropy, top_ids,
                    top_logp) == cudaSuccess
             ? BIL_OK
             : BIL_E_CUDA;
}

template <int DT>
int launch_topk(const TopkParams& p, bool ent, float* logp, float* lse, float* entropy, int64_t* top_ids,
                float* top_logp, cudaStream_t stream) {
  const bool vec = aligned_to(p.logits, 16) && (p.n_rows <= 1 || (p.ld * Elem<DT>::kBytes) % 16 == 0);
  if (vec)
    return ent ? launch_topk_t<DT, true, true>(p, logp, lse, entropy, top_ids, top_logp, stream)
               : launch_topk_t<DT, true, false>(p, logp, lse, entropy, top_ids, top_logp, stream);
  return ent ? launch_topk_t<DT, false, true>(p, logp, lse, entropy, top_ids, top_logp, stream)
             : launch_topk_t<DT, false, false>(p, logp, lse, entropy, top_ids, top_logp, stream);
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
  *bytes = static_cast<int64_t>(topk_workspace(dtype, n_rows, num_tiles, tile_v, entropy != 0).total);
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
  const TopkWorkspace w = topk_workspace(dtype, n_rows, num_tiles, tile_v, ent);
  if (workspace_bytes < static_cast<int64_t>(w.total)) return BIL_E_INVALID_ARG;
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
  p.tile_chunks = w.tile_chunks;
  p.targets = target_ids;
  p.ignore_index = ignore_index;
  p.rcp = rcp;
  p.k = k;
  p.chunk_max = ws;
  p.part_max = reinterpret_cast<float*>(ws + w.chunks);
  p.part_sum = reinterpret_cast<float*>(ws + w.chunks + w.part);
  p.part_ent = ent ? reinterpret_cast<float*>(ws + w.chunks + 2 * w.part) : nullptr;
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
