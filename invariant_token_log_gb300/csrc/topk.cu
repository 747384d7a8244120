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
//                       contract, and the maximum of every 64 columns (a
//                       chunk), which it reduces on the way to the tile's.
//   topk_row_kernel     the row.  The partials are merged in the one fixed
//                       order (merge_lse: logp, lse and the entropy are
//                       bil_logp_fwd's bits).  The columns are found by way of
//                       the chunks' maxima: of 128 (k > 32: 256) groups of
//                       chunks, the k-th largest maximum has k columns at or
//                       above it, and few chunks reach it (about 22 of 2374 for
//                       k = 20 of 151936 columns), so that only those are read
//                       again: 22 lines of 128 bytes.
//
// The choice of columns thus costs the pass over the logits little, whatever k
// is.  Measured otherwise, 4096 x 151936 bf16, k = 20: a list of the best
// columns kept by the streaming warp, sorted across its lanes, 437 to 528 us
// (most of its instructions went into columns that came in early and left
// again); chunks of a lane's 128 columns, whose maximum the lane has anyway, 240
// to 265 us (they lie in 16 places 512 bytes apart, and the row kernel was bound
// by the 45 KB of DRAM lines it read again per row).
//
// Up to 48 rows of a 16-bit type take one kernel that does both, a cluster of
// blocks a row (topk_cluster_kernel).
//
// Bound: HBM, one read of the logits.  4096 x 151936 bf16, k = 20, no row ignored:
// 212 us, 5.9 TB/s (0.86 of a plain copy's rate, whose time would be 183 us); with
// the entropy 214 us, where the forward without alternatives takes 196: the choice
// of columns adds 9%.  Rows 151939 apart 234 and 268 us.  float32 405 us, 6.1 TB/s
// (0.91).  4096 x 32000 60 us, 0.65: the row kernel's time is per row and weighs more
// on short ones.  One row: 7 us, the latency of the launch, of one tile and of the
// choice.
//
//   topk_grad_sum_kernel  g + sum_j gk_j, what the softmax term is scaled by;
//   (bil_logp_bwd)        d = -(g + sum gk) p - gh p (a + H), one pass;
//   topk_grad_fix_kernel  the k + 1 columns per row that have a term of their own.

#include "../../include/bil.h"
#include "device_common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "layout.h"
#include "logp_device.cuh"

#include <algorithm>

namespace {

using bil_layout::kTopkMaxWarps;
constexpr int kChunk = 64;        // columns of a chunk

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
  int tile_chunks; // chunks of a tile
  const int64_t* targets;
  int64_t ignore_index;
  float rcp;
  int k;
  float* part_max;  // [n_rows, num_tiles]
  float* part_sum;
  float* part_ent;
  unsigned char* chunk_max;  // [n_rows, num_tiles, tile_chunks] of the logits' type, -inf up to the row's pitch
  int64_t chunk_pitch;       // bytes of a row of chunk maxima, a multiple of 16
  unsigned stage_bytes;
};

// ---------------------------------------------------------------------------
// The pass over the logits.
// ---------------------------------------------------------------------------

// Where a warp is in its units: the tile, where the unit's tiles end, and the
// tile's first column.  Units of ignored rows are passed over.
struct UnitCursor {
  int64_t unit, row;
  const unsigned char* src;
  int tile, end;
  bool more;

  // the unit itself, or the next one at `stride` that is not of an ignored row
  __device__ __forceinline__ void settle(const TopkParams& p, int64_t stride, int eb) {
    for (; unit < p.n_rows * p.units; unit += stride) {
      row = p.units == 1 ? unit : unit / p.units;
      if (p.targets[row] == p.ignore_index) continue;
      tile = static_cast<int>(unit - row * p.units) * p.unit_tiles;
      end = min(tile + p.unit_tiles, p.num_tiles);
      src = p.logits + (row * p.ld + static_cast<int64_t>(tile) * p.tile_v) * eb;
      more = true;
      return;
    }
    more = false;
  }
  __device__ __forceinline__ void next(const TopkParams& p, int64_t stride, int eb) {
    if (++tile < end) {
      src += p.tile_v * eb;
      return;
    }
    unit += stride;
    settle(p, stride, eb);
  }
  __device__ __forceinline__ int valid(const TopkParams& p) const {
    return tile < p.num_tiles - 1 ? p.tile_v : static_cast<int>(p.vocab - static_cast<int64_t>(tile) * p.tile_v);
  }
};

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

// The chunk maxima of up to kMaxTile columns (16 groups of a 16-bit type a
// lane, 8 of float32).  Group i of lane l is columns 8 (l + 32 i) on, so chunk
// c + 4 i is group i of the eight lanes 8 c on.  Eight registers a lane, a
// 16-bit type's with the maxima of the groups 2 a and 2 a + 1; three exchanges
// within the eight lanes, each halving what a lane still holds, leave register
// l % 8 reduced in lane l: seven shuffles.
template <int DT>
struct ChunkMax {
  static constexpr int EB = Elem<DT>::kBytes;
  static constexpr int kW = Group<DT>::kW;
  static constexpr int kGroups = EB == 4 ? 8 : 16;
  static constexpr uint32_t kNone = EB == 4 ? Elem<DT>::kNegInf : Elem<DT>::kNegInf * 0x10001u;
  uint32_t r[8];

  __device__ static __forceinline__ uint32_t max_of(uint32_t a, uint32_t b) {
    if constexpr (EB == 4)
      return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    else
      return Elem<DT>::max2(a, b);
  }
  // a group's words to one (16-bit types: a pair whose halves are still to be compared)
  __device__ static __forceinline__ uint32_t group(const uint32_t (&w)[kW]) {
    uint32_t m = max_of(max_of(w[0], w[1]), max_of(w[2], w[3]));
    if constexpr (EB == 4) m = max_of(m, max_of(max_of(w[kW - 4], w[kW - 3]), max_of(w[kW - 2], w[kW - 1])));
    return m;
  }
  // groups 2 a and 2 a + 1 of a 16-bit type
  __device__ __forceinline__ void pair(int a, uint32_t even, uint32_t odd) {
    r[a] = max_of(__byte_perm(even, odd, 0x5410), __byte_perm(even, odd, 0x7632));
  }
  // Reduces, stores the chunks first + 0, 1, ... that are below `chunks`, and returns the lane's maximum.
  __device__ __forceinline__ float finish(unsigned char* out, int first, int chunks, int lane) {
#pragma unroll
    for (int half = 4; half > 0; half /= 2) {
      const bool upper = (lane & half) != 0;
#pragma unroll
      for (int q = 0; q < half; ++q) {
        const uint32_t give = upper ? r[q] : r[q + half], keep = upper ? r[q + half] : r[q];
        r[q] = max_of(keep, __shfl_xor_sync(0xffffffffu, give, half));
      }
    }
    const int a = lane % 8, c = lane / 8;
    if constexpr (EB == 4) {
      const float v = fmaxf(-INFINITY, __uint_as_float(r[0]));  // NaN never wins
      if (first + c + 4 * a < chunks) store_value<DT>(out, first + c + 4 * a, v);
      return v;
    } else {
      float lo, hi;
      Elem<DT>::pair(r[0], lo, hi);
      lo = fmaxf(-INFINITY, lo);
      hi = fmaxf(-INFINITY, hi);
      if (first + c + 8 * a < chunks) store_value<DT>(out, first + c + 8 * a, lo);
      if (first + c + 8 * a + 4 < chunks) store_value<DT>(out, first + c + 8 * a + 4, hi);
      return fmaxf(lo, hi);
    }
  }
};

// Group g of a tile whose first element lies `off` bytes past the 16-byte
// aligned `tile`.  Of a 16-bit type: 8-byte words from the boundary at or below
// the group, one selection and a funnel shift by what is left of the offset (one
// code for all eight offsets, which differ from row to row).  Of float32: the
// 16-byte units, a case an offset (8-byte reads 32 bytes apart would take the
// banks nearly twice as long).
template <int DT>
__device__ __forceinline__ void load_group_at(const unsigned char* tile, unsigned off, int g, uint32_t (&w)[Group<DT>::kW]) {
  constexpr int kW = Group<DT>::kW;
  if constexpr (Elem<DT>::kBytes == 4) {
    switch (off >> 2) {
      case 0: load_group<DT, 0>(tile, g, 0, w); break;
      case 1: load_group<DT, 1>(tile, g, 0, w); break;
      case 2: load_group<DT, 2>(tile, g, 0, w); break;
      default: load_group<DT, 3>(tile, g, 0, w); break;
    }
  } else {
    const int at = static_cast<int>(off & 8u) + g * kGroup * Elem<DT>::kBytes;
    uint32_t v[kW + 2];
#pragma unroll
    for (int q = 0; q < kW / 2 + 1; ++q) {
      const uint2 x = *reinterpret_cast<const uint2*>(tile + at + 8 * q);
      v[2 * q] = x.x;
      v[2 * q + 1] = x.y;
    }
    const bool word = (off & 4u) != 0;
#pragma unroll
    for (int j = 0; j < kW + 1; ++j) v[j] = word ? v[j + 1] : v[j];
#pragma unroll
    for (int j = 0; j < kW; ++j) w[j] = __funnelshift_r(v[j], v[j + 1], 8u * (off & 3u));
  }
}

// As load_group_at with the columns past the tile's `valid` as -inf; ALIGNED: off is 0.
template <int DT, bool ALIGNED>
__device__ __forceinline__ void stage_group(const unsigned char* tile, unsigned off, int g, int valid,
                                            uint32_t (&w)[Group<DT>::kW]) {
  if constexpr (ALIGNED)
    load_group<DT, -1>(tile, g, 0, w);
  else
    load_group_at<DT>(tile, off, g, w);
  if (valid - g * kGroup < kGroup) Group<DT>::mask_tail(w, valid - g * kGroup);
}

// The lane's groups of a staged tile off 16-byte boundaries, as tile_load_regs
// gives those of one on them.
template <int DT>
__device__ __forceinline__ void load_regs_at(const unsigned char* tile, unsigned off, int valid, int lane, TileRegs<DT>& r) {
#pragma unroll
  for (int i = 0; i < TileRegs<DT>::kMaxGroups; ++i) {
    const int g = lane + kLanes * i;
    if (g * kGroup < valid) {
      load_group_at<DT>(tile, off, g, r.w[i]);
      if (valid - g * kGroup < kGroup) Group<DT>::mask_tail(r.w[i], valid - g * kGroup);
    }
  }
}

// The same from global memory (16-bit types): the aligned 16-byte units that hold
// the tile, each read once, by the lane that has the group that begins in it; the
// rest of a group is in the next lane's unit.  (Each lane reading the three 8-byte
// words of its groups: 32 rows of 151936 columns, 151939 apart, 14.8 us; so 10.7.)
template <int DT>
__device__ __forceinline__ void load_regs_shifted(const unsigned char* tile, unsigned off, int valid, int lane,
                                                  TileRegs<DT>& r) {
  constexpr int kGroups = TileRegs<DT>::kMaxGroups;
  const uint4* units = reinterpret_cast<const uint4*>(tile);
  const int n = (static_cast<int>(off) + valid * Elem<DT>::kBytes + 15) / 16;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int g = lane + kLanes * i;
    const uint4 u = g < n ? units[g] : make_uint4(0u, 0u, 0u, 0u);
    r.w[i][0] = u.x, r.w[i][1] = u.y, r.w[i][2] = u.z, r.w[i][3] = u.w;
  }
  uint4 past = make_uint4(0u, 0u, 0u, 0u);
  if (lane == 0 && kGroups * kLanes < n) past = units[kGroups * kLanes];
  const bool two = (off & 8u) != 0, one = (off & 4u) != 0;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const uint32_t next[4] = {i + 1 < kGroups ? r.w[(i + 1) % kGroups][0] : past.x,
                              i + 1 < kGroups ? r.w[(i + 1) % kGroups][1] : past.y,
                              i + 1 < kGroups ? r.w[(i + 1) % kGroups][2] : past.z,
                              i + 1 < kGroups ? r.w[(i + 1) % kGroups][3] : past.w};
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = r.w[i][j];
      v[4 + j] = __shfl_sync(0xffffffffu, lane == 0 ? next[j] : r.w[i][j], (lane + 1) % kLanes);
    }
#pragma unroll
    for (int j = 0; j < 6; ++j) v[j] = two ? v[j + 2] : v[j];
#pragma unroll
    for (int j = 0; j < 5; ++j) v[j] = one ? v[j + 1] : v[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[i][j] = __funnelshift_r(v[j], v[j + 1], 8u * (off & 3u));
    const int left = valid - (lane + kLanes * i) * kGroup;
    if (left > 0 && left < kGroup) Group<DT>::mask_tail(r.w[i], left);
  }
}

// As in the streaming forward, a tile's entropy sum from a clamped pass over the
// logits (in global memory), where the plain one gave NaN; mx_all: the tile's
// maximum.  Off 16-byte boundaries two groups at a time: all of them, shifted, do
// not fit beside what the pass keeps.
template <int DT, bool ALIGNED>
__device__ __forceinline__ float clamped_entropy(const unsigned char* src, int valid, int lane, float mx_all, float rcp,
                                                 TileRegs<DT>& regs) {
  if constexpr (ALIGNED) {
    tile_load_regs<DT>(src, valid, lane, regs);
    return tile_reduce_regs<DT, true, true>(regs, valid, lane, rcp).u;
  }
  const float shift = (mx_all == -INFINITY) ? 0.0f : mx_all;
  const float c = __fmul_rn(rcp, kLog2e);
  const uint64_t shift2 = pk(shift, shift), c2 = pk(c, c);
  uint64_t a[4] = {0, 0, 0, 0}, u[4] = {0, 0, 0, 0};
#pragma unroll 2
  for (int g = lane; g * kGroup < valid; g += kLanes) {
    const int left = valid - g * kGroup;
    uint32_t w[Group<DT>::kW];
    // the 4-byte words that hold a column of the tile
    const uintptr_t at = reinterpret_cast<uintptr_t>(src) + g * kGroup * Elem<DT>::kBytes;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(at & ~static_cast<uintptr_t>(3));
    const uint32_t* end = reinterpret_cast<const uint32_t*>(src + valid * Elem<DT>::kBytes);
    uint32_t v[Group<DT>::kW + 1];
#pragma unroll
    for (int j = 0; j <= Group<DT>::kW; ++j) v[j] = q + j < end ? q[j] : 0u;
#pragma unroll
    for (int j = 0; j < Group<DT>::kW; ++j) w[j] = __funnelshift_r(v[j], v[j + 1], 8u * (at & 3u));
    if (left < kGroup) Group<DT>::mask_tail(w, left);
    Group<DT>::template sum_acc<true, true>(a, u, w, shift2, c2);
  }
  return finish_tile<true>(0.0f, a, u).u;
}

// A tile of a 16-bit type in registers: its chunk maxima, to `out`, and the
// lane's part of the tile's.
template <int DT, bool FULL>
__device__ __forceinline__ float regs_max(const TileRegs<DT>& t, int valid, int lane, unsigned char* out, int chunks) {
  using C = ChunkMax<DT>;
  const int ng = FULL ? TileRegs<DT>::kMaxGroups : lane_groups(valid, lane);
  C c;
#pragma unroll
  for (int a = 0; a < 8; ++a) {
    const uint32_t even = FULL || 2 * a < ng ? C::group(t.w[2 * a]) : C::kNone;
    const uint32_t odd = FULL || 2 * a + 1 < ng ? C::group(t.w[2 * a + 1]) : C::kNone;
    c.pair(a, even, odd);
  }
  return c.finish(out, 0, chunks, lane);
}

// A tile's last group where it is a part of one, for the lane that has it (of
// the lane's groups it is the last too): Group::sum_acc with nothing added for
// the columns that are not there.  As -inf, which they are in the maximum, they
// would make the entropy sum 0 * inf, and the tile would be summed again with
// the clamp (4096 x 32003 bf16, a row's last tile of eight: 114 us, and 85 so; 4096
// x 32000, whose last group is whole, 65).
template <int DT, bool ENT>
__device__ __forceinline__ void sum_tail(uint64_t (&a)[4], uint64_t (&u)[4], const uint32_t (&w)[Group<DT>::kW], int valid,
                                         int lane, uint64_t shift2, uint64_t c2) {
  const int rem = valid % kGroup;
  if (rem == 0 || (valid / kGroup) % kLanes != lane) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint64_t t = mul2(sub2(Group<DT>::xpair(w, k), shift2), c2);
    const float t0 = 2 * k < rem ? lo_of(t) : 0.0f, t1 = 2 * k + 1 < rem ? hi_of(t) : 0.0f;
    const uint64_t e = pk(2 * k < rem ? ex2_approx(t0) : 0.0f, 2 * k + 1 < rem ? ex2_approx(t1) : 0.0f);
    a[k] = add2(a[k], e);
    if (ENT) u[k] = fma2(e, pk(t0, t1), u[k]);
  }
}

// The sums for the tile's maximum (the operations of tile_reduce_regs_t, in its order).
template <int DT, bool FULL, bool ENT>
__device__ __forceinline__ TilePartial regs_sums(const TileRegs<DT>& r, int valid, int lane, float mx_all, float rcp) {
  const float m = rcp == 1.0f ? mx_all : __fmul_rn(mx_all, rcp);
  const float shift = (mx_all == -INFINITY) ? 0.0f : mx_all;
  const float c = __fmul_rn(rcp, kLog2e);
  const uint64_t shift2 = pk(shift, shift), c2 = pk(c, c);
  uint64_t a[4] = {0, 0, 0, 0}, u[4] = {0, 0, 0, 0};
  uint32_t tail[Group<DT>::kW];
#pragma unroll
  for (int i = 0; i < TileRegs<DT>::kMaxGroups; ++i) {
    const int left = valid - (lane + kLanes * i) * kGroup;
    if (FULL || left >= kGroup) {
      Group<DT>::template sum_acc<ENT, false>(a, u, r.w[i], shift2, c2);
    } else if (left > 0) {
#pragma unroll
      for (int j = 0; j < Group<DT>::kW; ++j) tail[j] = r.w[i][j];
    }
  }
  if (!FULL) sum_tail<DT, ENT>(a, u, tail, valid, lane, shift2, c2);
  return finish_tile<ENT>(m, a, u);
}

// The same of a tile in shared memory (tiles past what registers hold).
template <int DT, bool ALIGNED>
__device__ __forceinline__ float smem_max(const unsigned char* tile, int valid, int lane, unsigned off,
                                          unsigned char* out, int chunks) {
  using C = ChunkMax<DT>;
  float m = -INFINITY;
#pragma unroll 1
  for (int g0 = 0; g0 < chunks * (kChunk / kGroup); g0 += C::kGroups * kLanes) {
    C c;
    uint32_t last = 0;
#pragma unroll
    for (int i = 0; i < C::kGroups; ++i) {
      const int g = g0 + i * kLanes + lane;
      uint32_t now = C::kNone;
      if (g * kGroup < valid) {
        uint32_t w[Group<DT>::kW];
        stage_group<DT, ALIGNED>(tile, off, g, valid, w);
        now = C::group(w);
      }
      if constexpr (C::EB == 4)
        c.r[i % 8] = now;
      else if (i % 2 == 1)
        c.pair(i / 2, last, now);
      last = now;
    }
    m = fmaxf(m, c.finish(out, g0 / (kChunk / kGroup), chunks, lane));
  }
  return m;
}

// The sums of a tile in shared memory for its maximum (the operations of
// tile_reduce_smem_t, in its order).
template <int DT, bool ENT, bool ALIGNED>
__device__ __forceinline__ TilePartial smem_sums(const unsigned char* tile, int valid, int lane, float mx_all, float rcp,
                                                 unsigned off) {
  const int groups = (valid + kGroup - 1) / kGroup;
  const float m = rcp == 1.0f ? mx_all : __fmul_rn(mx_all, rcp);
  const float shift = (mx_all == -INFINITY) ? 0.0f : mx_all;
  const float c = __fmul_rn(rcp, kLog2e);
  const uint64_t shift2 = pk(shift, shift), c2 = pk(c, c);
  uint64_t a[4] = {0, 0, 0, 0}, u[4] = {0, 0, 0, 0};
#pragma unroll 4
  for (int g = lane; g < valid / kGroup; g += kLanes) {
    uint32_t w[Group<DT>::kW];
    stage_group<DT, ALIGNED>(tile, off, g, valid, w);
    Group<DT>::template sum_acc<ENT, false>(a, u, w, shift2, c2);
  }
  if (groups != valid / kGroup) {
    uint32_t w[Group<DT>::kW];
    stage_group<DT, ALIGNED>(tile, off, groups - 1, valid, w);
    sum_tail<DT, ENT>(a, u, w, valid, lane, shift2, c2);
  }
  TilePartial tp = finish_tile<ENT>(m, a, u);
  if (ENT && tp.u != tp.u) {  // NaN (warp-uniform): the entropy terms again, with the clamp
    uint64_t a2[4] = {0, 0, 0, 0}, u2[4] = {0, 0, 0, 0};
#pragma unroll 1
    for (int g = lane; g < groups; g += kLanes) {
      uint32_t w[Group<DT>::kW];
      stage_group<DT, ALIGNED>(tile, off, g, valid, w);
      Group<DT>::template sum_acc<ENT, true>(a2, u2, w, shift2, c2);
    }
    tp.u = finish_tile<ENT>(m, a2, u2).u;
  }
  return tp;
}

template <int DT, bool ALIGNED, bool ENT>
__global__ void __launch_bounds__(kTopkMaxWarps * kLanes, 2) topk_stream_kernel(const TopkParams p) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  __shared__ uint64_t full_bars[kTopkMaxWarps];
  __shared__ int abort_flag;
  constexpr int EB = Elem<DT>::kBytes;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x / kLanes), 0);
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
  UnitCursor at;
  at.unit = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;
  at.settle(p, stride, EB);

  // The copy of the tile at `at` into the warp's stage (its last reader is
  // done): the 16-byte aligned span that covers the tile, as in the streaming
  // forward.
  auto issue = [&]() {
    if (lane != 0 || !at.more) return;
    const unsigned off = ALIGNED ? 0u : static_cast<unsigned>(reinterpret_cast<uintptr_t>(at.src) & 15u);
    const unsigned bytes = (off + static_cast<unsigned>(at.valid(p)) * EB + 15u) & ~15u;
    mbar_arrive_expect_tx(full, bytes);
    bulk_g2s(stage, at.src - off, bytes, full, policy);
  };
  issue();

  unsigned parity = 0;
  bool ok = true;
  while (at.more) {
    ok = warp_wait(full, parity, abort, kWatchFull);
    if (!ok) break;
    parity ^= 1u;
    const UnitCursor now = at;
    at.next(p, stride, EB);
    const int valid = now.valid(p);
    const unsigned char* src = now.src;
    const unsigned off = ALIGNED ? 0u : static_cast<unsigned>(reinterpret_cast<uintptr_t>(src) & 15u);
    const int64_t o = now.row * p.num_tiles + now.tile;
    TilePartial tp;
    unsigned char* chunks = p.chunk_max + now.row * p.chunk_pitch + static_cast<int64_t>(now.tile) * p.tile_chunks * EB;
    bool done = false;
    // A 16-bit type's tile of up to 4096 columns in registers; any other in its stage, twice.  (Float32 has no
    // register form: half of its default tile would fit, and the code of both slowed either.)
    if constexpr (EB == 2) {
      if (p.tile_v <= TileRegs<DT>::kMaxTile) {
        const bool whole = valid == TileRegs<DT>::kMaxTile;
        TileRegs<DT> regs;
        if (ALIGNED)
          tile_load_regs<DT>(stage, valid, lane, regs);
        else
          load_regs_at<DT>(stage, off, valid, lane, regs);
        __syncwarp();  // the stage has been read
        issue();
        const float mx_all = warp_max(whole ? regs_max<DT, true>(regs, valid, lane, chunks, p.tile_chunks)
                                            : regs_max<DT, false>(regs, valid, lane, chunks, p.tile_chunks));
        tp = whole ? regs_sums<DT, true, ENT>(regs, valid, lane, mx_all, p.rcp)
                   : regs_sums<DT, false, ENT>(regs, valid, lane, mx_all, p.rcp);
        if (ENT && tp.u != tp.u) tp.u = clamped_entropy<DT, ALIGNED>(src, valid, lane, mx_all, p.rcp, regs);
        done = true;
      }
    }
    if (!done) {
      const float mx_all = warp_max(smem_max<DT, ALIGNED>(stage, valid, lane, off, chunks, p.tile_chunks));
      tp = smem_sums<DT, ENT, ALIGNED>(stage, valid, lane, mx_all, p.rcp, off);
      __syncwarp();
      issue();
    }
    if (now.tile == p.num_tiles - 1) {  // the rest of the row's last 16 bytes
      const int pad = p.num_tiles * p.tile_chunks + lane;
      if (pad < p.chunk_pitch / EB) store_value<DT>(p.chunk_max + now.row * p.chunk_pitch, pad, -INFINITY);
    }
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

// A row is taken by one warp where there are many rows (their latencies hide
// behind each other: 32 rows at a time on an SM), or by five where there are
// few (four choose the columns, one merges the partials).  SW: the warps that
// choose.
constexpr int kFewRowWarps = 4;
constexpr int kCandidates = 512;     // entries the selection holds
constexpr int kDigitBits = 10;       // of a pass of the radix selection
constexpr int kBins = 1 << kDigitBits;
constexpr int kStep = 4;             // 16-byte units of chunk maxima a lane looks at together
constexpr int kQueue = 320;          // chunks a warp holds between two rounds of reading
constexpr int kInFlight = 4;         // chunks eight lanes read at a time

template <int SW>
struct alignas(16) SelShared {
  union {
    u64 cand[kCandidates];
    uint32_t bins[kBins];
  };
  uint32_t group_max[SW == 1 ? 4 : 8 * kLanes];
  int queue[SW][kQueue];
  u64 merged[BIL_MAX_TOPK];
  float scratch[kMergeScratch];
  int count;
  uint32_t bound;
  int above;
  float lse;
};
static_assert(sizeof(uint32_t) * kBins <= sizeof(u64) * kCandidates, "the bins share the candidates' space");

// The warps that choose a row's columns wait for each other.
template <int SW>
__device__ __forceinline__ void sel_sync() {
  if constexpr (SW == 1)
    __syncwarp();
  else
    asm volatile("bar.sync 1, %0;" ::"n"(SW * kLanes) : "memory");
}

// The columns of one row by way of its chunks.
template <int DT, int SW>
struct RowColumns {
  static constexpr int EB = Elem<DT>::kBytes;
  const unsigned char* row;    // column 0
  const unsigned char* chunks; // the row's chunk maxima
  int units;                   // 16-byte units of them
  int vocab, tile_v, tile_chunks, num_tiles;
  int warp, lane;
  int* queue;

  static constexpr int kUnit = 16 / EB;  // maxima of a unit
  __device__ __forceinline__ uint4 unit(int u) const { return reinterpret_cast<const uint4*>(chunks)[u]; }
  // running maxima of the units a lane looks at: each of a unit's 8 (16-bit) in its own, or its 4
  // (float32) in the set `half`
  struct Maxima {
    uint32_t r[8];
    __device__ __forceinline__ void clear() {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = ChunkMax<DT>::kNone;
    }
    __device__ __forceinline__ void add(uint4 w, int half) {
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = EB == 4 ? 4 * half + j : j;
        r[at] = ChunkMax<DT>::max_of(r[at], x[j]);
      }
    }
    __device__ __forceinline__ void get(float (&m)[8]) const {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (EB == 4) {
          m[j] = __uint_as_float(r[j]);
        } else {
          float lo, hi;
          Elem<DT>::pair(r[j / 2], lo, hi);
          m[j] = j % 2 == 0 ? lo : hi;
        }
      }
    }
  };
  // A bound to compare stored words with (the smallest value of the type that is `least` or more), which of
  // a word's values reach it, and value `bit` of the words: one bit a value, a 16-bit type's upper halves
  // from bit 16 on.
  __device__ static __forceinline__ uint32_t bound_word(float least) {
    if constexpr (DT == BIL_F32) {
      return __float_as_uint(least);
    } else if constexpr (DT == BIL_BF16) {
      return __bfloat16_as_ushort(__float2bfloat16_ru(least)) * 0x10001u;
    } else {
      return __half_as_ushort(__float2half_ru(least)) * 0x10001u;
    }
  }
  template <int N>
  __device__ static __forceinline__ unsigned reach(const uint32_t (&w)[N], uint32_t bound) {
    unsigned t = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if constexpr (DT == BIL_F32)
        t |= __uint_as_float(w[j]) >= __uint_as_float(bound) ? 1u << j : 0u;
      else if constexpr (DT == BIL_BF16)
        t |= __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w[j]), *reinterpret_cast<const __nv_bfloat162*>(&bound)) &
             (0x10001u << j);
      else
        t |= __hge2_mask(*reinterpret_cast<const __half2*>(&w[j]), *reinterpret_cast<const __half2*>(&bound)) &
             (0x10001u << j);
    }
    return t;
  }
  __device__ static __forceinline__ int place(int bit) { return EB == 4 ? bit : 2 * (bit % 16) + bit / 16; }

  // whether a chunk of the tile reaches a key (every lane)
  __device__ __forceinline__ bool tile_reaches(int tile, uint32_t least) const {
    bool in = false;
    for (int c = lane; c < tile_chunks; c += kLanes)
      in |= order_key(Elem<DT>::one(chunks + (static_cast<int64_t>(tile) * tile_chunks + c) * EB)) >= least;
    return __any_sync(0xffffffffu, in) != 0;
  }
  static constexpr int kW = Group<DT>::kW;

  // the words of the `n` columns from column c0 (n <= 8)
  __device__ __forceinline__ void load8(int c0, int n, uint32_t (&w)[kW]) const {
    const unsigned char* p = row + static_cast<int64_t>(c0) * EB;
    if (n == kGroup && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
      Group<DT>::load(p, w);
    } else {
#pragma unroll
      for (int j = 0; j < kW; ++j) w[j] = 0;
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        if (j >= n) continue;
        if constexpr (EB == 4)
          w[j] = reinterpret_cast<const uint32_t*>(p)[j];
        else
          w[j / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[j]) << (16 * (j & 1));
      }
    }
  }
  // fn(value, column) for the columns that reach `bound` of the queue's first n
  // chunks: eight lanes a chunk, a lane a group of 8 columns, kInFlight chunks
  // at a time.
  template <typename F>
  __device__ __forceinline__ void read_queue(int n, uint32_t bound, F fn) const {
    const bool even = tile_v % kChunk == 0;  // chunks lie one after the other
    __syncwarp();
    for (int i = lane / 8; i < n; i += 4 * kInFlight) {
      uint32_t w[kInFlight][kW];
      int first[kInFlight], left[kInFlight];
#pragma unroll
      for (int q = 0; q < kInFlight; ++q) {
        left[q] = 0;
        if (i + 4 * q < n) {
          const int c = queue[i + 4 * q];
          if (even) {
            first[q] = c * kChunk + (lane % 8) * kGroup;
            left[q] = min(kGroup, vocab - first[q]);
          } else {
            const int tile = c / tile_chunks;
            const int e = (c - tile * tile_chunks) * kChunk + (lane % 8) * kGroup;
            first[q] = tile * tile_v + e;
            left[q] = min(kGroup, min(tile_v, vocab - tile * tile_v) - e);
          }
          if (left[q] > 0) load8(first[q], left[q], w[q]);
        }
      }
#pragma unroll
      for (int q = 0; q < kInFlight; ++q) {
        if (left[q] <= 0) continue;
        unsigned take = reach(w[q], bound);
        while (take != 0u) {
          const int bit = __ffs(take) - 1;
          take &= take - 1;
          const int j = place(bit);
          if (j >= left[q]) continue;
          const float x = Elem<DT>::one(row + (static_cast<int64_t>(first[q]) + j) * EB);  // a line just read
          fn(x, first[q] + j);
        }
      }
    }
    __syncwarp();
  }
  // fn(value, column) for every column that is `least` (above -inf) or more; the
  // row's warps share the chunks whose maximum is.
  template <typename F>
  __device__ __forceinline__ void visit(float least, F fn) const {
    const uint32_t bound = bound_word(least);
    int n = 0;
#pragma unroll 1
    for (int u0 = warp * kLanes; u0 < units; u0 += kStep * SW * kLanes) {
      uint4 w[kStep];
#pragma unroll
      for (int q = 0; q < kStep; ++q) {
        const int u = u0 + q * SW * kLanes + lane;
        w[q] = u < units ? unit(u) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll 1
      for (int q = 0; q < kStep; ++q) {
        const int u = u0 + q * SW * kLanes + lane;
        const uint4 now = q == 0 ? w[0] : q == 1 ? w[1] : q == 2 ? w[2] : w[3];
        const uint32_t x[4] = {now.x, now.y, now.z, now.w};
        unsigned take = u < units ? reach(x, bound) : 0u;
        for (;;) {
          const unsigned vote = __ballot_sync(0xffffffffu, take != 0u);
          if (vote == 0u) break;
          if (take != 0u) {
            queue[n + __popc(vote & ((1u << lane) - 1u))] = u * kUnit + place(__ffs(take) - 1);
            take &= take - 1;
          }
          n += __popc(vote);
        }
        const bool last = q == kStep - 1 && u0 + kStep * SW * kLanes >= units;
        if (n > kQueue - kUnit * kLanes || (last && n != 0)) {
          read_queue(n, bound, fn);
          n = 0;
        }
      }
    }
  }
};
static_assert(kStep == 4, "visit picks among four units");

// The row's k best columns, best first, into sm.merged (the row's SW warps).
template <int DT, int SW>
__device__ __forceinline__ void select_columns(const RowColumns<DT, SW>& cols, int k, SelShared<SW>& sm) {
  const int tid = cols.warp * kLanes + cols.lane;
  // 1. the maxima of 128 groups of chunks (k > 32: 256): which chunks make a group does not matter
  constexpr int kSets = 8 / SW;  // groups of a thread
  uint32_t key[8];
  {
    typename RowColumns<DT, SW>::Maxima maxima;
    maxima.clear();
#pragma unroll 1
    for (int u0 = tid; u0 < cols.units; u0 += 6 * SW * kLanes) {
      uint4 w[6];
#pragma unroll
      for (int q = 0; q < 6; ++q)
        if (u0 + q * SW * kLanes < cols.units) w[q] = cols.unit(u0 + q * SW * kLanes);
#pragma unroll
      for (int q = 0; q < 6; ++q)
        if (u0 + q * SW * kLanes < cols.units) maxima.add(w[q], q & 1);
    }
    float m[8];
    maxima.get(m);
#pragma unroll
    for (int q = kSets; q < 8; ++q) m[q % kSets] = fmaxf(m[q % kSets], m[q]);
    if (k <= kLanes) {
#pragma unroll
      for (int q = 0; q < kSets / 2; ++q) {
        m[q] = fmaxf(m[q], m[q + kSets / 2]);
        m[q + kSets / 2] = -INFINITY;
      }
    }
#pragma unroll
    for (int q = 0; q < kSets; ++q) {
      if constexpr (SW == 1)
        key[q] = order_key(m[q]);
      else
        sm.group_max[q * SW * kLanes + tid] = order_key(m[q]);
    }
    if (tid == 0) sm.count = 0;
  }
  sel_sync<SW>();
  // 2. the k-th largest of them, to the upper 16 bits of its key (all of a bfloat16): it has k columns at or
  // above it
  if (cols.warp == 0) {
    if constexpr (SW != 1) {
#pragma unroll
      for (int q = 0; q < 8; ++q) key[q] = sm.group_max[q * kLanes + cols.lane];
    }
    uint32_t bound = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 16; --bit) {
      const uint32_t up = bound | (1u << bit);
      int above = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) above += __popc(__ballot_sync(0xffffffffu, key[q] >= up));
      if (k > kLanes) {
#pragma unroll
        for (int q = 4; q < 8; ++q) above += __popc(__ballot_sync(0xffffffffu, key[q] >= up));
      }
      if (above >= k) bound = up;
      if (above == k) break;  // no tighter bound is needed
    }
    if (cols.lane == 0) sm.bound = bound;
  }
  sel_sync<SW>();
  // 3. The columns of that key or more, if there are no more of them than fit.  Else (many equal or
  // crowded columns), and where the bound is -inf, which says nothing (a chunk of NaN says -inf too): those
  // above it; if there are too many of these, a radix selection over their keys first, from the top digit.
  enum { kReach, kAbove, kDigits, kLast } step = kReach;
  uint32_t least = sm.bound;
  uint32_t prefix = 0;        // of the k-th key, `fixed` bits known; `taken` columns are above its range
  int fixed = 0, bits = 0, shift = 0, taken = 0, found = 0;
  if (least <= kKeyNegInf) {
    least = kKeyNegInf + 1;
    step = kAbove;
  }
#pragma unroll 1
  for (;;) {
    cols.visit(key_value(least), [&](float x, int c) {
      const uint32_t key = order_key(x);
      if (step == kDigits) {
        if (fixed == 0 || (key >> (32 - fixed)) == (prefix >> (32 - fixed)))
          atomicAdd(&sm.bins[(key >> shift) & ((1u << bits) - 1u)], 1u);
      } else {
        const int at = atomicAdd(&sm.count, 1);
        if (at < kCandidates) sm.cand[at] = entry_of(key, c);
      }
    });
    sel_sync<SW>();
    if (step != kDigits) {
      found = sm.count;
      sel_sync<SW>();  // every thread has read the count before any may change it
      if (found <= kCandidates || step == kLast) break;
      if (step == kReach) {
        ++least;
        step = kAbove;
      } else {
        step = kDigits;
      }
    } else {
      if (cols.warp == 0) {
        // from the highest bin down: the bin that holds the k-th column
        int sum = taken, digit = -1, before = 0, upto_digit = 0;
        for (int b0 = max((1 << bits) - kLanes, 0); b0 >= 0 && digit < 0; b0 -= kLanes) {
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
            upto_digit = sum + __shfl_sync(0xffffffffu, upto, src);
          }
          sum += __shfl_sync(0xffffffffu, upto, kLanes - 1);
        }
        if (cols.lane == 0) {
          sm.bound = prefix | (static_cast<uint32_t>(max(digit, 0)) << shift);
          sm.above = before;
          sm.count = upto_digit;
        }
      }
      sel_sync<SW>();
      prefix = sm.bound;
      taken = sm.above;
      found = sm.count;  // columns of `prefix` or more
      sel_sync<SW>();
      fixed += bits;
      least = max(least, prefix);
      if (found <= kCandidates || fixed == 32) {
        // too many even so (equal columns): those above it, fewer than k, and the rest is found below
        if (found > kCandidates) least = prefix + 1;
        step = kLast;
      }
    }
    if (step == kDigits) {
      bits = min(kDigitBits, 32 - fixed);
      shift = 32 - fixed - bits;
      for (int i = tid; i < kBins; i += SW * kLanes) sm.bins[i] = 0;
    } else if (tid == 0) {
      sm.count = 0;
    }
    sel_sync<SW>();
  }
  if (found < k) {
    // Equal columns just below `least`, then NaN, in column order: one warp, tile by tile.
    if (cols.warp == 0) {
      uint32_t want = least - 1;
      for (;;) {
        for (int tile = 0; tile < cols.num_tiles && found < k; ++tile) {
          if (!cols.tile_reaches(tile, max(want, kKeyNegInf))) continue;
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
    }
    found = k;
  }
  // 4. in order: an entry's place is the number of entries above it
  const int n = found;
  if (tid == 0 && n < kCandidates) sm.cand[n] = 0;  // the pair of the last one
  sel_sync<SW>();
  for (int i = tid; i < n; i += SW * kLanes) {
    const u64 mine = sm.cand[i];
    int above = 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 2) {
      const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&sm.cand[j]);
      above += (o.x > mine ? 1 : 0) + (o.y > mine ? 1 : 0);
    }
    if (above < k) sm.merged[above] = mine;
  }
}

struct TopkOut {
  float* logp;
  float* lse;
  float* entropy;
  int64_t* top_ids;
  float* top_logp;
};

// A row's results from its chunk maxima and partials (in global or in shared
// memory): one warp, or SW + 1 of a block.
template <int DT, bool ENT, int SW>
__device__ __forceinline__ void finish_row(const TopkParams& p, const TopkOut& out, int64_t row, int64_t t,
                                           const unsigned char* chunks, const float* part_max, const float* part_sum,
                                           const float* part_ent, SelShared<SW>& sm, int warp, int lane) {
  int64_t* ids = out.top_ids + row * p.k;
  float* top = out.top_logp + row * p.k;
  const int tid = SW == 1 ? lane : static_cast<int>(threadIdx.x);
  constexpr int kThreads = SW == 1 ? kLanes : (SW + 1) * kLanes;
  if (t == p.ignore_index) {
    for (int j = tid; j < p.k; j += kThreads) {
      ids[j] = -1;
      top[j] = 0.0f;
    }
    if (tid == 0) {
      out.logp[row] = 0.0f;
      if (out.lse != nullptr) out.lse[row] = 0.0f;
      if (ENT) out.entropy[row] = 0.0f;
    }
    return;
  }
  const unsigned char* src = p.logits + row * p.ld * Elem<DT>::kBytes;
  if (SW == 1 || warp != SW) {
    RowColumns<DT, SW> cols;
    cols.row = src;
    cols.num_tiles = p.num_tiles;
    cols.chunks = chunks;
    cols.units = static_cast<int>(p.chunk_pitch / 16);
    cols.vocab = static_cast<int>(p.vocab);
    cols.tile_v = p.tile_v;
    cols.tile_chunks = p.tile_chunks;
    cols.warp = SW == 1 ? 0 : warp;
    cols.lane = lane;
    cols.queue = sm.queue[SW == 1 ? 0 : warp];
    select_columns<DT, SW>(cols, p.k, sm);
  }
  if (SW == 1 || warp == SW) {
    float H = 0.0f;
    const float L = merge_lse<ENT, true>(part_max, part_sum, part_ent, p.num_tiles, lane, &H, sm.scratch);
    if (lane == 0) {
      sm.lse = L;
      float z = __int_as_float(0x7fc00000);
      if (t >= 0 && t < p.vocab) {
        z = Elem<DT>::one(src + t * Elem<DT>::kBytes);
        if (p.rcp != 1.0f) z = __fmul_rn(z, p.rcp);
      }
      out.logp[row] = __fsub_rn(z, L);
      if (out.lse != nullptr) out.lse[row] = L;
      if (ENT) out.entropy[row] = H;
    }
  }
  if constexpr (SW == 1)
    __syncwarp();
  else
    __syncthreads();
  for (int j = tid; j < p.k; j += kThreads) {
    const u64 e = sm.merged[j];
    float z = key_value(static_cast<uint32_t>(e >> 32));
    if (p.rcp != 1.0f) z = __fmul_rn(z, p.rcp);
    ids[j] = entry_column(e);
    top[j] = __fsub_rn(z, sm.lse);
  }
}


template <int DT, bool ENT, int SW>
__global__ void __launch_bounds__(SW == 1 ? 4 * kLanes : (SW + 1) * kLanes, SW == 1 ? 6 : 4)
    topk_row_kernel(const TopkParams p, const TopkOut out) {
  constexpr int kRows = SW == 1 ? 4 : 1;  // rows of a block
  __shared__ SelShared<SW> shared[kRows];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % kLanes, warp = threadIdx.x / kLanes;
  const int64_t row = SW == 1 ? static_cast<int64_t>(blockIdx.x) * kRows + warp : blockIdx.x;
  if (row >= p.n_rows) return;  // a warp of its own: no barrier follows
  const int64_t o = row * p.num_tiles;
  finish_row<DT, ENT, SW>(p, out, row, p.targets[row], p.chunk_max + row * p.chunk_pitch, p.part_max + o,
                          p.part_sum + o, ENT ? p.part_ent + o : nullptr, shared[SW == 1 ? warp : 0], warp, lane);
}

// ---------------------------------------------------------------------------
// Few rows of a 16-bit type: one kernel and no workspace.  A row is shared by a
// cluster of eight blocks, as in the small-batch forward: each warp reduces its
// tiles from global memory with the functions of the pass above, chunk maxima and
// partials go to the first block over distributed shared memory, and after the
// cluster's barrier that block ends the row.
// ---------------------------------------------------------------------------

constexpr int kClusterTiles = 256;            // most tiles of a row
constexpr size_t kClusterChunks = 24 * 1024;  // most bytes of a row's chunk maxima

// The address of `p` (a shared variable of this block) in the block of rank `rank`.
template <typename T>
__device__ __forceinline__ T* cluster_ptr(T* p, uint32_t rank) {
  uint64_t r;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
  return reinterpret_cast<T*>(r);
}

template <int DT, bool ALIGNED, bool ENT>
__global__ void __launch_bounds__((kFewRowWarps + 1) * kLanes, 3)
    topk_cluster_kernel(const TopkParams p, const TopkOut out) {
  extern __shared__ __align__(128) unsigned char smem_raw[];  // the row's chunk maxima (the first block's)
  __shared__ SelShared<kFewRowWarps> sm;
  __shared__ float part[3][kClusterTiles];
  constexpr int EB = Elem<DT>::kBytes;
  constexpr int kWarps = kFewRowWarps + 1;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % kLanes, warp = threadIdx.x / kLanes;
  const int rank = static_cast<int>(cluster_ctarank());
  const int64_t row = static_cast<int64_t>(blockIdx.x) / kSplitCtas;
  const int64_t t = p.targets[row];
  // the first block has to have started before the others write into it; the first tiles are loaded meanwhile
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  TileRegs<DT> regs;
  const unsigned char* src;
  int valid;
  unsigned off;
  const auto load = [&](int tile) {
    src = p.logits + (row * p.ld + static_cast<int64_t>(tile) * p.tile_v) * EB;
    valid = static_cast<int>(min(static_cast<int64_t>(p.tile_v), p.vocab - static_cast<int64_t>(tile) * p.tile_v));
    off = ALIGNED ? 0u : static_cast<unsigned>(reinterpret_cast<uintptr_t>(src) & 15u);
    if (ALIGNED)
      tile_load_regs<DT>(src, valid, lane, regs);
    else
      load_regs_shifted<DT>(src - off, off, valid, lane, regs);
  };
  int tile = t != p.ignore_index ? warp * kSplitCtas + rank : p.num_tiles;
  if (tile < p.num_tiles) load(tile);
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  unsigned char* chunks = cluster_ptr(smem_raw, 0);
  while (tile < p.num_tiles) {
    const bool whole = valid == TileRegs<DT>::kMaxTile;
    unsigned char* at = chunks + static_cast<int64_t>(tile) * p.tile_chunks * EB;
    const float mx_all = warp_max(whole ? regs_max<DT, true>(regs, valid, lane, at, p.tile_chunks)
                                        : regs_max<DT, false>(regs, valid, lane, at, p.tile_chunks));
    TilePartial tp = whole ? regs_sums<DT, true, ENT>(regs, valid, lane, mx_all, p.rcp)
                           : regs_sums<DT, false, ENT>(regs, valid, lane, mx_all, p.rcp);
    if (ENT && tp.u != tp.u) tp.u = clamped_entropy<DT, ALIGNED>(src, valid, lane, mx_all, p.rcp, regs);
    if (lane == 0) {
      *cluster_ptr(&part[0][tile], 0) = tp.m;
      *cluster_ptr(&part[1][tile], 0) = tp.s;
      if (ENT) *cluster_ptr(&part[2][tile], 0) = tp.u;
    }
    if (tile == p.num_tiles - 1) {  // the rest of the row's last 16 bytes
      const int pad = p.num_tiles * p.tile_chunks + lane;
      if (pad < p.chunk_pitch / EB) store_value<DT>(chunks, pad, -INFINITY);
    }
    tile += kSplitCtas * kWarps;
    if (tile < p.num_tiles) load(tile);
  }
  cluster_sync_all();
  if (rank != 0) return;
  finish_row<DT, ENT, kFewRowWarps>(p, out, row, t, smem_raw, part[0], part[1], part[2], sm, warp, lane);
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
  size_t pitch, chunks, part, total;  // bytes: a row of chunk maxima, all rows, one partial array, everything
};

TopkWorkspace topk_workspace(int dtype, int64_t n_rows, int64_t num_tiles, int tile_v, bool ent) {
  TopkWorkspace w;
  w.tile_chunks = (tile_v + kChunk - 1) / kChunk;
  w.pitch = static_cast<size_t>(align_up(static_cast<size_t>(num_tiles) * w.tile_chunks * bil_internal::elem_bytes(dtype), 16));
  w.chunks = round256(static_cast<size_t>(n_rows) * w.pitch);
  w.part = round256(static_cast<size_t>(n_rows) * num_tiles * sizeof(float));
  w.total = w.chunks + w.part * (ent ? 3 : 2);
  return w;
}

// Whether the forward takes the cluster kernel (and no workspace): rows of a
// 16-bit type with a tile or more for every block of a cluster, and all their
// blocks on the device at a time.  151936 columns of bfloat16, k = 20, in a CUDA
// graph: 1 row 7.1 us (the two kernels 8.1), 32 rows 8.7 (9.9), 48 rows 9.7 (10.8),
// 64 rows 13.0 (12.2), 128 rows 18.5 (15.8); rows off 16-byte boundaries 7.0 to 11.9
// (8.2 to 12.9) up to 48.  A call from Python: 20 us (27).
#ifndef BIL_TOPK_CLUSTER_ROWS
#define BIL_TOPK_CLUSTER_ROWS 48
#endif
bool use_cluster(int dtype, int64_t n_rows, int64_t num_tiles, int tile_v, const TopkWorkspace& w) {
  return dtype != BIL_F32 && n_rows <= BIL_TOPK_CLUSTER_ROWS && num_tiles >= kSplitCtas && num_tiles <= kClusterTiles &&
         tile_v <= 4096 && w.pitch <= kClusterChunks;
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
int launch_topk_t(TopkParams p, const TopkOut& out, cudaStream_t stream) {
  if (p.chunk_max == nullptr) {  // no workspace: few rows
    if constexpr (Elem<DT>::kBytes == 2) {
      return launch_pdl(topk_cluster_kernel<DT, ALIGNED, ENT>, p.n_rows * kSplitCtas, (kFewRowWarps + 1) * kLanes,
                        static_cast<size_t>(p.chunk_pitch), stream, kSplitCtas, p, out) == cudaSuccess
                 ? BIL_OK
                 : BIL_E_CUDA;
    }
    return BIL_E_INVALID_ARG;
  }
  int sms = 0, smem_optin = 0;
  if (int st = bil_internal::device_limits(&sms, &smem_optin)) return st;
  p.stage_bytes =
      static_cast<unsigned>(align_up(static_cast<size_t>(p.tile_v) * Elem<DT>::kBytes + (ALIGNED ? 0 : 16), 128));
  const size_t limit = bil_layout::dynamic_limit(smem_optin);
  int warps = 0, blocks = 0;
  bil_layout::topk_stream(p.stage_bytes, limit, &warps, &blocks);
  if (warps < 1) return BIL_E_UNSUPPORTED;
  const int64_t slots = static_cast<int64_t>(sms) * blocks;
  p.unit_tiles = unit_tiles(p.n_rows, p.num_tiles, slots * warps);
  p.units = (p.num_tiles + p.unit_tiles - 1) / p.unit_tiles;
  const int64_t units = p.n_rows * p.units;
  // few units: one warp a block, so that they spread over the SMs
  warps = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(warps, (units + slots - 1) / slots)));
  const int64_t grid = std::min<int64_t>(slots, (units + warps - 1) / warps);
  const size_t smem = static_cast<size_t>(warps) * p.stage_bytes;
  auto kernel = topk_stream_kernel<DT, ALIGNED, ENT>;
  // past what needs no opt-in (48 KB with the kernel's own variables)
  if (smem > 47 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(limit)) != cudaSuccess)
    return BIL_E_CUDA;
  if (launch_pdl(kernel, grid, warps * kLanes, smem, stream, 1, p) != cudaSuccess) return BIL_E_CUDA;
  // One warp a row from four rows an SM on.
  const cudaError_t e =
      p.n_rows >= 4 * static_cast<int64_t>(sms)
          ? launch_pdl(topk_row_kernel<DT, ENT, 1>, (p.n_rows + 3) / 4, 4 * kLanes, 0, stream, 1, p, out)
          : launch_pdl(topk_row_kernel<DT, ENT, kFewRowWarps>, p.n_rows, (kFewRowWarps + 1) * kLanes, 0, stream, 1, p,
                       out);
  return e == cudaSuccess ? BIL_OK : BIL_E_CUDA;
}

template <int DT>
int launch_topk(const TopkParams& p, bool ent, const TopkOut& out, cudaStream_t stream) {
  const bool vec = aligned_to(p.logits, 16) && (p.n_rows <= 1 || (p.ld * Elem<DT>::kBytes) % 16 == 0);
  if (vec)
    return ent ? launch_topk_t<DT, true, true>(p, out, stream)
               : launch_topk_t<DT, true, false>(p, out, stream);
  return ent ? launch_topk_t<DT, false, true>(p, out, stream)
             : launch_topk_t<DT, false, false>(p, out, stream);
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
  const TopkWorkspace w = topk_workspace(dtype, n_rows, num_tiles, tile_v, entropy != 0);
  *bytes = use_cluster(dtype, n_rows, num_tiles, tile_v, w) ? 0 : static_cast<int64_t>(w.total);
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
  const bool ent = entropy != nullptr;
  const TopkWorkspace w = topk_workspace(dtype, n_rows, num_tiles, tile_v, ent);
  const bool cluster = use_cluster(dtype, n_rows, num_tiles, tile_v, w);
  if (logits == nullptr || target_ids == nullptr || logp == nullptr || top_ids == nullptr || top_logp == nullptr ||
      (!cluster && workspace == nullptr))
    return BIL_E_INVALID_ARG;
  if (!aligned_to(logits, static_cast<size_t>(eb)) || !aligned_to(target_ids, 8) || !aligned_to(logp, 4) ||
      (lse && !aligned_to(lse, 4)) || (entropy && !aligned_to(entropy, 4)) || !aligned_to(top_ids, 8) ||
      !aligned_to(top_logp, 4) || (!cluster && !aligned_to(workspace, 256)))
    return BIL_E_ALIGN;
  if (!cluster && workspace_bytes < static_cast<int64_t>(w.total)) return BIL_E_INVALID_ARG;
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
  p.chunk_pitch = static_cast<int64_t>(w.pitch);
  p.targets = target_ids;
  p.ignore_index = ignore_index;
  p.rcp = rcp;
  p.k = k;
  if (!cluster) {
    p.chunk_max = ws;
    p.part_max = reinterpret_cast<float*>(ws + w.chunks);
    p.part_sum = reinterpret_cast<float*>(ws + w.chunks + w.part);
    p.part_ent = ent ? reinterpret_cast<float*>(ws + w.chunks + 2 * w.part) : nullptr;
  }
  const TopkOut out{logp, lse, entropy, top_ids, top_logp};
  switch (dtype) {
    case BIL_BF16: return launch_topk<BIL_BF16>(p, ent, out, s);
    case BIL_F16: return launch_topk<BIL_F16>(p, ent, out, s);
    default: return launch_topk<BIL_F32>(p, ent, out, s);
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
  if (dlogits == logits) return BIL_E_INVALID_ARG;  // the named columns' logits are read after the full pass
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
