// Embedding lookup with a scale, and the table's gradient by sorted tokens.  The C
// ABI is declared in include/bil.h.
//
//     y_i = round_T(scale * weight[id_i])
//     dweight[v] = round(scale * sum of dy_i over the i with id_i = v, in order of i)
//
// The gradient without atomics on floating-point numbers: the tokens' places are
// sorted by token (radix, stable, so a token's places stay in order), cut into
// segments of a fixed number of places, and each segment's sums are taken in order
// in float32 registers.  A token whose places lie in one segment is done with that;
// the sums of one that lies in several are parts which a second kernel adds up in
// order.  What a row's bits depend on is thus the tokens and their order alone, not
// the launch.  Tokens outside the table, and the padding token, sort behind the
// last row and are left out.

#include "launch.cuh"
#include "rows_device.cuh"

#include <algorithm>
#include <cmath>

namespace {

// ---------------------------------------------------------------------------
// Lookup.
// ---------------------------------------------------------------------------

constexpr int kLookupThreads = 128;

struct LookupParams {
  const int64_t* ids;
  const unsigned char* weight;
  unsigned char* out;
  int64_t n, vocab, ld_w, ld_out;
  int width, groups, row_threads, vec_out;
  float scale;
};

template <int DT, bool FULL>
__global__ void __launch_bounds__(kLookupThreads) embedding_lookup_kernel(const LookupParams p) {
  using R = Row<DT>;
  constexpr int kAhead = DT == BIL_F32 ? 2 : 4;
  griddep_wait();
  griddep_launch_dependents();
  const int per_block = kLookupThreads / p.row_threads;
  const int lane = static_cast<int>(threadIdx.x) & (p.row_threads - 1);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / p.row_threads; row < p.n;
       row += static_cast<int64_t>(gridDim.x) * per_block) {
    const int64_t id = p.ids[row];
    const bool ok = id >= 0 && id < p.vocab;
    const RowStart from(p.weight + (ok ? id : 0) * p.ld_w * R::EB);
    unsigned char* out = p.out + row * p.ld_out * R::EB;
    for (int g0 = lane; g0 < p.groups; g0 += kAhead * p.row_threads) {
      uint32_t w[kAhead][R::kW];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int g = g0 + i * p.row_threads;
        if (g < p.groups && ok) R::template load_path<FULL ? kFullRows : kAnyRows>(from.base, from.off, g, p.width, w[i]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int g = g0 + i * p.row_threads;
        if (g >= p.groups) continue;
        float v[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = ok ? __fmul_rn(R::get(w[i], j), p.scale) : __int_as_float(0x7fc00000);
        uint32_t o[R::kW];
        R::pack(v, o);
        R::template store_path<FULL ? kFullRows : kAnyRows>(out, g, p.width, p.vec_out != 0, o);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Sorting the places by token: least significant digit first.  A kernel counts the
// first digit in every tile; then one a digit moves each tile's places to where they
// belong and counts the next digit there (whole numbers: in any order).  A few
// blocks of small latency each; of the table's zeros, most of what the gradient
// writes, further blocks of the same launches store a part meanwhile.
// ---------------------------------------------------------------------------

constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / kLanes;
constexpr int kFewPer = 4, kManyPer = 16;               // places a thread (see sort_per)
constexpr int kDigitBits = 9;                           // 151936 tokens and the one behind them: two digits
constexpr int kDigits = 1 << kDigitBits;
static_assert(kDigits == 2 * kSortThreads, "a thread has two digits");

// Rows [begin, end) of the table's gradient to set to zero: row_bytes of each, ld bytes apart.
struct Zeros {
  unsigned char* to;
  int64_t ld, begin, end, row_bytes;
};

// Row `row`, by threads `thread` of `threads`: 16 bytes at a time where it starts on a boundary of them, and a rest.
__device__ __forceinline__ void store_zero_row(const Zeros& z, int64_t row, int thread, int threads) {
  unsigned char* to = z.to + row * z.ld;
  int64_t done = 0;
  if ((reinterpret_cast<uintptr_t>(to) & 15u) == 0) {
    done = z.row_bytes & ~static_cast<int64_t>(15);
    for (int64_t i = thread; i < done / 16; i += threads) reinterpret_cast<uint4*>(to)[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  for (int64_t i = done / 2 + thread; i < z.row_bytes / 2; i += threads) reinterpret_cast<uint16_t*>(to)[i] = 0;
}

struct SortParams {
  const int64_t* ids;     // of the first digit: the tokens themselves
  int64_t vocab, padding;
  const uint32_t* keys;   // of the others: the tokens and places so far
  const uint32_t* places;
  uint32_t* keys_out;
  uint32_t* places_out;
  uint32_t* counts;       // [tiles, kDigits] of this digit
  uint32_t* next_counts;  // of the next one, added to; NULL: this is the last
  uint32_t* zero_counts;  // what the next launch adds to, set to zero here; NULL: nothing
  int n, tiles, shift;
  Zeros zeros;            // by the blocks from `tiles` on
};

// All of the rows, by threads `thread` of `threads`.  Rows one after the other are one long row.
__device__ __forceinline__ void store_zeros(const Zeros& z, int64_t thread, int64_t threads) {
  if (z.ld == z.row_bytes && z.row_bytes % 16 == 0 && (reinterpret_cast<uintptr_t>(z.to) & 15u) == 0) {
    uint4* to = reinterpret_cast<uint4*>(z.to + z.begin * z.ld);
    const int64_t units = (z.end - z.begin) * (z.row_bytes / 16);
    for (int64_t i = thread; i < units; i += threads) to[i] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  for (int64_t row = z.begin + thread / kLanes; row < z.end; row += threads / kLanes)
    store_zero_row(z, row, static_cast<int>(thread % kLanes), kLanes);
}

template <bool FIRST>
__device__ __forceinline__ uint32_t sort_key(const SortParams& p, int i) {
  if (!FIRST) return p.keys[i];
  const int64_t id = p.ids[i];
  return static_cast<uint32_t>(id >= 0 && id < p.vocab && id != p.padding ? id : p.vocab);
}

template <int PER>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortParams p) {
  __shared__ uint32_t counts[kDigits];
  for (int d = threadIdx.x; d < kDigits; d += kSortThreads) counts[d] = 0;
  griddep_wait();
  griddep_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= p.tiles) {
    store_zeros(p.zeros, static_cast<int64_t>(blockIdx.x - p.tiles) * kSortThreads + threadIdx.x,
                static_cast<int64_t>(gridDim.x - p.tiles) * kSortThreads);
    return;
  }
  __syncthreads();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kSortThreads * PER);
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int64_t i = first + j * kSortThreads + threadIdx.x;
    if (i < p.n) atomicAdd(&counts[sort_key<true>(p, static_cast<int>(i)) & (kDigits - 1)], 1u);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < kDigits; d += kSortThreads) {
    p.counts[static_cast<int64_t>(blockIdx.x) * kDigits + d] = counts[d];
    if (p.zero_counts != nullptr) p.zero_counts[static_cast<int64_t>(blockIdx.x) * kDigits + d] = 0u;
  }
}

// A warp takes its 32 PER places in order, 32 at a time; those with one digit rank by
// lane.  Where a digit's places of this tile begin: the counts of the smaller digits
// in every tile, and of this one in the tiles before.
template <bool FIRST, int PER>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const SortParams p) {
  __shared__ uint32_t of_warp[kSortWarps][kDigits];  // counts, then where the warp's begin
  __shared__ uint32_t scan[kSortWarps];
  const int lane = threadIdx.x % kLanes, warp = threadIdx.x / kLanes;
  for (int d = threadIdx.x; d < kDigits * kSortWarps; d += kSortThreads) of_warp[d / kDigits][d % kDigits] = 0;
  griddep_wait();
  griddep_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= p.tiles) {
    store_zeros(p.zeros, static_cast<int64_t>(blockIdx.x - p.tiles) * kSortThreads + threadIdx.x,
                static_cast<int64_t>(gridDim.x - p.tiles) * kSortThreads);
    return;
  }
  if (p.zero_counts != nullptr)
    for (int d = threadIdx.x; d < kDigits; d += kSortThreads)
      p.zero_counts[static_cast<int64_t>(blockIdx.x) * kDigits + d] = 0u;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kSortThreads * PER) + warp * (PER * kLanes);
  uint32_t key[PER];
  uint32_t rank[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int64_t i = first + j * kLanes + lane;
    key[j] = i < p.n ? sort_key<FIRST>(p, static_cast<int>(i)) : 0u;
  }
  // this thread's two digits: their counts in all tiles and in those before this one
  uint32_t total[2] = {0, 0}, ahead[2] = {0, 0};
#pragma unroll 8
  for (int t = 0; t < p.tiles; ++t) {
    const uint2 c = *reinterpret_cast<const uint2*>(p.counts + static_cast<int64_t>(t) * kDigits + 2 * threadIdx.x);
    total[0] += c.x;
    total[1] += c.y;
    if (t < static_cast<int>(blockIdx.x)) {
      ahead[0] += c.x;
      ahead[1] += c.y;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const bool have = first + j * kLanes + lane < p.n;
    const uint32_t d = have ? (key[j] >> p.shift) & (kDigits - 1) : kDigits;  // kDigits: none
    const unsigned peers = __match_any_sync(0xffffffffu, d);
    const unsigned before = peers & ((1u << lane) - 1u);
    uint32_t at = 0;
    if (have) at = of_warp[warp][d];
    __syncwarp();
    if (have && before == 0) of_warp[warp][d] = at + static_cast<uint32_t>(__popc(peers));
    __syncwarp();
    rank[j] = at + static_cast<uint32_t>(__popc(before));
  }
  uint32_t sum = total[0] + total[1];
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == kLanes - 1) scan[warp] = sum;
  __syncthreads();  // of_warp's counts too
  uint32_t base = sum - total[0] - total[1];
  for (int w = 0; w < warp; ++w) base += scan[w];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t at = base + ahead[k];
    base += total[k];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t c = of_warp[w][2 * threadIdx.x + k];
      of_warp[w][2 * threadIdx.x + k] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int64_t i = first + j * kLanes + lane;
    if (i >= p.n) continue;
    const uint32_t to = of_warp[warp][(key[j] >> p.shift) & (kDigits - 1)] + rank[j];
    p.keys_out[to] = key[j];
    p.places_out[to] = FIRST ? static_cast<uint32_t>(i) : p.places[i];
    if (p.next_counts != nullptr)
      atomicAdd(p.next_counts + static_cast<int64_t>(to / (kSortThreads * PER)) * kDigits +
                    ((key[j] >> (p.shift + kDigitBits)) & (kDigits - 1)),
                1u);
  }
}

// ---------------------------------------------------------------------------
// The sums.
// ---------------------------------------------------------------------------

constexpr int kSumThreads = 128;

struct SumParams {
  const unsigned char* dy;
  const uint32_t* keys;    // sorted
  const uint32_t* places;
  int n, segment, segments;  // places a segment
  int64_t vocab, ld_dy, ld_dw;
  int width, groups, row_threads, slabs;  // row_threads: of a slab of a row, one group each
  float scale;
  unsigned char* dw;
  int vec_dw, accumulate;
  Zeros zeros;             // rows without a token among these
  int sum_blocks, zero_blocks;
  float* parts;            // [segments, 2, groups * 8]: a token's sum that goes on from the segment before, and
                           // one that begins here and goes on behind
};

// Row `key` of the gradient from a group's sum.
template <int OT>
__device__ __forceinline__ void put_sum(const SumParams& p, uint32_t key, int g, const float (&sum)[kVec]) {
  using R = Row<OT>;
  unsigned char* row = p.dw + static_cast<int64_t>(key) * p.ld_dw * R::EB;
  const int count = min(kVec, p.width - g * kVec);
  float v[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) v[j] = __fmul_rn(sum[j], p.scale);
  uint32_t w[R::kW];
  if (p.accumulate) {
    const RowStart at(row);
    R::load(at.base, at.off, g, count, w);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = __fadd_rn(R::get(w, j), v[j]);
  }
  R::pack(v, w);
  R::store(row, g, count, p.vec_dw != 0, w);
}

__device__ __forceinline__ void put_part(const SumParams& p, int segment, int which, int g, const float (&sum)[kVec]) {
  float4* o = reinterpret_cast<float4*>(p.parts + (static_cast<int64_t>(segment) * 2 + which) * p.groups * kVec + g * kVec);
  o[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
  o[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
}

// A thread's segment and group in block `block`; false: it has none.
__device__ __forceinline__ bool sum_unit(const SumParams& p, int64_t block, int& segment, int& g) {
  const int sub = static_cast<int>(threadIdx.x) / p.row_threads, per_block = kSumThreads / p.row_threads;
  const int64_t unit = block * per_block + sub;
  segment = static_cast<int>(unit / p.slabs);
  g = static_cast<int>(unit % p.slabs) * p.row_threads + static_cast<int>(threadIdx.x) - sub * p.row_threads;
  return sub < per_block && segment < p.segments && g < p.groups;
}

// Zeros in the rows of one block that have no token: 32 rows, a lane looking for each.
constexpr int kZeroRows = 32;
__device__ __forceinline__ void zero_rows(const SumParams& p, int64_t block) {
  const int64_t first = p.zeros.begin + block * kZeroRows;
  const int64_t mine = first + threadIdx.x % kLanes;
  int low = 0, high = p.n;  // the first place whose token is not below
  while (low < high) {
    const int mid = low + (high - low) / 2;
    if (static_cast<int64_t>(p.keys[mid]) < mine)
      low = mid + 1;
    else
      high = mid;
  }
  const bool none = mine < p.zeros.end && (low == p.n || static_cast<int64_t>(p.keys[low]) != mine);
  unsigned rows = __ballot_sync(0xffffffffu, none);
  while (rows != 0) {
    store_zero_row(p.zeros, first + __ffs(rows) - 1, threadIdx.x, kSumThreads);
    rows &= rows - 1;
  }
}

// One segment of places for one slab of columns: a group a thread.  The blocks that
// store zeros lie evenly among those that sum: the ones write while the others wait.
template <int DT, int OT, bool FULL>
__global__ void __launch_bounds__(kSumThreads) embedding_sum_kernel(const SumParams p) {
  using R = Row<DT>;
  constexpr int kAhead = DT == BIL_F32 ? 4 : 8;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t all = static_cast<int64_t>(p.sum_blocks) + p.zero_blocks, block = blockIdx.x;
  const int64_t zeros_before = block * p.zero_blocks / all;
  if ((block + 1) * p.zero_blocks / all != zeros_before) {
    zero_rows(p, zeros_before);
    return;
  }
  int segment, g;
  if (!sum_unit(p, block - zeros_before, segment, g)) return;
  const int begin = segment * p.segment;
  const int end = min(p.n, begin + p.segment);
  const uint32_t none = static_cast<uint32_t>(p.vocab);
  uint32_t now = p.keys[begin];
  if (now == none) return;
  bool from_before = begin > 0 && p.keys[begin - 1] == now;
  float sum[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) sum[j] = 0.0f;
  // The tokens and places of the next rows are loaded with the rows of these.
  uint32_t next_key[kAhead], next_place[kAhead];
  auto look = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      next_key[k] = i0 + k < end ? p.keys[i0 + k] : none;
      next_place[k] = i0 + k < end ? p.places[i0 + k] : 0u;
    }
  };
  look(begin);
  for (int i0 = begin; i0 < end; i0 += kAhead) {
    uint32_t key[kAhead];
    uint32_t w[kAhead][R::kW];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      key[k] = next_key[k];
      if (key[k] == none) continue;
      const RowStart row(p.dy + static_cast<int64_t>(next_place[k]) * p.ld_dy * R::EB);
      R::template load_path<FULL ? kFullRows : kAnyRows>(row.base, row.off, g, p.width, w[k]);
    }
    look(i0 + kAhead);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (i0 + k >= end) continue;
      if (key[k] != now) {  // the token before this one is done
        if (from_before)
          put_part(p, segment, 0, g, sum);
        else
          put_sum<OT>(p, now, g, sum);
        from_before = false;
        now = key[k];
        if (now == none) return;
#pragma unroll
        for (int j = 0; j < kVec; ++j) sum[j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) sum[j] = __fadd_rn(sum[j], R::get(w[k], j));
    }
  }
  const bool goes_on = end < p.n && p.keys[end] == now;
  if (from_before)
    put_part(p, segment, 0, g, sum);
  else if (goes_on)
    put_part(p, segment, 1, g, sum);
  else
    put_sum<OT>(p, now, g, sum);
}

// The tokens that begin in one segment and go on behind it: their parts in order.
template <int OT>
__global__ void __launch_bounds__(kSumThreads) embedding_join_kernel(const SumParams p) {
  griddep_wait();
  griddep_launch_dependents();
  int segment, g;
  if (!sum_unit(p, blockIdx.x, segment, g)) return;
  const int64_t begin = static_cast<int64_t>(segment) * p.segment, end = begin + p.segment;
  if (end >= p.n) return;
  const uint32_t key = p.keys[end - 1], behind = p.keys[end], before = begin > 0 ? p.keys[begin - 1] : ~0u;
  if (key == static_cast<uint32_t>(p.vocab) || behind != key || before == key) return;
  float sum[kVec];
  auto part = [&](int s, int which, float (&v)[kVec]) {
    const float4* o = reinterpret_cast<const float4*>(p.parts + (static_cast<int64_t>(s) * 2 + which) * p.groups * kVec + g * kVec);
    const float4 a = o[0], b = o[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  };
  part(segment, 1, sum);
  // the segments that begin with the token, a few at a time: their parts are loaded with their first tokens
  constexpr int kAhead = 8;
  for (int s0 = segment + 1; s0 < p.segments; s0 += kAhead) {
    uint32_t first[kAhead];
    float v[kAhead][kVec];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      first[k] = static_cast<uint32_t>(p.vocab);
      if (s0 + k >= p.segments) continue;
      first[k] = p.keys[static_cast<int64_t>(s0 + k) * p.segment];
      part(s0 + k, 0, v[k]);  // (of another token: not used)
    }
    bool more = true;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      more = more && first[k] == key;
      if (!more) continue;
#pragma unroll
      for (int j = 0; j < kVec; ++j) sum[j] = __fadd_rn(sum[j], v[k][j]);
    }
    if (!more) break;
  }
  put_sum<OT>(p, key, g, sum);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------

size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

// Places a segment: 16, or as many as leave 512 segments (of a power of two).  More segments would be more parts of
// the most frequent tokens, which are joined one after the other.
int segment_places(int64_t n) {
  int s = 16;
  while (static_cast<int64_t>(s) * 512 < n) s *= 2;
  return s;
}

// Places a thread of the sort's tiles: few, so that a short sort has blocks for more SMs (16384 tokens: 16); many
// from 64 such tiles on, since every tile reads the counts of all.
int sort_per(int64_t n) { return n <= 64 * kSortThreads * kFewPer ? kFewPer : kManyPer; }
int64_t sort_tiles(int64_t n) {
  const int64_t tile = static_cast<int64_t>(kSortThreads) * sort_per(n);
  return (n + tile - 1) / tile;
}

constexpr int64_t kEarlyZeros = 48 << 20;  // bytes of zeros in a launch of the sort: its seven microseconds at 6.6 TB/s

constexpr int kMaxDigits = 4;  // of 31 bits

struct Layout {
  size_t keys, counts, parts, total;
};

Layout layout_of(int64_t n, int64_t width) {
  Layout l;
  const int64_t tiles = sort_tiles(n), segments = (n + segment_places(n) - 1) / segment_places(n);
  l.keys = round256(static_cast<size_t>(n) * 4);
  l.counts = round256(static_cast<size_t>(tiles) * kDigits * 4);
  l.parts = round256(static_cast<size_t>(segments) * 2 * static_cast<size_t>((width + kVec - 1) / kVec * kVec) * 4);
  l.total = 4 * l.keys + kMaxDigits * l.counts + l.parts;
  return l;
}

int check_sizes(int64_t n, int64_t vocab, int64_t width) {
  if (n < 0 || vocab < 1 || width < 1) return BIL_E_INVALID_ARG;
  if (n > INT32_MAX - 65536 || vocab > INT32_MAX - 1 || width > INT32_MAX / 16) return BIL_E_UNSUPPORTED;
  return BIL_OK;
}

int pow2_threads(int groups, int most) {
  int t = 8;
  while (t < most && t < groups) t *= 2;
  return t;
}

template <int DT, int OT>
cudaError_t launch_sums(const SumParams& p, bool full, cudaStream_t s) {
  cudaError_t e = launch_pdl(full ? embedding_sum_kernel<DT, OT, true> : embedding_sum_kernel<DT, OT, false>,
                             static_cast<int64_t>(p.sum_blocks) + p.zero_blocks, kSumThreads, 0, s, 1, p);
  if (e != cudaSuccess || p.segments < 2) return e;
  return launch_pdl(embedding_join_kernel<OT>, p.sum_blocks, kSumThreads, 0, s, 1, p);
}

}  // namespace

extern "C" {

int bil_embedding_fwd(const int64_t* ids, int64_t n, const void* weight, int dtype, int64_t vocab, int64_t width,
                      int64_t ld_weight, float scale, void* out, int64_t ld_out, bil_stream_t stream) {
  bil_internal::NvtxRange nvtx_range("bil_embedding_fwd");
  const int eb = bil_internal::elem_bytes(dtype);
  if (eb == 0) return BIL_E_DTYPE;
  if (int st = check_sizes(n, vocab, width)) return st;
  if (!std::isfinite(scale)) return BIL_E_INVALID_ARG;
  if (int st = check_rows(weight, vocab, width, ld_weight, eb)) return st;
  if (int st = check_rows(out, n, width, ld_out, eb)) return st;
  if (n == 0) return BIL_OK;
  if (ids == nullptr) return BIL_E_INVALID_ARG;
  if (!aligned_to(ids, 8)) return BIL_E_ALIGN;
  LookupParams p{};
  p.ids = ids;
  p.weight = static_cast<const unsigned char*>(weight);
  p.out = static_cast<unsigned char*>(out);
  p.n = n;
  p.vocab = vocab;
  p.ld_w = ld_weight;
  p.ld_out = ld_out;
  p.width = static_cast<int>(width);
  p.groups = (p.width + kVec - 1) / kVec;
  p.vec_out = rows_start_on(out, n, ld_out * eb, 16);
  p.scale = scale;
  const int ahead = dtype == BIL_F32 ? 2 : 4;
  p.row_threads = pow2_threads((p.groups + ahead - 1) / ahead, kLookupThreads);
  const bool full = p.vec_out && width % kVec == 0 && rows_start_on(weight, vocab, ld_weight * eb, 16);
  void (*kernel)(LookupParams) =
      dtype == BIL_F32    ? (full ? embedding_lookup_kernel<BIL_F32, true> : embedding_lookup_kernel<BIL_F32, false>)
      : dtype == BIL_BF16 ? (full ? embedding_lookup_kernel<BIL_BF16, true> : embedding_lookup_kernel<BIL_BF16, false>)
                          : (full ? embedding_lookup_kernel<BIL_F16, true> : embedding_lookup_kernel<BIL_F16, false>);
  const int per_block = kLookupThreads / p.row_threads;
  const int64_t grid = std::min<int64_t>((n + per_block - 1) / per_block, INT32_MAX);
  return launch_pdl(kernel, grid, kLookupThreads, 0, reinterpret_cast<cudaStream_t>(stream), 1, p) == cudaSuccess
             ? BIL_OK
             : BIL_E_CUDA;
}

int bil_embedding_bwd_workspace_bytes(int64_t n, int64_t width, int64_t* bytes) {
  if (bytes == nullptr) return BIL_E_INVALID_ARG;
  if (int st = check_sizes(n, 1, width)) return st;
  *bytes = static_cast<int64_t>(layout_of(n, width).total);
  return BIL_OK;
}

int bil_embedding_bwd(const void* dy, int dtype, int64_t n, int64_t width, int64_t ld_dy, const int64_t* ids,
                      int64_t vocab, float scale, int64_t padding_idx, void* dweight, int dweight_dtype,
                      int64_t ld_dweight, int accumulate, void* workspace, int64_t workspace_bytes,
                      bil_stream_t stream) {
  bil_internal::NvtxRange nvtx_range("bil_embedding_bwd");
  const int eb = bil_internal::elem_bytes(dtype), ob = bil_internal::elem_bytes(dweight_dtype);
  if (eb == 0 || ob == 0 || (dweight_dtype != dtype && dweight_dtype != BIL_F32)) return BIL_E_DTYPE;
  if (int st = check_sizes(n, vocab, width)) return st;
  if (!std::isfinite(scale)) return BIL_E_INVALID_ARG;
  if (int st = check_rows(dy, n, width, ld_dy, eb)) return st;
  if (int st = check_rows(dweight, vocab, width, ld_dweight, ob)) return st;
  if (n > 0) {
    if (ids == nullptr || workspace == nullptr || dweight == dy) return BIL_E_INVALID_ARG;  // (dy is read to the end)
    if (!aligned_to(ids, 8) || !aligned_to(workspace, 256)) return BIL_E_ALIGN;
    if (workspace_bytes < static_cast<int64_t>(layout_of(n, width).total)) return BIL_E_INVALID_ARG;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (n == 0) {
    return accumulate || cudaMemset2DAsync(dweight, static_cast<size_t>(ld_dweight) * ob, 0, static_cast<size_t>(width) * ob,
                                           static_cast<size_t>(vocab), s) == cudaSuccess
               ? BIL_OK
               : BIL_E_CUDA;
  }
  int sms = 0, smem_optin = 0;
  if (int st = bil_internal::device_limits(&sms, &smem_optin)) return st;
  const Layout l = layout_of(n, width);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  uint32_t* buf[4];
  for (int i = 0; i < 4; ++i) buf[i] = reinterpret_cast<uint32_t*>(ws + i * l.keys);

  SortParams q{};
  q.ids = ids;
  q.vocab = vocab;
  q.padding = padding_idx;
  q.n = static_cast<int>(n);
  q.tiles = static_cast<int>(sort_tiles(n));
  Zeros zeros{static_cast<unsigned char*>(dweight), ld_dweight * ob, 0, accumulate ? 0 : vocab, width * ob};
  int digits = 1;
  while ((vocab >> (digits * kDigitBits)) != 0) ++digits;
  const int launches = digits + 1;
  // What the sort's launches have time for; the sums' launch stores the others.
  const int64_t early = std::min(zeros.end, launches * (kEarlyZeros / zeros.row_bytes + 1));
  const bool few = sort_per(n) == kFewPer;
  auto counts_of = [&](int digit) {
    return digit < digits ? reinterpret_cast<uint32_t*>(ws + 4 * l.keys + static_cast<size_t>(digit) * l.counts) : nullptr;
  };
  int at = 0;  // the pair of buffers that the next digit is written to
  for (int i = 0; i < launches; ++i) {
    const int digit = i == 0 ? 0 : i - 1;
    q.shift = digit * kDigitBits;
    q.counts = counts_of(digit);
    q.next_counts = counts_of(digit + 1);
    q.zero_counts = counts_of(i == 0 ? 1 : digit + 2);
    q.keys = buf[at ^ 2];
    q.places = buf[(at ^ 2) + 1];
    q.keys_out = buf[at];
    q.places_out = buf[at + 1];
    q.zeros = zeros;
    q.zeros.begin = early * i / launches;
    q.zeros.end = early * (i + 1) / launches;
    const int64_t units = ((q.zeros.end - q.zeros.begin) * q.zeros.row_bytes / 16 + kSortThreads - 1) / kSortThreads;
    const int64_t zero_blocks = early == 0 ? 0 : std::max<int64_t>(1, std::min<int64_t>(units, 8 * static_cast<int64_t>(sms)));
    void (*kernel)(SortParams) =
        i == 0   ? (few ? sort_count_kernel<kFewPer> : sort_count_kernel<kManyPer>)
        : i == 1 ? (few ? sort_place_kernel<true, kFewPer> : sort_place_kernel<true, kManyPer>)
                 : (few ? sort_place_kernel<false, kFewPer> : sort_place_kernel<false, kManyPer>);
    if (launch_pdl(kernel, q.tiles + zero_blocks, kSortThreads, 0, s, 1, q) != cudaSuccess) return BIL_E_CUDA;
    if (i > 0) at ^= 2;
  }

  SumParams p{};
  p.dy = static_cast<const unsigned char*>(dy);
  p.keys = buf[at ^ 2];
  p.places = buf[(at ^ 2) + 1];
  p.n = q.n;
  p.segment = segment_places(n);
  p.segments = (q.n + p.segment - 1) / p.segment;
  p.vocab = vocab;
  p.ld_dy = ld_dy;
  p.ld_dw = ld_dweight;
  p.width = static_cast<int>(width);
  p.groups = (p.width + kVec - 1) / kVec;
  p.slabs = (p.groups + kSumThreads - 1) / kSumThreads;  // as even as can be
  p.row_threads = ((p.groups + p.slabs - 1) / p.slabs + 7) / 8 * 8;
  p.scale = scale;
  p.dw = static_cast<unsigned char*>(dweight);
  p.vec_dw = rows_start_on(dweight, vocab, ld_dweight * ob, 16);
  p.accumulate = accumulate != 0;
  p.parts = reinterpret_cast<float*>(ws + 4 * l.keys + kMaxDigits * l.counts);
  const bool full = width % kVec == 0 && rows_start_on(dy, n, ld_dy * eb, 16);
  const int per_block = kSumThreads / p.row_threads;
  zeros.begin = early;
  p.zeros = zeros;
  const int64_t sum_blocks = (static_cast<int64_t>(p.segments) * p.slabs + per_block - 1) / per_block;
  const int64_t zero_blocks = (zeros.end - zeros.begin + kZeroRows - 1) / kZeroRows;
  if (sum_blocks + zero_blocks > INT32_MAX) return BIL_E_UNSUPPORTED;
  p.sum_blocks = static_cast<int>(sum_blocks);
  p.zero_blocks = static_cast<int>(zero_blocks);
  cudaError_t e;
  if (dtype == BIL_F32)
    e = launch_sums<BIL_F32, BIL_F32>(p, full, s);
  else if (dtype == BIL_BF16)
    e = dweight_dtype == BIL_F32 ? launch_sums<BIL_BF16, BIL_F32>(p, full, s)
                                 : launch_sums<BIL_BF16, BIL_BF16>(p, full, s);
  else
    e = dweight_dtype == BIL_F32 ? launch_sums<BIL_F16, BIL_F32>(p, full, s)
                                 : launch_sums<BIL_F16, BIL_F16>(p, full, s);
  return e == cudaSuccess ? BIL_OK : BIL_E_CUDA;
}

}  // extern "C"
