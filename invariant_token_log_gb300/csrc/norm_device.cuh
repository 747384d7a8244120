// The norms' kernels and their launches, shared by norm.cu (root-mean-square) and
// layer_norm.cu (layer norm): rows in registers or through a ring of bulk copies,
// their reductions, the weights' gradients.  What a kernel computes is said where
// its entry points are.  Everything is in an anonymous namespace: each
// translation unit has the instances that it launches and a watchdog word.
#pragma once

#include "launch.cuh"
#include "philox.cuh"
#include "rows_device.cuh"

#include <algorithm>
#include <cmath>

namespace {

using bil_layout::kMaxGroups;
using bil_layout::kMaxRowThreads;
using bil_layout::kMaxStages;
using bil_layout::row_shape;
using bil_layout::slot_bytes;
static_assert(bil_layout::kWarp == kLanes, "the layouts count in the same warps");

__device__ unsigned int g_watchdog_norm;
constexpr unsigned kWatchNorm = 1024u;  // the wait for a row of a ring
constexpr int kDrained = 2;             // of a block's abort flag: nothing is in flight any more
constexpr float kE4m3Max = 448.0f;
constexpr float kMinAmax = 7.888609052210118e-31f;  // 2^-100
static_assert(2 * (kMaxRowThreads / kLanes) * sizeof(float2) + kMaxStages * sizeof(uint64_t) + sizeof(DropKeys) + 32 <=
                  bil_layout::kNormStatics,
              "what the kernels declare beside their ring");
static_assert(BIL_MAX_NORM_WIDTH == kMaxRowThreads * kMaxGroups * kVec, "the widest row a block holds");

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// A row's reductions: a butterfly in each warp, then (more than one warp a row)
// one over the warps' results.  Every thread gets the same values.  Two rows'
// reductions in turn use a buffer of their own: the barrier of the one keeps a
// thread from writing the other's before every thread has read it.
struct RowReduce {
  float2* red;   // [2][kMaxRowThreads / kLanes]
  int warps;     // of the row
  int which = 0;

  // the sum of s and the maximum (a NaN wins) of m, which is >= 0
  template <bool SUM, bool MAX>
  __device__ __forceinline__ void run(float& s, float& m) {
    butterfly<SUM, MAX>(s, m);
    if (warps == 1) return;
    float2* buf = red + which * (kMaxRowThreads / kLanes);
    which ^= 1;
    const int lane = threadIdx.x % kLanes;
    if (lane == 0) buf[threadIdx.x / kLanes] = make_float2(s, m);
    __syncthreads();
    const float2 v = lane < warps ? buf[lane] : make_float2(0.0f, 0.0f);
    s = v.x;
    m = v.y;
    butterfly<SUM, MAX>(s, m);
  }
  // The layer norm's, with less latency: the sums of a and of b, the two halves of a warp taking one each from the
  // first step on, and the warps' results added up by every thread itself (more than one warp a row).
  __device__ __forceinline__ void sums(float& a, float& b) {
    const int lane = threadIdx.x % kLanes;
    const bool upper = lane >= 16;
    float mine = __fadd_rn(upper ? b : a, __shfl_xor_sync(0xffffffffu, upper ? a : b, 16));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) mine = __fadd_rn(mine, __shfl_xor_sync(0xffffffffu, mine, o));
    if (warps == 1) {
      a = __shfl_sync(0xffffffffu, mine, 0);
      b = __shfl_sync(0xffffffffu, mine, 16);
      return;
    }
    float2* buf = red + which * (kMaxRowThreads / kLanes);
    which ^= 1;
    if (lane % 16 == 0) (upper ? buf[threadIdx.x / kLanes].y : buf[threadIdx.x / kLanes].x) = mine;
    __syncthreads();
    a = b = 0.0f;
    for (int w = 0; w < warps; ++w) {
      const float2 v = buf[w];
      a = __fadd_rn(a, v.x);
      b = __fadd_rn(b, v.y);
    }
  }
  // the sum of a alone
  __device__ __forceinline__ void sum(float& a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = __fadd_rn(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (warps == 1) return;
    float2* buf = red + which * (kMaxRowThreads / kLanes);
    which ^= 1;
    if (threadIdx.x % kLanes == 0) buf[threadIdx.x / kLanes].x = a;
    __syncthreads();
    a = 0.0f;
    for (int w = 0; w < warps; ++w) a = __fadd_rn(a, buf[w].x);
  }
  template <bool SUM, bool MAX>
  __device__ static __forceinline__ void butterfly(float& s, float& m) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (SUM) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
      if (MAX) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
  }
};

// 1-D bulk copy global -> shared, completion counted on `bar` in bytes (16-byte aligned, a multiple of 16).
__device__ __forceinline__ void bulk_copy(void* dst, const void* src, unsigned bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// The 8 elements of a group times their factor, in pairs.
template <typename R>
__device__ __forceinline__ void drop_pairs(const uint4& bits, const Dropout& drop, const uint32_t (&w)[R::kW], float (&v)[kVec]) {
#pragma unroll
  for (int j = 0; j < kVec / 2; ++j) {
    const uint64_t x = mul2(R::pair(w, j), pk(drop.times, drop.times));
    v[2 * j] = drop_keeps(bits, 2 * j, drop.border) ? lo_of(x) : 0.0f;
    v[2 * j + 1] = drop_keeps(bits, 2 * j + 1, drop.border) ? hi_of(x) : 0.0f;
  }
}

struct NormParams {
  const unsigned char* x;
  const unsigned char* residual;  // NULL: none
  const unsigned char* weight;    // NULL: the quantisation alone, y = x
  int64_t n_rows;
  int width, groups;
  int64_t ld_x, ld_r, ld_y, ld_h;  // elements (ld_y of an 8-bit output: bytes)
  float eps;
  unsigned char* y;
  unsigned char* h;   // NULL: not stored
  float* rstd;        // NULL: not stored
  float* scale;       // 8-bit output
  int vec_y, vec_h;   // the output's rows start on 16-byte (8-bit: 8-byte) boundaries
  int row_threads;    // TPR
  // backward
  const unsigned char* dy;
  const unsigned char* dh;        // NULL: none
  int64_t ld_dy, ld_dh, ld_dx;
  unsigned char* dx;
  int vec_dx;
  float* dw_part;  // [parts, width]
  int stages;      // of the ring, where there is one
  // layer norm
  const unsigned char* bias;      // NULL: none
  float* mean;                    // of the forward: NULL: not stored
  unsigned char* dr;              // backward with dropout: the residual's gradient (NULL: not stored)
  int64_t ld_dr;
  int vec_dr;
  int need_bias;                  // the backward's parts hold the bias's sums besides: [parts, 2 width]
  Dropout drop;
};

// A block's ring of stages, each the rows of up to three operands in slots of
// their own, which one thread fills with bulk copies of the 16-byte aligned spans
// that hold them.
struct RowRing {
  unsigned char* smem;
  uint64_t* full;
  unsigned slot, stage_bytes;
  int row_bytes;

  __device__ __forceinline__ void fill(int s, const unsigned char* a, const unsigned char* b, const unsigned char* c) {
    const unsigned char* src[3] = {a, b, c};
    unsigned bytes[3], total = 0;
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const unsigned off = static_cast<unsigned>(reinterpret_cast<uintptr_t>(src[q]) & 15u);
      bytes[q] = (off + static_cast<unsigned>(row_bytes) + 15u) & ~15u;
      if (src[q] != nullptr) {
        src[q] -= off;
        total += bytes[q];
      }
    }
    mbar_arrive_expect_tx(&full[s], total);
    unsigned at = 0;
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      if (src[q] == nullptr) continue;
      bulk_copy(smem + static_cast<size_t>(s) * stage_bytes + at, src[q], bytes[q], &full[s]);
      at += slot;
    }
  }
  // Where the wait for stage s (phase `parity`) gave up: the thread that fills waits (bounded) for the copies
  // that may still be in flight, those of the `ahead` rows from this one on, once; no stage is filled after.
  __device__ __forceinline__ void drain(int s, unsigned parity, int stages, int64_t ahead, volatile int* abort) {
    if (*abort == kDrained) return;
    for (int k = 0; k < stages && k < ahead; ++k) {
      const int t = s + k < stages ? s + k : s + k - stages;
      if (!thread_wait_watch(&full[t], s + k < stages ? parity : parity ^ 1u, abort, kWatchNorm, &g_watchdog_norm, false))
        break;
    }
    *abort = kDrained;
  }
};

enum NormMode { kNormPlain = 0, kNormQuant = 1, kQuantOnly = 2, kLayer = 3, kLayerDrop = 4 };

// Two float32 values to e4m3, to nearest even, at most 448 in magnitude, a in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
  return r;
}

// Rows of whole units: a block takes its rows (eight of one warp each, or one)
// and is done.  Any rows: one row a block at a time through the ring, a stage
// refilled as soon as its row is in registers (the registers could not hold
// the two units a group lies in until they are shifted).
template <int DT, int NG, int MODE, int PATH>
__global__ void __launch_bounds__(kMaxRowThreads) norm_fwd_kernel(const NormParams p) {
  using R = Row<DT>;
  constexpr bool BULK = PATH < kFullRows;
  constexpr bool LAYER = MODE == kLayer || MODE == kLayerDrop;
  extern __shared__ __align__(128) unsigned char ring_smem[];
  __shared__ float2 red[2 * (kMaxRowThreads / kLanes)];
  __shared__ uint64_t full[kMaxStages];
  __shared__ int abort_flag;
  volatile int* abort = &abort_flag;
  const int tpr = p.row_threads;
  const int r = static_cast<int>(threadIdx.x) % tpr;
  int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  RowReduce reduce{red, tpr / kLanes};
  RowRing ring{ring_smem, full, slot_bytes(p.width * R::EB), 0, p.width * R::EB};
  ring.stage_bytes = ring.slot * (p.residual != nullptr ? 2u : 1u);
  auto fill = [&](int64_t of, int s) {
    ring.fill(s, p.x + of * p.ld_x * R::EB, p.residual != nullptr ? p.residual + of * p.ld_r * R::EB : nullptr, nullptr);
  };
  if (BULK) {
    if (threadIdx.x == 0) {
      for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], 1);
      *abort = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
  }
  griddep_wait();
  griddep_launch_dependents();
  __shared__ DropKeys drop_keys;
  if (MODE == kLayerDrop) {
    drop_keys.make(p.drop);
    __syncthreads();
  }
  if (row >= p.n_rows) return;  // whole units, one warp a row: no barrier follows
  if (BULK && threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s)
      if (row + static_cast<int64_t>(s) * gridDim.x < p.n_rows) fill(row + static_cast<int64_t>(s) * gridDim.x, s);
  }
  int stage = 0;
  unsigned parity = 0;
  do {
  RowStart x(p.x + row * p.ld_x * R::EB);
  RowStart res(p.residual != nullptr ? p.residual + row * p.ld_r * R::EB : nullptr);
  if (BULK) {
    // (A wait that ran out has set the watchdog's bit; the block goes on to its end with what is there, its
    // barriers still met by every thread, and fills no further stage.)
    if (!warp_wait_watch(&full[stage], parity, abort, kWatchNorm, &g_watchdog_norm) && threadIdx.x == 0)
      ring.drain(stage, parity, p.stages, (p.n_rows - row + gridDim.x - 1) / gridDim.x, abort);
    x.base = ring_smem + static_cast<size_t>(stage) * ring.stage_bytes;
    res.base = x.base + ring.slot;
  }
  uint32_t w[NG][R::kW];  // the row's h
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int g = r + i * tpr;
    if (g < p.groups) R::template load_path<PATH>(x.base, x.off, g, p.width, w[i]);
  }
  if (MODE != kQuantOnly && (MODE == kLayerDrop || p.residual != nullptr)) {
    uint32_t q[NG][R::kW];
    if (MODE != kLayerDrop || p.residual != nullptr) {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const int g = r + i * tpr;
        if (g < p.groups) R::template load_path<PATH>(res.base, res.off, g, p.width, q[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g >= p.groups) continue;
      float v[kVec];
      if constexpr (MODE == kLayerDrop) {
        const uint4 bits = drop_keys.bits(static_cast<uint64_t>(row) * static_cast<uint64_t>(p.groups) + g);
        drop_pairs<R>(bits, p.drop, w[i], v);
        if (p.residual != nullptr) {
#pragma unroll
          for (int j = 0; j < kVec; ++j) v[j] = __fadd_rn(v[j], R::get(q[i], j));
        }
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = __fadd_rn(R::get(w[i], j), R::get(q[i], j));
      }
      R::pack(v, w[i]);
      if (p.h != nullptr)
        R::template store_path<PATH>(p.h + row * p.ld_h * R::EB, g, p.width, p.vec_h != 0, w[i]);
    }
  }
  float ss = 0.0f, amax = 0.0f;
  uint64_t sums = 0;
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int g = r + i * tpr;
    if (g >= p.groups) continue;
    if constexpr (LAYER) {  // in pairs, half of the instructions
#pragma unroll
      for (int j = 0; j < kVec / 2; ++j) sums = add2(sums, R::pair(w[i], j));
      continue;
    }
    Weight<DT, PATH> wt;
    if (MODE == kNormQuant) wt.load(p.weight, g, p.width);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {  // missing elements are zero, and so are their weights
      const float v = R::get(w[i], j);
      if (MODE != kQuantOnly) ss = __fmaf_rn(v, v, ss);
      if (MODE == kNormQuant) amax = max_nan(amax, fabsf(__fmul_rn(v, wt.get(j))));
      if (MODE == kQuantOnly) amax = max_nan(amax, fabsf(v));
    }
  }
  if (LAYER) {
    ss = __fadd_rn(lo_of(sums), hi_of(sums));
    reduce.sum(ss);
  } else {
    reduce.run<MODE != kQuantOnly, MODE != kNormPlain>(ss, amax);
  }
  if (BULK) {  // every thread has the row: its stage takes another
    if (reduce.warps == 1) __syncwarp();
    const int64_t refill = row + static_cast<int64_t>(p.stages) * gridDim.x;
    if (threadIdx.x == 0 && refill < p.n_rows && *abort == 0) fill(refill, stage);
    if (++stage == p.stages) {
      stage = 0;
      parity ^= 1u;
    }
  }
  float rstd = 1.0f, mean = 0.0f;
  if constexpr (LAYER) {  // the squares of what is left of the row without its mean
    mean = __fdiv_rn(ss, static_cast<float>(p.width));
    if (r == 0 && p.mean != nullptr) p.mean[row] = mean;
    sums = 0;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g >= p.groups) continue;
      const int count = PATH >= kFullRows ? kVec : min(kVec, p.width - g * kVec);
#pragma unroll
      for (int j = 0; j < kVec / 2; ++j) {
        uint64_t v = sub2(R::pair(w[i], j), pk(mean, mean));
        if (2 * j >= count) v = 0;
        if (2 * j + 1 >= count) v = pk(lo_of(v), 0.0f);
        sums = fma2(v, v, sums);
      }
    }
    ss = __fadd_rn(lo_of(sums), hi_of(sums));
    reduce.sum(ss);
  }
  if (MODE != kQuantOnly) {
    const float ms = __fdiv_rn(ss, static_cast<float>(p.width));
    rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(ms, p.eps)));
    if (r == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
  }
  if constexpr (LAYER) {
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g >= p.groups) continue;
      Weight<DT, PATH> wt, bias;
      wt.load(p.weight, g, p.width);
      float v[kVec];
      const uint64_t mean2 = pk(mean, mean), rstd2 = pk(rstd, rstd);
      if (p.bias != nullptr) bias.load(p.bias, g, p.width);
#pragma unroll
      for (int j = 0; j < kVec / 2; ++j) {
        const uint64_t u = mul2(sub2(R::pair(w[i], j), mean2), rstd2);
        const uint64_t y = p.bias != nullptr ? fma2(u, wt.pair(j), bias.pair(j)) : mul2(u, wt.pair(j));
        v[2 * j] = lo_of(y);
        v[2 * j + 1] = hi_of(y);
      }
      uint32_t o[R::kW];
      R::pack(v, o);
      R::template store_path<PATH>(p.y + row * p.ld_y * R::EB, g, p.width, p.vec_y != 0, o);
    }
  } else if constexpr (MODE == kNormPlain) {
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g >= p.groups) continue;
      Weight<DT, PATH> wt;
      wt.load(p.weight, g, p.width);
      float v[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[j] = __fmul_rn(__fmul_rn(R::get(w[i], j), rstd), wt.get(j));
      uint32_t o[R::kW];
      R::pack(v, o);
      R::template store_path<PATH>(p.y + row * p.ld_y * R::EB, g, p.width, p.vec_y != 0, o);
    }
  } else {
    if (MODE == kNormQuant) amax = __fmul_rn(amax, rstd);
    amax = max_nan(amax, kMinAmax);
    const float inv = __fdiv_rn(kE4m3Max, amax);
    if (r == 0) p.scale[row] = __fdiv_rn(amax, kE4m3Max);
    unsigned char* out = p.y + row * p.ld_y;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g >= p.groups) continue;
      const int count = min(kVec, p.width - g * kVec);
      float y[kVec];
      if (MODE == kNormQuant) {
        Weight<DT, PATH> wt;
        wt.load(p.weight, g, p.width);
#pragma unroll
        for (int j = 0; j < kVec; ++j) y[j] = __fmul_rn(__fmul_rn(R::get(w[i], j), rstd), wt.get(j));
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) y[j] = R::get(w[i], j);
      }
      uint32_t q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        q[j] = e4m3x2(__fmul_rn(y[2 * j], inv), __fmul_rn(y[2 * j + 1], inv));
      unsigned char* o = out + static_cast<int64_t>(g) * kVec;
      if (PATH >= kFullRows || (p.vec_y != 0 && count == kVec)) {
        *reinterpret_cast<uint2*>(o) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (j < count) o[j] = static_cast<unsigned char>(q[j / 2] >> (8 * (j & 1)));
      }
    }
  }
  row += gridDim.x;
  } while (BULK && row < p.n_rows);
}

// Backward.  A block takes the rows b, b + blocks, ... (a warp takes its
// block's rows in turn where a warp has a row) and keeps its columns' sums of
// dy u in registers; they go to dw_part as one row a block (the warps' added up
// in order), which norm_dw_kernel adds up in order.
// BULK (one row a block): the rows of h, dy and dh come through p.stages stages
// of shared memory, each operand's 16-byte aligned span in a slot of its own; a
// stage is refilled once every thread has passed the next row's reduction, when
// all are done with it.
enum NormKind { kRms = 0, kLayerNorm = 1, kLayerNormDrop = 2 };

template <int DT, int NG, bool BULK, int PATH, int KIND>
__global__ void __launch_bounds__(kMaxRowThreads) norm_bwd_kernel(const NormParams p) {
  using R = Row<DT>;
  constexpr bool LAYER = KIND != kRms;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ float2 red[2 * (kMaxRowThreads / kLanes)];
  __shared__ uint64_t full[kMaxStages];
  __shared__ int abort_flag;
  const int tpr = p.row_threads;
  const int r = static_cast<int>(threadIdx.x) % tpr;
  const int64_t part = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  const int64_t parts = static_cast<int64_t>(gridDim.x) * (blockDim.x / tpr);
  RowReduce reduce{red, tpr / kLanes};
  volatile int* abort = &abort_flag;
  if (BULK) {
    if (threadIdx.x == 0) {
      for (int s = 0; s < p.stages; ++s) mbar_init(&full[s], 1);
      *abort = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
  }
  griddep_wait();
  griddep_launch_dependents();
  RowRing rows{ring, full, slot_bytes(p.width * R::EB), 0, p.width * R::EB};
  rows.stage_bytes = rows.slot * (p.dh != nullptr ? 3u : 2u);
  auto fill = [&](int64_t row, int s) {
    rows.fill(s, p.x + row * p.ld_x * R::EB, p.dy + row * p.ld_dy * R::EB,
              p.dh != nullptr ? p.dh + row * p.ld_dh * R::EB : nullptr);
  };
  if (BULK && threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s)
      if (part + s * parts < p.n_rows) fill(part + s * parts, s);
  }
  Weight<DT, PATH> wt[NG];  // stays in registers, packed
#pragma unroll
  for (int i = 0; i < NG; ++i)
    if (r + i * tpr < p.groups) wt[i].load(p.weight, r + i * tpr, p.width);
  float dw[NG][kVec];
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) dw[i][j] = 0.0f;
  uint64_t dw2[NG][kVec / 2], db2[NG][kVec / 2];  // the layer norm's, in pairs
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int j = 0; j < kVec / 2; ++j) dw2[i][j] = db2[i][j] = 0;
  __shared__ DropKeys drop_keys;
  if (KIND == kLayerNormDrop) {
    drop_keys.make(p.drop);
    __syncthreads();
  }
  const float inv_width = __fdiv_rn(1.0f, static_cast<float>(p.width));
  int stage = 0;
  unsigned parity = 0;
  // The layer norm's statistics of a row are loaded a row ahead.
  float next_rstd = 0.0f, next_mean = 0.0f;
  if (LAYER && part < p.n_rows) {
    next_rstd = p.rstd[part];
    next_mean = p.mean[part];
  }
  for (int64_t row = part; row < p.n_rows; row += parts) {
    // where the rows lie in memory and (BULK, as far past a 16-byte boundary) in the stage
    RowStart h(p.x + row * p.ld_x * R::EB), dy(p.dy + row * p.ld_dy * R::EB);
    RowStart dh(p.dh != nullptr ? p.dh + row * p.ld_dh * R::EB : nullptr);
    const float rstd = LAYER ? next_rstd : p.rstd[row];
    // The layer norm works on pairs of elements, half of the instructions; an element of the normed row is
    // h rstd - (mean rstd) there, whose rounding is far below the mean's own.
    const float off = LAYER ? -__fmul_rn(next_mean, rstd) : 0.0f;
    if (LAYER && row + parts < p.n_rows) {
      next_rstd = p.rstd[row + parts];
      next_mean = p.mean[row + parts];
    }
    const uint64_t rstd2 = pk(rstd, rstd), off2 = pk(off, off);
    if (BULK) {
      // (A wait that ran out has set the watchdog's bit; the block goes on to its end with what is there, its
      // barriers still met by every thread, and fills no further stage.)
      if (!warp_wait_watch(&full[stage], parity, abort, kWatchNorm, &g_watchdog_norm) && threadIdx.x == 0)
        rows.drain(stage, parity, p.stages, row == part ? p.stages : p.stages - 1, abort);
      h.base = ring + static_cast<size_t>(stage) * rows.stage_bytes;
      dy.base = h.base + rows.slot;
      dh.base = h.base + 2 * rows.slot;
    }
    // The row in registers between the two passes, or (BULK) in its stage: then a group at a time.
    constexpr int kHeld = BULK ? 1 : NG;
    uint32_t wh[kHeld][R::kW], wd[kHeld][R::kW], wg[kHeld][R::kW];
    float dot = 0.0f, sum = 0.0f;
    uint64_t dots = 0, sums = 0;
    if (!BULK) {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const int g = r + i * tpr;
        if (g >= p.groups) continue;
        R::template load_path<PATH>(h.base, h.off, g, p.width, wh[i % kHeld]);
        R::template load_path<PATH>(dy.base, dy.off, g, p.width, wd[i % kHeld]);
        if (p.dh != nullptr) R::template load_path<PATH>(dh.base, dh.off, g, p.width, wg[i % kHeld]);
      }
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g >= p.groups) continue;
      if (BULK) {
        R::template load_path<PATH>(h.base, h.off, g, p.width, wh[0]);
        R::template load_path<PATH>(dy.base, dy.off, g, p.width, wd[0]);
      }
      if constexpr (LAYER) {
#pragma unroll
        for (int j = 0; j < kVec / 2; ++j) {  // (a missing element's d and weight are zero)
          const uint64_t u = fma2(R::pair(wh[i % kHeld], j), rstd2, off2), d = R::pair(wd[i % kHeld], j);
          const uint64_t v = mul2(d, wt[i].pair(j));
          dots = fma2(v, u, dots);
          sums = add2(sums, v);
          dw2[i][j] = fma2(d, u, dw2[i][j]);
          db2[i][j] = add2(db2[i][j], d);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const float u = __fmul_rn(R::get(wh[i % kHeld], j), rstd), d = R::get(wd[i % kHeld], j);
          dot = __fmaf_rn(__fmul_rn(d, wt[i].get(j)), u, dot);
          dw[i][j] = __fmaf_rn(d, u, dw[i][j]);
        }
      }
    }
    float none = 0.0f;
    if (LAYER) {
      dot = __fadd_rn(lo_of(dots), hi_of(dots));
      sum = __fadd_rn(lo_of(sums), hi_of(sums));
      reduce.sums(dot, sum);
    } else {
      reduce.run<true, false>(dot, none);
    }
    const float c = LAYER ? 0.0f : __fdiv_rn(dot, static_cast<float>(p.width));
    // of the layer norm's rstd (v - c1 - u c2)
    const float f1 = LAYER ? -__fmul_rn(__fmul_rn(sum, inv_width), rstd) : 0.0f;
    const float f2 = LAYER ? -__fmul_rn(__fmul_rn(dot, inv_width), rstd) : 0.0f;
    const uint64_t f1s = pk(f1, f1), f2s = pk(f2, f2);
    if (BULK) {
      // every thread is done with the stage of the row before this one
      const int64_t refill = row + static_cast<int64_t>(p.stages - 1) * parts;
      if (threadIdx.x == 0 && row != part && refill < p.n_rows && *abort == 0)
        fill(refill, stage == 0 ? p.stages - 1 : stage - 1);
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g >= p.groups) continue;
      float v[kVec];
      if (BULK) {
        R::template load_path<PATH>(h.base, h.off, g, p.width, wh[0]);
        R::template load_path<PATH>(dy.base, dy.off, g, p.width, wd[0]);
      }
      if (BULK && p.dh != nullptr) R::template load_path<PATH>(dh.base, dh.off, g, p.width, wg[0]);
      if constexpr (LAYER) {
        uint64_t v2[kVec / 2];
#pragma unroll
        for (int j = 0; j < kVec / 2; ++j) {
          const uint64_t u = fma2(R::pair(wh[i % kHeld], j), rstd2, off2);
          v2[j] = fma2(mul2(R::pair(wd[i % kHeld], j), wt[i].pair(j)), rstd2, fma2(u, f2s, f1s));
        }
        if (p.dh != nullptr) {
#pragma unroll
          for (int j = 0; j < kVec / 2; ++j) v2[j] = add2(v2[j], R::pair(wg[i % kHeld], j));
        }
#pragma unroll
        for (int j = 0; j < kVec / 2; ++j) {
          v[2 * j] = lo_of(v2[j]);
          v[2 * j + 1] = hi_of(v2[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const float u = __fmul_rn(R::get(wh[i % kHeld], j), rstd);
          v[j] = __fmul_rn(rstd, __fmaf_rn(-u, c, __fmul_rn(R::get(wd[i % kHeld], j), wt[i].get(j))));
        }
        if (p.dh != nullptr) {
#pragma unroll
          for (int j = 0; j < kVec; ++j) v[j] = __fadd_rn(v[j], R::get(wg[i % kHeld], j));
        }
      }
      uint32_t o[R::kW];
      if constexpr (KIND == kLayerNormDrop) {
        if (p.dr != nullptr) {
          R::pack(v, o);
          R::template store_path<PATH>(p.dr + row * p.ld_dr * R::EB, g, p.width, p.vec_dr != 0, o);
        }
        const uint4 bits = drop_keys.bits(static_cast<uint64_t>(row) * static_cast<uint64_t>(p.groups) + g);
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          v[j] = drop_keeps(bits, j, p.drop.border) ? __fmul_rn(v[j], p.drop.times) : 0.0f;
      }
      R::pack(v, o);
      R::template store_path<PATH>(p.dx + row * p.ld_dx * R::EB, g, p.width, p.vec_dx != 0, o);
    }
    if (++stage == p.stages) {
      stage = 0;
      parity ^= 1u;
    }
  }
  // (the barrier in it is met by every thread)
  auto put = [&](float* out, const float (&sums_of)[NG][kVec]) {
    if (BULK || tpr == static_cast<int>(blockDim.x)) {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const int g = r + i * tpr;
        if (g >= p.groups) continue;
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (g * kVec + j < p.width) out[g * kVec + j] = sums_of[i][j];
      }
    } else {  // the block's warps: each row of `ring` is one warp's sums
      float* sums = reinterpret_cast<float*>(ring);
      const int pitch = p.groups * kVec, warps = blockDim.x / tpr;
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const int g = r + i * tpr;
        if (g >= p.groups) continue;
#pragma unroll
        for (int j = 0; j < kVec; ++j) sums[static_cast<int>(threadIdx.x) / tpr * pitch + g * kVec + j] = sums_of[i][j];
      }
      __syncthreads();
      for (int col = threadIdx.x; col < p.width; col += blockDim.x) {
        float v = sums[col];
        for (int q = 1; q < warps; ++q) v = __fadd_rn(v, sums[q * pitch + col]);
        out[col] = v;
      }
    }
  };
  float* out = p.dw_part + static_cast<int64_t>(blockIdx.x) * p.width * (LAYER && p.need_bias ? 2 : 1);
  auto apart = [&](const uint64_t (&pairs)[NG][kVec / 2]) {
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int j = 0; j < kVec / 2; ++j) {
        dw[i][2 * j] = lo_of(pairs[i][j]);
        dw[i][2 * j + 1] = hi_of(pairs[i][j]);
      }
  };
  if (LAYER) apart(dw2);
  put(out, dw);
  if (LAYER && p.need_bias) {
    apart(db2);
    __syncthreads();
    put(out + p.width, dw);
  }
}

// dw[c] = the parts' sum in a fixed order: warp w of the block adds parts w,
// w + 16, ... of its 32 columns in order, and the sums are added in order.  The
// columns from `width` on, where a part has more, are db's.
constexpr int kDwWarps = 16;

__global__ void __launch_bounds__(kDwWarps * kLanes) norm_dw_kernel(const float* __restrict__ part, int64_t parts,
                                                                    int width, float* __restrict__ dw,
                                                                    int columns, float* __restrict__ db) {
  __shared__ float sums[kDwWarps][kLanes];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % kLanes, warp = threadIdx.x / kLanes;
  const int c = static_cast<int>(blockIdx.x) * kLanes + lane;
  float s = 0.0f;
  if (c < columns) {
#pragma unroll 8
    for (int64_t i = warp; i < parts; i += kDwWarps) s = __fadd_rn(s, part[i * columns + c]);
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= columns) return;
  s = sums[0][lane];
  for (int w = 1; w < kDwWarps; ++w) s = __fadd_rn(s, sums[w][lane]);
  if (c < width)
    dw[c] = s;
  else
    db[c - width] = s;
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------

constexpr int kFwdGroups = 4, kBwdGroups = 2;

// Threads of a block: one row, or eight rows of one warp each.
int block_threads(int row_threads) { return row_threads == kLanes ? 8 * kLanes : row_threads; }

typedef void (*NormKernel)(NormParams);

template <int DT, int MODE, int PATH>
NormKernel fwd_kernel_ng(int ng) {
  return ng == 1 ? norm_fwd_kernel<DT, 1, MODE, PATH>
                 : ng == 2 ? norm_fwd_kernel<DT, 2, MODE, PATH> : norm_fwd_kernel<DT, 4, MODE, PATH>;
}

template <int DT, int MODE>
NormKernel fwd_kernel_dt(int ng, int path) {
  if (path == kFullRows) return fwd_kernel_ng<DT, MODE, kFullRows>(ng);
  if constexpr (DT != BIL_F32 && MODE != kQuantOnly) {
    if (path == kFullRowsF32Weight) return fwd_kernel_ng<DT, MODE, kFullRowsF32Weight>(ng);
    if (path == kAnyRowsF32Weight) return fwd_kernel_ng<DT, MODE, kAnyRowsF32Weight>(ng);
  }
  return fwd_kernel_ng<DT, MODE, kAnyRows>(ng);
}

template <int MODE>
NormKernel fwd_kernel(int dtype, int ng, int path) {
  return dtype == BIL_F32    ? fwd_kernel_dt<BIL_F32, MODE>(ng, path)
         : dtype == BIL_BF16 ? fwd_kernel_dt<BIL_BF16, MODE>(ng, path)
                             : fwd_kernel_dt<BIL_F16, MODE>(ng, path);
}

template <int DT, int PATH, int KIND>
NormKernel bwd_kernel_ng(int ng, bool bulk) {
  if (bulk) return ng <= 2 ? norm_bwd_kernel<DT, 2, true, PATH, KIND> : norm_bwd_kernel<DT, 4, true, PATH, KIND>;
  // Rows too wide for the ring (past 9636 elements with dh, 14460 without) in registers, which do not hold them:
  // 472 bytes a thread are spilled, 1028 where rows lie anywhere.  4096 x 16000 with dh 293 us, 0.53 of a copy's rate.
  if constexpr (DT == BIL_F32)
    if (ng == 4) return norm_bwd_kernel<DT, 4, false, PATH, KIND>;
  return ng == 1 ? norm_bwd_kernel<DT, 1, false, PATH, KIND> : norm_bwd_kernel<DT, 2, false, PATH, KIND>;
}

template <int DT, int KIND>
NormKernel bwd_kernel_dt(int ng, bool bulk, int path) {
  if (path == kFullRows) return bwd_kernel_ng<DT, kFullRows, KIND>(ng, bulk);
  if constexpr (DT != BIL_F32) {
    if (path == kFullRowsF32Weight) return bwd_kernel_ng<DT, kFullRowsF32Weight, KIND>(ng, bulk);
    if (path == kAnyRowsF32Weight) return bwd_kernel_ng<DT, kAnyRowsF32Weight, KIND>(ng, bulk);
  }
  return bwd_kernel_ng<DT, kAnyRows, KIND>(ng, bulk);
}

template <int KIND>
NormKernel bwd_kernel(int dtype, int ng, bool bulk, int path) {
  return dtype == BIL_F32    ? bwd_kernel_dt<BIL_F32, KIND>(ng, bulk, path)
         : dtype == BIL_BF16 ? bwd_kernel_dt<BIL_BF16, KIND>(ng, bulk, path)
                             : bwd_kernel_dt<BIL_F16, KIND>(ng, bulk, path);
}

int check_common(int dtype, int64_t n_rows, int64_t width) {
  if (bil_internal::elem_bytes(dtype) == 0) return BIL_E_DTYPE;
  if (n_rows < 0 || width < 1) return BIL_E_INVALID_ARG;
  if (width > BIL_MAX_NORM_WIDTH) return BIL_E_UNSUPPORTED;
  return BIL_OK;
}

int check_weight(const void* weight, int dtype, int weight_dtype) {
  if (weight_dtype != dtype && weight_dtype != BIL_F32) return BIL_E_DTYPE;
  if (weight == nullptr) return BIL_E_INVALID_ARG;
  return aligned_to(weight, 16) ? BIL_OK : BIL_E_ALIGN;
}

int launch_fwd(NormKernel kernel, NormParams& p, int path, int eb, cudaStream_t s) {
  if (path >= kFullRows) {
    const int threads = block_threads(p.row_threads);
    const int64_t rows_per_block = threads / p.row_threads;
    const int64_t grid = (p.n_rows + rows_per_block - 1) / rows_per_block;
    if (grid > INT32_MAX) return BIL_E_UNSUPPORTED;
    return launch_pdl(kernel, grid, threads, 0, s, 1, p) == cudaSuccess ? BIL_OK : BIL_E_CUDA;
  }
  int sms = 0, smem_optin = 0;
  if (int st = bil_internal::device_limits(&sms, &smem_optin)) return st;
  const size_t limit = bil_layout::dynamic_limit(smem_optin);
  const size_t stage_bytes = static_cast<size_t>(slot_bytes(p.width * eb)) * (p.residual != nullptr ? 2 : 1);
  int per_sm = 0;
  bil_layout::fwd_ring(stage_bytes, p.row_threads, eb, limit, &per_sm, &p.stages);
  if (p.stages < 1) return BIL_E_UNSUPPORTED;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(limit)) != cudaSuccess)
    return BIL_E_CUDA;
  const int64_t grid = std::min<int64_t>(p.n_rows, static_cast<int64_t>(sms) * per_sm);
  return launch_pdl(kernel, grid, p.row_threads, stage_bytes * p.stages, s, 1, p) == cudaSuccess ? BIL_OK : BIL_E_CUDA;
}

// Blocks of the backward: per_sm a multiprocessor, at most one a row (eight
// rows a block where a warp takes a row).
int64_t bwd_blocks(int64_t n_rows, int row_threads, int sms, int per_sm) {
  const int64_t rows_per_block = block_threads(row_threads) / row_threads;
  return std::max<int64_t>(1, std::min<int64_t>((n_rows + rows_per_block - 1) / rows_per_block,
                                                static_cast<int64_t>(sms) * per_sm));
}

// The backward's partial sums, at most: one row of `width` a block.
int bwd_parts(int64_t n_rows, int64_t width, bool layer, int64_t* parts) {
  int sms = 0, smem = 0;
  if (int st = bil_internal::device_limits(&sms, &smem)) return st;
  int threads = 0, ng = 0;
  row_shape(static_cast<int>(width), kBwdGroups, &threads, &ng);
  *parts = bwd_blocks(n_rows, threads, sms, layer ? bil_layout::layer_bwd_per_sm(threads) : bil_layout::bwd_per_sm(threads, ng));
  return BIL_OK;
}

// The backward: the rows' kernel, then the weights' sums.  p: the operands, their
// strides and alignments, n_rows, width, groups, dw_part.  `full`: every row starts
// on a 16-byte boundary.  need_bias: dbias besides, from parts twice as wide.
template <int KIND>
int launch_bwd(NormParams& p, int dtype, int weight_dtype, bool full, float* dweight, float* dbias, cudaStream_t s) {
  const int eb = bil_internal::elem_bytes(dtype);
  int ng = 0;
  row_shape(p.width, kBwdGroups, &p.row_threads, &ng);
  const int threads = block_threads(p.row_threads);
  // Rows of more than one warp come through the ring.
  int sms = 0, smem_optin = 0;
  if (int st = bil_internal::device_limits(&sms, &smem_optin)) return st;
  const size_t limit = bil_layout::dynamic_limit(smem_optin);
  const size_t stage_bytes = static_cast<size_t>(slot_bytes(p.width * eb)) * (p.dh != nullptr ? 3 : 2);
  const int most = KIND != kRms ? bil_layout::layer_bwd_per_sm(p.row_threads) : bil_layout::bwd_per_sm(p.row_threads, ng);
  int per_sm = most;
  if (p.row_threads > kLanes) bil_layout::bwd_ring(stage_bytes, limit, &per_sm, &p.stages);
  const bool bulk = p.stages != 0;
  if (!bulk) per_sm = most;
  const int64_t grid = bwd_blocks(p.n_rows, p.row_threads, sms, per_sm);
  const int path = row_path(p.width, full, weight_dtype == dtype);
  NormKernel kernel = bwd_kernel<KIND>(dtype, ng, bulk, path);
  const size_t smem = bulk                       ? stage_bytes * p.stages
                      : threads == p.row_threads ? 0  // the warps' sums
                                                 : static_cast<size_t>(threads / kLanes) * p.groups * kVec * sizeof(float);
  if (bulk && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(limit)) !=
                      cudaSuccess)
    return BIL_E_CUDA;
  if (launch_pdl(kernel, grid, threads, smem, s, 1, p) != cudaSuccess) return BIL_E_CUDA;
  const int columns = p.width * (dbias != nullptr ? 2 : 1);
  return launch_pdl(norm_dw_kernel, (columns + kLanes - 1) / kLanes, kDwWarps * kLanes, 0, s, 1,
                    static_cast<const float*>(p.dw_part), grid, p.width, dweight, columns, dbias) == cudaSuccess
             ? BIL_OK
             : BIL_E_CUDA;
}

}  // namespace
