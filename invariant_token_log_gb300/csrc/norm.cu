// Root-mean-square norm of a residual stream, with the residual's addition and
// an output in 8 bits with a scale per row: what produces the LM head's
// hidden states.  The C ABI is declared in include/bil.h.
//
//     h = round_T(x + r)          (r optional: h = x)
//     rstd = 1 / sqrt(mean_c h_c^2 + eps)
//     y = (h rstd) w              stored in h's type T, or as
//     a = max(rstd max_c |h_c w_c|, 2^-100),  scale = a / 448,  q = e4m3(y * (448 / a))
// and the backward of y (and of h, which goes on as the residual stream):
//     u = h rstd,  v = dy w,  c = mean(v u)
//     dx = dr = rstd (v - u c) + dh,    dw = sum over rows of dy u
//
// Everything is float32 between the loads and the stores.  h is rounded to T
// before it is normed: the stream that the next layer and the backward read is
// the one the norm saw, so the norm of the sum and the norm of the stored sum
// are the same bits.  q is the float32 y rounded once, to 8 bits.  Its scale
// comes from the products h w, before rstd is known, so that the row's sum of
// squares and its maximum are one reduction; 2^-100 keeps an all-zero row's
// scale positive.
//
// Bound: HBM.  Every element is read once and written once.  16384 x 4096 bf16 (a
// plain copy's rate would be 6.8 TB/s): the forward with a residual 537 MB, 78 us,
// 6.85 TB/s; to 8 bits 470 MB, 70 us, 6.7 TB/s; the backward with dh 537 MB, 87 us,
// 6.2 TB/s, 8 us of it the weight's sums over the blocks (norm_dw_kernel: a block for
// every 32 columns, too few for the SMs; it weighs most on narrow rows: 16384 x 1024
// 33 us, 0.59 of the copy's rate, 65536 x 512 55 us, 0.72).  Rows off 16-byte
// boundaries (16384 x 4097): 97, 119 and 171 us.  A row is held between its
// reduction and its output: thread r of the row's TPR threads has the 8-element
// groups r, r + TPR, ... (at most 4).  TPR and the sums' order follow from the
// width alone, so a row's bits do not depend on the batch.  The forward keeps
// the row in registers, packed, four groups a lane: as many bytes in flight for
// as few registers and barriers as can be.  The backward, whose registers hold
// the weight's sums, has two groups a lane and streams its rows through shared
// memory with bulk copies, a few rows ahead (but for rows of one warp, and float32
// rows of which not two stages fit).  A row that does not start on a
// 16-byte boundary is read by the 16-byte units that hold its elements, shifted
// into place.

#include "../../include/bil.h"
#include "device_common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "layout.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

namespace {

using bil_layout::kMaxGroups;
using bil_layout::kMaxRowThreads;
using bil_layout::kMaxStages;
using bil_layout::kVec;
using bil_layout::row_shape;
using bil_layout::slot_bytes;
static_assert(bil_layout::kWarp == kLanes, "the layouts count in the same warps");

__device__ unsigned int g_watchdog_norm;
constexpr unsigned kWatchNorm = 1024u;  // the wait for a row of a ring
constexpr int kDrained = 2;             // of a block's abort flag: nothing is in flight any more
constexpr float kE4m3Max = 448.0f;
constexpr float kMinAmax = 7.888609052210118e-31f;  // 2^-100
static_assert(BIL_MAX_NORM_WIDTH == kMaxRowThreads * kMaxGroups * kVec, "the widest row a block holds");

// How a kernel reads its rows: from anywhere, of any width, or (without the tests
// that takes, half of the instructions) rows of a multiple of 8 elements on
// 16-byte boundaries, outputs too; the weight in the rows' type or in float32.
enum RowPath { kAnyRows = 0, kAnyRowsF32Weight = 1, kFullRows = 2, kFullRowsF32Weight = 3 };

template <int DT>
struct Row {
  static constexpr int EB = DT == BIL_F32 ? 4 : 2;
  static constexpr int kW = kVec * EB / 4;    // 32-bit words of a group
  static constexpr int kUnits = kW / 4;       // 16-byte units of an aligned group

  // Group g of a row that starts `off` bytes past the 16-byte boundary `base`:
  // `count` of its 8 elements exist (the others come out as +0).  Reads only
  // 16-byte units that hold one of them.  The offset is the row's: the branch on
  // it is uniform.
  __device__ static __forceinline__ void load(const unsigned char* base, unsigned off, int g, int count,
                                              uint32_t (&w)[kW]) {
    const unsigned char* p = base + static_cast<int64_t>(g) * kVec * EB;
    switch (off >> 2) {
      case 0: load_from<0>(p, off, count, w); break;
      case 1: load_from<1>(p, off, count, w); break;
      case 2: load_from<2>(p, off, count, w); break;
      default: load_from<3>(p, off, count, w); break;
    }
    if (count < kVec) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        if (j < count) continue;
        if (EB == 4)
          w[j] = 0u;
        else
          w[j / 2] &= (j & 1) ? 0x0000ffffu : 0xffff0000u;
      }
    }
  }
  // the group's words, WOFF words and off % 4 bytes into the units from p on
  template <int WOFF>
  __device__ static __forceinline__ void load_from(const unsigned char* p, unsigned off, int count, uint32_t (&w)[kW]) {
    uint32_t v[4 * (kUnits + 1)];
    const int units = (static_cast<int>(off) + count * EB + 15) / 16;
#pragma unroll
    for (int u = 0; u <= kUnits; ++u) {
      uint4 q = make_uint4(0u, 0u, 0u, 0u);
      if (u < units) q = *reinterpret_cast<const uint4*>(p + 16 * u);
      v[4 * u] = q.x;
      v[4 * u + 1] = q.y;
      v[4 * u + 2] = q.z;
      v[4 * u + 3] = q.w;
    }
    if constexpr (EB == 4) {
#pragma unroll
      for (int j = 0; j < kW; ++j) w[j] = v[j + WOFF];
    } else {
      const unsigned sh = 8u * (off & 3u);
#pragma unroll
      for (int j = 0; j < kW; ++j) w[j] = __funnelshift_r(v[j + WOFF], v[j + WOFF + 1], sh);
    }
  }

  // As load and store; no part of a unit to leave out where every row starts on a
  // 16-byte boundary and the width is a multiple of 8.
  template <int PATH>
  __device__ static __forceinline__ void load_path(const unsigned char* base, unsigned off, int g, int width,
                                                   uint32_t (&w)[kW]) {
    if constexpr (PATH == kAnyRows || PATH == kAnyRowsF32Weight) {
      load(base, off, g, min(kVec, width - g * kVec), w);
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(base) + g * kUnits;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const uint4 q = p[u];
        w[4 * u] = q.x;
        w[4 * u + 1] = q.y;
        w[4 * u + 2] = q.z;
        w[4 * u + 3] = q.w;
      }
    }
  }
  template <int PATH>
  __device__ static __forceinline__ void store_path(unsigned char* row, int g, int width, bool vec,
                                                    const uint32_t (&w)[kW]) {
    if constexpr (PATH == kAnyRows || PATH == kAnyRowsF32Weight) {
      store(row, g, min(kVec, width - g * kVec), vec, w);
    } else {
      uint4* p = reinterpret_cast<uint4*>(row) + g * kUnits;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) p[u] = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
    }
  }

  __device__ static __forceinline__ float get(const uint32_t (&w)[kW], int j) {
    if constexpr (DT == BIL_F32) {
      return __uint_as_float(w[j]);
    } else if constexpr (DT == BIL_BF16) {
      return __uint_as_float((j & 1) ? (w[j / 2] & 0xffff0000u) : (w[j / 2] << 16));
    } else {
      const __half2 h = *reinterpret_cast<const __half2*>(&w[j / 2]);
      return (j & 1) ? __high2float(h) : __low2float(h);
    }
  }

  // Words of the 8 values rounded to the type (to nearest even).
  __device__ static __forceinline__ void pack(const float (&v)[kVec], uint32_t (&w)[kW]) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      if constexpr (DT == BIL_F32) {
        w[j] = __float_as_uint(v[j]);
      } else if ((j & 1) == 0) {
        if constexpr (DT == BIL_BF16) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[j], v[j + 1]);
          w[j / 2] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __half2 h = __floats2half2_rn(v[j], v[j + 1]);
          w[j / 2] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
    }
  }

  // Store the first `count` elements of a group; vec: the row's start is
  // 16-byte aligned.
  __device__ static __forceinline__ void store(unsigned char* row, int g, int count, bool vec, const uint32_t (&w)[kW]) {
    unsigned char* p = row + static_cast<int64_t>(g) * kVec * EB;
    if (vec && count == kVec) {
#pragma unroll
      for (int u = 0; u < kUnits; ++u)
        *reinterpret_cast<uint4*>(p + 16 * u) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
      return;
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      if (j >= count) continue;
      if constexpr (EB == 4)
        reinterpret_cast<uint32_t*>(p)[j] = w[j];
      else
        reinterpret_cast<uint16_t*>(p)[j] = static_cast<uint16_t>((j & 1) ? (w[j / 2] >> 16) : (w[j / 2] & 0xffffu));
    }
  }
};

// The weight's words of group g, and its values.
template <int DT, int PATH>
struct Weight {
  using W = Row<PATH == kFullRows || PATH == kAnyRows ? DT : BIL_F32>;
  uint32_t w[W::kW];

  __device__ __forceinline__ void load(const unsigned char* weight, int g, int width) {
    W::template load_path<PATH>(weight, 0, g, width, w);
  }
  __device__ __forceinline__ float get(int j) const { return W::get(w, j); }
};

// A row's 16-byte boundary and how far past it the row starts.
struct RowStart {
  const unsigned char* base;
  unsigned off;
  __device__ __forceinline__ RowStart(const unsigned char* row)
      : off(static_cast<unsigned>(reinterpret_cast<uintptr_t>(row) & 15u)) {
    base = row - off;
  }
};

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

enum NormMode { kNormPlain = 0, kNormQuant = 1, kQuantOnly = 2 };

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
  if (MODE != kQuantOnly && p.residual != nullptr) {
    uint32_t q[NG][R::kW];
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g < p.groups) R::template load_path<PATH>(res.base, res.off, g, p.width, q[i]);
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g >= p.groups) continue;
      float v[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[j] = __fadd_rn(R::get(w[i], j), R::get(q[i], j));
      R::pack(v, w[i]);
      if (p.h != nullptr)
        R::template store_path<PATH>(p.h + row * p.ld_h * R::EB, g, p.width, p.vec_h != 0, w[i]);
    }
  }
  float ss = 0.0f, amax = 0.0f;
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int g = r + i * tpr;
    if (g >= p.groups) continue;
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
  reduce.run<MODE != kQuantOnly, MODE != kNormPlain>(ss, amax);
  if (BULK) {  // every thread has the row: its stage takes another
    if (reduce.warps == 1) __syncwarp();
    const int64_t refill = row + static_cast<int64_t>(p.stages) * gridDim.x;
    if (threadIdx.x == 0 && refill < p.n_rows && *abort == 0) fill(refill, stage);
    if (++stage == p.stages) {
      stage = 0;
      parity ^= 1u;
    }
  }
  float rstd = 1.0f;
  if (MODE != kQuantOnly) {
    const float ms = __fdiv_rn(ss, static_cast<float>(p.width));
    rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(ms, p.eps)));
    if (r == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
  }
  if constexpr (MODE == kNormPlain) {
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
template <int DT, int NG, bool BULK, int PATH>
__global__ void __launch_bounds__(kMaxRowThreads) norm_bwd_kernel(const NormParams p) {
  using R = Row<DT>;
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
  int stage = 0;
  unsigned parity = 0;
  for (int64_t row = part; row < p.n_rows; row += parts) {
    // where the rows lie in memory and (BULK, as far past a 16-byte boundary) in the stage
    RowStart h(p.x + row * p.ld_x * R::EB), dy(p.dy + row * p.ld_dy * R::EB);
    RowStart dh(p.dh != nullptr ? p.dh + row * p.ld_dh * R::EB : nullptr);
    const float rstd = p.rstd[row];
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
    float dot = 0.0f;
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
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float u = __fmul_rn(R::get(wh[i % kHeld], j), rstd), d = R::get(wd[i % kHeld], j);
        dot = __fmaf_rn(__fmul_rn(d, wt[i].get(j)), u, dot);
        dw[i][j] = __fmaf_rn(d, u, dw[i][j]);
      }
    }
    float none = 0.0f;
    reduce.run<true, false>(dot, none);
    const float c = __fdiv_rn(dot, static_cast<float>(p.width));
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
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float u = __fmul_rn(R::get(wh[i % kHeld], j), rstd);
        v[j] = __fmul_rn(rstd, __fmaf_rn(-u, c, __fmul_rn(R::get(wd[i % kHeld], j), wt[i].get(j))));
      }
      if (p.dh != nullptr) {
        if (BULK) R::template load_path<PATH>(dh.base, dh.off, g, p.width, wg[0]);
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = __fadd_rn(v[j], R::get(wg[i % kHeld], j));
      }
      uint32_t o[R::kW];
      R::pack(v, o);
      R::template store_path<PATH>(p.dx + row * p.ld_dx * R::EB, g, p.width, p.vec_dx != 0, o);
    }
    if (++stage == p.stages) {
      stage = 0;
      parity ^= 1u;
    }
  }
  float* out = p.dw_part + static_cast<int64_t>(blockIdx.x) * p.width;
  if (BULK || tpr == static_cast<int>(blockDim.x)) {
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g >= p.groups) continue;
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (g * kVec + j < p.width) out[g * kVec + j] = dw[i][j];
    }
  } else {  // the block's warps: each row of `ring` is one warp's sums
    float* sums = reinterpret_cast<float*>(ring);
    const int pitch = p.groups * kVec, warps = blockDim.x / tpr;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g >= p.groups) continue;
#pragma unroll
      for (int j = 0; j < kVec; ++j) sums[static_cast<int>(threadIdx.x) / tpr * pitch + g * kVec + j] = dw[i][j];
    }
    __syncthreads();
    for (int col = threadIdx.x; col < p.width; col += blockDim.x) {
      float v = sums[col];
      for (int q = 1; q < warps; ++q) v = __fadd_rn(v, sums[q * pitch + col]);
      out[col] = v;
    }
  }
}

// dw[c] = the parts' sum in a fixed order: warp w of the block adds parts w,
// w + 16, ... of its 32 columns in order, and the sums are added in order.
constexpr int kDwWarps = 16;

__global__ void __launch_bounds__(kDwWarps * kLanes) norm_dw_kernel(const float* __restrict__ part, int64_t parts,
                                                                    int width, float* __restrict__ dw) {
  __shared__ float sums[kDwWarps][kLanes];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % kLanes, warp = threadIdx.x / kLanes;
  const int c = static_cast<int>(blockIdx.x) * kLanes + lane;
  float s = 0.0f;
  if (c < width) {
#pragma unroll 8
    for (int64_t i = warp; i < parts; i += kDwWarps) s = __fadd_rn(s, part[i * width + c]);
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= width) return;
  s = sums[0][lane];
  for (int w = 1; w < kDwWarps; ++w) s = __fadd_rn(s, sums[w][lane]);
  dw[c] = s;
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool rows_start_on(const void* p, int64_t n_rows, int64_t ld_bytes, size_t a) {
  return aligned_to(p, a) && (n_rows <= 1 || ld_bytes % static_cast<int64_t>(a) == 0);
}

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

template <int DT, int PATH>
NormKernel bwd_kernel_ng(int ng, bool bulk) {
  if (bulk) return ng <= 2 ? norm_bwd_kernel<DT, 2, true, PATH> : norm_bwd_kernel<DT, 4, true, PATH>;
  // Rows too wide for the ring (past 9636 elements with dh, 14460 without) in registers, which do not hold them:
  // 472 bytes a thread are spilled, 1028 where rows lie anywhere.  4096 x 16000 with dh 293 us, 0.53 of a copy's rate.
  if constexpr (DT == BIL_F32)
    if (ng == 4) return norm_bwd_kernel<DT, 4, false, PATH>;
  return ng == 1 ? norm_bwd_kernel<DT, 1, false, PATH> : norm_bwd_kernel<DT, 2, false, PATH>;
}

template <int DT>
NormKernel bwd_kernel_dt(int ng, bool bulk, int path) {
  if (path == kFullRows) return bwd_kernel_ng<DT, kFullRows>(ng, bulk);
  if constexpr (DT != BIL_F32) {
    if (path == kFullRowsF32Weight) return bwd_kernel_ng<DT, kFullRowsF32Weight>(ng, bulk);
    if (path == kAnyRowsF32Weight) return bwd_kernel_ng<DT, kAnyRowsF32Weight>(ng, bulk);
  }
  return bwd_kernel_ng<DT, kAnyRows>(ng, bulk);
}

// The rows' path: `full` says that every row starts on a 16-byte boundary.
int row_path(int64_t width, bool full, bool same_type) {
  if (!full || width % kVec != 0) return same_type ? kAnyRows : kAnyRowsF32Weight;
  return same_type ? kFullRows : kFullRowsF32Weight;
}

// Rows' extent and alignment of one [n_rows, ld] operand of eb-byte elements.
int check_rows(const void* p, int64_t n_rows, int64_t width, int64_t ld, int eb) {
  if (ld < width) return BIL_E_INVALID_ARG;
  if (!bil_internal::extent_ok(n_rows, ld, eb)) return BIL_E_UNSUPPORTED;
  if (n_rows > 0 && p == nullptr) return BIL_E_INVALID_ARG;
  if (!aligned_to(p, static_cast<size_t>(eb))) return BIL_E_ALIGN;
  return BIL_OK;
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
int bwd_parts(int64_t n_rows, int64_t width, int64_t* parts) {
  int sms = 0, smem = 0;
  if (int st = bil_internal::device_limits(&sms, &smem)) return st;
  int threads = 0, ng = 0;
  row_shape(static_cast<int>(width), kBwdGroups, &threads, &ng);
  *parts = bwd_blocks(n_rows, threads, sms, bil_layout::bwd_per_sm(threads, ng));
  return BIL_OK;
}

}  // namespace

namespace bil_internal {

int norm_watchdog(unsigned int* flags, int clear) {
  if (cudaMemcpyFromSymbol(flags, g_watchdog_norm, sizeof(unsigned int)) != cudaSuccess) return BIL_E_CUDA;
  if (clear) {
    const unsigned int zero = 0;
    if (cudaMemcpyToSymbol(g_watchdog_norm, &zero, sizeof(unsigned int)) != cudaSuccess) return BIL_E_CUDA;
  }
  return BIL_OK;
}

}  // namespace bil_internal

extern "C" {

int bil_rms_norm_fwd(const void* x, const void* residual, const void* weight, int dtype, int weight_dtype,
                     int64_t n_rows, int64_t width, int64_t ld_x, int64_t ld_residual, float eps, void* y,
                     int64_t ld_y, void* h, int64_t ld_h, float* rstd, bil_stream_t stream) {
  bil_internal::NvtxRange nvtx_range("bil_rms_norm_fwd");
  if (int st = check_common(dtype, n_rows, width)) return st;
  if (!(eps >= 0.0f) || std::isinf(eps)) return BIL_E_INVALID_ARG;
  if ((residual == nullptr) != (h == nullptr) && n_rows > 0) return BIL_E_INVALID_ARG;
  if (int st = check_weight(weight, dtype, weight_dtype)) return st;
  const int eb = bil_internal::elem_bytes(dtype);
  if (int st = check_rows(x, n_rows, width, ld_x, eb)) return st;
  if (int st = check_rows(y, n_rows, width, ld_y, eb)) return st;
  if (residual != nullptr) {
    if (int st = check_rows(residual, n_rows, width, ld_residual, eb)) return st;
    if (int st = check_rows(h, n_rows, width, ld_h, eb)) return st;
  }
  if (!aligned_to(rstd, 4)) return BIL_E_ALIGN;
  if (n_rows == 0) return BIL_OK;
  NormParams p{};
  p.x = static_cast<const unsigned char*>(x);
  p.residual = static_cast<const unsigned char*>(residual);
  p.weight = static_cast<const unsigned char*>(weight);
  p.n_rows = n_rows;
  p.width = static_cast<int>(width);
  p.groups = (p.width + kVec - 1) / kVec;
  p.ld_x = ld_x;
  p.ld_r = ld_residual;
  p.ld_y = ld_y;
  p.ld_h = ld_h;
  p.eps = eps;
  p.y = static_cast<unsigned char*>(y);
  p.h = static_cast<unsigned char*>(h);
  p.rstd = rstd;
  p.vec_y = rows_start_on(y, n_rows, ld_y * eb, 16);
  p.vec_h = rows_start_on(h, n_rows, ld_h * eb, 16);
  int ng = 0;
  row_shape(p.width, kFwdGroups, &p.row_threads, &ng);
  const bool full = rows_start_on(x, n_rows, ld_x * eb, 16) && p.vec_y &&
                    (residual == nullptr || (rows_start_on(residual, n_rows, ld_residual * eb, 16) && p.vec_h));
  const int path = row_path(width, full, weight_dtype == dtype);
  return launch_fwd(fwd_kernel<kNormPlain>(dtype, ng, path), p, path, eb, reinterpret_cast<cudaStream_t>(stream));
}

int bil_rms_norm_quant(const void* x, const void* residual, const void* weight, int dtype, int weight_dtype,
                       int64_t n_rows, int64_t width, int64_t ld_x, int64_t ld_residual, float eps, void* q,
                       int64_t ld_q, float* scale, void* h, int64_t ld_h, bil_stream_t stream) {
  bil_internal::NvtxRange nvtx_range("bil_rms_norm_quant");
  if (int st = check_common(dtype, n_rows, width)) return st;
  if (!(eps >= 0.0f) || std::isinf(eps)) return BIL_E_INVALID_ARG;
  if ((residual == nullptr) != (h == nullptr) && n_rows > 0) return BIL_E_INVALID_ARG;
  if (int st = check_weight(weight, dtype, weight_dtype)) return st;
  const int eb = bil_internal::elem_bytes(dtype);
  if (int st = check_rows(x, n_rows, width, ld_x, eb)) return st;
  if (int st = check_rows(q, n_rows, width, ld_q, 1)) return st;
  if (residual != nullptr) {
    if (int st = check_rows(residual, n_rows, width, ld_residual, eb)) return st;
    if (int st = check_rows(h, n_rows, width, ld_h, eb)) return st;
  }
  if (n_rows == 0) return BIL_OK;
  if (scale == nullptr) return BIL_E_INVALID_ARG;
  if (!aligned_to(scale, 4)) return BIL_E_ALIGN;
  NormParams p{};
  p.x = static_cast<const unsigned char*>(x);
  p.residual = static_cast<const unsigned char*>(residual);
  p.weight = static_cast<const unsigned char*>(weight);
  p.n_rows = n_rows;
  p.width = static_cast<int>(width);
  p.groups = (p.width + kVec - 1) / kVec;
  p.ld_x = ld_x;
  p.ld_r = ld_residual;
  p.ld_y = ld_q;
  p.ld_h = ld_h;
  p.eps = eps;
  p.y = static_cast<unsigned char*>(q);
  p.h = static_cast<unsigned char*>(h);
  p.scale = scale;
  p.vec_y = rows_start_on(q, n_rows, ld_q, 8);
  p.vec_h = rows_start_on(h, n_rows, ld_h * eb, 16);
  int ng = 0;
  row_shape(p.width, kFwdGroups, &p.row_threads, &ng);
  const bool full = rows_start_on(x, n_rows, ld_x * eb, 16) && p.vec_y &&
                    (residual == nullptr || (rows_start_on(residual, n_rows, ld_residual * eb, 16) && p.vec_h));
  const int path = row_path(width, full, weight_dtype == dtype);
  return launch_fwd(fwd_kernel<kNormQuant>(dtype, ng, path), p, path, eb, reinterpret_cast<cudaStream_t>(stream));
}

int bil_quantize_rows(const void* x, int dtype, int64_t n_rows, int64_t width, int64_t ld_x, void* q, int64_t ld_q,
                      float* scale, bil_stream_t stream) {
  bil_internal::NvtxRange nvtx_range("bil_quantize_rows");
  if (int st = check_common(dtype, n_rows, width)) return st;
  const int eb = bil_internal::elem_bytes(dtype);
  if (int st = check_rows(x, n_rows, width, ld_x, eb)) return st;
  if (int st = check_rows(q, n_rows, width, ld_q, 1)) return st;
  if (n_rows == 0) return BIL_OK;
  if (scale == nullptr) return BIL_E_INVALID_ARG;
  if (!aligned_to(scale, 4)) return BIL_E_ALIGN;
  NormParams p{};
  p.x = static_cast<const unsigned char*>(x);
  p.n_rows = n_rows;
  p.width = static_cast<int>(width);
  p.groups = (p.width + kVec - 1) / kVec;
  p.ld_x = ld_x;
  p.ld_y = ld_q;
  p.y = static_cast<unsigned char*>(q);
  p.scale = scale;
  p.vec_y = rows_start_on(q, n_rows, ld_q, 8);
  int ng = 0;
  row_shape(p.width, kFwdGroups, &p.row_threads, &ng);
  const bool full = rows_start_on(x, n_rows, ld_x * eb, 16) && p.vec_y;
  const int path = row_path(width, full, true);
  return launch_fwd(fwd_kernel<kQuantOnly>(dtype, ng, path), p, path, eb, reinterpret_cast<cudaStream_t>(stream));
}

int bil_rms_norm_bwd_workspace_bytes(int64_t n_rows, int64_t width, int64_t* bytes) {
  if (n_rows < 0 || width < 1 || bytes == nullptr) return BIL_E_INVALID_ARG;
  if (width > BIL_MAX_NORM_WIDTH) return BIL_E_UNSUPPORTED;
  int64_t parts = 0;
  if (int st = bwd_parts(n_rows, width, &parts)) return st;
  *bytes = parts * width * static_cast<int64_t>(sizeof(float));
  return BIL_OK;
}

int bil_rms_norm_bwd(const void* dy, const void* h, const void* weight, const float* rstd, const void* dh, int dtype,
                     int weight_dtype, int64_t n_rows, int64_t width, int64_t ld_dy, int64_t ld_h, int64_t ld_dh,
                     void* dx, int64_t ld_dx, float* dweight, void* workspace, int64_t workspace_bytes,
                     bil_stream_t stream) {
  bil_internal::NvtxRange nvtx_range("bil_rms_norm_bwd");
  if (int st = check_common(dtype, n_rows, width)) return st;
  if (int st = check_weight(weight, dtype, weight_dtype)) return st;
  const int eb = bil_internal::elem_bytes(dtype);
  if (int st = check_rows(dy, n_rows, width, ld_dy, eb)) return st;
  if (int st = check_rows(h, n_rows, width, ld_h, eb)) return st;
  if (int st = check_rows(dx, n_rows, width, ld_dx, eb)) return st;
  if (dh != nullptr) {
    if (int st = check_rows(dh, n_rows, width, ld_dh, eb)) return st;
  }
  if (dweight == nullptr) return BIL_E_INVALID_ARG;
  if (!aligned_to(dweight, 4) || !aligned_to(rstd, 4)) return BIL_E_ALIGN;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (n_rows == 0)  // a sum over no rows
    return cudaMemsetAsync(dweight, 0, static_cast<size_t>(width) * sizeof(float), s) == cudaSuccess ? BIL_OK
                                                                                                     : BIL_E_CUDA;
  if (rstd == nullptr || workspace == nullptr) return BIL_E_INVALID_ARG;
  if (!aligned_to(workspace, 16)) return BIL_E_ALIGN;
  int64_t parts = 0;
  if (int st = bwd_parts(n_rows, width, &parts)) return st;
  if (workspace_bytes < parts * width * static_cast<int64_t>(sizeof(float))) return BIL_E_INVALID_ARG;
  NormParams p{};
  p.x = static_cast<const unsigned char*>(h);
  p.weight = static_cast<const unsigned char*>(weight);
  p.n_rows = n_rows;
  p.width = static_cast<int>(width);
  p.groups = (p.width + kVec - 1) / kVec;
  p.ld_x = ld_h;
  p.rstd = const_cast<float*>(rstd);
  p.dy = static_cast<const unsigned char*>(dy);
  p.dh = static_cast<const unsigned char*>(dh);
  p.ld_dy = ld_dy;
  p.ld_dh = ld_dh;
  p.ld_dx = ld_dx;
  p.dx = static_cast<unsigned char*>(dx);
  p.vec_dx = rows_start_on(dx, n_rows, ld_dx * eb, 16);
  p.dw_part = static_cast<float*>(workspace);
  int ng = 0;
  row_shape(p.width, kBwdGroups, &p.row_threads, &ng);
  const int threads = block_threads(p.row_threads);
  // Rows of more than one warp come through the ring.
  int sms = 0, smem_optin = 0;
  if (int st = bil_internal::device_limits(&sms, &smem_optin)) return st;
  const size_t limit = bil_layout::dynamic_limit(smem_optin);
  const size_t stage_bytes = static_cast<size_t>(slot_bytes(p.width * eb)) * (dh != nullptr ? 3 : 2);
  int per_sm = bil_layout::bwd_per_sm(p.row_threads, ng);
  if (p.row_threads > kLanes) bil_layout::bwd_ring(stage_bytes, limit, &per_sm, &p.stages);
  const bool bulk = p.stages != 0;
  if (!bulk) per_sm = bil_layout::bwd_per_sm(p.row_threads, ng);
  const int64_t grid = bwd_blocks(n_rows, p.row_threads, sms, per_sm);
  parts = grid;
  const bool full = rows_start_on(h, n_rows, ld_h * eb, 16) && rows_start_on(dy, n_rows, ld_dy * eb, 16) && p.vec_dx &&
                    (dh == nullptr || rows_start_on(dh, n_rows, ld_dh * eb, 16));
  const int path = row_path(width, full, weight_dtype == dtype);
  NormKernel kernel = dtype == BIL_F32    ? bwd_kernel_dt<BIL_F32>(ng, bulk, path)
                      : dtype == BIL_BF16 ? bwd_kernel_dt<BIL_BF16>(ng, bulk, path)
                                          : bwd_kernel_dt<BIL_F16>(ng, bulk, path);
  const size_t smem = bulk                            ? stage_bytes * p.stages
                      : threads == p.row_threads ? 0  // the warps' sums
                                                 : static_cast<size_t>(threads / kLanes) * p.groups * kVec * sizeof(float);
  if (bulk && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(limit)) !=
                      cudaSuccess)
    return BIL_E_CUDA;
  if (launch_pdl(kernel, grid, threads, smem, s, 1, p) != cudaSuccess) return BIL_E_CUDA;
  return launch_pdl(norm_dw_kernel, (width + kLanes - 1) / kLanes, kDwWarps * kLanes, 0, s, 1,
                    static_cast<const float*>(p.dw_part), parts, p.width, dweight) == cudaSuccess
             ? BIL_OK
             : BIL_E_CUDA;
}

}  // extern "C"
