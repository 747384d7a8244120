// Root-mean-square norm of a residual stream, with the residual's addition and
// an output in 8 bits with a scale per row: what produces the LM head's
// hidden states.  The C ABI is declared in include/bil.h.
//
//     h = round_T(x + r)          (r optional: h = x)
//     rstd = 1 / sqrt(mean_c h_c^2 + eps)
//     y = (h rstd) w              stored in h's type T, or as
//     scale = max(max_c |y_c|, 2^-100) / 448,  q = e4m3(y * (448 / max))
// and the backward of y (and of h, which goes on as the residual stream):
//     u = h rstd,  v = dy w,  c = mean(v u)
//     dx = dr = rstd (v - u c) + dh,    dw = sum over rows of dy u
//
// Everything is float32 between the loads and the stores.  h is rounded to T
// before it is normed: the stream that the next layer and the backward read is
// the one the norm saw, so the norm of the sum and the norm of the stored sum
// are the same bits.  q's scale comes from the float32 y, which is then
// rounded once, to 8 bits; 2^-100 keeps an all-zero row's scale positive.
//
// Bound: HBM.  Every element is read once and written once (16384 x 4096 bf16:
// 537 MB, 79 us at the measured copy rate).  A row stays in registers
// between the reductions: thread r of the row's TPR threads holds the 8-element
// groups r, r + TPR, ... (at most 4), as the 16-byte units they are read in.
// TPR and the sums' order follow from the width alone, so a row's bits do not
// depend on the batch.  A row that does not start on a 16-byte boundary is read
// by the 16-byte units that hold its elements, shifted into place.

#include "../../include/bil.h"
#include "device_common.cuh"
#include "internal.h"
#include "launch.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

namespace {

constexpr int kVec = 8;             // elements of a group
constexpr int kMaxGroups = 4;       // groups a thread holds
constexpr int kMaxRowThreads = 512;
constexpr float kE4m3Max = 448.0f;
constexpr float kMinAmax = 7.888609052210118e-31f;  // 2^-100
static_assert(BIL_MAX_NORM_WIDTH == kMaxRowThreads * kMaxGroups * kVec, "the widest row a block holds");

template <int DT>
struct Row {
  static constexpr int EB = DT == BIL_F32 ? 4 : 2;
  static constexpr int kW = kVec * EB / 4;    // 32-bit words of a group
  static constexpr int kUnits = kW / 4;       // 16-byte units of an aligned group

  // Group g of the row at `row`: `count` of its 8 elements exist (the others
  // come out as +0).  Reads only 16-byte units that hold one of them.
  __device__ static __forceinline__ void load(const unsigned char* row, int g, int count, uint32_t (&w)[kW]) {
    const unsigned char* p = row + static_cast<int64_t>(g) * kVec * EB;
    const unsigned off = static_cast<unsigned>(reinterpret_cast<uintptr_t>(p) & 15u);
    if (off == 0) {
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        if (count * EB > 16 * u) q = *reinterpret_cast<const uint4*>(p + 16 * u);
        w[4 * u] = q.x;
        w[4 * u + 1] = q.y;
        w[4 * u + 2] = q.z;
        w[4 * u + 3] = q.w;
      }
    } else {
      uint32_t v[kW + 4];
#pragma unroll
      for (int u = 0; u <= kUnits; ++u) {
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        if (static_cast<int>(off) + count * EB > 16 * u) q = *reinterpret_cast<const uint4*>(p - off + 16 * u);
        v[4 * u] = q.x;
        v[4 * u + 1] = q.y;
        v[4 * u + 2] = q.z;
        v[4 * u + 3] = q.w;
      }
      // the group's first word sits off / 4 words in, then off % 4 bytes down
#pragma unroll
      for (int i = 0; i + 2 < kW + 4; ++i)
        if (off & 8u) v[i] = v[i + 2];
#pragma unroll
      for (int i = 0; i + 1 < kW + 2; ++i)
        if (off & 4u) v[i] = v[i + 1];
      const unsigned sh = 8u * (off & 3u);
#pragma unroll
      for (int j = 0; j < kW; ++j) w[j] = __funnelshift_r(v[j], v[j + 1], sh);
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

// The weight's 8 values of group g, in the rows' type or float32.
template <int DT>
__device__ __forceinline__ void load_weight(const unsigned char* weight, bool f32, int g, int count, float (&w)[kVec]) {
  if (DT == BIL_F32 || f32) {
    uint32_t q[Row<BIL_F32>::kW];
    Row<BIL_F32>::load(weight, g, count, q);
#pragma unroll
    for (int j = 0; j < kVec; ++j) w[j] = Row<BIL_F32>::get(q, j);
  } else {
    uint32_t q[Row<DT>::kW];
    Row<DT>::load(weight, g, count, q);
#pragma unroll
    for (int j = 0; j < kVec; ++j) w[j] = Row<DT>::get(q, j);
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The row's reductions: a butterfly in each warp, then (more than one warp a
// row) one over the warps' results.  Every thread gets the same value.  Both
// reductions of a row use a buffer of their own; the barrier of the one keeps
// a thread from writing the other's before every thread has read it.
struct RowReduce {
  float* red;    // [2][kMaxRowThreads / kLanes]
  int warps;     // of the row
  int which = 0;

  template <typename Op>
  __device__ __forceinline__ float run(float v, Op op, float none) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (warps == 1) return v;
    float* buf = red + which * (kMaxRowThreads / kLanes);
    which ^= 1;
    const int lane = threadIdx.x % kLanes;
    if (lane == 0) buf[threadIdx.x / kLanes] = v;
    __syncthreads();
    v = lane < warps ? buf[lane] : none;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
  __device__ __forceinline__ float sum(float v) {
    return run(v, [](float a, float b) { return __fadd_rn(a, b); }, 0.0f);
  }
  __device__ __forceinline__ float max_abs(float v) {
    return run(v, [](float a, float b) { return max_nan(a, b); }, 0.0f);
  }
};

struct NormParams {
  const unsigned char* x;
  const unsigned char* residual;  // NULL: none
  const unsigned char* weight;    // NULL: the quantisation alone, y = x
  int weight_f32;
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
};

enum NormMode { kNormPlain = 0, kNormQuant = 1, kQuantOnly = 2 };

// Two float32 values to e4m3, to nearest even, at most 448 in magnitude, a in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
  return r;
}

template <int DT, int NG, int MODE>
__global__ void __launch_bounds__(kMaxRowThreads) norm_fwd_kernel(const NormParams p) {
  using R = Row<DT>;
  __shared__ float red[2 * (kMaxRowThreads / kLanes)];
  griddep_wait();
  griddep_launch_dependents();
  const int tpr = p.row_threads;
  const int r = static_cast<int>(threadIdx.x) % tpr;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  if (row >= p.n_rows) return;  // one warp a row: no barrier follows
  RowReduce reduce{red, tpr / kLanes};
  const unsigned char* x = p.x + row * p.ld_x * R::EB;

  uint32_t w[NG][R::kW];  // the row's h
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int g = r + i * tpr;
    if (g < p.groups) R::load(x, g, min(kVec, p.width - g * kVec), w[i]);
  }
  if (MODE != kQuantOnly && p.residual != nullptr) {
    const unsigned char* res = p.residual + row * p.ld_r * R::EB;
    uint32_t q[NG][R::kW];
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g < p.groups) R::load(res, g, min(kVec, p.width - g * kVec), q[i]);
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
        R::store(p.h + row * p.ld_h * R::EB, g, min(kVec, p.width - g * kVec), p.vec_h != 0, w[i]);
    }
  }
  float rstd = 1.0f;
  if (MODE != kQuantOnly) {
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      if (r + i * tpr >= p.groups) continue;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float v = R::get(w[i], j);
        ss = __fmaf_rn(v, v, ss);
      }
    }
    ss = reduce.sum(ss);
    const float ms = __fdiv_rn(ss, static_cast<float>(p.width));
    rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(ms, p.eps)));
    if (r == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
  }
  if constexpr (MODE == kNormPlain) {
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g >= p.groups) continue;
      const int count = min(kVec, p.width - g * kVec);
      float wt[kVec], v[kVec];
      load_weight<DT>(p.weight, p.weight_f32 != 0, g, count, wt);
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[j] = __fmul_rn(__fmul_rn(R::get(w[i], j), rstd), wt[j]);
      uint32_t o[R::kW];
      R::pack(v, o);
      R::store(p.y + row * p.ld_y * R::EB, g, count, p.vec_y != 0, o);
    }
  } else {
    float y[NG][kVec];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
#pragma unroll
      for (int j = 0; j < kVec; ++j) y[i][j] = 0.0f;
      if (g >= p.groups) continue;
      if (MODE == kNormQuant) {
        float wt[kVec];
        load_weight<DT>(p.weight, p.weight_f32 != 0, g, min(kVec, p.width - g * kVec), wt);
#pragma unroll
        for (int j = 0; j < kVec; ++j) y[i][j] = __fmul_rn(__fmul_rn(R::get(w[i], j), rstd), wt[j]);
        if (p.width - g * kVec < kVec) {  // a missing element is no part of the maximum (0 * inf would be)
#pragma unroll
          for (int j = 0; j < kVec; ++j)
            if (j >= p.width - g * kVec) y[i][j] = 0.0f;
        }
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) y[i][j] = R::get(w[i], j);
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) amax = max_nan(amax, fabsf(y[i][j]));
    }
    amax = max_nan(reduce.max_abs(amax), kMinAmax);
    const float inv = __fdiv_rn(kE4m3Max, amax);
    if (r == 0) p.scale[row] = __fdiv_rn(amax, kE4m3Max);
    unsigned char* out = p.y + row * p.ld_y;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g >= p.groups) continue;
      const int count = min(kVec, p.width - g * kVec);
      uint32_t q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        q[j] = e4m3x2(__fmul_rn(y[i][2 * j], inv), __fmul_rn(y[i][2 * j + 1], inv));
      unsigned char* o = out + static_cast<int64_t>(g) * kVec;
      if (p.vec_y != 0 && count == kVec) {
        *reinterpret_cast<uint2*>(o) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (j < count) o[j] = static_cast<unsigned char>(q[j / 2] >> (8 * (j & 1)));
      }
    }
  }
}

// Backward.  A block takes the rows b, b + blocks, ... and keeps its columns'
// sums of dy u in registers; they go to dw_part as one row a block (a row a
// warp where a warp takes a row), which norm_dw_kernel adds up in order.
template <int DT, int NG>
__global__ void __launch_bounds__(kMaxRowThreads) norm_bwd_kernel(const NormParams p) {
  using R = Row<DT>;
  __shared__ float red[2 * (kMaxRowThreads / kLanes)];
  const int tpr = p.row_threads;
  const int r = static_cast<int>(threadIdx.x) % tpr;
  const int64_t part = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  const int64_t parts = static_cast<int64_t>(gridDim.x) * (blockDim.x / tpr);
  RowReduce reduce{red, tpr / kLanes};
  float dw[NG][kVec];
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int j = 0; j < kVec; ++j) dw[i][j] = 0.0f;
  for (int64_t row = part; row < p.n_rows; row += parts) {
    const unsigned char* h = p.x + row * p.ld_x * R::EB;
    const unsigned char* dy = p.dy + row * p.ld_dy * R::EB;
    const float rstd = p.rstd[row];
    uint32_t wh[NG][R::kW], wd[NG][R::kW];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g >= p.groups) continue;
      const int count = min(kVec, p.width - g * kVec);
      R::load(h, g, count, wh[i]);
      R::load(dy, g, count, wd[i]);
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g >= p.groups) continue;
      float wt[kVec];
      load_weight<DT>(p.weight, p.weight_f32 != 0, g, min(kVec, p.width - g * kVec), wt);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float u = __fmul_rn(R::get(wh[i], j), rstd), d = R::get(wd[i], j);
        dot = __fmaf_rn(__fmul_rn(d, wt[j]), u, dot);
        dw[i][j] = __fmaf_rn(d, u, dw[i][j]);
      }
    }
    const float c = __fdiv_rn(reduce.sum(dot), static_cast<float>(p.width));
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int g = r + i * tpr;
      if (g >= p.groups) continue;
      const int count = min(kVec, p.width - g * kVec);
      float wt[kVec], v[kVec];
      load_weight<DT>(p.weight, p.weight_f32 != 0, g, count, wt);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float u = __fmul_rn(R::get(wh[i], j), rstd);
        v[j] = __fmul_rn(rstd, __fmaf_rn(-u, c, __fmul_rn(R::get(wd[i], j), wt[j])));
      }
      if (p.dh != nullptr) {
        uint32_t q[R::kW];
        R::load(p.dh + row * p.ld_dh * R::EB, g, count, q);
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = __fadd_rn(v[j], R::get(q, j));
      }
      uint32_t o[R::kW];
      R::pack(v, o);
      R::store(p.dx + row * p.ld_dx * R::EB, g, count, p.vec_dx != 0, o);
    }
  }
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int g = r + i * tpr;
    if (g >= p.groups) continue;
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (g * kVec + j < p.width) p.dw_part[part * p.width + g * kVec + j] = dw[i][j];
  }
}

// dw[c] = the parts' sum in a fixed order: warp w of the block adds parts w,
// w + 8, ... of its 32 columns in order, and the eight sums are added in order.
constexpr int kDwWarps = 8;

__global__ void __launch_bounds__(kDwWarps * kLanes) norm_dw_kernel(const float* __restrict__ part, int64_t parts,
                                                                    int width, float* __restrict__ dw) {
  __shared__ float sums[kDwWarps][kLanes];
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

// A row's threads and the groups each holds, by the width alone: a warp up to
// 1024 elements (four groups a lane), then the fewest threads, in powers of
// two up to 512, that hold the row in two groups each; past 8192 elements 512
// threads hold up to four.
void row_shape(int width, int* threads, int* per_thread) {
  const int groups = (width + kVec - 1) / kVec;
  if (groups <= kLanes * kMaxGroups) {
    *threads = kLanes;
  } else {
    int t = 2 * kLanes;
    while (t < kMaxRowThreads && t * 2 < groups) t *= 2;
    *threads = t;
  }
  const int need = (groups + *threads - 1) / *threads;
  *per_thread = need <= 1 ? 1 : need <= 2 ? 2 : 4;
}

// Threads of a block: one row, or eight rows of one warp each.
int block_threads(int row_threads) { return row_threads == kLanes ? 8 * kLanes : row_threads; }

typedef void (*NormKernel)(NormParams);

template <int MODE>
NormKernel fwd_kernel(int dtype, int ng) {
  switch (dtype) {
    case BIL_F32:
      return ng == 1 ? norm_fwd_kernel<BIL_F32, 1, MODE> : ng == 2 ? norm_fwd_kernel<BIL_F32, 2, MODE>
                                                                  : norm_fwd_kernel<BIL_F32, 4, MODE>;
    case BIL_BF16:
      return ng == 1 ? norm_fwd_kernel<BIL_BF16, 1, MODE> : ng == 2 ? norm_fwd_kernel<BIL_BF16, 2, MODE>
                                                                    : norm_fwd_kernel<BIL_BF16, 4, MODE>;
    default:
      return ng == 1 ? norm_fwd_kernel<BIL_F16, 1, MODE> : ng == 2 ? norm_fwd_kernel<BIL_F16, 2, MODE>
                                                                   : norm_fwd_kernel<BIL_F16, 4, MODE>;
  }
}

NormKernel bwd_kernel_of(int dtype, int ng) {
  switch (dtype) {
    case BIL_F32:
      return ng == 1 ? norm_bwd_kernel<BIL_F32, 1> : ng == 2 ? norm_bwd_kernel<BIL_F32, 2> : norm_bwd_kernel<BIL_F32, 4>;
    case BIL_BF16:
      return ng == 1 ? norm_bwd_kernel<BIL_BF16, 1>
                     : ng == 2 ? norm_bwd_kernel<BIL_BF16, 2> : norm_bwd_kernel<BIL_BF16, 4>;
    default:
      return ng == 1 ? norm_bwd_kernel<BIL_F16, 1> : ng == 2 ? norm_bwd_kernel<BIL_F16, 2> : norm_bwd_kernel<BIL_F16, 4>;
  }
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
  return aligned_to(weight, static_cast<size_t>(bil_internal::elem_bytes(weight_dtype))) ? BIL_OK : BIL_E_ALIGN;
}

int launch_fwd(NormKernel kernel, NormParams& p, cudaStream_t s) {
  const int threads = block_threads(p.row_threads);
  const int64_t rows_per_block = threads / p.row_threads;
  const int64_t grid = (p.n_rows + rows_per_block - 1) / rows_per_block;
  if (grid > INT32_MAX) return BIL_E_UNSUPPORTED;
  return launch_pdl(kernel, grid, threads, 0, s, 1, p) == cudaSuccess ? BIL_OK : BIL_E_CUDA;
}

// Blocks of the backward: four a multiprocessor, at most one a row (eight rows
// a block where a warp takes a row).
int64_t bwd_blocks(int64_t n_rows, int row_threads, int sms) {
  const int64_t rows_per_block = block_threads(row_threads) / row_threads;
  return std::max<int64_t>(1, std::min<int64_t>((n_rows + rows_per_block - 1) / rows_per_block,
                                                static_cast<int64_t>(sms) * 4));
}

// The backward's partial sums: one row of `width` a block, or a warp.
int bwd_parts(int64_t n_rows, int64_t width, int64_t* parts) {
  int sms = 0, smem = 0;
  if (int st = bil_internal::device_limits(&sms, &smem)) return st;
  int threads = 0, ng = 0;
  row_shape(static_cast<int>(width), &threads, &ng);
  *parts = bwd_blocks(n_rows, threads, sms) * (block_threads(threads) / threads);
  return BIL_OK;
}

}  // namespace

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
  p.weight_f32 = weight_dtype == BIL_F32;
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
  row_shape(p.width, &p.row_threads, &ng);
  return launch_fwd(fwd_kernel<kNormPlain>(dtype, ng), p, reinterpret_cast<cudaStream_t>(stream));
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
  p.weight_f32 = weight_dtype == BIL_F32;
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
  row_shape(p.width, &p.row_threads, &ng);
  return launch_fwd(fwd_kernel<kNormQuant>(dtype, ng), p, reinterpret_cast<cudaStream_t>(stream));
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
  row_shape(p.width, &p.row_threads, &ng);
  return launch_fwd(fwd_kernel<kQuantOnly>(dtype, ng), p, reinterpret_cast<cudaStream_t>(stream));
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
  p.weight_f32 = weight_dtype == BIL_F32;
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
  row_shape(p.width, &p.row_threads, &ng);
  const int threads = block_threads(p.row_threads);
  bwd_kernel_of(dtype, ng)<<<static_cast<unsigned>(parts / (threads / p.row_threads)), threads, 0, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return BIL_E_CUDA;
  norm_dw_kernel<<<static_cast<unsigned>((width + kLanes - 1) / kLanes), kDwWarps * kLanes, 0, s>>>(
      p.dw_part, parts, p.width, dweight);
  return cudaGetLastError() == cudaSuccess ? BIL_OK : BIL_E_CUDA;
}

}  // extern "C"
