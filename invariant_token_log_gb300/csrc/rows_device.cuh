// Rows of float32, bfloat16 or float16 in groups of 8 elements: loads and stores
// of rows that may start anywhere, and the host's checks of their operands.
// Shared by the norms, dropout and the embedding.
#pragma once

#include "../../include/bil.h"
#include "device_common.cuh"
#include "internal.h"
#include "layout.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace {

using bil_layout::kVec;

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

  // Values 2k and 2k + 1 as a packed pair.
  __device__ static __forceinline__ uint64_t pair(const uint32_t (&w)[kW], int k) { return pk(get(w, 2 * k), get(w, 2 * k + 1)); }

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
  __device__ __forceinline__ uint64_t pair(int k) const { return W::pair(w, k); }
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

// ---- host ----

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool rows_start_on(const void* p, int64_t n_rows, int64_t ld_bytes, size_t a) {
  return aligned_to(p, a) && (n_rows <= 1 || ld_bytes % static_cast<int64_t>(a) == 0);
}

// Rows' extent and alignment of one [n_rows, ld] operand of eb-byte elements.
int check_rows(const void* p, int64_t n_rows, int64_t width, int64_t ld, int eb) {
  if (ld < width) return BIL_E_INVALID_ARG;
  if (!bil_internal::extent_ok(n_rows, ld, eb)) return BIL_E_UNSUPPORTED;
  if (n_rows > 0 && p == nullptr) return BIL_E_INVALID_ARG;
  if (!aligned_to(p, static_cast<size_t>(eb))) return BIL_E_ALIGN;
  return BIL_OK;
}

// The rows' path: `full` says that every row starts on a 16-byte boundary.
int row_path(int64_t width, bool full, bool same_type) {
  if (!full || width % kVec != 0) return same_type ? kAnyRows : kAnyRowsF32Weight;
  return same_type ? kFullRows : kFullRowsF32Weight;
}

}  // namespace
