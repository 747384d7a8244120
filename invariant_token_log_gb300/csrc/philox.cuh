// The counter-based generator behind dropout's masks: Philox4x32-10 (J. Salmon,
// M. Moraes, R. Dror, D. Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// 2011).  A mask is a function of its seed, its step and an element's place, so
// the backward pass makes it again and nothing stores it.
//
// A group is 8 consecutive elements of a row, from a multiple of 8 on (the row's
// last may be cut off).  Group j of row r of [rows, width] has the counter
// (r * ceil(width / 8) + j, step), 64 bits each, lower word first, under the seed
// as key; its elements take the eight 16-bit parts of the four result words, each
// word's lower part first.  An element is dropped when its part is below
// border = p * 65536 rounded to nearest even, the others are multiplied by
// 65536 / (65536 - border): the share that stays is known to the bit, and so the
// mean of the outputs is the inputs'.  (16 bits and not 32: one call of about 55
// instructions serves 8 elements, which keeps the passes bound by memory.)
#pragma once

#include "../../include/bil.h"

#include <stdint.h>

#include <cmath>

namespace {

struct Dropout {
  const int64_t* rng;  // NULL, or two words on the device: the seed, and what is added to the step
  uint64_t seed, step;
  uint32_t border;
  float times;
};

// What a thread holds of it.
struct DropKey {
  uint2 key, step;
  __device__ __forceinline__ explicit DropKey(const Dropout& d) {
    uint64_t k = d.seed, s = d.step;
    if (d.rng != nullptr) {
      k = static_cast<uint64_t>(d.rng[0]);
      s += static_cast<uint64_t>(d.rng[1]);
    }
    key = make_uint2(static_cast<uint32_t>(k), static_cast<uint32_t>(k >> 32));
    step = make_uint2(static_cast<uint32_t>(s), static_cast<uint32_t>(s >> 32));
  }
  // the eight 16-bit parts of a group
  __device__ __forceinline__ uint4 bits(uint64_t group) const {
    uint4 c = make_uint4(static_cast<uint32_t>(group), static_cast<uint32_t>(group >> 32), step.x, step.y);
    uint2 k = key;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const uint32_t h0 = __umulhi(0xD2511F53u, c.x), l0 = 0xD2511F53u * c.x;
      const uint32_t h1 = __umulhi(0xCD9E8D57u, c.z), l1 = 0xCD9E8D57u * c.z;
      c = make_uint4(h1 ^ c.y ^ k.x, l1, h0 ^ c.w ^ k.y, l0);
      k.x += 0x9E3779B9u;
      k.y += 0xBB67AE85u;
    }
    return c;
  }
};

// The same for the threads of a block, in shared memory: the ten rounds' keys, made
// once (a quarter of a call's instructions), and the step.
struct DropKeys {
  uint2 key[10];
  uint2 step;
  __device__ __forceinline__ void make(const Dropout& d) {  // a barrier has to follow
    if (threadIdx.x >= 10) return;
    const DropKey k(d);
    key[threadIdx.x] = make_uint2(k.key.x + threadIdx.x * 0x9E3779B9u, k.key.y + threadIdx.x * 0xBB67AE85u);
    if (threadIdx.x == 0) step = k.step;
  }
  __device__ __forceinline__ uint4 bits(uint64_t group) const {
    uint4 c = make_uint4(static_cast<uint32_t>(group), static_cast<uint32_t>(group >> 32), step.x, step.y);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const uint32_t h0 = __umulhi(0xD2511F53u, c.x), l0 = 0xD2511F53u * c.x;
      const uint32_t h1 = __umulhi(0xCD9E8D57u, c.z), l1 = 0xCD9E8D57u * c.z;
      c = make_uint4(h1 ^ c.y ^ key[i].x, l1, h0 ^ c.w ^ key[i].y, l0);
    }
    return c;
  }
};

// Whether element j of a group stays.
__device__ __forceinline__ bool drop_keeps(const uint4& bits, int j, uint32_t border) {
  const uint32_t w = j < 2 ? bits.x : j < 4 ? bits.y : j < 6 ? bits.z : bits.w;
  return ((j & 1) ? w : w << 16) >= border << 16;  // (a 16-bit part in the upper half: what lies below does not count)
}

// ---- host ----

// The dropout of a call; p is checked here.
int make_dropout(double p, uint64_t seed, uint64_t step, const int64_t* rng, Dropout* d) {
  if (!(p >= 0.0 && p < 1.0)) return BIL_E_INVALID_ARG;
  const double border = std::nearbyint(p * 65536.0);
  if (border >= 65536.0) return BIL_E_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(rng) & 7u) != 0) return BIL_E_ALIGN;
  d->rng = rng;
  d->seed = seed;
  d->step = step;
  d->border = static_cast<uint32_t>(border);
  d->times = static_cast<float>(65536.0 / (65536.0 - border));
  return BIL_OK;
}

}  // namespace
