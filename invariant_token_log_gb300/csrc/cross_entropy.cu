// The LM head's projection with softmax cross entropy, and the gradients of the
// hidden states and the weight, without the logits.  The C ABI is declared in
// include/bil.h.
//
//     z = hidden . weight^T,   lse_r = log sum_c exp(z_rc)
//     loss_r = lse_r - (1 - e) z_rt - (e / V) sum_c z_rc + f lse_r^2
//     dz_rc = g_r ((1 + 2 f lse_r) exp(z_rc - lse_r) - (1 - e) [c = t] - e / V)
//     dhidden = dz . weight,   dweight = dz^T . hidden
// over the rows whose target is not ignored.  Those are copied together first, and
// everything after works on them alone: an ignored row costs nothing, and what it
// holds, a NaN too, reaches no result.  Their number stays on the device: the
// kernels are launched for every row and stop behind the last.
//
// The forward keeps a maximum, a sum of exponentials (and of logits, with e > 0) for
// each row and 128 columns, out of a matrix product's accumulators, and joins them.
// The backward goes over the vocabulary in pieces: a piece's logits are computed
// again and leave the accumulators as dz in 16 bits, [rows, piece], whose two
// products follow; dhidden is added up over the pieces in float32.  So the scratch is
// a piece wide however large the vocabulary is, for four products in place of three.
//
// dz is stored times 2^12 / max_r |g_r (1 - e)| and the products' results are scaled
// back.  With the mean's 1/N in them the values would lie among float16's subnormals;
// and where all rows have one g, the -g (1 - e) at a target, the largest value of
// nearly every row, is -2^12 to the bit: as any other number it would carry the same
// rounding error, up to 2^-9, into every row.
//
// The tensor cores round an accumulator towards zero at each step of 16 products: of
// K = 4096 in one accumulation a logit comes out 4e-6 of itself too small, and every
// lse with it (the mean loss 2.7e-6 of itself, 7e-7 at K = 1104).  So a logit is
// accumulated in even segments of at most 16 K blocks, whose sums are added up in float32
// in the epilogue's registers: the error goes with a segment's steps, 8e-7 of the loss
// at any K (with 12 blocks 6e-7, and 3% more time at 4096 x 151936 x 4096, with 16 0.2%).
// (The gradients' products, rounded to 16 bits, are one accumulation.)
//
// One GEMM body, C = A . B^T on pairs of blocks (cta_group::2, 256 x 256 a pair, K
// blocks of 64 in a ring of six stages, two accumulators in tensor memory, so that a
// tile's epilogue runs under the next tile's products):
//   warp 0      copies: this block's 128 rows of A and 128 of B (K-major in one box,
//               MN-major in two of 64);
//   warp 1      of the pair's first block: issues the products;
//   warps 2-9   epilogue: a quarter of the block's rows and half of the columns each;
//               what it stores goes through two boxes of 32 128-byte lines a warp and TMA
//               (a stage of the ring is theirs).

#include "launch.cuh"
#include "tc_device.cuh"

#include <cuda_fp16.h>

#include <cmath>

namespace {

__device__ unsigned int g_watchdog_xent;

constexpr unsigned kWatchAccFull = 32u;    // as linear.cu's
constexpr unsigned kWatchStageFree = 64u;
constexpr unsigned kWatchMma = 128u;
constexpr unsigned kWatchOwnDrain = 256u;

constexpr int kMaxStages = 6;
constexpr unsigned kStageBytes = 2 * kStageABytes;  // 128 rows of A, 128 of B
constexpr int kUnitRows = 2 * kBM;                  // of a pair
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int kHalf = kBN / 2;                      // columns of an epilogue warp
constexpr int kSegment = 16;                        // K blocks of an accumulation, at most (see below)
constexpr uint32_t kBoxBytes = 32 * 128;            // of a store: 32 rows of a 128-byte line
constexpr uint32_t kStagingBytes = 2 * kBoxBytes;   // of a warp

struct alignas(8) PairSmem {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};

// kProducts: two products in one launch, dhidden's (float32, stored or added to what is there) and dweight's.
enum Epilogue { kStats = 0, kGrad = 1, kProducts = 2 };
constexpr size_t kRingBytes = (kMaxStages - 1) * size_t(kStageBytes) + kEpiWarps * size_t(kStagingBytes);
static_assert(kRingBytes >= kMaxStages * size_t(kStageBytes), "either layout");
constexpr size_t kSmemBytes = 1024 + kRingBytes + sizeof(PairSmem);
static_assert(kSmemBytes <= 227 * 1024, "a block's shared memory");

struct GemmParams {
  const int* n_active;   // rows of hidden that count
  int m_rows;            // rows of A; -1: n_active
  int num_n;             // column tiles
  int k_blocks;          // -1: of n_active
  int splits;            // of K, each with a slice of C of its own
  int m_group;           // row units of a raster group
  int64_t cols;          // columns of C
  int c_rows;            // rows of it (of a slice) that may be stored
  uint32_t idesc;
  const int* targets;    // of the rows that count: the target, -1 for none
  int64_t col0;          // vocabulary column of column 0
  // kStats: [column half-tiles, ld_part]
  float* part_max;
  float* part_sum;
  float* part_z;         // NULL: not needed
  int64_t ld_part;
  float* target_logit;
  // kGrad
  const float4* coef;    // of a row: a, b, c, lse:  dz = a exp(z - lse) - c - [c = t] b
  // kProducts
  const float* scale;    // NULL: 1
  int slice_rows;
  int add;
};

__device__ __forceinline__ void umma_f16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16 columns of this thread's tensor-memory lane, waited for (few registers beside the sums that they are added to).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// As tma_store_2d, added to what is there.
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, int c0, int c1, const void* src) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(smem_u32(src))
               : "memory");
}
// A warp's box of 32 rows of 128 bytes, a lane's row in eight 16-byte words which lie
// where TMA's 128-byte swizzle has them (word j of row i at j ^ (i mod 8): eight lanes'
// writes meet eight different banks), handed to TMA for column x, row y.  Two buffers
// in turn.
__device__ __forceinline__ void put_box(unsigned char* staging, const CUtensorMap* map, int x, int y, int lane,
                                        uint32_t& issued, const uint32_t (&w)[32], bool add) {
  unsigned char* box = staging + (issued & 1u) * kBoxBytes;
  if (lane == 0) bulk_wait_read_1();
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (add)
      tma_add_2d(map, x, y, box);
    else
      tma_store_2d(map, x, y, box);
    bulk_commit();
  }
  ++issued;
}

// Two values rounded to the 16-bit type, the first in the low half.
template <int DT>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (DT == BIL_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// What a launch works on, from the number of rows that count.
struct Shape {
  int active, m_rows, num_m, k_blocks, k_split;
  int64_t per_split, total;
  __device__ __forceinline__ explicit Shape(const GemmParams& p) {
    active = *p.n_active;
    m_rows = p.m_rows < 0 ? active : p.m_rows;
    num_m = (m_rows + kUnitRows - 1) / kUnitRows;
    k_blocks = p.k_blocks < 0 ? (active + kBK - 1) / kBK : p.k_blocks;
    k_split = (k_blocks + p.splits - 1) / p.splits;
    per_split = static_cast<int64_t>(num_m) * p.num_n;
    total = per_split * p.splits;
  }
  __device__ __forceinline__ void unit(const GemmParams& p, int64_t u, int& m, int& n, int& split, int& k0, int& k1) const {
    split = p.splits == 1 ? 0 : static_cast<int>(u / per_split);
    unit_coords(u - split * per_split, num_m, p.num_n, p.m_group, m, n);
    k0 = split * k_split;
    k1 = min(k_blocks, k0 + k_split);
  }
};

// The statistics of one row's 128 columns (vcols of them exist), from the accumulator in registers:
//   mx = max z,  s = sum 2^((z - mx) log2 e) in eight slots, and with SUM the sum of z in eight slots.
template <bool SUM, bool CUT>
__device__ __forceinline__ void half_stats(const uint32_t (&r)[4][kChunk], int vcols, float& mx, float& s, float& zs) {
  float m8[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) m8[j] = -INFINITY;
  uint64_t z2[4] = {0, 0, 0, 0}, a2[4] = {0, 0, 0, 0};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
#pragma unroll
    for (int j = 0; j < kChunk; ++j)
      if (!CUT || c * kChunk + j < vcols) m8[j % 8] = fmaxf(m8[j % 8], __uint_as_float(r[c][j]));
    if (SUM) {
#pragma unroll
      for (int j = 0; j < kChunk; j += 2) {
        const float lo = !CUT || c * kChunk + j < vcols ? __uint_as_float(r[c][j]) : 0.0f;
        const float hi = !CUT || c * kChunk + j + 1 < vcols ? __uint_as_float(r[c][j + 1]) : 0.0f;
        z2[j / 2 % 4] = add2(z2[j / 2 % 4], pk(lo, hi));
      }
    }
  }
  mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])), fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
  const float shift = mx == -INFINITY ? 0.0f : mx;
  const uint64_t shift2 = pk(shift, shift), c2 = pk(kLog2e, kLog2e);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
#pragma unroll
    for (int j = 0; j < kChunk; j += 2) {
      const uint64_t z = static_cast<uint64_t>(r[c][j]) | (static_cast<uint64_t>(r[c][j + 1]) << 32);
      const uint64_t t = mul2(sub2(z, shift2), c2);
      float e0 = ex2_approx(lo_of(t)), e1 = ex2_approx(hi_of(t));
      if (CUT) {
        if (c * kChunk + j >= vcols) e0 = 0.0f;
        if (c * kChunk + j + 1 >= vcols) e1 = 0.0f;
      }
      a2[j / 2 % 4] = add2(a2[j / 2 % 4], pk(e0, e1));
    }
  }
  const uint64_t a = add2(add2(a2[0], a2[1]), add2(a2[2], a2[3]));
  s = __fadd_rn(lo_of(a), hi_of(a));
  const uint64_t z = add2(add2(z2[0], z2[1]), add2(z2[2], z2[3]));
  zs = SUM ? __fadd_rn(lo_of(z), hi_of(z)) : 0.0f;
}

struct Maps {
  CUtensorMap a, b, c;
};

// SUM: kStats the sums of z too.  DT: the 16-bit type of dz, or dweight's type.  The second product (kProducts alone)
// has its units behind the first's; the first's A is K-major, all else that kProducts reads MN-major.
template <int EPI, bool SUM, int DT>
__global__ void __launch_bounds__(kThreads, 1)
    xent_gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Maps maps2, const GemmParams p,
                     const GemmParams p2) {
  constexpr int kStages = EPI == kStats ? kMaxStages : kMaxStages - 1;  // the last is the boxes'
  extern __shared__ unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* staging = base + kStages * size_t(kStageBytes);  // (kStats: none)
  PairSmem& sm = *reinterpret_cast<PairSmem*>(base + kRingBytes);
  volatile int* abort = &sm.abort;
  const int warp = threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  const int rank = static_cast<int>(cluster_rank());

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.acc_full[b], 1);
      mbar_init(&sm.acc_empty[b], 2 * kEpiWarps);
    }
    mbar_init(&sm.mma_done, 1);
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();  // both blocks' barriers and tensor memory are there
  tc_fence_after();
  const uint32_t tmem_base = sm.tmem_base;
  griddep_wait();
  griddep_launch_dependents();
  asm volatile("fence.proxy.async;" ::: "memory");  // what the kernels before stored, before TMA reads it

  const Shape shape(p), shape2(p2);
  // K blocks of a segment: as even as can be.
  const int segments = (shape.k_blocks + kSegment - 1) / kSegment;
  const int segment = EPI == kProducts ? INT32_MAX : (shape.k_blocks + segments - 1) / max(1, segments);
  const int64_t total = shape.total + (EPI == kProducts ? shape2.total : 0);
  auto unit = [&](int64_t u, int& m, int& n, int& split, int& k0, int& k1) {  // true: of the second product
    const bool second = EPI == kProducts && u >= shape.total;
    if (second)
      shape2.unit(p2, u - shape.total, m, n, split, k0, k1);
    else
      shape.unit(p, u, m, n, split, k0, k1);
    return second;
  };
  const int64_t pair0 = blockIdx.x / 2, pairs = gridDim.x / 2;

  if (warp == 0) {
    if (lane == 0) {
      // ---- this block's half of the pair's copies ----
      int64_t it = 0;
      bool ok = true;
      for (int64_t u = pair0; u < total && ok; u += pairs) {
        int m, n, split, k0, k1;
        const bool second = unit(u, m, n, split, k0, k1);
        const CUtensorMap* tmap_a = second ? &maps2.a : &maps.a;
        const CUtensorMap* tmap_b = second ? &maps2.b : &maps.b;
        const int a_row = (2 * m + rank) * kBM, b_row = n * kBN + rank * kHalf;
        for (int kb = k0; kb < k1; ++kb, ++it) {
          const int s = static_cast<int>(it % kStages);
          const unsigned ph = static_cast<unsigned>((it / kStages) & 1);
          if (!thread_wait_watch(&sm.empty[s], ph ^ 1u, abort, kWatchStageFree, &g_watchdog_xent, true)) {
            ok = false;
            break;
          }
          const uint32_t bar = cluster_smem(&sm.full[s], 0);
          if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * kStageBytes);
          unsigned char* a_dst = base + s * size_t(kStageBytes);
          unsigned char* b_dst = a_dst + kStageABytes;
          if (second) {
            tma_load_2d_pair(a_dst, tmap_a, a_row, kb * kBK, bar);
            tma_load_2d_pair(a_dst + kMnBoxBytes, tmap_a, a_row + kMnBox, kb * kBK, bar);
          } else {
            tma_load_2d_pair(a_dst, tmap_a, kb * kBK, a_row, bar);
          }
          if (EPI == kProducts) {
            tma_load_2d_pair(b_dst, tmap_b, b_row, kb * kBK, bar);
            tma_load_2d_pair(b_dst + kMnBoxBytes, tmap_b, b_row + kMnBox, kb * kBK, bar);
          } else {
            tma_load_2d_pair(b_dst, tmap_b, kb * kBK, b_row, bar);
          }
        }
      }
      // The leader waits (bounded, whatever happened) for the pair's copies still in flight; both stay until the
      // leader's last commits have arrived here (see linear.cu's pairs).
      const int64_t last = it > kStages ? it - kStages : 0;
      if (rank == 0) {
        for (int64_t i = last; i < it; ++i) {
          if (!thread_wait_watch(&sm.full[i % kStages], static_cast<unsigned>((i / kStages) & 1), abort, kWatchOwnDrain,
                                 &g_watchdog_xent, false))
            break;
        }
      }
      for (int64_t i = last; i < it; ++i) {
        if (!thread_wait_watch(&sm.empty[i % kStages], static_cast<unsigned>((i / kStages) & 1), abort, kWatchOwnDrain,
                               &g_watchdog_xent, false))
          break;
      }
      if (rank != 0) thread_wait_watch(&sm.mma_done, 0u, abort, kWatchOwnDrain, &g_watchdog_xent, false);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ---- the pair's products ----
      int64_t it = 0;
      int local = 0;
      bool ok = true;
      for (int64_t u = pair0; u < total && ok; u += pairs) {
        int m, n, split, k0, k1;
        const bool second = unit(u, m, n, split, k0, k1);
        const uint32_t idesc = second ? p2.idesc : p.idesc;
        int s0 = k0;
        do {  // a segment: an accumulator of its own
          const int s1 = k1 - s0 > segment ? s0 + segment : k1;
          const int b = local & 1;
          const unsigned use = static_cast<unsigned>(local >> 1);
          if (!thread_wait_cluster_watch(&sm.acc_empty[b], (use & 1u) ^ 1u, abort, kWatchMma, &g_watchdog_xent)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(b * kAccCols);
          for (int kb = s0; kb < s1; ++kb, ++it) {
            const int s = static_cast<int>(it % kStages);
            const unsigned ph = static_cast<unsigned>((it / kStages) & 1);
            if (!thread_wait_watch(&sm.full[s], ph, abort, kWatchMma, &g_watchdog_xent, true)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a_addr = smem_u32(base + s * size_t(kStageBytes)), b_addr = a_addr + kStageABytes;
#pragma unroll
            for (int k = 0; k < kBK / kUmmaK; ++k) {
              // a K step: 32 bytes along a K-major line, 16 lines of an MN-major box
              const uint64_t adesc = second ? smem_desc_mn(a_addr + k * kUmmaK * 128) : smem_desc(a_addr + k * kUmmaK * 2);
              const uint64_t bdesc =
                  EPI == kProducts ? smem_desc_mn(b_addr + k * kUmmaK * 128) : smem_desc(b_addr + k * kUmmaK * 2);
              umma_f16_pair(d_tmem, adesc, bdesc, idesc, kb != s0 || k != 0 ? 1u : 0u);
            }
            umma_commit_pair(&sm.empty[s]);
          }
          if (!ok) break;
          umma_commit_pair(&sm.acc_full[b]);
          ++local;
          s0 = s1;
        } while (s0 < k1);
      }
      umma_commit_pair(&sm.mma_done);  // every product completes before the blocks free tensor memory
      thread_wait_watch(&sm.mma_done, 0u, abort, kWatchOwnDrain, &g_watchdog_xent, false);
    }
  } else {
    // ---- epilogue: a quarter of this block's 128 rows, half of the columns ----
    const int q = warp & 3, half = (warp - 2) / 4;
    unsigned char* boxes = staging + (warp - 2) * size_t(kStagingBytes);
    const float scale2 = EPI == kProducts ? *p2.scale : 1.0f;
    int local = 0;
    uint32_t issued = 0;
    for (int64_t u = pair0; u < total; u += pairs) {
      int m, n, split, k0, k1;
      const bool second = unit(u, m, n, split, k0, k1);
      const int row0 = (2 * m + rank) * kBM + q * 32, row = row0 + lane;
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * kHalf);
      const int64_t first = static_cast<int64_t>(n) * kBN + half * kHalf;  // column of C
      const int vcols = static_cast<int>(p.cols - first < kHalf ? p.cols - first : kHalf);  // <= 0: none
      auto release = [&](int b) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0)
          asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                           cluster_smem(&sm.acc_empty[b], 0))
                       : "memory");
      };
      float4 coef = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      int tcol = -1;  // the target's column in this warp's half
      if constexpr (EPI != kProducts) {
        if (row < shape.m_rows) {
          if (EPI == kGrad) coef = p.coef[row];
          const int64_t t = p.targets[row];
          if (t >= p.col0 + first && t < p.col0 + first + vcols) tcol = static_cast<int>(t - p.col0 - first);
        }
      }
      // The warp's columns into registers, a segment after the other, and the accumulator back at once: where K is
      // short the next tile's products wait for it (64 x 151936 x 4096, the whole backward: 757 us, and 783 with the
      // accumulator held to the end).
      uint32_t acc[4][kChunk];
      if constexpr (EPI != kProducts) {
#pragma unroll
        for (int c = 0; c < 4 * kChunk; ++c) acc[c / kChunk][c % kChunk] = 0u;
      }
      bool ok = true;
      int s0 = k0;
      do {
        const int s1 = k1 - s0 > segment ? s0 + segment : k1;
        const int b = local & 1;
        const unsigned use = static_cast<unsigned>(local >> 1);
        ok = warp_wait_watch(&sm.acc_full[b], use & 1u, abort, kWatchAccFull, &g_watchdog_xent);
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = taddr + static_cast<uint32_t>(b * kAccCols);
        if constexpr (EPI == kProducts) {
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32_issue(at + c * kChunk, acc[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_wait(acc[c]);
        } else {
#pragma unroll
          for (int c = 0; c < 4 * kChunk; c += 16) {
            uint32_t r[16];
            tmem_ld16(at + c, r);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              uint32_t& a = acc[c / kChunk][c % kChunk + j];
              a = __float_as_uint(__fadd_rn(__uint_as_float(a), __uint_as_float(r[j])));
            }
          }
        }
        release(b);
        ++local;
        s0 = s1;
      } while (s0 < k1);
      if (!ok) break;
      if constexpr (EPI == kStats) {
        if (row0 >= shape.m_rows || vcols <= 0) continue;
        if (__any_sync(0xffffffffu, tcol >= 0)) {
          float tl = 0.0f;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < kChunk; ++j)
              if (c * kChunk + j == tcol) tl = __uint_as_float(acc[c][j]);
          if (tcol >= 0) p.target_logit[row] = tl;
        }
        float mx, s, zs;
        if (vcols == kHalf)
          half_stats<SUM, false>(acc, vcols, mx, s, zs);
        else
          half_stats<SUM, true>(acc, vcols, mx, s, zs);
        if (row < shape.m_rows) {
          const int64_t at = (2 * static_cast<int64_t>(n) + half) * p.ld_part + row;
          p.part_max[at] = mx;
          p.part_sum[at] = s;
          if (SUM) p.part_z[at] = zs;
        }
      } else {
        // dz has zeros up to the end of a K block of the rows, which the product with them reads.
        const int rows = EPI == kGrad ? min(p.c_rows, (shape.m_rows + kBK - 1) / kBK * kBK)
                                      : second ? shape2.m_rows : shape.m_rows;
        const int chunks = vcols <= 0 || row0 >= rows ? 0 : (vcols + kChunk - 1) / kChunk;
        const bool none = EPI == kGrad && coef.x == 0.0f && coef.y == 0.0f && coef.z == 0.0f;
        const bool wide = EPI == kProducts && (DT == BIL_F32 || !second);  // 32 columns a box, not 64
        const int x0 = static_cast<int>(first), y = (second ? 0 : split * p.slice_rows) + row0;
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < kHalf / kChunk; ++c) {
          uint32_t (&r)[kChunk] = acc[c];
          if (EPI == kProducts && k0 >= k1) {  // a sum over nothing
#pragma unroll
            for (int j = 0; j < kChunk; ++j) r[j] = 0u;
          }
          if (c >= chunks + (wide ? 0 : chunks & 1)) continue;  // (a box begun is filled)
          if constexpr (EPI == kGrad) {
            const int t = tcol - c * kChunk;
#pragma unroll
            for (int j = 0; j < kChunk; j += 2) {
              float d[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float e = contract_exp(__fsub_rn(__uint_as_float(r[j + k]), coef.w));
                d[k] = __fmaf_rn(coef.x, e, -coef.z);
                if (j + k == t) d[k] = __fsub_rn(d[k], coef.y);
                if (none) d[k] = 0.0f;
              }
              w[c % 2 * 16 + j / 2] = pack16<DT>(d[0], d[1]);
            }
            if (c % 2 == 1) put_box(boxes, &maps.c, x0 + (c - 1) * kChunk, y, lane, issued, w, false);
          } else if (!second) {
            put_box(boxes, &maps.c, x0 + c * kChunk, y, lane, issued, r, p.add != 0);
          } else if constexpr (DT == BIL_F32) {
#pragma unroll
            for (int j = 0; j < kChunk; ++j) w[j] = __float_as_uint(__fmul_rn(__uint_as_float(r[j]), scale2));
            put_box(boxes, &maps2.c, x0 + c * kChunk, y, lane, issued, w, false);
          } else {
#pragma unroll
            for (int j = 0; j < kChunk; j += 2)
              w[c % 2 * 16 + j / 2] =
                  pack16<DT>(__fmul_rn(__uint_as_float(r[j]), scale2), __fmul_rn(__uint_as_float(r[j + 1]), scale2));
            if (c % 2 == 1) put_box(boxes, &maps2.c, x0 + (c - 1) * kChunk, y, lane, issued, w, false);
          }
        }
      }
    }
    if (lane == 0 && issued != 0) bulk_wait_all();  // the boxes stay in use until then
  }

  tc_fence_before();
  __syncwarp();
  cluster_sync();  // neither block leaves while the other may still reach into it
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols)
                 : "memory");
  }
}

// ---------------------------------------------------------------------------
// The rows that count.
// ---------------------------------------------------------------------------

enum Reduction { kNone = 0, kMean = 1, kSum = 2 };

struct RowsParams {
  const int64_t* targets;
  int64_t ignore_index, vocab;
  int n;
  int* n_active;
  int* rows;          // the row of each that counts
  int* targets_out;   // its target; -1: outside the vocabulary
  // forward: what ignored rows give
  float* lse;         // [n]
  float* loss;        // [n] or NULL
  // backward
  const float* lse_in;
  const float* grad;  // one, or one a row
  int reduction;
  float smoothing, z_loss;
  int* place;         // [n] each row's place among those that count, -1: none
  float4* coef;       // by place (see GemmParams)
  float* scale;       // of the products' results
  // the copy of the rows that count (xent_gather_kernel's, or this kernel's where the rows are few)
  const unsigned char* hidden;
  int64_t ld_bytes;
  int width;
  unsigned char* compact;
  unsigned* done;     // forward: blocks of the join that are through, set to 0
};

// Row c of the copy, from row r of hidden; r < 0: zeros.
__device__ __forceinline__ void copy_row(const RowsParams& p, int r, int c, int thread, int threads) {
  const int units = p.width / 8, tail = p.width % 8, pitch = (p.width + 7) / 8 * 16;
  uint4* dst = reinterpret_cast<uint4*>(p.compact + static_cast<int64_t>(c) * pitch);
  if (r >= 0) {
    const uint4* src = reinterpret_cast<const uint4*>(p.hidden + r * p.ld_bytes);
    for (int i = thread; i < units; i += threads) dst[i] = src[i];
    if (thread < tail)  // nothing is read behind a row
      reinterpret_cast<uint16_t*>(dst + units)[thread] = reinterpret_cast<const uint16_t*>(src + units)[thread];
  } else {
    for (int i = thread; i < pitch / 16; i += threads) dst[i] = make_uint4(0u, 0u, 0u, 0u);
  }
}

constexpr int kRowsThreads = 1024;
constexpr int kRowsPer = 8;
constexpr int kRowsShare = 128;  // of a block's rows, at most

__device__ __forceinline__ void row_coefs(const RowsParams& p, int r, int count, float4& c) {
  float g = p.grad[p.reduction == kNone ? r : 0];
  if (p.reduction == kMean) g = __fdiv_rn(g, static_cast<float>(count));
  const float lse = p.lse_in[r];
  c.x = __fmul_rn(g, __fmaf_rn(2.0f * p.z_loss, lse, 1.0f));
  c.y = __fmul_rn(g, __fsub_rn(1.0f, p.smoothing));
  c.z = __fdiv_rn(__fmul_rn(g, p.smoothing), static_cast<float>(p.vocab));
  c.w = lse;
}

// The rows keep their order.  One block; or, for at most kRowsThreads * kRowsPer rows,
// as many as there are SMs or rows, each of which finds every row's place, and copies its
// share of them (the first alone writes the lists).
template <bool BWD>
__global__ void __launch_bounds__(kRowsThreads) xent_rows_kernel(const RowsParams p) {
  __shared__ int counts[kRowsThreads / kLanes];
  __shared__ float maxima[kRowsThreads / kLanes];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % kLanes, warp = threadIdx.x / kLanes;
  const bool lists = blockIdx.x == 0, copies = p.compact != nullptr;
  const int share = (p.n + gridDim.x - 1) / gridDim.x, share0 = blockIdx.x * share;  // this block's rows
  __shared__ int place_of[kRowsShare];
  if (!BWD && lists && threadIdx.x == 0) *p.done = 0u;
  int total = 0;
  float times = 1.0f;
  if (BWD) {
    int count = 0;
#pragma unroll 8
    for (int64_t r = threadIdx.x; r < p.n; r += kRowsThreads) count += p.targets[r] != p.ignore_index ? 1 : 0;
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) counts[warp] = count;
    __syncthreads();
    total = __reduce_add_sync(0xffffffffu, counts[lane]);
    float most_a = 0.0f, most_b = 0.0f;
#pragma unroll 4
    for (int64_t r = threadIdx.x; r < p.n; r += kRowsThreads) {
      if (p.targets[r] == p.ignore_index) continue;
      float4 c;
      row_coefs(p, static_cast<int>(r), total, c);
      const float a = fabsf(c.x), b = fabsf(c.y);
      if (a < INFINITY) most_a = fmaxf(most_a, a);
      if (b < INFINITY) most_b = fmaxf(most_b, b);
    }
    auto across = [&](float& most) {
      for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      __syncthreads();
      if (lane == 0) maxima[warp] = most;
      __syncthreads();
      most = maxima[lane];
      for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    };
    across(most_a);
    across(most_b);
    // (Where the smoothing leaves little on the target, the other terms are the larger.)
    const float most = most_a <= 8.0f * most_b ? most_b : most_a;
    const bool usual = most > 1e-30f && most < 1e30f;
    times = usual ? __fdiv_rn(4096.0f, most) : most >= 1e30f ? 1e-30f : most > 0.0f ? 1e30f : 1.0f;
    if (lists && threadIdx.x == 0) *p.scale = usual ? __fdiv_rn(most, 4096.0f) : most >= 1e30f ? 1e30f : most > 0.0f ? 1e-30f : 1.0f;
    __syncthreads();
  }
  int before = 0;  // rows that count in the chunks so far
  for (int64_t first = 0; first < p.n; first += kRowsThreads * kRowsPer) {
    const int64_t r0 = first + threadIdx.x * kRowsPer;
    int64_t t[kRowsPer];
    int mine = 0;
#pragma unroll
    for (int j = 0; j < kRowsPer; ++j) {
      t[j] = r0 + j < p.n ? p.targets[r0 + j] : p.ignore_index;
      mine += t[j] != p.ignore_index ? 1 : 0;
    }
    int upto = mine;
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == kLanes - 1) counts[warp] = upto;
    __syncthreads();
    const int c = counts[lane];
    const int all = __reduce_add_sync(0xffffffffu, c);
    int at = before + upto - mine + __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
#pragma unroll
    for (int j = 0; j < kRowsPer; ++j) {
      const int64_t r = r0 + j;
      if (r >= p.n) continue;
      const bool counts_in = t[j] != p.ignore_index;
      if (copies && r >= share0 && r < share0 + share) place_of[r - share0] = counts_in ? at : -1;
      if (!lists) {
        at += counts_in ? 1 : 0;
        continue;
      }
      const bool bad = t[j] < 0 || t[j] >= p.vocab;
      if (BWD) p.place[r] = counts_in ? at : -1;
      if (!counts_in) {
        if (!BWD) {
          if (p.lse != nullptr) p.lse[r] = 0.0f;
          if (p.loss != nullptr) p.loss[r] = 0.0f;
        }
        continue;
      }
      p.rows[at] = static_cast<int>(r);
      p.targets_out[at] = bad ? -1 : static_cast<int>(t[j]);
      if (BWD) {
        float4 c4;
        row_coefs(p, static_cast<int>(r), total, c4);
        c4.x = __fmul_rn(c4.x, times);
        c4.y = __fmul_rn(c4.y, times);
        c4.z = __fmul_rn(c4.z, times);
        if (bad) c4.x = __int_as_float(0x7fc00000);
        p.coef[at] = c4;
      }
      ++at;
    }
    before += all;
    __syncthreads();
  }
  if (lists && threadIdx.x == 0) *p.n_active = before;
  if (!copies) return;
  for (int k = warp; k < share && share0 + k < p.n; k += kRowsThreads / kLanes)
    if (place_of[k] >= 0) copy_row(p, share0 + k, place_of[k], lane, kLanes);
  const int end = min(p.n, (before + kUnitRows - 1) / kUnitRows * kUnitRows);
  for (int c = before + blockIdx.x * (kRowsThreads / kLanes) + warp; c < end; c += gridDim.x * (kRowsThreads / kLanes))
    copy_row(p, -1, c, lane, kLanes);
}

// The rows of hidden that count, one after the other; behind the last, zeros up to the end of its unit.
__global__ void __launch_bounds__(128) xent_gather_kernel(const RowsParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int active = *p.n_active;
  const int end = min(p.n, (active + kUnitRows - 1) / kUnitRows * kUnitRows);
  for (int c = blockIdx.x; c < end; c += gridDim.x) copy_row(p, c < active ? p.rows[c] : -1, c, threadIdx.x, 128);
}

// ---------------------------------------------------------------------------
// The forward's end: a row's statistics joined, its loss.
// ---------------------------------------------------------------------------

struct JoinParams {
  const int* n_active;
  const int* rows;
  const int* targets;
  const float* part_max;
  const float* part_sum;
  const float* part_z;
  const float* target_logit;
  int64_t ld_part, vocab;
  int parts;
  float smoothing, z_loss;
  float* lse;       // [n] NULL: not stored
  float* loss;      // [n] by row, or NULL
  float* row_loss;  // by place among the rows that count
  int reduction;
  float* total;     // the losses' sum or mean
  unsigned* done;
};

constexpr int kJoinSlices = 32;  // of a row's parts: a thread each, lanes along the rows

__global__ void __launch_bounds__(kJoinSlices * kLanes) xent_join_kernel(const JoinParams p) {
  __shared__ float sm[3][kJoinSlices][kLanes];
  griddep_wait();
  griddep_launch_dependents();
  const int active = *p.n_active;
  const int lane = threadIdx.x % kLanes, slice = threadIdx.x / kLanes;
  const int row = static_cast<int>(blockIdx.x) * kLanes + lane;
  if (blockIdx.x != 0 && static_cast<int>(blockIdx.x) * kLanes >= active) return;  // (over no rows: the first block)
  float m = -INFINITY, s = 0.0f, z = 0.0f;
  auto add = [&](float pm, float ps) {  // (m, s) and another part
    const float top = fmaxf(m, pm), at = top == -INFINITY ? 0.0f : top;
    s = __fadd_rn(__fmul_rn(s, contract_exp(__fsub_rn(m, at))), __fmul_rn(ps, contract_exp(__fsub_rn(pm, at))));
    m = top;
  };
  const int per = (p.parts + kJoinSlices - 1) / kJoinSlices;
  if (row < active) {
#pragma unroll 4
    for (int t = slice * per; t < min(p.parts, (slice + 1) * per); ++t) {
      const int64_t at = t * p.ld_part + row;
      add(p.part_max[at], p.part_sum[at]);
      if (p.part_z != nullptr) z = __fadd_rn(z, p.part_z[at]);
    }
  }
  sm[0][slice][lane] = m;
  sm[1][slice][lane] = s;
  sm[2][slice][lane] = z;
  __syncthreads();
  if (slice == 0 && row < active) {
    for (int k = 1; k < kJoinSlices; ++k) {
      add(sm[0][k][lane], sm[1][k][lane]);
      z = __fadd_rn(z, sm[2][k][lane]);
    }
    const float lse = __fadd_rn(m, logf(s));
    const int t = p.targets[row];
    float loss = __int_as_float(0x7fc00000);  // a target outside the vocabulary
    if (t >= 0) {
      const float tl = p.target_logit[row];
      if (p.smoothing == 0.0f) {
        loss = __fsub_rn(lse, tl);
      } else {
        // (1 - e) (lse - z_t) + e (lse - mean z)
        const float mean = __fdiv_rn(z, static_cast<float>(p.vocab));
        loss = __fmaf_rn(p.smoothing, __fsub_rn(lse, mean), __fmul_rn(__fsub_rn(1.0f, p.smoothing), __fsub_rn(lse, tl)));
      }
      loss = __fmaf_rn(__fmul_rn(p.z_loss, lse), lse, loss);
    }
    const int r = p.rows[row];
    if (p.lse != nullptr) p.lse[r] = lse;
    if (p.loss != nullptr)
      p.loss[r] = loss;
    else
      p.row_loss[row] = loss;
  }
  if (p.reduction == kNone) return;
  // The last block to come here adds up every row's loss, in an order that their number fixes.
  __shared__ bool last;
  __threadfence();
  __syncthreads();
  const unsigned blocks = static_cast<unsigned>(max(1, (active + kLanes - 1) / kLanes));
  if (threadIdx.x == 0) last = atomicAdd(p.done, 1u) == blocks - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  float sum = 0.0f;
#pragma unroll 4
  for (int i = threadIdx.x; i < active; i += kJoinSlices * kLanes) sum = __fadd_rn(sum, __ldcg(p.row_loss + i));
  for (int o = 16; o > 0; o >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
  if (lane == 0) sm[0][0][slice] = sum;
  __syncthreads();
  if (slice != 0) return;
  sum = sm[0][0][lane];
  for (int o = 16; o > 0; o >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
  if (lane == 0) *p.total = p.reduction == kMean ? __fdiv_rn(sum, static_cast<float>(max(active, 1))) : sum;
}

// The backward's end: dhidden's slices added in order, scaled, rounded, each row to its place; zeros where a row
// does not count.
template <int OT>
__global__ void __launch_bounds__(128) xent_spread_kernel(const float* __restrict__ slices, int splits, int64_t slice_rows,
                                                          int64_t ld, const int* __restrict__ place,
                                                          const float* __restrict__ scale, int n, int width, int chunks,
                                                          unsigned char* __restrict__ out, int64_t ld_out) {
  griddep_wait();
  griddep_launch_dependents();
  const float times = *scale;
  for (int64_t unit = blockIdx.x; unit < static_cast<int64_t>(n) * chunks; unit += gridDim.x) {
    const int r = static_cast<int>(unit / chunks);
    const int c = place[r];
    const int x = (static_cast<int>(unit % chunks) * 128 + static_cast<int>(threadIdx.x)) * 4;
    if (x < width) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (c >= 0) {
        const float* from = slices + c * ld + x;
        v = *reinterpret_cast<const float4*>(from);
#pragma unroll 8
        for (int s = 1; s < splits; ++s) {
          const float4 w = *reinterpret_cast<const float4*>(from + s * slice_rows * ld);
          v = make_float4(__fadd_rn(v.x, w.x), __fadd_rn(v.y, w.y), __fadd_rn(v.z, w.z), __fadd_rn(v.w, w.w));
        }
        v = make_float4(__fmul_rn(v.x, times), __fmul_rn(v.y, times), __fmul_rn(v.z, times), __fmul_rn(v.w, times));
      }
      if constexpr (OT == BIL_F32) {
        float* o = reinterpret_cast<float*>(out) + r * ld_out + x;
        if (x + 4 <= width) {
          *reinterpret_cast<float4*>(o) = v;
        } else {
          const float e[4] = {v.x, v.y, v.z, v.w};
          for (int j = 0; j < width - x; ++j) o[j] = e[j];
        }
      } else {
        uint16_t* o = reinterpret_cast<uint16_t*>(out) + r * ld_out + x;
        const uint2 w = make_uint2(pack16<OT>(v.x, v.y), pack16<OT>(v.z, v.w));
        if (x + 4 <= width) {
          *reinterpret_cast<uint2*>(o) = w;
        } else {
          for (int j = 0; j < width - x; ++j)
            o[j] = static_cast<uint16_t>((j < 2 ? w.x : w.y) >> (16 * (j & 1)));
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------

size_t round256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }
int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// tcgen05.mma kind::f16 of a pair: M = 256 (see linear.cu's make_idesc).
uint32_t pair_idesc(int dtype, bool a_mn, bool b_mn) {
  const uint32_t bf16 = dtype == BIL_BF16 ? 1u : 0u;
  return (1u << 4) | (bf16 << 7) | (bf16 << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(kBN >> 3) << 17) | (static_cast<uint32_t>(kUnitRows >> 4) << 24);
}

// The map of put_box's boxes: 32 rows of 128 bytes.
int make_box_map(CUtensorMap* map, void* ptr, int dtype, int64_t rows, int64_t cols, int64_t ld) {
  const int eb = dtype == BIL_F32 ? 4 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * eb};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / eb), 32};
  return encode_2d(map, map_type(dtype), ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE)
             ? BIL_OK
             : BIL_E_CUDA;
}

typedef void (*GemmKernel)(Maps, Maps, GemmParams, GemmParams);

// units: the launch's work at most.
int launch_gemm(GemmKernel kernel, const Maps& maps, const Maps& maps2, const GemmParams& p, const GemmParams& p2,
                int64_t units, cudaStream_t s) {
  int sms = 0, smem_optin = 0;
  if (int st = bil_internal::device_limits(&sms, &smem_optin)) return st;
  if (static_cast<size_t>(smem_optin) < kSmemBytes) return BIL_E_UNSUPPORTED;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes)) != cudaSuccess)
    return BIL_E_CUDA;
  const int64_t grid = 2 * std::max<int64_t>(1, std::min<int64_t>(units, sms / 2));
  return launch_pdl(kernel, grid, kThreads, kSmemBytes, s, 2, maps, maps2, p, p2) == cudaSuccess ? BIL_OK : BIL_E_CUDA;
}

// Row units of a raster group: of the products whose columns are the vocabulary, and of those whose columns are the
// hidden size.  (16384 x 151936 x 4096: the forward 11.88 ms with 16, 12.54 with 8, 12.37 with 32; the backward is the
// same within 1% with 4, 8 and 16.)
constexpr int kRowGroup = 16, kColumnGroup = 8;

// Slices of dhidden's product (its K is the piece): those that take the least time, in cycles of 512 for a K block of
// a unit and 3500 bytes for the slices' traffic (written, and read or added to, for each piece), if that is 5% less
// than one slice takes.  Few rows make few units: 64 x 32003 x 1104 has 5 of 501 K blocks for 76 pairs, in 15 slices
// 75 of 34; 2048 x 151936 x 4096 has 128, two rounds of 76, in 4 slices 512, seven rounds a quarter as long.
int dhidden_splits(int64_t n_rows, int64_t hidden_size, int64_t vocab, int64_t piece, int pairs) {
  const int64_t tiles = (n_rows + kUnitRows - 1) / kUnitRows * ((hidden_size + kBN - 1) / kBN);
  const int64_t k_blocks = (std::min(piece, vocab) + kBK - 1) / kBK;
  int best = 1;
  double least = 0.0;
  for (int s = 1; s <= 16 && s <= k_blocks && s * up(n_rows, kUnitRows) <= INT32_MAX; ++s) {
    const double rounds = static_cast<double>((tiles * s + pairs - 1) / pairs);
    const double cycles = rounds * static_cast<double>((k_blocks + s - 1) / s) * 512.0 +
                          s * static_cast<double>(n_rows) * static_cast<double>(hidden_size) * 8.0 / 3500.0;
    if (s == 1)
      least = 0.95 * cycles;
    else if (cycles < least) {
      least = cycles;
      best = s;
    }
  }
  return best;
}

// Columns of a piece: the vocabulary, or what keeps dz within a gigabyte (4096 at least), in as many tiles as give
// dweight's product whole rounds of the pairs.  (16384 x 151936 x 4096, the whole step: 47.8 ms in pieces of 9728,
// 47.4 of 19456, 47.2 of 38912 columns: each piece adds to dhidden in float32, and ends three products.)
int64_t piece_columns(int64_t n_rows, int64_t hidden_size, int64_t vocab, int64_t piece, int pairs) {
  if (piece == 0) {
    piece = (int64_t(1) << 29) / std::max<int64_t>(1, n_rows);
    if (piece >= vocab) return up(vocab, kBN);
    int64_t a = pairs, b = (hidden_size + kBN - 1) / kBN;
    while (b != 0) {
      const int64_t rest = a % b;
      a = b;
      b = rest;
    }
    const int64_t step = pairs / a * kBN;
    piece = piece >= step ? piece / step * step : std::max<int64_t>(4096, piece / kBN * kBN);
  }
  return up(std::min(piece, vocab), kBN);
}

struct FwdLayout {
  size_t rows, part, at_part, total;
  int64_t padded, parts;
};

FwdLayout fwd_layout(int64_t n, int64_t hidden_size, int64_t vocab, bool smoothing) {
  FwdLayout l;
  l.padded = up(n, kUnitRows);
  l.parts = (vocab + kHalf - 1) / kHalf;
  l.rows = round256(static_cast<size_t>(l.padded) * 4);
  l.part = round256(static_cast<size_t>(l.parts) * static_cast<size_t>(l.padded) * 4);
  // n_active | rows | targets | target logits | row losses | hidden | parts
  l.at_part = 256 + 4 * l.rows + round256(static_cast<size_t>(n) * static_cast<size_t>(up(hidden_size, 8)) * 2);
  l.total = l.at_part + (smoothing ? 3 : 2) * l.part;
  return l;
}

struct BwdLayout {
  size_t rows, coef, hidden, dz, total;
  int64_t padded, piece, ld_slice;
  int splits;
};

int bwd_layout(int64_t n, int64_t hidden_size, int64_t vocab, int64_t piece, BwdLayout* l) {
  int sms = 0, smem = 0;
  if (int st = bil_internal::device_limits(&sms, &smem)) return st;
  l->padded = up(n, kUnitRows);
  l->piece = piece_columns(n, hidden_size, vocab, piece, sms / 2);
  l->splits = dhidden_splits(n, hidden_size, vocab, l->piece, sms / 2);
  l->ld_slice = up(hidden_size, 8);
  l->rows = round256(static_cast<size_t>(l->padded) * 4);
  l->coef = round256(static_cast<size_t>(l->padded) * sizeof(float4));
  l->hidden = round256(static_cast<size_t>(n) * static_cast<size_t>(up(hidden_size, 8)) * 2);
  l->dz = round256(static_cast<size_t>(n) * static_cast<size_t>(l->piece) * 2);
  // n_active, scale | rows | targets | places | coefficients | hidden | dz | slices
  l->total = 256 + 3 * l->rows + l->coef + l->hidden + l->dz +
             round256(static_cast<size_t>(l->splits) * static_cast<size_t>(l->padded) * static_cast<size_t>(l->ld_slice) * 4);
  return BIL_OK;
}

int check_sizes(int dtype, int64_t n, int64_t hidden_size, int64_t vocab) {
  if (dtype != BIL_BF16 && dtype != BIL_F16) return BIL_E_DTYPE;
  if (n < 0 || hidden_size < 1 || vocab < 1) return BIL_E_INVALID_ARG;
  if (n > INT32_MAX - 65536 || hidden_size > (1 << 24) || vocab > INT32_MAX - 65536) return BIL_E_UNSUPPORTED;
  return bil_internal::extent_ok(n, (vocab + kHalf - 1) / kHalf, 4) ? BIL_OK : BIL_E_UNSUPPORTED;
}

// What both directions take.
int check_call(const void* hidden, const void* weight, int dtype, int64_t n, int64_t hidden_size, int64_t ld_hidden,
               int64_t vocab, int64_t ld_weight, const int64_t* targets, float smoothing, float z_loss, int reduction) {
  if (int st = check_sizes(dtype, n, hidden_size, vocab)) return st;
  if (ld_hidden < hidden_size || ld_weight < hidden_size) return BIL_E_INVALID_ARG;
  if (!(smoothing >= 0.0f && smoothing <= 1.0f) || !std::isfinite(z_loss)) return BIL_E_INVALID_ARG;
  if (reduction != kNone && reduction != kMean && reduction != kSum) return BIL_E_INVALID_ARG;
  if (!bil_internal::extent_ok(n, ld_hidden, 2) || !bil_internal::extent_ok(vocab, ld_weight, 2)) return BIL_E_UNSUPPORTED;
  if (weight == nullptr) return BIL_E_INVALID_ARG;
  if (!rows16(weight, ld_weight, 2)) return BIL_E_ALIGN;
  if (n == 0) return BIL_OK;
  if (hidden == nullptr || targets == nullptr) return BIL_E_INVALID_ARG;
  if (!rows16(hidden, ld_hidden, 2) || !aligned_to(targets, 8)) return BIL_E_ALIGN;
  return BIL_OK;
}

// The lists and the copy of the rows that count.
template <bool BWD>
int launch_rows(const RowsParams& r, int sms, cudaStream_t s) {
  const int blocks = std::min(r.n, sms);
  if (r.n <= kRowsThreads * kRowsPer && (r.n + blocks - 1) / blocks <= kRowsShare)
    return launch_pdl(xent_rows_kernel<BWD>, blocks, kRowsThreads, 0, s, 1, r) == cudaSuccess ? BIL_OK : BIL_E_CUDA;
  RowsParams lists = r;
  lists.compact = nullptr;
  if (launch_pdl(xent_rows_kernel<BWD>, 1, kRowsThreads, 0, s, 1, lists) != cudaSuccess) return BIL_E_CUDA;
  return launch_pdl(xent_gather_kernel, std::min<int64_t>(r.n, 1 << 20), 128, 0, s, 1, r) == cudaSuccess ? BIL_OK
                                                                                                        : BIL_E_CUDA;
}

}  // namespace

namespace bil_internal {

int xent_watchdog(unsigned int* flags, int clear) {
  if (cudaMemcpyFromSymbol(flags, g_watchdog_xent, sizeof(unsigned int)) != cudaSuccess) return BIL_E_CUDA;
  if (clear) {
    const unsigned int zero = 0;
    if (cudaMemcpyToSymbol(g_watchdog_xent, &zero, sizeof(unsigned int)) != cudaSuccess) return BIL_E_CUDA;
  }
  return BIL_OK;
}

}  // namespace bil_internal

extern "C" {

int bil_linear_cross_entropy_fwd_workspace_bytes(int64_t n_rows, int64_t hidden_size, int64_t vocab, int smoothing,
                                                 int64_t* bytes) {
  if (bytes == nullptr) return BIL_E_INVALID_ARG;
  if (int st = check_sizes(BIL_BF16, n_rows, hidden_size, vocab)) return st;
  *bytes = static_cast<int64_t>(fwd_layout(n_rows, hidden_size, vocab, smoothing != 0).total);
  return BIL_OK;
}

int bil_linear_cross_entropy_fwd(const void* hidden, const void* weight, int dtype, int64_t n_rows, int64_t hidden_size,
                                 int64_t ld_hidden, int64_t vocab, int64_t ld_weight, const int64_t* target_ids,
                                 int64_t ignore_index, float label_smoothing, float z_loss, int reduction, float* loss,
                                 float* lse, void* workspace, int64_t workspace_bytes, int validate,
                                 bil_stream_t stream) {
  bil_internal::NvtxRange nvtx_range("bil_linear_cross_entropy_fwd");
  if (int st = check_call(hidden, weight, dtype, n_rows, hidden_size, ld_hidden, vocab, ld_weight, target_ids,
                          label_smoothing, z_loss, reduction))
    return st;
  if (!aligned_to(loss, 4) || !aligned_to(lse, 4)) return BIL_E_ALIGN;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (n_rows == 0) {
    if (reduction == kNone) return BIL_OK;
    if (loss == nullptr) return BIL_E_INVALID_ARG;
    return cudaMemsetAsync(loss, 0, sizeof(float), s) == cudaSuccess ? BIL_OK : BIL_E_CUDA;
  }
  if (loss == nullptr || workspace == nullptr) return BIL_E_INVALID_ARG;
  if (!aligned_to(workspace, 256)) return BIL_E_ALIGN;
  const bool smooth = label_smoothing > 0.0f;
  const FwdLayout l = fwd_layout(n_rows, hidden_size, vocab, smooth);
  if (workspace_bytes < static_cast<int64_t>(l.total)) return BIL_E_INVALID_ARG;
  if (validate) {
    if (int st = bil_internal::check_targets_host(target_ids, n_rows, ignore_index, vocab, s)) return st;
  }
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  unsigned char* compact = ws + 256 + 4 * l.rows;
  Maps maps;
  if (int st = make_map(&maps.a, compact, dtype, n_rows, hidden_size, up(hidden_size, 8), kBM)) return st;
  if (int st = make_map(&maps.b, weight, dtype, vocab, hidden_size, ld_weight, kHalf)) return st;
  maps.c = maps.b;  // not used
  RowsParams r{};
  r.targets = target_ids;
  r.ignore_index = ignore_index;
  r.vocab = vocab;
  r.n = static_cast<int>(n_rows);
  r.n_active = reinterpret_cast<int*>(ws);
  r.rows = reinterpret_cast<int*>(ws + 256);
  r.targets_out = reinterpret_cast<int*>(ws + 256 + l.rows);
  r.lse = lse;
  r.loss = reduction == kNone ? loss : nullptr;
  r.hidden = static_cast<const unsigned char*>(hidden);
  r.ld_bytes = ld_hidden * 2;
  r.width = static_cast<int>(hidden_size);
  r.compact = compact;
  r.done = reinterpret_cast<unsigned*>(ws + 64);
  int sms = 0, smem = 0;
  if (int st = bil_internal::device_limits(&sms, &smem)) return st;
  if (int st = launch_rows<false>(r, sms, s)) return st;
  GemmParams p{};
  p.n_active = r.n_active;
  p.m_rows = -1;
  p.num_n = static_cast<int>((vocab + kBN - 1) / kBN);
  p.k_blocks = static_cast<int>((hidden_size + kBK - 1) / kBK);
  p.splits = 1;
  p.m_group = kRowGroup;
  p.cols = vocab;
  p.idesc = pair_idesc(dtype, false, false);
  p.targets = r.targets_out;
  p.part_max = reinterpret_cast<float*>(ws + l.at_part);
  p.part_sum = reinterpret_cast<float*>(ws + l.at_part + l.part);
  p.part_z = smooth ? reinterpret_cast<float*>(ws + l.at_part + 2 * l.part) : nullptr;
  p.ld_part = l.padded;
  p.target_logit = reinterpret_cast<float*>(ws + 256 + 2 * l.rows);
  if (int st = launch_gemm(smooth ? xent_gemm_kernel<kStats, true, 0> : xent_gemm_kernel<kStats, false, 0>, maps, maps, p, p,
                           l.padded / kUnitRows * p.num_n, s))
    return st;
  JoinParams j{};
  j.n_active = r.n_active;
  j.rows = r.rows;
  j.targets = r.targets_out;
  j.part_max = p.part_max;
  j.part_sum = p.part_sum;
  j.part_z = p.part_z;
  j.target_logit = p.target_logit;
  j.ld_part = l.padded;
  j.vocab = vocab;
  j.parts = static_cast<int>(l.parts);
  j.smoothing = label_smoothing;
  j.z_loss = z_loss;
  j.lse = lse;
  j.loss = r.loss;
  j.row_loss = reinterpret_cast<float*>(ws + 256 + 3 * l.rows);
  j.reduction = reduction;
  j.total = loss;
  j.done = r.done;
  return launch_pdl(xent_join_kernel, (n_rows + kLanes - 1) / kLanes, kJoinSlices * kLanes, 0, s, 1, j) == cudaSuccess
             ? BIL_OK
             : BIL_E_CUDA;
}

int bil_linear_cross_entropy_bwd_workspace_bytes(int64_t n_rows, int64_t hidden_size, int64_t vocab, int64_t piece,
                                                 int64_t* bytes) {
  if (bytes == nullptr || piece < 0) return BIL_E_INVALID_ARG;
  if (int st = check_sizes(BIL_BF16, n_rows, hidden_size, vocab)) return st;
  BwdLayout l;
  if (int st = bwd_layout(n_rows, hidden_size, vocab, piece, &l)) return st;
  *bytes = static_cast<int64_t>(l.total);
  return BIL_OK;
}

int bil_linear_cross_entropy_bwd(const void* hidden, const void* weight, int dtype, int64_t n_rows, int64_t hidden_size,
                                 int64_t ld_hidden, int64_t vocab, int64_t ld_weight, const int64_t* target_ids,
                                 int64_t ignore_index, float label_smoothing, float z_loss, int reduction,
                                 const float* lse, const float* grad_loss, int64_t piece, void* dhidden,
                                 int dhidden_dtype, int64_t ld_dhidden, void* dweight, int dweight_dtype,
                                 int64_t ld_dweight, void* workspace, int64_t workspace_bytes, bil_stream_t stream) {
  bil_internal::NvtxRange nvtx_range("bil_linear_cross_entropy_bwd");
  if (int st = check_call(hidden, weight, dtype, n_rows, hidden_size, ld_hidden, vocab, ld_weight, target_ids,
                          label_smoothing, z_loss, reduction))
    return st;
  for (int ot : {dhidden_dtype, dweight_dtype})
    if (ot != BIL_F32 && ot != dtype) return BIL_E_DTYPE;
  if (piece < 0 || (dhidden == nullptr && dweight == nullptr && n_rows > 0)) return BIL_E_INVALID_ARG;
  const int64_t eh = dhidden_dtype == BIL_F32 ? 4 : 2, ew = dweight_dtype == BIL_F32 ? 4 : 2;
  if (dhidden != nullptr) {
    if (ld_dhidden < hidden_size) return BIL_E_INVALID_ARG;
    if (!bil_internal::extent_ok(n_rows, ld_dhidden, eh)) return BIL_E_UNSUPPORTED;
    if (!rows16(dhidden, ld_dhidden, eh)) return BIL_E_ALIGN;
  }
  if (dweight != nullptr) {
    if (ld_dweight < hidden_size || dweight == weight) return BIL_E_INVALID_ARG;  // (the weight is read to the end)
    if (!bil_internal::extent_ok(vocab, ld_dweight, ew)) return BIL_E_UNSUPPORTED;
    if (!rows16(dweight, ld_dweight, ew)) return BIL_E_ALIGN;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (n_rows == 0) {  // dweight is a sum over no rows
    if (dweight == nullptr) return BIL_OK;
    return cudaMemset2DAsync(dweight, static_cast<size_t>(ld_dweight * ew), 0, static_cast<size_t>(hidden_size * ew),
                             static_cast<size_t>(vocab), s) == cudaSuccess
               ? BIL_OK
               : BIL_E_CUDA;
  }
  if (lse == nullptr || grad_loss == nullptr || workspace == nullptr) return BIL_E_INVALID_ARG;
  if (!aligned_to(lse, 4) || !aligned_to(grad_loss, 4) || !aligned_to(workspace, 256)) return BIL_E_ALIGN;
  BwdLayout l;
  if (int st = bwd_layout(n_rows, hidden_size, vocab, piece, &l)) return st;
  if (workspace_bytes < static_cast<int64_t>(l.total)) return BIL_E_INVALID_ARG;
  int sms = 0, smem = 0;
  if (int st = bil_internal::device_limits(&sms, &smem)) return st;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  unsigned char* at = ws + 256;
  auto take = [&](size_t bytes) {
    unsigned char* p = at;
    at += bytes;
    return p;
  };
  RowsParams r{};
  r.targets = target_ids;
  r.ignore_index = ignore_index;
  r.vocab = vocab;
  r.n = static_cast<int>(n_rows);
  r.n_active = reinterpret_cast<int*>(ws);
  r.scale = reinterpret_cast<float*>(ws + 128);
  r.rows = reinterpret_cast<int*>(take(l.rows));
  r.targets_out = reinterpret_cast<int*>(take(l.rows));
  r.place = reinterpret_cast<int*>(take(l.rows));
  r.coef = reinterpret_cast<float4*>(take(l.coef));
  unsigned char* compact = take(l.hidden);
  unsigned char* dz = take(l.dz);
  float* slices = reinterpret_cast<float*>(at);
  r.lse_in = lse;
  r.grad = grad_loss;
  r.reduction = reduction;
  r.smoothing = label_smoothing;
  r.z_loss = z_loss;
  const int64_t ld_compact = up(hidden_size, 8);

  // Of every piece: hidden, and dhidden's slices.
  Maps grad, dh, dw;
  if (int st = make_map(&grad.a, compact, dtype, n_rows, hidden_size, ld_compact, kBM)) return st;
  if (int st = operand_map(&dw.b, compact, dtype, hidden_size, n_rows, ld_compact, true, 0)) return st;
  if (int st = make_box_map(&dh.c, slices, BIL_F32, l.padded * l.splits, hidden_size, l.ld_slice)) return st;

  r.hidden = static_cast<const unsigned char*>(hidden);
  r.ld_bytes = ld_hidden * 2;
  r.width = static_cast<int>(hidden_size);
  r.compact = compact;
  if (int st = launch_rows<true>(r, sms, s)) return st;

  const int64_t row_units = l.padded / kUnitRows;
  const int num_h = static_cast<int>((hidden_size + kBN - 1) / kBN);
  for (int64_t col0 = 0; col0 < vocab; col0 += l.piece) {
    const int64_t cols = std::min(l.piece, vocab - col0);
    const int num_v = static_cast<int>((cols + kBN - 1) / kBN);
    const unsigned char* w = static_cast<const unsigned char*>(weight) + col0 * ld_weight * 2;
    if (int st = make_map(&grad.b, w, dtype, cols, hidden_size, ld_weight, kHalf)) return st;
    if (int st = make_box_map(&grad.c, dz, dtype, n_rows, cols, l.piece)) return st;
    if (int st = make_map(&dh.a, dz, dtype, n_rows, cols, l.piece, kBM)) return st;
    if (int st = operand_map(&dh.b, w, dtype, hidden_size, cols, ld_weight, true, 0)) return st;
    if (int st = operand_map(&dw.a, dz, dtype, cols, n_rows, l.piece, true, 0)) return st;
    dw.c = dw.a;
    if (dweight != nullptr) {
      unsigned char* out = static_cast<unsigned char*>(dweight) + col0 * ld_dweight * ew;
      if (int st = make_box_map(&dw.c, out, dweight_dtype, cols, hidden_size, ld_dweight)) return st;
    }
    GemmParams p{};
    p.n_active = r.n_active;
    p.splits = 1;
    // the piece's dz
    GemmParams z = p;
    z.m_rows = -1;
    z.num_n = num_v;
    z.k_blocks = static_cast<int>((hidden_size + kBK - 1) / kBK);
    z.m_group = kRowGroup;
    z.cols = cols;
    z.c_rows = r.n;
    z.idesc = pair_idesc(dtype, false, false);
    z.targets = r.targets_out;
    z.col0 = col0;
    z.coef = r.coef;
    if (int st = launch_gemm(dtype == BIL_BF16 ? xent_gemm_kernel<kGrad, false, BIL_BF16>
                                               : xent_gemm_kernel<kGrad, false, BIL_F16>,
                             grad, grad, z, z, row_units * num_v, s))
      return st;
    // dz . weight, K the piece's columns, and dz^T . hidden, K the rows
    p.num_n = num_h;
    p.m_group = kColumnGroup;
    p.cols = hidden_size;
    p.scale = r.scale;
    GemmParams p2 = p;
    p.m_rows = dhidden != nullptr ? -1 : 0;
    p.k_blocks = static_cast<int>((cols + kBK - 1) / kBK);
    p.splits = l.splits;
    p.idesc = pair_idesc(dtype, false, true);
    p.slice_rows = static_cast<int>(l.padded);
    p.add = col0 != 0;
    p2.m_rows = dweight != nullptr ? static_cast<int>(cols) : 0;
    p2.k_blocks = -1;
    p2.idesc = pair_idesc(dtype, true, true);
    GemmKernel k = dweight == nullptr || dweight_dtype == BIL_F32 ? xent_gemm_kernel<kProducts, false, BIL_F32>
                   : dweight_dtype == BIL_BF16                   ? xent_gemm_kernel<kProducts, false, BIL_BF16>
                                                                 : xent_gemm_kernel<kProducts, false, BIL_F16>;
    if (int st = launch_gemm(k, dh, dw, p, p2, row_units * num_h * l.splits + static_cast<int64_t>(num_v) * num_h, s))
      return st;
  }
  if (dhidden == nullptr) return BIL_OK;
  auto spread = dhidden_dtype == BIL_F32    ? xent_spread_kernel<BIL_F32>
                : dhidden_dtype == BIL_BF16 ? xent_spread_kernel<BIL_BF16>
                                            : xent_spread_kernel<BIL_F16>;
  const int chunks = static_cast<int>((hidden_size + 511) / 512);  // of a row, a block each
  return launch_pdl(spread, std::min<int64_t>(n_rows * chunks, 1 << 20), 128, 0, s, 1, static_cast<const float*>(slices), l.splits,
                    l.padded, l.ld_slice, static_cast<const int*>(r.place), static_cast<const float*>(r.scale), r.n,
                    static_cast<int>(hidden_size), chunks, static_cast<unsigned char*>(dhidden), ld_dhidden) == cudaSuccess
             ? BIL_OK
             : BIL_E_CUDA;
}

}  // extern "C"
