// Tensor-core building blocks of the GEMM kernels (linear.cu, cross_entropy.cu):
// tile sizes, shared-memory descriptors, TMA copies and stores, tensor-memory loads,
// pairs of blocks, and on the host the tensor maps.
#pragma once

#include "../../include/bil.h"
#include "device_common.cuh"
#include "internal.h"

#include <cuda.h>  // CUtensorMap and its enums (types only; the encoder is fetched at run time)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

namespace {

constexpr int kBM = 128;      // rows per tile: one tensor-memory lane per row
constexpr int kBN = 256;      // vocabulary columns per tile = the operator's tile width here
constexpr int kBK = 64;       // K per stage: 64 x 16 bits = one 128-byte swizzle row
constexpr int kUmmaK = 16;    // K of one tcgen05.mma kind::f16
constexpr unsigned kStageABytes = kBM * kBK * 2;  // 16 KB
constexpr int kAccCols = kBN;            // one 32-bit tensor-memory column per output column
constexpr uint32_t kTmemCols = 2 * kAccCols;  // two accumulator buffers: 512 columns
constexpr int kChunk = 32;               // columns per tensor-memory load
constexpr int kStoreBox = 32;  // rows and columns of one dZ store box: a warp's rows, one TMEM chunk
constexpr uint32_t kStoreBoxBytes = kStoreBox * kStoreBox * 2;           // 2 KB of 16-bit elements

// Shared-memory matrix descriptor of a K-major operand stored the way a TMA
// load with 128-byte swizzle writes it: rows of 128 bytes (64 elements of K),
// 8-row groups 1024 bytes apart (stride byte offset), start address >> 4 in
// bits 0-13, leading byte offset (unused for this layout) 16 bytes, the fixed
// 0b001 in bits 46-48, swizzle mode 2 (128 bytes) in bits 61-63.  The 8-row
// groups start on 1024-byte boundaries, so the base offset is 0; a K step
// within the 128-byte row advances the start address by 32 bytes.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(16 >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

// The same for an MN-major operand (rows contiguous in memory), as TMA loads
// with 128-byte swizzle write it in boxes of 64 rows x 64 K: each K index is
// one 128-byte line of 64 consecutive rows, 8 K indices make a 1024-byte
// swizzle atom (stride byte offset between the atoms along K), and the next
// 64 rows are the next box, kMnBoxBytes further on (leading byte offset).  A
// K step of 16 advances the start address by 16 lines = 2048 bytes, two whole
// atoms.
constexpr int kMnBox = 64;                                // rows (and K) per box of an MN-major operand
constexpr uint32_t kMnBoxBytes = kMnBox * kBK * 2;        // 8 KB
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(kMnBoxBytes >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

// One box from shared memory to global memory (the tensor map's box; parts
// past the matrix are not written), in this thread's current bulk group.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int c0, int c1, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Until at most one of this thread's bulk groups still reads shared memory.
__device__ __forceinline__ void bulk_wait_read_1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
// Until all of this thread's bulk groups have completed.
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 consecutive 32-bit columns of this thread's tensor-memory lane, waited
// for in the same statement (so no use of the registers can be scheduled
// before the data has arrived).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[kChunk]) {
  __syncwarp();  // the load is warp-wide (.sync.aligned): the warp must be converged
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// The same load without the wait, and the wait for every load issued so far
// (which hands out the registers of one of them, so that no use of these can be
// scheduled before it): what comes between the two runs while the data is on
// its way.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t (&r)[kChunk]) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[kChunk]) {
  __syncwarp();
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// Row tile m and column tile n of work unit u: groups of `group` row tiles;
// within a group the row tile varies fastest, so the blocks working at one
// time share a few B tiles (and their A tiles) through L2.
__device__ __forceinline__ void unit_coords(int64_t u, int num_m, int num_n, int group, int& m, int& n) {
  const int64_t per_group = static_cast<int64_t>(group) * num_n;
  const int g = static_cast<int>(u / per_group);
  const int r = static_cast<int>(u - g * per_group);
  const int m0 = g * group;
  const int gm = min(group, num_m - m0);
  n = r / gm;
  m = m0 + (r - n * gm);
}

// A warp hands one 2 KB box (32 rows of 64 bytes: 32 16-bit or 16 float32
// values per row) to TMA: each lane writes its row's four 16-byte words into
// the warp's next staging buffer (two, used in turn), and lane 0 stores the
// box at (column x, row y) of `map` once the store that used the buffer before
// has read it.  `issued` counts the warp's boxes.
__device__ __forceinline__ void store_box(unsigned char* staging, const CUtensorMap* map, int x, int y, int lane,
                                          uint32_t& issued, const uint32_t (&w)[16]) {
  unsigned char* box = staging + (issued & 1u) * kStoreBoxBytes;
  if (lane == 0) bulk_wait_read_1();
  __syncwarp();
  uint4* dst = reinterpret_cast<uint4*>(box + lane * 64);
#pragma unroll
  for (int j = 0; j < 4; ++j) dst[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  fence_proxy_async_smem();  // the writes above, before the bulk copy reads them
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, x, y, box);
    bulk_commit();
  }
  ++issued;
}

// ---- pairs of blocks (cta_group::2) ----

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The shared::cluster address of `p` (a shared variable of this block) in the block of rank `rank`.
__device__ __forceinline__ uint32_t cluster_smem(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// One box into this block's shared memory, completion counted on a barrier of either block of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
// Arrive once on `bar` in both blocks when every tcgen05 operation this thread issued so far has completed.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------

// cuTensorMapEncodeTiled, fetched from the driver at run time (no link-time
// dependency on the driver library).
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// Whether another try is worth it: the encoder wants a current context, and a thread that has made no runtime call yet
// (a backward pass's) has none until its device is set.
bool context_made() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess;
}

CUtensorMapDataType map_type(int dtype) {
  return dtype == BIL_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
         : dtype == BIL_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// A row-major map of 2 dimensions: dims, box and strides as cuTensorMapEncodeTiled takes them.
bool encode_2d(CUtensorMap* map, CUtensorMapDataType type, void* ptr, const cuuint64_t* dims, const cuuint64_t* strides,
               const cuuint32_t* box, CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promotion) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint32_t estr[2] = {1, 1};
  auto encode = [&] {
    return fn(map, type, 2, ptr, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promotion,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  return encode() || (context_made() && encode());
}

// A 2-D tensor map over a row-major [rows, cols] matrix of 16-bit elements
// (row stride ld elements), box = box_rows x 64 elements, 128-byte swizzle;
// reads past the matrix fill zeros.
int make_map(CUtensorMap* map, const void* ptr, int dtype, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kBK), static_cast<cuuint32_t>(box_rows)};
  return encode_2d(map, dtype == BIL_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                   const_cast<void*>(ptr), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B)
             ? BIL_OK
             : BIL_E_CUDA;
}

// The tensor map an epilogue stores a [rows, cols] output (row stride ld
// elements) through from the warps' staging boxes: 32 rows of 64 bytes, i.e.
// 32 columns of a 16-bit type or 16 of float32, no swizzle (a box in shared
// memory is row-major).
int make_store_map(CUtensorMap* map, void* ptr, int dtype, int64_t rows, int64_t cols, int64_t ld) {
  const int eb = dtype == BIL_F32 ? 4 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * eb};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(64 / eb), static_cast<cuuint32_t>(kStoreBox)};
  return encode_2d(map, map_type(dtype), ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE)
             ? BIL_OK
             : BIL_E_CUDA;
}

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A 16-byte aligned base and a row stride of a multiple of 16 bytes (what TMA
// and the epilogues' vector stores need).
bool rows16(const void* p, int64_t ld, int64_t elem_bytes) {
  return aligned_to(p, 16) && (ld * elem_bytes) % 16 == 0;
}

// A store GEMM operand with `rows` rows (M or N) over K = k: stored [rows, k]
// (K-major) and copied in boxes of box_rows x 64 K, or stored [k, rows] (mn:
// MN-major) and copied in boxes of 64 rows x 64 K.
int operand_map(CUtensorMap* map, const void* ptr, int dtype, int64_t rows, int64_t k, int64_t ld, bool mn,
                int box_rows) {
  return mn ? make_map(map, ptr, dtype, k, rows, ld, kMnBox) : make_map(map, ptr, dtype, rows, k, ld, box_rows);
}

}  // namespace
