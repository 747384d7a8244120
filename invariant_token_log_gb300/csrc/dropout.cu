// Dropout with a mask made from a seed, a step and an element's place (philox.cuh),
// with the residual's addition or without.  The C ABI is declared in include/bil.h.
//
//     y = round_T(x f + r),   f = 65536 / (65536 - border) or 0
// The gradient of x is the same call on the gradient of y, without a residual; that
// of r is y's own.  A dropped element's x adds nothing whatever it is (an infinity
// or a NaN among them).
//
// Bound: HBM, and next the instructions of the generator (about 55 for 8 elements,
// 10 rounds of two 32 x 32 -> 64 bit products each).  A thread has its groups' loads
// in flight before it makes their masks.

#include "launch.cuh"
#include "philox.cuh"
#include "rows_device.cuh"

#include <algorithm>

namespace {

struct DropParams {
  const unsigned char* x;
  const unsigned char* residual;  // NULL: none
  unsigned char* y;
  int64_t n_rows;
  int width, groups;  // a row's groups
  int64_t ld_x, ld_r, ld_y;
  int vec_y;
  int row_threads;    // of drop_rows_kernel
  int64_t total;      // groups of all rows
  Dropout drop;
};

constexpr int kDropThreads = 256;

template <int DT>
__device__ __forceinline__ void drop_group(const DropParams& p, const DropKey& key, uint64_t group,
                                           uint32_t (&x)[Row<DT>::kW], const uint32_t (&r)[Row<DT>::kW]) {
  using R = Row<DT>;
  const uint4 bits = key.bits(group);
  float v[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j)
    v[j] = drop_keeps(bits, j, p.drop.border) ? __fmul_rn(R::get(x, j), p.drop.times) : 0.0f;
  if (p.residual != nullptr) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = __fadd_rn(v[j], R::get(r, j));
  }
  R::pack(v, x);
}

// Rows one after the other without a gap, from 16-byte boundaries on: groups in
// the order of memory, kAhead of them a thread.
template <int DT>
__global__ void __launch_bounds__(kDropThreads) drop_flat_kernel(const DropParams p) {
  using R = Row<DT>;
  constexpr int kAhead = DT == BIL_F32 ? 2 : 4;
  griddep_wait();
  griddep_launch_dependents();
  const DropKey key(p.drop);
  constexpr int64_t kBlock = static_cast<int64_t>(kDropThreads) * kAhead;
  for (int64_t b = blockIdx.x * kBlock; b < p.total; b += gridDim.x * kBlock) {
    uint32_t x[kAhead][R::kW], r[kAhead][R::kW];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t g = b + i * kDropThreads + threadIdx.x;
      if (g >= p.total) continue;
      R::template load_path<kFullRows>(p.x + g * kVec * R::EB, 0, 0, kVec, x[i]);
      if (p.residual != nullptr) R::template load_path<kFullRows>(p.residual + g * kVec * R::EB, 0, 0, kVec, r[i]);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t g = b + i * kDropThreads + threadIdx.x;
      if (g >= p.total) continue;
      drop_group<DT>(p, key, static_cast<uint64_t>(g), x[i], r[i]);
      R::template store_path<kFullRows>(p.y + g * kVec * R::EB, 0, kVec, true, x[i]);
    }
  }
}

// Any rows: row_threads (a power of two) threads a row.
template <int DT>
__global__ void __launch_bounds__(kDropThreads) drop_rows_kernel(const DropParams p) {
  using R = Row<DT>;
  griddep_wait();
  griddep_launch_dependents();
  const DropKey key(p.drop);
  const int per_block = kDropThreads / p.row_threads;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * per_block + threadIdx.x / p.row_threads; row < p.n_rows;
       row += static_cast<int64_t>(gridDim.x) * per_block) {
    const RowStart x_at(p.x + row * p.ld_x * R::EB);
    const RowStart r_at(p.residual != nullptr ? p.residual + row * p.ld_r * R::EB : nullptr);
    unsigned char* out = p.y + row * p.ld_y * R::EB;
    for (int g = static_cast<int>(threadIdx.x) & (p.row_threads - 1); g < p.groups; g += p.row_threads) {
      const int count = min(kVec, p.width - g * kVec);
      uint32_t x[R::kW], r[R::kW];
      R::load(x_at.base, x_at.off, g, count, x);
      if (p.residual != nullptr) R::load(r_at.base, r_at.off, g, count, r);
      drop_group<DT>(p, key, static_cast<uint64_t>(row) * static_cast<uint64_t>(p.groups) + g, x, r);
      R::store(out, g, count, p.vec_y != 0, x);
    }
  }
}

}  // namespace

extern "C" {

int bil_dropout(const void* x, const void* residual, int dtype, int64_t n_rows, int64_t width, int64_t ld_x,
                int64_t ld_residual, double p_drop, uint64_t seed, uint64_t step, const int64_t* rng, void* y,
                int64_t ld_y, bil_stream_t stream) {
  bil_internal::NvtxRange nvtx_range("bil_dropout");
  const int eb = bil_internal::elem_bytes(dtype);
  if (eb == 0) return BIL_E_DTYPE;
  if (n_rows < 0 || width < 1) return BIL_E_INVALID_ARG;
  if (width > INT32_MAX - kVec) return BIL_E_UNSUPPORTED;
  DropParams p{};
  if (int st = make_dropout(p_drop, seed, step, rng, &p.drop)) return st;
  if (int st = check_rows(x, n_rows, width, ld_x, eb)) return st;
  if (int st = check_rows(y, n_rows, width, ld_y, eb)) return st;
  if (residual != nullptr)
    if (int st = check_rows(residual, n_rows, width, ld_residual, eb)) return st;
  if (n_rows == 0) return BIL_OK;
  p.x = static_cast<const unsigned char*>(x);
  p.residual = static_cast<const unsigned char*>(residual);
  p.y = static_cast<unsigned char*>(y);
  p.n_rows = n_rows;
  p.width = static_cast<int>(width);
  p.groups = (p.width + kVec - 1) / kVec;
  p.ld_x = ld_x;
  p.ld_r = ld_residual;
  p.ld_y = ld_y;
  p.vec_y = rows_start_on(y, n_rows, ld_y * eb, 16);
  p.total = n_rows * p.groups;
  int sms = 0, smem_optin = 0;
  if (int st = bil_internal::device_limits(&sms, &smem_optin)) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto dense = [&](const void* q, int64_t ld) { return q == nullptr || (aligned_to(q, 16) && (ld == width || n_rows == 1)); };
  const bool flat = width % kVec == 0 && dense(x, ld_x) && dense(residual, ld_residual) && dense(y, ld_y);
  void (*kernel)(DropParams) = flat ? (dtype == BIL_F32    ? drop_flat_kernel<BIL_F32>
                                       : dtype == BIL_BF16 ? drop_flat_kernel<BIL_BF16>
                                                           : drop_flat_kernel<BIL_F16>)
                                    : (dtype == BIL_F32    ? drop_rows_kernel<BIL_F32>
                                       : dtype == BIL_BF16 ? drop_rows_kernel<BIL_BF16>
                                                           : drop_rows_kernel<BIL_F16>);
  int64_t blocks;
  if (flat) {
    const int64_t per = static_cast<int64_t>(kDropThreads) * (dtype == BIL_F32 ? 2 : 4);
    blocks = (p.total + per - 1) / per;
  } else {
    p.row_threads = 8;
    while (p.row_threads < kDropThreads && p.row_threads < p.groups) p.row_threads *= 2;
    const int per = kDropThreads / p.row_threads;
    blocks = (n_rows + per - 1) / per;
  }
  const int64_t grid = std::min<int64_t>(blocks, INT32_MAX);
  return launch_pdl(kernel, grid, kDropThreads, 0, s, 1, p) == cudaSuccess ? BIL_OK : BIL_E_CUDA;
}

}  // extern "C"
