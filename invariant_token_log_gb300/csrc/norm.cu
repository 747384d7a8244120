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

#include "norm_device.cuh"

#include <cmath>

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
  if (int st = bwd_parts(n_rows, width, false, &parts)) return st;
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
  if (int st = bwd_parts(n_rows, width, false, &parts)) return st;
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
  const bool full = rows_start_on(h, n_rows, ld_h * eb, 16) && rows_start_on(dy, n_rows, ld_dy * eb, 16) && p.vec_dx &&
                    (dh == nullptr || rows_start_on(dh, n_rows, ld_dh * eb, 16));
  return launch_bwd<kRms>(p, dtype, weight_dtype, full, dweight, nullptr, s);
}

}  // extern "C"
