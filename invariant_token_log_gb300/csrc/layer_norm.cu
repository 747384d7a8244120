// Layer norm of a residual stream, with dropout of what joins the stream and the
// residual's addition.  The C ABI is declared in include/bil.h.
//
//     h = round_T(drop(x) + r)          (no dropout, no residual: h = x)
//     mean = sum_c h_c / H,  rstd = 1 / sqrt(sum_c (h_c - mean)^2 / H + eps)
//     u = (h - mean) rstd,   y = u w + b
// and the backward of y (and of h, which goes on as the residual stream):
//     v = dy w,  c1 = mean(v),  c2 = mean(v u)
//     dr = rstd (v - c1 - u c2) + dh,   dx = drop'(dr)
//     dw = sum over rows of dy u,       db = sum over rows of dy
// drop multiplies by 65536 / (65536 - border) or by 0 (see philox.cuh), drop'
// by the same factors, made again from the seed.
//
// Everything is float32 between the loads and the stores.  The row stays in
// registers for both of its sums, so the squares are those of the centred row: a
// row far from zero keeps its variance.  h is rounded to T before it is normed,
// as in norm.cu.  The kernels are norm.cu's with the mean, the bias and the mask
// (norm_device.cuh).

#include "norm_device.cuh"

namespace bil_internal {

int layer_norm_watchdog(unsigned int* flags, int clear) {
  if (cudaMemcpyFromSymbol(flags, g_watchdog_norm, sizeof(unsigned int)) != cudaSuccess) return BIL_E_CUDA;
  if (clear) {
    const unsigned int zero = 0;
    if (cudaMemcpyToSymbol(g_watchdog_norm, &zero, sizeof(unsigned int)) != cudaSuccess) return BIL_E_CUDA;
  }
  return BIL_OK;
}

}  // namespace bil_internal

extern "C" {

int bil_layer_norm_fwd(const void* x, const void* residual, const void* weight, const void* bias, int dtype,
                       int weight_dtype, int64_t n_rows, int64_t width, int64_t ld_x, int64_t ld_residual, float eps,
                       double p_drop, uint64_t seed, uint64_t step, const int64_t* rng, void* y, int64_t ld_y, void* h,
                       int64_t ld_h, float* mean, float* rstd, bil_stream_t stream) {
  bil_internal::NvtxRange nvtx_range("bil_layer_norm_fwd");
  if (int st = check_common(dtype, n_rows, width)) return st;
  if (!(eps >= 0.0f) || std::isinf(eps)) return BIL_E_INVALID_ARG;
  NormParams p{};
  if (int st = make_dropout(p_drop, seed, step, rng, &p.drop)) return st;
  const bool drop = p_drop > 0.0;
  if ((residual != nullptr || drop) != (h != nullptr) && n_rows > 0) return BIL_E_INVALID_ARG;
  if (int st = check_weight(weight, dtype, weight_dtype)) return st;
  if (!aligned_to(bias, 16)) return BIL_E_ALIGN;
  const int eb = bil_internal::elem_bytes(dtype);
  if (int st = check_rows(x, n_rows, width, ld_x, eb)) return st;
  if (int st = check_rows(y, n_rows, width, ld_y, eb)) return st;
  if (residual != nullptr)
    if (int st = check_rows(residual, n_rows, width, ld_residual, eb)) return st;
  if (h != nullptr)
    if (int st = check_rows(h, n_rows, width, ld_h, eb)) return st;
  if (!aligned_to(rstd, 4) || !aligned_to(mean, 4)) return BIL_E_ALIGN;
  if (n_rows == 0) return BIL_OK;
  p.x = static_cast<const unsigned char*>(x);
  p.residual = static_cast<const unsigned char*>(residual);
  p.weight = static_cast<const unsigned char*>(weight);
  p.bias = static_cast<const unsigned char*>(bias);
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
  p.mean = mean;
  p.rstd = rstd;
  p.vec_y = rows_start_on(y, n_rows, ld_y * eb, 16);
  p.vec_h = rows_start_on(h, n_rows, ld_h * eb, 16);
  int ng = 0;
  row_shape(p.width, kFwdGroups, &p.row_threads, &ng);
  const bool full = rows_start_on(x, n_rows, ld_x * eb, 16) && p.vec_y && (h == nullptr || p.vec_h) &&
                    (residual == nullptr || rows_start_on(residual, n_rows, ld_residual * eb, 16));
  const int path = row_path(width, full, weight_dtype == dtype);
  return launch_fwd(drop ? fwd_kernel<kLayerDrop>(dtype, ng, path) : fwd_kernel<kLayer>(dtype, ng, path), p, path, eb,
                    reinterpret_cast<cudaStream_t>(stream));
}

int bil_layer_norm_bwd_workspace_bytes(int64_t n_rows, int64_t width, int need_bias, int64_t* bytes) {
  if (n_rows < 0 || width < 1 || bytes == nullptr) return BIL_E_INVALID_ARG;
  if (width > BIL_MAX_NORM_WIDTH) return BIL_E_UNSUPPORTED;
  int64_t parts = 0;
  if (int st = bwd_parts(n_rows, width, true, &parts)) return st;
  *bytes = parts * width * static_cast<int64_t>(sizeof(float)) * (need_bias ? 2 : 1);
  return BIL_OK;
}

int bil_layer_norm_bwd(const void* dy, const void* h, const void* weight, const float* mean, const float* rstd,
                       const void* dh, int dtype, int weight_dtype, int64_t n_rows, int64_t width, int64_t ld_dy,
                       int64_t ld_h, int64_t ld_dh, double p_drop, uint64_t seed, uint64_t step, const int64_t* rng,
                       void* dx, int64_t ld_dx, void* dresidual, int64_t ld_dresidual, float* dweight, float* dbias,
                       void* workspace, int64_t workspace_bytes, bil_stream_t stream) {
  bil_internal::NvtxRange nvtx_range("bil_layer_norm_bwd");
  if (int st = check_common(dtype, n_rows, width)) return st;
  NormParams p{};
  if (int st = make_dropout(p_drop, seed, step, rng, &p.drop)) return st;
  const bool drop = p_drop > 0.0;
  if (dresidual != nullptr && !drop) return BIL_E_INVALID_ARG;  // it is dx
  if (dresidual != nullptr && dresidual == dx) return BIL_E_INVALID_ARG;
  if (int st = check_weight(weight, dtype, weight_dtype)) return st;
  const int eb = bil_internal::elem_bytes(dtype);
  if (int st = check_rows(dy, n_rows, width, ld_dy, eb)) return st;
  if (int st = check_rows(h, n_rows, width, ld_h, eb)) return st;
  if (int st = check_rows(dx, n_rows, width, ld_dx, eb)) return st;
  if (dh != nullptr)
    if (int st = check_rows(dh, n_rows, width, ld_dh, eb)) return st;
  if (dresidual != nullptr)
    if (int st = check_rows(dresidual, n_rows, width, ld_dresidual, eb)) return st;
  if (dweight == nullptr) return BIL_E_INVALID_ARG;
  if (!aligned_to(dweight, 4) || !aligned_to(dbias, 4) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return BIL_E_ALIGN;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (n_rows == 0) {  // sums over no rows
    for (float* sums : {dweight, dbias})
      if (sums != nullptr &&
          cudaMemsetAsync(sums, 0, static_cast<size_t>(width) * sizeof(float), s) != cudaSuccess)
        return BIL_E_CUDA;
    return BIL_OK;
  }
  if (mean == nullptr || rstd == nullptr || workspace == nullptr) return BIL_E_INVALID_ARG;
  if (!aligned_to(workspace, 16)) return BIL_E_ALIGN;
  int64_t need = 0;
  if (int st = bil_layer_norm_bwd_workspace_bytes(n_rows, width, dbias != nullptr, &need)) return st;
  if (workspace_bytes < need) return BIL_E_INVALID_ARG;
  p.x = static_cast<const unsigned char*>(h);
  p.weight = static_cast<const unsigned char*>(weight);
  p.n_rows = n_rows;
  p.width = static_cast<int>(width);
  p.groups = (p.width + kVec - 1) / kVec;
  p.ld_x = ld_h;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.dy = static_cast<const unsigned char*>(dy);
  p.dh = static_cast<const unsigned char*>(dh);
  p.ld_dy = ld_dy;
  p.ld_dh = ld_dh;
  p.ld_dx = ld_dx;
  p.dx = static_cast<unsigned char*>(dx);
  p.vec_dx = rows_start_on(dx, n_rows, ld_dx * eb, 16);
  p.dr = static_cast<unsigned char*>(dresidual);
  p.ld_dr = ld_dresidual;
  p.vec_dr = rows_start_on(dresidual, n_rows, ld_dresidual * eb, 16);
  p.dw_part = static_cast<float*>(workspace);
  p.need_bias = dbias != nullptr;
  const bool full = rows_start_on(h, n_rows, ld_h * eb, 16) && rows_start_on(dy, n_rows, ld_dy * eb, 16) && p.vec_dx &&
                    (dh == nullptr || rows_start_on(dh, n_rows, ld_dh * eb, 16)) && (dresidual == nullptr || p.vec_dr);
  return drop ? launch_bwd<kLayerNormDrop>(p, dtype, weight_dtype, full, dweight, dbias, s)
              : launch_bwd<kLayerNorm>(p, dtype, weight_dtype, full, dweight, dbias, s);
}

}  // extern "C"
