// C-ABI host layer of the operators around the routed layer: the norm in front
// of it, tokens sorted by expert and back, and the gradients.  Argument checks
// and launches only.
#include "pw_internal.h"

using namespace pw;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

pw_status hip_status(hipError_t e) { return e == hipSuccess ? PW_OK : PW_ERR_HIP; }

// Bytes of an element of a row type, 0 if it is none.
int64_t row_type_bytes(int32_t dtype) { return dtype == PW_F32 ? 4 : (dtype == PW_F16 || dtype == PW_BF16) ? 2 : 0; }

// A matrix of T rows of H elements: 16-byte aligned rows `stride` elements
// apart.  Rows that are written must not overlap.
pw_status check_rows(const void* p, int64_t stride, int64_t T, int64_t H, int64_t bytes, bool written) {
  if (!p) return PW_ERR_INVALID_ARG;
  if (stride < 0 || (written && T > 1 && stride < H)) return PW_ERR_INVALID_ARG;
  if (!aligned(p, 16) || (stride * bytes) % 16) return PW_ERR_ALIGNMENT;
  return PW_OK;
}

pw_status check_norm_shape(int32_t T, int32_t H, int32_t dtype, float eps) {
  if (T < 0 || H <= 0 || !row_type_bytes(dtype)) return PW_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || eps > 1e30f) return PW_ERR_INVALID_ARG;
  if (H % 8 || H > kMaxNormHidden) return PW_ERR_UNSUPPORTED_SHAPE;
  return PW_OK;
}

#define PW_TRY(expr)                     \
  do {                                   \
    const pw_status st_ = (expr);        \
    if (st_ != PW_OK) return st_;        \
  } while (0)

pw_status unpermute(const pw_moe_shape* shape, int32_t T, int32_t dtype, const void* rows, int64_t rows_stride,
                    const int32_t* inv, const float* w, void* y, int64_t y_stride, void* stream) {
  PW_TRY(pw_check_shape(shape, T));
  const int64_t bytes = row_type_bytes(dtype);
  if (!bytes) return PW_ERR_INVALID_ARG;
  if (T == 0) return PW_OK;
  if (!inv) return PW_ERR_INVALID_ARG;
  PW_TRY(check_rows(rows, rows_stride, (int64_t)T * shape->top_k, shape->hidden, bytes, false));
  PW_TRY(check_rows(y, y_stride, T, shape->hidden, bytes, true));
  if (!aligned(inv, 4) || !aligned(w, 4)) return PW_ERR_ALIGNMENT;
  UnpermuteArgs a{T, shape->hidden, shape->top_k, rows, rows_stride, inv, w, y, y_stride};
  return hip_status(launch_unpermute(a, dtype, (hipStream_t)stream));
}

}  // namespace

extern "C" {

pw_status pw_rmsnorm(int32_t T, int32_t H, int32_t dtype, const void* x, int64_t x_stride, const void* residual,
                     int64_t residual_stride, void* residual_out, int64_t residual_out_stride, const void* weight,
                     float eps, int32_t y_dtype, void* y, int64_t y_stride, float* scale, int32_t group,
                     void* stream) {
  PW_TRY(check_norm_shape(T, H, dtype, eps));
  const bool e4m3 = y_dtype == PW_E4M3;
  if (!e4m3 && y_dtype != dtype) return PW_ERR_INVALID_ARG;
  if (e4m3 ? (group != 0 && group != kNormGroup) : (group != 0 || scale != nullptr)) return PW_ERR_INVALID_ARG;
  if (T == 0) return PW_OK;
  const int64_t bytes = row_type_bytes(dtype);
  PW_TRY(check_rows(x, x_stride, T, H, bytes, false));
  if (residual) PW_TRY(check_rows(residual, residual_stride, T, H, bytes, false));
  if (residual_out) {
    if (!residual) return PW_ERR_INVALID_ARG;
    PW_TRY(check_rows(residual_out, residual_out_stride, T, H, bytes, true));
  }
  PW_TRY(check_rows(weight, H, 1, H, 16, false));
  PW_TRY(check_rows(y, y_stride, T, H, e4m3 ? 2 : bytes, true));   // 8-bit rows start on 8-byte boundaries
  if (e4m3 && !scale) return PW_ERR_INVALID_ARG;
  if (!aligned(scale, 4)) return PW_ERR_ALIGNMENT;
  NormArgs a{T, H, x, x_stride, residual, residual_stride, residual_out, residual_out_stride, weight, eps,
             y, y_stride, scale, group};
  return hip_status(launch_rmsnorm(a, dtype, e4m3, (hipStream_t)stream));
}

size_t pw_rmsnorm_backward_workspace_bytes(int32_t T, int32_t H) {
  if (T < 0 || H <= 0 || H % 8 || H > kMaxNormHidden) return 0;
  return align_up(norm_grad_parts(T) * (size_t)H * sizeof(float) + 1, kAlign);
}

pw_status pw_rmsnorm_backward(int32_t T, int32_t H, int32_t dtype, const void* dy, int64_t dy_stride, const void* r,
                              int64_t r_stride, const void* weight, float eps, const void* dresidual,
                              int64_t dresidual_stride, void* dx, int64_t dx_stride, float* dweight, void* workspace,
                              size_t workspace_bytes, void* stream) {
  PW_TRY(check_norm_shape(T, H, dtype, eps));
  const int64_t bytes = row_type_bytes(dtype);
  if (dweight) {
    if (!aligned(dweight, 16)) return PW_ERR_ALIGNMENT;
    if (T == 0) return hip_status(launch_fill_zero(dweight, (size_t)H * sizeof(float), (hipStream_t)stream));
  }
  if (T == 0) return PW_OK;
  PW_TRY(check_rows(dy, dy_stride, T, H, bytes, false));
  PW_TRY(check_rows(r, r_stride, T, H, bytes, false));
  PW_TRY(check_rows(weight, H, 1, H, 16, false));
  if (dresidual) PW_TRY(check_rows(dresidual, dresidual_stride, T, H, bytes, false));
  PW_TRY(check_rows(dx, dx_stride, T, H, bytes, true));
  if (dweight) {
    if (!workspace) return PW_ERR_INVALID_ARG;
    if (!aligned(workspace, kAlign)) return PW_ERR_ALIGNMENT;
    if (workspace_bytes < pw_rmsnorm_backward_workspace_bytes(T, H)) return PW_ERR_WORKSPACE;
  }
  NormGradArgs a{T, H, dy, dy_stride, r, r_stride, weight, eps, dresidual, dresidual_stride, dx, dx_stride,
                 dweight ? static_cast<float*>(workspace) : nullptr};
  return hip_status(launch_rmsnorm_grad(a, dtype, dweight, (hipStream_t)stream));
}

size_t pw_moe_permute_workspace_bytes(const pw_moe_shape* shape, int32_t T_max) {
  if (pw_check_shape(shape, T_max) != PW_OK) return 0;
  return align_up(sizeof(int32_t) * permute_count_ints(T_max, shape->top_k, shape->num_experts), kAlign);
}

pw_status pw_moe_permute(const pw_moe_shape* shape, int32_t T, int32_t dtype, const void* x, int64_t x_stride,
                         const float* x_scale, int32_t groups, const int32_t* ids, void* xs, int64_t xs_stride,
                         float* xs_scale, int32_t* offsets, int32_t* inv, int32_t* perm, uint32_t* status,
                         void* workspace, size_t workspace_bytes, void* stream) {
  PW_TRY(pw_check_shape(shape, T));
  const int64_t bytes = dtype == PW_E4M3 ? 1 : row_type_bytes(dtype);
  if (!bytes || groups < 0 || (groups > 0) != (x_scale != nullptr) || (groups > 0) != (xs_scale != nullptr))
    return PW_ERR_INVALID_ARG;
  if (!offsets) return PW_ERR_INVALID_ARG;
  if (!aligned(offsets, 4)) return PW_ERR_ALIGNMENT;
  const int64_t S = (int64_t)T * shape->top_k;
  if (T == 0)
    return hip_status(launch_fill_zero(offsets, sizeof(int32_t) * ((size_t)shape->num_experts + 1),
                                       (hipStream_t)stream));
  if (!ids || !inv || !workspace) return PW_ERR_INVALID_ARG;
  PW_TRY(check_rows(x, x_stride, T, shape->hidden, bytes, false));
  PW_TRY(check_rows(xs, xs_stride, S, shape->hidden, bytes, true));
  if (!aligned(ids, 4) || !aligned(inv, 4) || !aligned(perm, 4) || !aligned(status, 4) || !aligned(x_scale, 4) ||
      !aligned(xs_scale, 4) || !aligned(workspace, kAlign))
    return PW_ERR_ALIGNMENT;
  if (workspace_bytes < pw_moe_permute_workspace_bytes(shape, T)) return PW_ERR_WORKSPACE;
  PermuteArgs a{};
  a.T = T;
  a.k = shape->top_k;
  a.E = shape->num_experts;
  a.x = static_cast<const uint8_t*>(x);
  a.xs = static_cast<uint8_t*>(xs);
  a.row_bytes = shape->hidden * bytes;
  a.x_stride = x_stride * bytes;
  a.xs_stride = xs_stride * bytes;
  a.x_scale = x_scale;
  a.xs_scale = xs_scale;
  a.groups = groups;
  a.ids = ids;
  a.offsets = offsets;
  a.inv = inv;
  a.perm = perm;
  a.status = status;
  a.counts = static_cast<int32_t*>(workspace);
  return hip_status(launch_permute(a, (hipStream_t)stream));
}

pw_status pw_moe_unpermute(const pw_moe_shape* shape, int32_t T, int32_t dtype, const void* rows, int64_t rows_stride,
                           const int32_t* inv, const float* w, void* y, int64_t y_stride, void* stream) {
  return unpermute(shape, T, dtype, rows, rows_stride, inv, w, y, y_stride, stream);
}

pw_status pw_moe_permute_backward(const pw_moe_shape* shape, int32_t T, int32_t dtype, const void* dxs,
                                  int64_t dxs_stride, const int32_t* inv, void* dx, int64_t dx_stride, void* stream) {
  return unpermute(shape, T, dtype, dxs, dxs_stride, inv, nullptr, dx, dx_stride, stream);
}

pw_status pw_moe_unpermute_backward(const pw_moe_shape* shape, int32_t T, int32_t dtype, const void* dy,
                                    int64_t dy_stride, const void* rows, int64_t rows_stride, const int32_t* inv,
                                    const float* w, void* drows, int64_t drows_stride, float* dw, void* stream) {
  PW_TRY(pw_check_shape(shape, T));
  const int64_t bytes = row_type_bytes(dtype);
  if (!bytes) return PW_ERR_INVALID_ARG;
  if (T == 0) return PW_OK;
  const int64_t S = (int64_t)T * shape->top_k;
  if (!inv || (dw && !rows)) return PW_ERR_INVALID_ARG;
  PW_TRY(check_rows(dy, dy_stride, T, shape->hidden, bytes, false));
  if (dw) PW_TRY(check_rows(rows, rows_stride, S, shape->hidden, bytes, false));
  PW_TRY(check_rows(drows, drows_stride, S, shape->hidden, bytes, true));
  if (!aligned(inv, 4) || !aligned(w, 4) || !aligned(dw, 4)) return PW_ERR_ALIGNMENT;
  UnpermuteGradArgs a{T, shape->hidden, shape->top_k, dy, dy_stride, rows, rows_stride, inv, w, drows, drows_stride,
                      dw};
  return hip_status(launch_unpermute_grad(a, dtype, (hipStream_t)stream));
}

size_t pw_router_backward_workspace_bytes(const pw_moe_shape* shape, int32_t T_max) {
  if (pw_check_shape(shape, T_max) != PW_OK) return 0;
  return router_grad_plan(shape->hidden, shape->num_experts, shape->top_k, T_max).bytes;
}

pw_status pw_router_backward(const pw_moe_shape* shape, int32_t T, const uint16_t* x, const uint16_t* router_w,
                             const int32_t* ids, const float* w, const float* dw, const uint16_t* dx_add, uint16_t* dx,
                             float* drouter_w, void* workspace, size_t workspace_bytes, void* stream) {
  PW_TRY(pw_check_shape(shape, T));
  if (shape->top_k > kMaxRouterTopK) return PW_ERR_UNSUPPORTED_SHAPE;
  if (!drouter_w) return PW_ERR_INVALID_ARG;
  if (!aligned(drouter_w, 16)) return PW_ERR_ALIGNMENT;
  const int H = shape->hidden, E = shape->num_experts, k = shape->top_k;
  if (T == 0) return hip_status(launch_fill_zero(drouter_w, sizeof(float) * (size_t)E * H, (hipStream_t)stream));
  if (!x || !router_w || !ids || !w || !dw || !dx || !workspace) return PW_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(router_w, 16) || !aligned(dx_add, 16) || !aligned(dx, 16) || !aligned(ids, 4) ||
      !aligned(w, 4) || !aligned(dw, 4) || !aligned(workspace, kAlign))
    return PW_ERR_ALIGNMENT;
  const RouterGradPlan p = router_grad_plan(H, E, k, T);
  if (workspace_bytes < p.bytes) return PW_ERR_WORKSPACE;
  RouterGradArgs a{T, H, E, k, x, router_w, ids, w, dw, dx_add, dx, drouter_w, static_cast<float*>(workspace),
                   p.splits, p.split_slots, p.shift, p.cshift};
  return hip_status(launch_router_grad(a, (hipStream_t)stream));
}

pw_status pw_moe_forward_block(const pw_moe_shape* shape, int32_t T, const uint16_t* x, uint16_t* residual,
                               const uint16_t* norm_w, float eps, const uint16_t* router_w,
                               const pw_block_desc* blocks, const uint8_t* q, uint16_t* y, uint32_t* stat_count,
                               float* stat_mass, void* workspace, size_t workspace_bytes, const pw_moe_options* opts,
                               void* stream) {
  PW_TRY(pw_check_shape(shape, T));
  if (shape->top_k > kMaxRouterTopK) return PW_ERR_UNSUPPORTED_SHAPE;
  PW_TRY(check_norm_shape(T, shape->hidden, PW_F16, eps));
  if (T == 0) return PW_OK;
  if (!x || !residual || !norm_w || !router_w || !blocks || !q || !y || !workspace) return PW_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(norm_w, 16) || !aligned(router_w, 16) || !aligned(y, 16) ||
      !aligned(blocks, 8) || !aligned(stat_count, 4) || !aligned(stat_mass, 4) || !aligned(workspace, kAlign))
    return PW_ERR_ALIGNMENT;
  const int H = shape->hidden;
  const WsLayout W = ws_layout(H, shape->inter, shape->num_experts, shape->top_k, T);
  if (workspace_bytes < W.total) return PW_ERR_WORKSPACE;
  pw_path_info info;   // options the layer would refuse are refused before the norm runs
  PW_TRY(pw_moe_path_info(shape, T, opts, &info));
  if (opts && opts->event_mode != PW_EVENTS_STAGES && opts->event_mode != PW_EVENTS_KERNELS) return PW_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint16_t* xn = reinterpret_cast<uint16_t*>(ws + W.xl);
  if (!norm_router_fits(T, H)) {
    PW_TRY(pw_rmsnorm(T, H, PW_F16, x, H, residual, H, residual, H, norm_w, eps, PW_F16, xn, H, nullptr, 0, stream));
    return pw_moe_forward_routed(shape, T, xn, router_w, blocks, q, y, stat_count, stat_mass, workspace,
                                 workspace_bytes, opts, stream);
  }
  int32_t* ids = reinterpret_cast<int32_t*>(ws + W.rids);
  float* w = reinterpret_cast<float*>(ws + W.rw);
  PW_TRY(hip_status(launch_norm_router(x, residual, norm_w, eps, xn, router_w, T, H, shape->num_experts, shape->top_k,
                                       ids, w, stat_count, stat_mass, (hipStream_t)stream)));
  return pw_moe_forward(shape, T, xn, ids, w, blocks, q, y, workspace, workspace_bytes, opts, stream);
}

}  // extern "C"
