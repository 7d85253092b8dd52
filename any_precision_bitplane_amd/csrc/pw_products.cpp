// C-ABI host layer of the expert products in 16 bits.  Argument checks and the
// order of the launches only.
#include "pw_checks.h"

using namespace pw;

namespace {

constexpr int64_t kMaxRowStride = (int64_t)1 << 22;   // a tile's rows are addressed with 31-bit byte offsets
constexpr int64_t kMaxMatrix = (int64_t)1 << 30;
constexpr int64_t kMaxRows = 0x7FFFFFFF - 255;           // rows rounded up to a tile's are 32-bit numbers

bool sixteen(int32_t dtype) { return dtype == PW_F16 || dtype == PW_BF16; }

// Sizes of a product; PW_OK if a call may have them.
pw_status check_product(int32_t E, int64_t S, int64_t N, int64_t K) {
  if (E < 1 || S < 0 || N < 1 || K < 1) return PW_ERR_INVALID_ARG;
  if (E > kMaxExperts || S > kMaxRows || N % 8 || K % 8 || N > kMaxRowStride || K > kMaxRowStride || N * K > kMaxMatrix)
    return PW_ERR_UNSUPPORTED_SHAPE;
  return PW_OK;
}

// The shape's hidden size, inter size and number of experts (its top_k plays no part).
pw_status check_ffn(const pw_moe_shape* shape, int32_t S) {
  if (!shape) return PW_ERR_INVALID_ARG;
  pw_moe_shape one = *shape;
  one.top_k = 1;
  PW_TRY(pw_check_shape(&one, S));
  // rows of h and of the gradient of gate and up are a tile's rows too
  return shape->hidden > kMaxRowStride || 2 * (int64_t)shape->inter > kMaxRowStride ? PW_ERR_UNSUPPORTED_SHAPE : PW_OK;
}

pw_status check_wide_rows(const void* p, int64_t stride, int64_t S, int64_t n, int64_t bytes, bool written) {
  if (stride >= kMaxRowStride + (S == 1)) return PW_ERR_UNSUPPORTED_SHAPE;   // a row of the largest size, alone
  return check_rows(p, stride, S, n, bytes, written);
}

pw_status check_matrix(const void* p) {
  if (!p) return PW_ERR_INVALID_ARG;
  return aligned(p, 16) ? PW_OK : PW_ERR_ALIGNMENT;
}

pw_status check_offsets(const int32_t* offsets, int32_t E) {
  if (!offsets && E != 1) return PW_ERR_INVALID_ARG;
  return aligned(offsets, 4) ? PW_OK : PW_ERR_ALIGNMENT;
}

pw_status check_scratch(const void* workspace, size_t have, size_t need) {
  if (!need) return PW_OK;
  if (!workspace) return PW_ERR_INVALID_ARG;
  if (!aligned(workspace, kAlign)) return PW_ERR_ALIGNMENT;
  return have < need ? PW_ERR_WORKSPACE : PW_OK;
}

// The checkpoint of gate and up.
pw_status check_kept(int32_t dtype, int32_t z_dtype, const void* z, int64_t z_stride, const float* z_scale, int64_t S,
                     int64_t I, bool written) {
  const bool z8 = z_dtype == PW_E4M3;
  if (!z8 && z_dtype != dtype) return PW_ERR_INVALID_ARG;
  if (z8 != (z_scale != nullptr)) return PW_ERR_INVALID_ARG;
  if (!aligned(z_scale, 4)) return PW_ERR_ALIGNMENT;
  return check_wide_rows(z, z_stride, S, 2 * I, z8 ? 1 : 2, written);
}

int kept_groups(int I) { return (I + 127) / 128; }

pw_status run_product(const ProductArgs& a, int dtype, int kind, void* stream) {
  const hipStream_t s = (hipStream_t)stream;
  return hip_status(few_rows(a, kind) ? launch_few(a, dtype, kind, s) : launch_product(a, dtype, kind, s));
}

size_t dz_bytes(int64_t S, int64_t N) { return align_up((size_t)S * (size_t)N * 2, kAlign); }
size_t dz_sum_bytes(int E, int64_t S, int N) { return align_up(sizeof(float) * dz_part_floats(E, S, N), kAlign); }
size_t h_bytes(int64_t S, int64_t I) { return align_up((size_t)S * (size_t)I * 2 + 1, kAlign); }

// Scratch of a forward call's cut tiles, whose largest matrix has so many elements:
// none for few rows, whose products have no tiles (no more rows have tiles then).
// Gate and up of few rows with 8-bit copies do have tiles, which are not cut (one
// expert, H 2048, I 1408, 8 rows fp16 28.6 us where 14.7 without copies).
size_t forward_part_bytes(int E, int64_t S, int64_t matrix) {
  return few_rows_for(E, S, matrix) ? 0 : product_part_bytes(E, S);
}
float* forward_parts(uint8_t* at, int E, int64_t S, int64_t matrix) {
  return forward_part_bytes(E, S, matrix) ? reinterpret_cast<float*>(at) : nullptr;
}

// Scratch of a backward call's cut products, one after another in the same place.
size_t backward_part_bytes(int E, int64_t S, int64_t M, int64_t N, int64_t M2 = 0, int64_t N2 = 0) {
  size_t bytes = product_part_bytes(E, S);
  const size_t outer = outer_part_bytes(E, S, M, N), second = M2 ? outer_part_bytes(E, S, M2, N2) : 0;
  if (outer > bytes) bytes = outer;
  return second > bytes ? second : bytes;
}

}  // namespace

extern "C" {

size_t pw_moe_product_workspace_bytes(int32_t E, int32_t S_max, int32_t N, int32_t K) {
  return check_product(E, S_max, N, K) == PW_OK ? kAlign + forward_part_bytes(E, S_max, (int64_t)N * K) : 0;
}

size_t pw_moe_product_backward_workspace_bytes(int32_t E, int32_t S_max, int32_t N, int32_t K) {
  if (check_product(E, S_max, N, K) != PW_OK) return 0;
  return dz_bytes(S_max, N) + dz_sum_bytes(E, S_max, N) + backward_part_bytes(E, S_max, N, K);
}

pw_status pw_moe_product(int32_t E, int32_t S, int32_t N, int32_t K, int32_t dtype, const void* x, int64_t x_stride,
                         const int32_t* offsets, const void* w, const void* bias, int32_t act, const void* residual,
                         int64_t residual_stride, void* pre, int64_t pre_stride, void* y, int64_t y_stride,
                         void* workspace, size_t workspace_bytes, void* stream) {
  PW_TRY(check_product(E, S, N, K));
  if (!sixteen(dtype) || act < PW_ACT_NONE || act > PW_ACT_GELU) return PW_ERR_INVALID_ARG;
  PW_TRY(check_offsets(offsets, E));
  if (S == 0) return PW_OK;
  PW_TRY(check_wide_rows(x, x_stride, S, K, 2, false));
  PW_TRY(check_matrix(w));
  if (!aligned(bias, 16)) return PW_ERR_ALIGNMENT;
  if (residual) PW_TRY(check_wide_rows(residual, residual_stride, S, N, 2, false));
  if (pre) PW_TRY(check_wide_rows(pre, pre_stride, S, N, 2, true));
  PW_TRY(check_wide_rows(y, y_stride, S, N, 2, true));
  PW_TRY(check_scratch(workspace, workspace_bytes, pw_moe_product_workspace_bytes(E, S, N, K)));
  ProductArgs a{};
  a.E = E; a.S = S; a.N = N; a.K = K;
  a.offsets = offsets;
  a.x = x; a.x_stride = x_stride;
  a.w = w; a.w_expert = (int64_t)N * K;
  a.bias = bias;
  a.residual = residual; a.residual_stride = residual_stride;
  a.pre = pre; a.pre_stride = pre_stride;
  a.y = y; a.y_stride = y_stride;
  a.act = act;
  a.part = forward_parts(static_cast<uint8_t*>(workspace), E, S, (int64_t)N * K);
  return run_product(a, dtype, kProductAct, stream);
}

pw_status pw_moe_product_backward(int32_t E, int32_t S, int32_t N, int32_t K, int32_t dtype, const void* dy,
                                  int64_t dy_stride, const void* x, int64_t x_stride, const int32_t* offsets,
                                  const void* w, int32_t act, const void* pre, int64_t pre_stride, void* dx,
                                  int64_t dx_stride, void* dw, void* dbias, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  PW_TRY(check_product(E, S, N, K));
  if (!sixteen(dtype) || act < PW_ACT_NONE || act > PW_ACT_GELU) return PW_ERR_INVALID_ARG;
  if (act == PW_ACT_NONE ? pre != nullptr : S > 0 && !pre) return PW_ERR_INVALID_ARG;
  PW_TRY(check_offsets(offsets, E));
  if (!aligned(dw, 16) || !aligned(dbias, 16)) return PW_ERR_ALIGNMENT;
  const hipStream_t s = (hipStream_t)stream;
  if (S > 0) {
    PW_TRY(check_wide_rows(dy, dy_stride, S, N, 2, false));
    if (pre) PW_TRY(check_wide_rows(pre, pre_stride, S, N, 2, false));
    if (dw) PW_TRY(check_wide_rows(x, x_stride, S, K, 2, false));
    if (dx) {
      PW_TRY(check_matrix(w));
      PW_TRY(check_wide_rows(dx, dx_stride, S, K, 2, true));
    }
    PW_TRY(check_scratch(workspace, workspace_bytes, pw_moe_product_backward_workspace_bytes(E, S, N, K)));
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool through = S > 0 && pre && (dx || dw);   // dz differs from dy and is read again
  DzArgs z{};
  z.E = E; z.S = S; z.N = N; z.act = act;
  z.offsets = offsets;
  z.dy = dy; z.dy_stride = dy_stride;
  z.pre = pre; z.pre_stride = pre_stride;
  z.dz = through ? ws : nullptr;
  z.part = dbias ? reinterpret_cast<float*>(ws + dz_bytes(S, N)) : nullptr;
  z.dbias = dbias;
  if (through || dbias) PW_TRY(hip_status(launch_dz(z, dtype, s)));
  float* const part = reinterpret_cast<float*>(ws + dz_bytes(S, N) + dz_sum_bytes(E, S, N));
  const void* dz = through ? ws : dy;
  const int64_t dz_stride = through ? N : dy_stride;
  if (dx && S > 0) {
    ProductArgs a{};
    a.E = E; a.S = S; a.N = K; a.K = N;
    a.offsets = offsets;
    a.x = dz; a.x_stride = dz_stride;
    a.w = w; a.w_expert = (int64_t)N * K;
    a.y = dx; a.y_stride = dx_stride;
    a.part = part;
    PW_TRY(run_product(a, dtype, kProductBack, stream));
  }
  if (!dw) return PW_OK;
  OuterArgs o{};
  o.E = E; o.S = S; o.M = N; o.N = K;
  o.offsets = offsets;
  o.p = dz; o.p_stride = dz_stride;
  o.q = x; o.q_stride = x_stride;
  o.out = dw;
  o.part = part;
  return hip_status(launch_outer(o, dtype, s));
}

size_t pw_moe_ffn_workspace_bytes(const pw_moe_shape* shape, int32_t S_max) {
  if (check_ffn(shape, S_max) != PW_OK) return 0;
  return h_bytes(S_max, shape->inter) +
         forward_part_bytes(shape->num_experts, S_max, 2 * (int64_t)shape->inter * shape->hidden);
}

size_t pw_moe_ffn_backward_workspace_bytes(const pw_moe_shape* shape, int32_t S_max) {
  if (check_ffn(shape, S_max) != PW_OK) return 0;
  return dz_bytes(S_max, 2 * (int64_t)shape->inter) + h_bytes(S_max, shape->inter) +
         backward_part_bytes(shape->num_experts, S_max, shape->hidden, shape->inter, 2 * (int64_t)shape->inter, shape->hidden);
}

pw_status pw_moe_ffn(const pw_moe_shape* shape, int32_t S, int32_t dtype, const void* x, int64_t x_stride,
                     const int32_t* offsets, const void* w_gate_up, const void* w_down, int32_t act, int32_t z_dtype,
                     void* z, int64_t z_stride, float* z_scale, void* y, int64_t y_stride, void* workspace,
                     size_t workspace_bytes, void* stream) {
  PW_TRY(check_ffn(shape, S));
  if (!sixteen(dtype) || (act != PW_ACT_SILU && act != PW_ACT_GELU)) return PW_ERR_INVALID_ARG;
  const int H = shape->hidden, I = shape->inter, E = shape->num_experts;
  PW_TRY(check_offsets(offsets, E));
  if (S == 0) return PW_OK;
  if (!z && z_scale) return PW_ERR_INVALID_ARG;
  PW_TRY(check_wide_rows(x, x_stride, S, H, 2, false));
  PW_TRY(check_matrix(w_gate_up));
  PW_TRY(check_matrix(w_down));
  if (z) PW_TRY(check_kept(dtype, z_dtype, z, z_stride, z_scale, S, I, true));
  PW_TRY(check_wide_rows(y, y_stride, S, H, 2, true));
  PW_TRY(check_scratch(workspace, workspace_bytes, pw_moe_ffn_workspace_bytes(shape, S)));
  ProductArgs a{};
  a.E = E; a.S = S; a.N = I; a.K = H;
  a.offsets = offsets;
  a.x = x; a.x_stride = x_stride;
  a.w = w_gate_up; a.w_expert = 2 * (int64_t)I * H;
  a.y = workspace; a.y_stride = I;
  a.act = act;
  a.z = z; a.z_stride = z_stride;
  a.z_scale = z_scale; a.groups = kept_groups(I);
  a.z8 = z && z_dtype == PW_E4M3;
  a.part = forward_parts(static_cast<uint8_t*>(workspace) + h_bytes(S, I), E, S, 2 * (int64_t)I * H);
  PW_TRY(run_product(a, dtype, kProductGate, stream));
  ProductArgs d{};
  d.E = E; d.S = S; d.N = H; d.K = I;
  d.offsets = offsets;
  d.x = workspace; d.x_stride = I;
  d.w = w_down; d.w_expert = (int64_t)I * H;
  d.y = y; d.y_stride = y_stride;
  d.act = PW_ACT_NONE;
  d.part = a.part;
  return run_product(d, dtype, kProductAct, stream);
}

pw_status pw_moe_ffn_backward(const pw_moe_shape* shape, int32_t S, int32_t dtype, const void* dy, int64_t dy_stride,
                              const void* x, int64_t x_stride, const int32_t* offsets, const void* w_gate_up,
                              const void* w_down, int32_t act, int32_t z_dtype, const void* z, int64_t z_stride,
                              const float* z_scale, void* dx, int64_t dx_stride, void* dw_gate_up, void* dw_down,
                              void* workspace, size_t workspace_bytes, void* stream) {
  PW_TRY(check_ffn(shape, S));
  if (!sixteen(dtype) || (act != PW_ACT_SILU && act != PW_ACT_GELU)) return PW_ERR_INVALID_ARG;
  const int H = shape->hidden, I = shape->inter, E = shape->num_experts;
  PW_TRY(check_offsets(offsets, E));
  if (!aligned(dw_gate_up, 16) || !aligned(dw_down, 16)) return PW_ERR_ALIGNMENT;
  if (S > 0) {
    PW_TRY(check_wide_rows(dy, dy_stride, S, H, 2, false));
    if (dw_gate_up) PW_TRY(check_wide_rows(x, x_stride, S, H, 2, false));
    if (dx) {
      PW_TRY(check_matrix(w_gate_up));
      PW_TRY(check_wide_rows(dx, dx_stride, S, H, 2, true));
    }
    PW_TRY(check_matrix(w_down));
    PW_TRY(check_kept(dtype, z_dtype, z, z_stride, z_scale, S, I, false));
    PW_TRY(check_scratch(workspace, workspace_bytes, pw_moe_ffn_backward_workspace_bytes(shape, S)));
  }
  const hipStream_t s = (hipStream_t)stream;
  uint8_t* dz = static_cast<uint8_t*>(workspace);
  uint8_t* h = dz + dz_bytes(S, 2 * (int64_t)I);
  float* const part = reinterpret_cast<float*>(h + h_bytes(S, I));
  if (S > 0 && (dx || dw_gate_up || dw_down)) {
    ProductArgs a{};
    a.E = E; a.S = S; a.N = I; a.K = H;
    a.offsets = offsets;
    a.x = dy; a.x_stride = dy_stride;
    a.w = w_down; a.w_expert = (int64_t)I * H;
    a.pre = dz; a.pre_stride = 2 * (int64_t)I;
    a.y = dw_down ? h : nullptr; a.y_stride = I;
    a.act = act;
    a.z = const_cast<void*>(z); a.z_stride = z_stride;
    a.z_scale = const_cast<float*>(z_scale); a.groups = kept_groups(I);
    a.z8 = z_dtype == PW_E4M3;
    a.part = part;
    PW_TRY(run_product(a, dtype, kProductGateGrad, stream));
  }
  OuterArgs o{};
  o.E = E; o.S = S;
  o.offsets = offsets;
  o.part = part;
  if (dw_down) {
    o.M = H; o.N = I;
    o.p = dy; o.p_stride = dy_stride;
    o.q = h; o.q_stride = I;
    o.out = dw_down;
    PW_TRY(hip_status(launch_outer(o, dtype, s)));
  }
  if (dx && S > 0) {
    ProductArgs a{};
    a.E = E; a.S = S; a.N = H; a.K = 2 * I;
    a.offsets = offsets;
    a.x = dz; a.x_stride = 2 * (int64_t)I;
    a.w = w_gate_up; a.w_expert = 2 * (int64_t)I * H;
    a.y = dx; a.y_stride = dx_stride;
    a.part = part;
    PW_TRY(run_product(a, dtype, kProductBack, stream));
  }
  if (!dw_gate_up) return PW_OK;
  o.M = 2 * I; o.N = H;
  o.p = dz; o.p_stride = 2 * (int64_t)I;
  o.q = x; o.q_stride = x_stride;
  o.out = dw_gate_up;
  return hip_status(launch_outer(o, dtype, s));
}

}  // extern "C"
