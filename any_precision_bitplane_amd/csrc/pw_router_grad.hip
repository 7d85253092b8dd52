// Gradient of the top-k softmax router, the selection held fixed.
//
// w[t][j] is the softmax over token t's selected logits l[t][j] = <x[t],
// Wr[e_j]>, e_j = ids[t][j], so with dw the gradient of w
//   dl[t][j] = w[t][j] (dw[t][j] - sum_i w[t][i] dw[t][i])
//   dx[t]    = dx_add[t] + sum_j dl[t][j] Wr[e_j]
//   dWr[e]   = sum over the slots of expert e of dl x[t]
// in fp32.  A dropped slot (id outside [0, E)) takes no part, in the inner sum
// either.
//
// Three kernels.  dx: one pass over dx_add and dx, the router's rows coming
// from L2; it leaves each slot's dl and expert behind.  dWr: a wave owns 128
// columns and a stretch of tokens and keeps dWr[0..E) of its columns in LDS,
// so x is read once whatever k is and no two lanes ever add to the same
// word (no atomics: the same inputs give the same bits).  Then the stretches'
// shares are summed in order.
#include "pw_rows.h"

namespace pw {

namespace {

constexpr unsigned kMaxGrid = 1u << 20;
constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void router_grad_x_kernel(RouterGradArgs a, int shift) {
  using R = Row<PW_F16>;
  const int C = a.H / 8;
  const int lanes = 1 << shift;
  const int per_block = kThreads >> shift;
  const int lane = (int)threadIdx.x & (lanes - 1);
  for (int64_t t = (int64_t)blockIdx.x * per_block + ((int)threadIdx.x >> shift); t < a.T;
       t += (int64_t)gridDim.x * per_block) {
    const int32_t* ids = a.ids + t * a.k;
    const float* w = a.w + t * a.k;
    const float* dw = a.dw + t * a.k;
    float mean = 0.f;
    for (int j = 0; j < a.k; ++j)
      if ((uint32_t)ids[j] < (uint32_t)a.E) mean = __builtin_fmaf(w[j], dw[j], mean);
    for (int c = lane; c < C; c += lanes) {
      floatx8 acc = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (a.dx_add) acc = R::wide(R::load(reinterpret_cast<const _Float16*>(a.dx_add) + t * a.H + 8 * c));
      for (int j = 0; j < a.k; ++j) {
        const int32_t e = ids[j];
        if ((uint32_t)e >= (uint32_t)a.E) continue;
        const float dl = w[j] * (dw[j] - mean);
        acc += dl * R::wide(R::load(reinterpret_cast<const _Float16*>(a.router_w) + (int64_t)e * a.H + 8 * c));
      }
      R::store(reinterpret_cast<_Float16*>(a.dx) + t * a.H + 8 * c, R::narrow(acc));
    }
    // a token that lists an expert twice keeps the sum in the first of the two slots
    for (int j = lane; j < a.k; j += lanes) {
      int32_t e = (uint32_t)ids[j] < (uint32_t)a.E ? ids[j] : -1;
      float dl = 0.f;
      for (int i = 0; i < a.k; ++i) {
        if (e < 0 || ids[i] != e) continue;
        if (i < j) {
          e = -1;
          break;
        }
        dl += w[i] * (dw[i] - mean);
      }
      a.slot_e[t * a.k + j] = e;
      a.slot_dl[t * a.k + j] = dl;
    }
  }
}

// One wave: columns [128 cb, 128 cb + 128), two a lane, tokens [t0, t1).
__global__ __launch_bounds__(kWave) void router_grad_w_kernel(RouterGradArgs a) {
  extern __shared__ float acc[];   // [E][128]
  typedef float floatx2 __attribute__((ext_vector_type(2)));
  constexpr int U = 16;            // tokens requested together
  const int lane = threadIdx.x;
  const int col = (int)blockIdx.x * 128 + 2 * lane;
  const bool in = col < a.H;
  const int64_t t0 = (int64_t)blockIdx.y * a.split_tokens;
  const int64_t t1 = t0 + a.split_tokens < a.T ? t0 + a.split_tokens : a.T;
  floatx2* mine = reinterpret_cast<floatx2*>(acc) + lane;
  for (int e = 0; e < a.E; ++e) mine[e * kWave] = floatx2{0.f, 0.f};
  const _Float16* x = reinterpret_cast<const _Float16*>(a.x) + (in ? col : 0);
  for (int64_t tb = t0; tb < t1; tb += U) {
    half2_t v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = tb + u < t1 ? tb + u : t1 - 1;
      v[u] = *reinterpret_cast<const half2_t*>(x + t * a.H);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (tb + u >= t1) break;
      const floatx2 xv = {(float)v[u][0], (float)v[u][1]};
      const int64_t s = (tb + u) * a.k;
      for (int j = 0; j < a.k; ++j) {
        const int e = a.slot_e[s + j];
        if (e < 0) continue;
        mine[e * kWave] += a.slot_dl[s + j] * xv;
      }
    }
  }
  if (!in) return;
  float* out = a.part + (size_t)blockIdx.y * a.E * a.H + col;
  for (int e = 0; e < a.E; ++e) *reinterpret_cast<floatx2*>(out + (size_t)e * a.H) = mine[e * kWave];
}

__global__ __launch_bounds__(kThreads) void router_grad_join_kernel(RouterGradArgs a) {
  const int64_t n = (int64_t)a.E * a.H;
  const int64_t i = 4 * ((int64_t)blockIdx.x * kThreads + threadIdx.x);
  if (i >= n) return;
  floatx4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int p = 0; p < a.splits; ++p) s += *reinterpret_cast<const floatx4*>(a.part + p * n + i);
  *reinterpret_cast<floatx4*>(a.drouter_w + i) = s;
}

}  // namespace

hipError_t launch_router_grad(const RouterGradArgs& a, hipStream_t s) {
  int shift = 0;
  while ((1 << shift) < a.H / 8 && (1 << shift) < kThreads) ++shift;
  const int per_block = kThreads >> shift;
  const int64_t blocks = ((int64_t)a.T + per_block - 1) / per_block;
  hipLaunchKernelGGL(router_grad_x_kernel, dim3((unsigned)(blocks < (int64_t)kMaxGrid ? blocks : (int64_t)kMaxGrid)),
                     dim3(kThreads), 0, s, a, shift);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(router_grad_w_kernel, dim3((a.H + 127) / 128, a.splits), dim3(kWave),
                     (size_t)a.E * 128 * sizeof(float), s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t quads = (int64_t)a.E * a.H / 4;
  hipLaunchKernelGGL(router_grad_join_kernel, dim3((unsigned)((quads + kThreads - 1) / kThreads)), dim3(kThreads), 0, s,
                     a);
  return hipGetLastError();
}

}  // namespace pw
