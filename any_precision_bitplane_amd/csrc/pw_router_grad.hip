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
// One launch for both.  dWr: a block takes one expert, 2048 columns and a
// stretch of tokens; its waves list the tokens that the expert serves, with
// their dl, in LDS, then each sums 512 columns of the listed rows in registers
// (no atomics: the same inputs give the same bits).  A row is read by each of
// its k experts, so the blocks of one stretch and its columns go to one XCD,
// whose L2 serves all but the first.  dx: a wave takes a token; the router's
// rows come from L2.  With several stretches a second launch sums their shares
// in order.
#include "pw_rows.h"

namespace pw {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kListed = 512;             // tokens whose matches a block lists at a time
constexpr int kSegment = kListed / kWaves;
constexpr int kXcds = 8;                 // consecutive blocks go to the XCDs in turn

struct Listed {
  int32_t t;
  float dl;
};

// The token's dl for expert e, summed over the slots that hold e (`hit`: there is one).
__device__ __forceinline__ float token_dl(const RouterGradArgs& a, int64_t t, int e, bool& hit) {
  const int32_t* ids = a.ids + t * a.k;
  const float* w = a.w + t * a.k;
  const float* dw = a.dw + t * a.k;
  hit = false;
  float mean = 0.f, sum_w = 0.f, sum_wdw = 0.f;
#pragma unroll 4
  for (int j = 0; j < a.k; ++j) {
    const int32_t id = ids[j];
    const float wj = w[j], wdw = wj * dw[j];
    if ((uint32_t)id < (uint32_t)a.E) mean += wdw;
    if (id == e) {
      hit = true;
      sum_w += wj;
      sum_wdw += wdw;
    }
  }
  return sum_wdw - sum_w * mean;
}

__device__ __forceinline__ void router_grad_w(const RouterGradArgs& a, int block) {
  using R = Row<PW_F16>;
  __shared__ Listed list[kWaves][kSegment];
  __shared__ int listed[kWaves];
  const int wave = uniform((int)threadIdx.x / kWave), lane = (int)threadIdx.x & (kWave - 1);
  const int columns = (a.H + 2047) / 2048;
  const int r = block / kXcds;
  const int e = r % a.E;
  const int tile = r / a.E * kXcds + block % kXcds;
  if (tile >= columns * a.splits) return;
  const int split = tile / columns;
  const int col = (tile % columns) * 2048 + wave * 512 + 8 * lane;
  const bool in = col < a.H;
  const int64_t t0 = (int64_t)split * a.split_tokens;
  const int64_t t1 = t0 + a.split_tokens < a.T ? t0 + a.split_tokens : a.T;
  const _Float16* x = reinterpret_cast<const _Float16*>(a.x) + (in ? col : 0);
  floatx8 sum = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t c0 = t0; c0 < t1; c0 += kListed) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kSegment / kWave; ++i) {
      const int64_t t = c0 + wave * kSegment + i * kWave + lane;
      bool hit = false;
      float dl = 0.f;
      if (t < t1) dl = token_dl(a, t, e, hit);
      const unsigned long long mask = __ballot(hit);
      if (hit) list[wave][n + __popcll(mask & ((1ull << lane) - 1ull))] = Listed{(int32_t)t, dl};
      n += __popcll(mask);
    }
    if (lane == 0) listed[wave] = n;
    __syncthreads();
    floatx8 acc = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};   // of at most kListed rows
    for (int s = 0; s < kWaves; ++s) {
      const int m = uniform(listed[s]);
      constexpr int U = 8;   // rows requested together
      for (int i = 0; i < m; i += U) {
        typename R::chunk v[U];
        float dl[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const Listed l = list[s][i + u < m ? i + u : m - 1];
          dl[u] = i + u < m ? l.dl : 0.f;
          v[u] = R::load(x + (int64_t)uniform(l.t) * a.H);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (i + u < m) acc += dl[u] * R::wide(v[u]);
      }
    }
    sum += acc;
    __syncthreads();
  }
  if (in) Row<PW_F32>::store((a.splits > 1 ? a.part : a.drouter_w) + ((int64_t)split * a.E + e) * a.H + col, sum);
}

// Lane j holds slot j (k <= 64): its expert and dl, handed to the wave one by one.
__device__ __forceinline__ void router_grad_x(const RouterGradArgs& a, int64_t t) {
  using R = Row<PW_F16>;
  const int lane = (int)threadIdx.x & (kWave - 1);
  const int C = a.H / 8;
  int32_t id = -1;
  float w = 0.f, wdw = 0.f;
  if (lane < a.k) {
    id = a.ids[t * a.k + lane];
    w = a.w[t * a.k + lane];
    wdw = w * a.dw[t * a.k + lane];
  }
  const bool kept = (uint32_t)id < (uint32_t)a.E;
  const _Float16* add = reinterpret_cast<const _Float16*>(a.dx_add) + t * a.H;
  const _Float16* wr = reinterpret_cast<const _Float16*>(a.router_w);
  _Float16* dx = reinterpret_cast<_Float16*>(a.dx) + t * a.H;
  constexpr int U = 4;   // chunks of a row requested together
  typename R::chunk v[U];
  if (a.dx_add)
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (lane + u * kWave < C) v[u] = R::load(add + 8 * (lane + u * kWave));
  const float mean = wave_sum(kept ? wdw : 0.f);
  const float dl = kept ? wdw - w * mean : 0.f;
  for (int c0 = lane; c0 - lane < C; c0 += U * kWave) {
    floatx8 acc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (a.dx_add && c0 >= U * kWave && c0 + u * kWave < C) v[u] = R::load(add + 8 * (c0 + u * kWave));
      acc[u] = floatx8{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (a.dx_add && c0 + u * kWave < C) acc[u] = R::wide(v[u]);
    }
    for (int j = 0; j < a.k; ++j) {
      const int32_t e = __builtin_amdgcn_readlane(id, j);
      if ((uint32_t)e >= (uint32_t)a.E) continue;
      const float f = row_lane(dl, j);
      const _Float16* row = wr + (int64_t)e * a.H;
      typename R::chunk m[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + u * kWave < C) m[u] = R::load(row + 8 * (c0 + u * kWave));
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + u * kWave < C) acc[u] += f * R::wide(m[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * kWave < C) R::store(dx + 8 * (c0 + u * kWave), R::narrow(acc[u]));
  }
}

__global__ __launch_bounds__(kThreads) void router_grad_kernel(RouterGradArgs a, int w_blocks) {
  if ((int)blockIdx.x < w_blocks) {
    router_grad_w(a, (int)blockIdx.x);
    return;
  }
  const int64_t step = (int64_t)(gridDim.x - w_blocks) * kWaves;
  for (int64_t t = (int64_t)(blockIdx.x - w_blocks) * kWaves + uniform((int)threadIdx.x / kWave); t < a.T; t += step)
    router_grad_x(a, t);
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
  const int columns = (a.H + 2047) / 2048;
  const int w_blocks = (columns * a.splits + kXcds - 1) / kXcds * kXcds * a.E;
  const int64_t x_blocks = ((int64_t)a.T + kWaves - 1) / kWaves;
  constexpr int64_t kMost = 1 << 20;
  hipLaunchKernelGGL(router_grad_kernel, dim3((unsigned)(w_blocks + (x_blocks < kMost ? x_blocks : kMost))),
                     dim3(kThreads), 0, s, a, w_blocks);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t quads = (int64_t)a.E * a.H / 4;
  hipLaunchKernelGGL(router_grad_join_kernel, dim3((unsigned)((quads + kThreads - 1) / kThreads)), dim3(kThreads), 0, s,
                     a);
  return hipGetLastError();
}

}  // namespace pw
