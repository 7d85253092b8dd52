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
// One launch for both.  dWr: a block takes one expert, up to 2048 columns and a
// stretch of the slots; its waves list the slots that the expert serves, with
// their token and dl, in LDS, then sum 512 columns each of the listed rows in
// registers (no atomics: the same inputs give the same bits).  A row is read by
// each of its k experts, so the blocks of one stretch and its columns go to one
// XCD, whose L2 serves all but the first.  dx: a wave takes a token; the
// router's rows come from L2, and dx is stored past it.  With several stretches
// a second launch sums their shares in order.
// Bound by memory: T = 16384, H = 4096, E = 8, k = 2 80 us, 5.0 TB/s of x, dx_add
// and dx; from E = 60 on also by the L2s, which serve each row of x and of the
// router k times (T = 32768, H = 2048, E = 60, k = 4 111 us, 3.6 TB/s; E = 256,
// k = 8 103 us for half the tokens).  With skewed routing by the hot expert's
// blocks, each of which sums all rows that its expert has in a stretch (136 us
// and 169 us for the same two).
#include "pw_rows.h"

namespace pw {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kLoads = 8;                // wave-wide loads of ids requested together
constexpr int kSegment = kLoads * kWave; // slots a wave looks at, and lists at most, at a time
constexpr int kListed = kWaves * kSegment;
constexpr int kXcds = 8;                 // consecutive blocks go to the XCDs in turn

struct __align__(8) Listed {
  int32_t t;
  float dl;
};

// dl of slot s, whose id is kept.
__device__ __forceinline__ Listed slot_dl(const RouterGradArgs& a, int64_t s) {
  const int64_t t = s / a.k;
  const int32_t* ids = a.ids + t * a.k;
  const float* w = a.w + t * a.k;
  const float* dw = a.dw + t * a.k;
  const int64_t j = s - t * a.k;
  const float mine = w[j], mine_dw = dw[j];
  float mean = 0.f;
#pragma unroll 4
  for (int i = 0; i < a.k; ++i) {
    const float wdw = w[i] * dw[i];
    mean += (uint32_t)ids[i] < (uint32_t)a.E ? wdw : 0.f;
  }
  return Listed{(int32_t)t, mine * mine_dw - mine * mean};
}

// WIDE: a wave takes 512 columns of a row (H >= 512); else the wave's lanes
// form 64 >> shift groups that each take a whole row.  1 << cshift waves of the
// block go to different columns, the others to different rows.
template <bool WIDE>
__device__ __forceinline__ void router_grad_w(const RouterGradArgs& a, int block) {
  using R = Row<PW_F16>;
  __shared__ __align__(32) Listed list[kListed];   // a segment a wave
  __shared__ int listed[kWaves];
  static_assert(sizeof(list) >= kThreads * sizeof(floatx8), "the waves' sums take the list's place at the end");
  const int wave = uniform((int)threadIdx.x / kWave), lane = (int)threadIdx.x & (kWave - 1);
  Listed* mine = list + wave * kSegment;
  const int cw = 1 << a.cshift, lanes = WIDE ? kWave : 1 << a.shift;
  const int groups = WIDE ? 1 : kWave >> a.shift;
  const int columns = (a.H + 512 * cw - 1) / (512 * cw);
  const int r = block / kXcds;
  const int e = r % a.E;
  const int tile = r / a.E * kXcds + block % kXcds;
  if (tile >= columns * a.splits) return;
  const int split = tile / columns;
  const int col = ((tile % columns) * cw + (wave & (cw - 1))) * 512 + 8 * (lane & (lanes - 1));
  const bool in = col < a.H;
  const int parts = (kWaves >> a.cshift) * groups;                   // rows go to the parts in turn
  const int part = (wave >> a.cshift) * groups + (WIDE ? 0 : lane >> a.shift);
  const int64_t S = (int64_t)a.T * a.k;
  const int64_t s0 = split * a.split_slots;
  const int64_t s1 = s0 + a.split_slots < S ? s0 + a.split_slots : S;
  const _Float16* x = reinterpret_cast<const _Float16*>(a.x) + (in ? col : 0);
  floatx8 sum = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t c0 = s0; c0 < s1; c0 += kListed) {
    // the wave's slots c0 + 64 (wave + 4 i) + lane that hold e, first as slots ...
    int32_t id[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int64_t s = c0 + (wave + kWaves * i) * kWave + lane;
      id[i] = s < s1 ? a.ids[s] : -1;
    }
    int n = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const unsigned long long mask = __ballot(id[i] == e);
      if (id[i] == e) mine[n + __popcll(mask & ((1ull << lane) - 1ull))].t = (wave + kWaves * i) * kWave + lane;
      n += __popcll(mask);
    }
    wave_lds_order();
    // ... then as tokens with their dl
    for (int i = lane; i < n; i += kWave) mine[i] = slot_dl(a, c0 + mine[i].t);
    if (lane == 0) listed[wave] = n;
    __syncthreads();
    const int n1 = uniform(listed[0]), n2 = n1 + uniform(listed[1]), n3 = n2 + uniform(listed[2]);
    const int rows = n3 + uniform(listed[3]);
    floatx8 acc = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};   // of this list alone
    // rows a part requests together (narrow rows have up to 64 parts: T = 31973, E = 129, H = 224 eight 58 us, four 39)
    constexpr int U = WIDE ? 8 : 4;
    for (int i0 = 0; i0 < rows; i0 += U * parts) {
      typename R::chunk v[U];
      float dl[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = i0 + u * parts + part;
        const int i = at < rows ? at : rows - 1;
        const int from = i < n1 ? 0 : i < n2 ? kSegment - n1 : i < n3 ? 2 * kSegment - n2 : 3 * kSegment - n3;
        const Listed l = list[from + i];
        dl[u] = l.dl;
        v[u] = R::load(x + (int64_t)(WIDE ? uniform(l.t) : l.t) * a.H);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * parts + part < rows) acc += dl[u] * R::wide(v[u]);
    }
    sum += acc;
    __syncthreads();
  }
  if (parts > 1) {
    floatx8* sums = reinterpret_cast<floatx8*>(list);
    sums[threadIdx.x] = sum;
    __syncthreads();
    if (part != 0) return;
    for (int q = 1; q < parts; ++q)
      sum += sums[((q / groups << a.cshift) + wave) * kWave + q % groups * lanes + lane];
  }
  if (in) Row<PW_F32>::store((a.splits > 1 ? a.part : a.drouter_w) + ((int64_t)split * a.E + e) * a.H + col, sum);
}

// dx of one token over `kXChunks` chunks a lane from chunk c0 on.  Lane j holds
// slot j (k <= 64): its expert and dl, handed to the wave a few at a time, so
// that the rows of kXSlots slots are requested together.
constexpr int kXChunks = 2, kXSlots = 2;

__device__ __forceinline__ void router_grad_x(const RouterGradArgs& a, int64_t t, int c0) {
  using R = Row<PW_F16>;
  const int lane = (int)threadIdx.x & (kWave - 1);
  const int C = a.H / 8;
  int c[kXChunks];
  bool in[kXChunks];
  typename R::chunk add[kXChunks];
  const _Float16* wr = reinterpret_cast<const _Float16*>(a.router_w);
#pragma unroll
  for (int u = 0; u < kXChunks; ++u) {
    c[u] = c0 + u * kWave + lane;
    in[u] = c[u] < C;
    if (!in[u]) c[u] = 0;
    if (a.dx_add) add[u] = R::load(reinterpret_cast<const _Float16*>(a.dx_add) + t * a.H + 8 * c[u]);
  }
  int32_t id = -1;
  float w = 0.f, wdw = 0.f;
  if (lane < a.k) {
    id = a.ids[t * a.k + lane];
    w = a.w[t * a.k + lane];
    wdw = w * a.dw[t * a.k + lane];
  }
  const bool kept = (uint32_t)id < (uint32_t)a.E;
  if (!kept) id = 0;                       // read, with dl 0
  const float mean = wave_sum(kept ? wdw : 0.f);
  const float dl = kept ? wdw - w * mean : 0.f;
  const unsigned long long slots = __ballot(kept);
  floatx8 acc[kXChunks];
#pragma unroll
  for (int u = 0; u < kXChunks; ++u)
    acc[u] = a.dx_add ? R::wide(add[u]) : floatx8{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < a.k; j0 += kXSlots) {
    typename R::chunk m[kXSlots][kXChunks];
#pragma unroll
    for (int j = 0; j < kXSlots; ++j) {
      const int64_t row = (int64_t)__builtin_amdgcn_readlane(id, (j0 + j) & (kWave - 1)) * a.H;
#pragma unroll
      for (int u = 0; u < kXChunks; ++u) m[j][u] = R::load(wr + row + 8 * c[u]);
    }
#pragma unroll
    for (int j = 0; j < kXSlots; ++j) {
      if (!(slots >> ((j0 + j) & (kWave - 1)) & 1)) continue;   // a dropped slot adds nothing, whatever the row holds
      const float f = row_lane(dl, (j0 + j) & (kWave - 1));
#pragma unroll
      for (int u = 0; u < kXChunks; ++u) acc[u] += f * R::wide(m[j][u]);
    }
  }
#pragma unroll
  for (int u = 0; u < kXChunks; ++u)
    if (in[u]) R::store_once(reinterpret_cast<_Float16*>(a.dx) + t * a.H + 8 * c[u], R::narrow(acc[u]));
}

// dx where a wave's lanes form groups that each take a token's whole row: every
// lane finds its token's dl by itself.
__device__ __forceinline__ void router_grad_x_narrow(const RouterGradArgs& a, int64_t t, int lane) {
  using R = Row<PW_F16>;
  if (t >= a.T || 8 * lane >= a.H) return;
  const int32_t* ids = a.ids + t * a.k;
  const float* w = a.w + t * a.k;
  const float* dw = a.dw + t * a.k;
  floatx8 acc = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (a.dx_add) acc = R::wide(R::load(reinterpret_cast<const _Float16*>(a.dx_add) + t * a.H + 8 * lane));
  float mean = 0.f;
#pragma unroll 4
  for (int j = 0; j < a.k; ++j) {
    const float wdw = w[j] * dw[j];
    mean += (uint32_t)ids[j] < (uint32_t)a.E ? wdw : 0.f;
  }
#pragma unroll 4
  for (int j = 0; j < a.k; ++j) {
    const int32_t e = ids[j];
    const bool kept = (uint32_t)e < (uint32_t)a.E;
    const float wj = w[j], dl = wj * dw[j] - wj * mean;
    const _Float16* row = reinterpret_cast<const _Float16*>(a.router_w) + (int64_t)(kept ? e : 0) * a.H + 8 * lane;
    const floatx8 v = R::wide(R::load(row));
    if (kept) acc += dl * v;
  }
  R::store_once(reinterpret_cast<_Float16*>(a.dx) + t * a.H + 8 * lane, R::narrow(acc));
}

template <bool WIDE>
__global__ __launch_bounds__(kThreads) void router_grad_kernel(RouterGradArgs a, int w_blocks) {
  if ((int)blockIdx.x < w_blocks) {
    router_grad_w<WIDE>(a, (int)blockIdx.x);
    return;
  }
  const int64_t block = blockIdx.x - w_blocks, blocks = gridDim.x - w_blocks;
  if constexpr (WIDE) {
    const int pieces = (a.H / 8 + kXChunks * kWave - 1) / (kXChunks * kWave);
    const int64_t n = (int64_t)a.T * pieces;
    for (int64_t i = block * kWaves + uniform((int)threadIdx.x / kWave); i < n; i += blocks * kWaves)
      router_grad_x(a, i / pieces, (int)(i % pieces) * kXChunks * kWave);
  } else {
    const int tokens = kThreads >> a.shift;
    for (int64_t t = block * tokens; t < a.T; t += blocks * tokens)
      router_grad_x_narrow(a, t + ((int)threadIdx.x >> a.shift), (int)threadIdx.x & ((1 << a.shift) - 1));
  }
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
  constexpr int64_t kMost = 1 << 20;
  const int columns = (a.H + (512 << a.cshift) - 1) / (512 << a.cshift);
  const int w_blocks = (columns * a.splits + kXcds - 1) / kXcds * kXcds * a.E;
  const bool wide = a.H >= 512;
  const int pieces = (a.H / 8 + kXChunks * kWave - 1) / (kXChunks * kWave);
  const int tokens = kThreads >> a.shift;
  int64_t x_blocks = wide ? ((int64_t)a.T * pieces + kWaves - 1) / kWaves : ((int64_t)a.T + tokens - 1) / tokens;
  if (x_blocks > kMost) x_blocks = kMost;
  const dim3 grid((unsigned)(w_blocks + x_blocks));
  if (wide) hipLaunchKernelGGL(router_grad_kernel<true>, grid, dim3(kThreads), 0, s, a, w_blocks);
  else hipLaunchKernelGGL(router_grad_kernel<false>, grid, dim3(kThreads), 0, s, a, w_blocks);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t quads = (int64_t)a.E * a.H / 4;
  hipLaunchKernelGGL(router_grad_join_kernel, dim3((unsigned)((quads + kThreads - 1) / kThreads)), dim3(kThreads), 0, s,
                     a);
  return hipGetLastError();
}

}  // namespace pw
