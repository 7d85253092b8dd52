// The experts' products for few rows (decoding): what bounds them is reading
// every reached matrix once, so nothing is staged.  A block takes 16 rows of W
// (gated: 16 of g and the same 16 of u) and up to 64 rows of x of one expert;
// its eight waves take every eighth 64 steps of the reduction each, with the
// loads of several such pieces in flight, straight into the operands of the
// matrix cores, and add their sums through LDS in the order of the waves.  H 2048,
// I 1408, E 60, 16 rows over 14 experts: 240 MB in 49 us, 5 TB/s.  One row through
// one expert of I 5632: gate and up, 46 MB, 12.5 us, down, 23 MB, 9.3 (2.5 TB/s: its
// 128 blocks leave half of the CUs without one, and the loads of a round of pieces
// are waited for before the next round's are asked for).
#include "pw_product.h"

namespace pw {

namespace {

constexpr int kFewWaves = 8;
constexpr int kFewAhead = 2;   // pieces of 64 steps in flight (4: 52 us for 49, 4 rows each 167 for 154)

// RT: tiles of 16 rows of x
template <int DT, int EPI, int RT>
__global__ __launch_bounds__(kFewWaves * kWave) void few_kernel(ProductArgs a) {
  using elem = typename RowType<DT>::elem;
  constexpr bool kGate = EPI == kProductGate;
  constexpr int NF = kGate ? 2 : 1;
  __shared__ float part[kFewWaves][NF][RT][256];
  const Tile t = find_tile<RT * 16>(a.offsets, a.E, a.S, a.NT);
  if (t.rows <= 0) return;
  const int wave = uniform((int)threadIdx.x / kWave), lane = (int)threadIdx.x & (kWave - 1);
  const int n0 = t.nt * 16, r = lane & 15;
  const int K = a.K;
  // lane l holds row l % 16 and steps 8 (l / 16) .. + 7 and 32 more of a piece, the same ones of x and of W
  const char* w[NF];
  const char* x[RT];
  const int col = min(n0 + r, a.N - 1);
#pragma unroll
  for (int f = 0; f < NF; ++f)
    w[f] = static_cast<const char*>(a.w) + ((int64_t)t.e * a.w_expert + (int64_t)(f * a.N + col) * K) * 2;
#pragma unroll
  for (int i = 0; i < RT; ++i)
    x[i] = static_cast<const char*>(a.x) + (int64_t)(t.row0 + min(i * 16 + r, t.rows - 1)) * a.x_stride * 2;
  f32x4 acc[NF][RT];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[f][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const s16x8 zero = {0, 0, 0, 0, 0, 0, 0, 0};
  const int own = (lane >> 4) * 8;
  constexpr int kStep = kFewWaves * 64;
  for (int base = wave * 64; base < K; base += kStep * kFewAhead) {
    s16x8 wf[kFewAhead][NF][2], xf[kFewAhead][RT][2];
#pragma unroll
    for (int u = 0; u < kFewAhead; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = base + u * kStep + own + 32 * h;
        const bool in = k < K;
        const int at = in ? k * 2 : 0;
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          wf[u][f][h] = *reinterpret_cast<const s16x8*>(w[f] + at);
          if (!in) wf[u][f][h] = zero;
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          xf[u][i][h] = *reinterpret_cast<const s16x8*>(x[i] + at);
          if (!in) xf[u][i][h] = zero;
        }
      }
    __builtin_amdgcn_sched_barrier(0);   // every load before the first product
#pragma unroll
    for (int u = 0; u < kFewAhead; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
          for (int i = 0; i < RT; ++i) acc[f][i] = Mma<DT>::mma(wf[u][f][h], xf[u][i][h], acc[f][i]);
  }
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) part[wave][f][i][j * kWave + lane] = acc[f][i][j];
  __syncthreads();
  const int rows = min(t.rows, RT * 16);
  for (int it = threadIdx.x; it < RT * 256; it += kFewWaves * kWave) {
    const int c = it & 15, own_row = it / 16, i = own_row / 16, n = n0 + c;
    if (own_row >= rows || n >= a.N) continue;
    const int at = (c & 3) * kWave + (c / 4) * 16 + (own_row & 15);
    float v[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      v[f] = part[0][f][i][at];
#pragma unroll
      for (int k = 1; k < kFewWaves; ++k) v[f] += part[k][f][i][at];
    }
    const int64_t row = t.row0 + own_row;
    float y;
    if constexpr (kGate) {
      if (a.z) {
        elem* z = static_cast<elem*>(a.z) + row * a.z_stride + n;
        z[0] = (elem)v[0];
        z[a.N] = (elem)v[1];
      }
      y = act_of(v[0], a.act) * v[1];
    } else {
      y = v[0];
      if (a.bias) y += (float)static_cast<const elem*>(a.bias)[(int64_t)t.e * a.N + n];
      if (a.pre) static_cast<elem*>(a.pre)[row * a.pre_stride + n] = (elem)y;
      y = act_of(y, a.act);
      if (a.residual) y += (float)static_cast<const elem*>(a.residual)[row * a.residual_stride + n];
    }
    static_cast<elem*>(a.y)[row * a.y_stride + n] = (elem)y;
  }
}

// Tiles of 16 rows of x that a block takes.
int row_pieces(int E, int64_t S) {
  const int64_t experts = S < E ? S : E, mean = S / experts;
  return mean > 16 ? 4 : mean > 4 ? 2 : 1;
}
int64_t blocks_of(const ProductArgs& a, int pieces) {
  return product_grid(product_row_tiles(a.offsets != nullptr, a.E, a.S, pieces * 16), (a.N + 15) / 16);
}

template <int DT, int EPI, int RT>
hipError_t run(ProductArgs a, hipStream_t s) {
  a.NT = (a.N + 15) / 16;
  const int64_t grid = blocks_of(a, RT);
  hipLaunchKernelGGL((few_kernel<DT, EPI, RT>), dim3((unsigned)grid), dim3(kFewWaves * kWave), 0, s, a);
  return hipGetLastError();
}

template <int DT, int EPI>
hipError_t pick(const ProductArgs& a, hipStream_t s) {
  switch (row_pieces(a.E, a.S)) {
    case 4: return run<DT, EPI, 4>(a, s);
    case 2: return run<DT, EPI, 2>(a, s);
    default: return run<DT, EPI, 1>(a, s);
  }
}

}  // namespace

// No 8-bit copies: a block has 16 columns of a group of 128.  Matrices so long that
// their blocks are more than a launch has (256 rows over 256 experts, N 2^20) take tiles.
bool few_rows(const ProductArgs& a, int kind) {
  if ((kind != kProductAct && kind != kProductGate) || a.z8) return false;
  return few_rows_for(a.E, a.S, (int64_t)a.N * a.K * (kind == kProductGate ? 2 : 1)) &&
         launch_fits(blocks_of(a, row_pieces(a.E, a.S)), kFewWaves * kWave);
}

hipError_t launch_few(const ProductArgs& a, int dtype, int kind, hipStream_t s) {
  if (kind == kProductGate)
    return dtype == PW_F16 ? pick<PW_F16, kProductGate>(a, s) : pick<PW_BF16, kProductGate>(a, s);
  return dtype == PW_F16 ? pick<PW_F16, kProductAct>(a, s) : pick<PW_BF16, kProductAct>(a, s);
}

}  // namespace pw
