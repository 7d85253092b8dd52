// Gradients of the experts' products that run over an expert's rows:
//
//   dW[n][k] = sum_s dz[s][n] x[s][k]        dz = dy act'(pre)
//   dbias[n] = sum_s dz[s][n]
//
// The weight's gradient is a product whose reduction runs over the rows, so both
// operands are transposed on their way from LDS to the matrix cores.  Rows past
// the expert's last read as zero in both operands, so what lies behind (NaN too)
// adds nothing.  What bounds it: the matrix cores with many rows an expert (8192
// rows over 8, 28672 x 4096 fp16 1.9 ms, 1010 TFLOP/s), writing the result with
// few (E 60, 17 rows each, 2816 x 2048, 692 MB in 178 us).
#include "pw_product.h"

namespace pw {

namespace {

// Tiles of 256 x 256 of eight waves, one block a CU; or of TM x 128 of four, in
// steps of 32, two or more blocks a CU, which is faster for few rows an expert,
// where a tile is mostly its first copies and its stores (E 60, 17 rows each,
// H 2048, I 1408: 440 us for the whole gradient against 466), and where there are
// few tiles, and slower otherwise (its tiles read half as much again: E 8, 1024
// rows each, H 4096, I 14336 5.53 ms against 5.31; between them: outer_is_short).
template <int TM, int TN>
struct OuterShape {
  static constexpr bool kShort = TN == 128;
  static constexpr int WM = 2, WN = TN / 64, kWaves = WM * WN, RI = TM / 16 / WM, CJ = TN / 16 / WN;
  static constexpr int kStep = kShort ? 32 : kProdK, kLds = (kShort ? 3 * (TM + TN) : 3 * TM + 2 * TN) * kStep * 2;
  static_assert(CJ == 4 && kWaves * Sums::kBytes <= kLds, "64 columns a wave");
};

template <int DT, int TM, int TN>
__global__ __launch_bounds__((OuterShape<TM, TN>::kWaves * kWave), 2) void outer_kernel(OuterArgs a) {
  using R = Row<DT>;
  using elem = typename R::elem;
  using Sh = OuterShape<TM, TN>;
  __shared__ __align__(1024) char lds[Sh::kLds];
  // Every expert's tiles are dealt to the eight XCDs, in a contiguous stretch each: experts differ in their rows.
  const unsigned per = (unsigned)(a.MT * a.NT), share = (per + 7) / 8, i = blockIdx.x / 8;
  const int e = (int)(i / share), local = (int)(blockIdx.x % 8 * share + i - (unsigned)e * share);
  if (local >= (int)per) return;
  const int group = local / (kProdGroup * a.NT), rem = local - group * kProdGroup * a.NT;
  const int here = min(kProdGroup, a.MT - group * kProdGroup);
  const int nt = rem / here, mt = group * kProdGroup + rem - nt * here;
  int row0, rows;
  expert_rows(a.offsets, e, a.S, row0, rows);
  row0 = uniform(row0);
  rows = uniform(rows);
  if (a.parts > 1) {   // this block's stretch of the rows
    const int all = (rows + Sh::kStep - 1) / Sh::kStep, p = (int)blockIdx.y;
    const int from = (int)((int64_t)all * p / a.parts) * Sh::kStep, to = (int)((int64_t)all * (p + 1) / a.parts) * Sh::kStep;
    row0 += from;
    rows = min(rows, to) - from;
  }
  const int wave = uniform((int)threadIdx.x / kWave), lane = (int)threadIdx.x & (kWave - 1);
  const int wm = wave / Sh::WN, wn = wave % Sh::WN;
  ColsOperand<TM, Sh::kWaves, Sh::kStep> po;
  ColsOperand<TN, Sh::kWaves, Sh::kStep> qo;
  po.init(static_cast<const char*>(a.p) + ((int64_t)row0 * a.p_stride + mt * TM) * 2, rows, wave, lane, a.p_stride * 2,
          (a.M - mt * TM + 7) / 8);
  qo.init(static_cast<const char*>(a.q) + ((int64_t)row0 * a.q_stride + nt * TN) * 2, rows, wave, lane, a.q_stride * 2,
          (a.N - nt * TN + 7) / 8);
  f32x4 acc[Sh::RI][Sh::CJ];
  const int steps = (rows + Sh::kStep - 1) / Sh::kStep;
  const int live = nt * TN + wn * 64 < a.N ? (a.M - mt * TM - wm * Sh::RI * 16 + 15) / 16 : 0;
  if constexpr (Sh::kShort)
    sum_short_steps<DT, Sh::RI, Sh::CJ, TM, TN>(acc, lds, steps, live, wave, wm, wn, lane, po, qo);
  else
    sum_steps<DT, Sh::RI, Sh::CJ, TM, TN, false, true, true, 3>(acc, lds, steps, live, wave, wm, wn, lane, po, qo);
  elem* out = static_cast<elem*>(a.out) + (int64_t)e * a.M * a.N;
  Sums sums(lds, wave, lane);
  const int n = nt * TN + wn * 64 + (lane & 7) * 8;
#pragma unroll
  for (int mi = 0; mi < Sh::RI / 2; ++mi) {
    sums.put(acc[2 * mi], acc[2 * mi + 1]);
#pragma unroll
    for (int r = lane / 8; r < 32; r += 8) {
      const int m = mt * TM + (wm * (Sh::RI / 2) + mi) * 32 + r;
      const floatx8 v = sums.get(r, lane & 7);
      if (a.parts > 1) {
        float* const to = a.part + (((int64_t)blockIdx.y * a.E + e) * per + local) * (TM * TN);
        *reinterpret_cast<floatx8*>(to + (m - mt * TM) * TN + n - nt * TN) = v;
        continue;
      }
      if (m < a.M && n < a.N) R::store_once(out + (int64_t)m * a.N + n, R::narrow(v));
    }
  }
}

// Adds the stretches' sums, in their order: sixteen lanes a row of a tile.
template <int DT>
__global__ __launch_bounds__(256) void outer_join_kernel(OuterArgs a) {
  using R = Row<DT>;
  constexpr int T = 128;
  const unsigned per = (unsigned)(a.MT * a.NT), e = blockIdx.x / per, local = blockIdx.x - e * per;
  // as outer_kernel numbers them
  const int group = (int)local / (kProdGroup * a.NT), rem = (int)local - group * kProdGroup * a.NT;
  const int here = min(kProdGroup, a.MT - group * kProdGroup), nt = rem / here, mt = group * kProdGroup + rem - nt * here;
  const int r = (int)blockIdx.y * 16 + (int)threadIdx.x / 16, c = ((int)threadIdx.x & 15) * 8;
  if (mt * T + r >= a.M || nt * T + c >= a.N) return;
  const float* from = a.part + ((int64_t)e * per + local) * (T * T) + r * T + c;
  floatx8 v = *reinterpret_cast<const floatx8*>(from);
  for (int p = 1; p < a.parts; ++p) v += *reinterpret_cast<const floatx8*>(from + (int64_t)p * a.E * per * (T * T));
  R::store_once(static_cast<typename R::elem*>(a.out) + ((int64_t)e * a.M + mt * T + r) * a.N + nt * T + c, R::narrow(v));
}

// dz and the columns' sums of stretches of kDzRows rows of one expert: a block
// has 256 columns, a wave two rows at a time.  dz is rounded to the rows' type, as
// the matrix cores of both products that read it take it (bf16 error against 64
// bits 2.3e-3 for 1.7e-3); the columns' sums are of the unrounded values.
constexpr int kDzRows = 128;
constexpr int kDzThreads = 256;

template <int DT>
__global__ __launch_bounds__(kDzThreads) void dz_kernel(DzArgs a) {
  using R = Row<DT>;
  using elem = typename R::elem;
  __shared__ float part[kDzThreads / 32][256];
  const Tile t = find_tile<kDzRows>(a.offsets, a.E, a.S, (a.N + 255) / 256);
  if (t.rows <= 0) return;
  const int lane = threadIdx.x & 31, own = threadIdx.x / 32;
  const int n = t.nt * 256 + lane * 8;
  floatx8 sum = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (n < a.N) {
    const int rows = min(t.rows, kDzRows);
    for (int r = own; r < rows; r += kDzThreads / 32) {
      const int64_t row = t.row0 + r;
      floatx8 d = R::wide(R::load(static_cast<const elem*>(a.dy) + row * a.dy_stride + n));
      if (a.act != PW_ACT_NONE) {
        const floatx8 z = R::wide(R::load(static_cast<const elem*>(a.pre) + row * a.pre_stride + n));
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] *= act_slope(z[j], a.act);
        if (a.dz) R::store(static_cast<elem*>(a.dz) + row * a.N + n, R::narrow(d));
      }
      sum += d;
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) part[own][lane * 8 + j] = sum[j];
  __syncthreads();
  const int c = t.nt * 256 + (int)threadIdx.x;
  if (c >= a.N) return;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kDzThreads / 32; ++i) s += part[i][threadIdx.x];
  // an expert's first stretch lies behind those of the experts before it
  a.part[((int64_t)t.row0 / kDzRows + t.e) * a.N + c] = s;
}

template <int DT>
__global__ __launch_bounds__(kDzThreads) void bias_grad_kernel(DzArgs a) {
  using elem = typename RowType<DT>::elem;
  const int c = (int)(blockIdx.x * kDzThreads + threadIdx.x), e = (int)blockIdx.y;
  if (c >= a.N) return;
  int row0, rows;
  expert_rows(a.offsets, e, a.S, row0, rows);
  float s = 0.f;
  for (int r = 0; r < rows; r += kDzRows) s += a.part[((int64_t)(row0 + r) / kDzRows + e) * a.N + c];
  static_cast<elem*>(a.dbias)[(int64_t)e * a.N + c] = (elem)s;
}

template <int DT, int TM, int TN>
hipError_t run_outer(OuterArgs a, hipStream_t s) {
  a.MT = (a.M + TM - 1) / TM;
  a.NT = (a.N + TN - 1) / TN;
  const int64_t grid = ((int64_t)a.MT * a.NT + 7) / 8 * 8 * a.E;
  if (!launch_fits(grid, OuterShape<TM, TN>::kWaves * kWave)) return hipErrorInvalidValue;
  a.parts = TM == 128 ? outer_parts(a.E, a.S, a.M, a.N) : 1;
  hipLaunchKernelGGL((outer_kernel<DT, TM, TN>), dim3((unsigned)grid, (unsigned)a.parts),
                     dim3(OuterShape<TM, TN>::kWaves * kWave), 0, s, a);
  if (a.parts > 1)
    hipLaunchKernelGGL(outer_join_kernel<DT>, dim3((unsigned)(a.MT * a.NT * a.E), 8), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int DT>
hipError_t pick_outer(const OuterArgs& a, hipStream_t s) {
  if (outer_is_small(a.E, a.M, a.N)) return run_outer<DT, 128, 128>(a, s);
  return outer_is_short(a.E, a.S) ? run_outer<DT, 256, 128>(a, s) : run_outer<DT, 256, 256>(a, s);
}

template <int DT>
hipError_t run_dz(const DzArgs& a, hipStream_t s) {
  if (a.S > 0) {
    const int64_t grid = product_grid(product_row_tiles(a.offsets != nullptr, a.E, a.S, kDzRows), (a.N + 255) / 256);
    if (!launch_fits(grid, kDzThreads)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(dz_kernel<DT>, dim3((unsigned)grid), dim3(kDzThreads), 0, s, a);
  }
  if (a.dbias)
    hipLaunchKernelGGL(bias_grad_kernel<DT>, dim3((unsigned)((a.N + kDzThreads - 1) / kDzThreads), (unsigned)a.E),
                       dim3(kDzThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

size_t dz_part_floats(int E, int64_t S, int N) { return (size_t)(S / kDzRows + E) * (size_t)N; }

hipError_t launch_outer(const OuterArgs& a, int dtype, hipStream_t s) {
  return dtype == PW_F16 ? pick_outer<PW_F16>(a, s) : pick_outer<PW_BF16>(a, s);
}

hipError_t launch_dz(const DzArgs& a, int dtype, hipStream_t s) {
  return dtype == PW_F16 ? run_dz<PW_F16>(a, s) : run_dz<PW_BF16>(a, s);
}

}  // namespace pw
