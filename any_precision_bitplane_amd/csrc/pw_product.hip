// Products of every expert's rows with its matrix, with what follows them:
//
//   product        z = x W^T + bias,  y = act(z) + residual          W [N][K]
//   gated          [g | u] = x W^T,   h = act(g) u                   W [2N][K]
//   back           dx = dz W                                         W [K][N]
//   gated, back    dh = dy W,  dg = dh u act'(g),  du = dh act(g),  h = act(g) u
//
// in tiles of 32 to 256 rows by 256 columns (gated: 128 of g and the same 128 of
// u, so that a lane holds both for its columns).
#include "pw_product.h"

namespace pw {

namespace {

// WM x WN waves, each with 32 MI rows and 128 / WN columns in either half.
template <int MI, int WM, int WN>
struct Shape {
  static constexpr int RI = 2 * MI, CJ = 16 / WN;   // pieces of 16 rows and of 16 columns
  static constexpr int kRows = MI * WM * 32;
  static constexpr int kWaves = WM * WN;
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int kABytes = kRows * kProdK * 2;
  static constexpr int kXBuffers = MI * WM == 2 ? 2 : 3;   // two blocks a CU with tiles of 32 and 64 rows
  static constexpr int kLds = kXBuffers * kABytes + 2 * kProdN * kProdK * 2;
  static_assert(kWaves * Sums<CJ>::kBytes + 2 * kRows * WN * 4 <= kLds, "LDS of what follows the products");
};

template <int DT, int EPI, int MI, int WM, int WN>
__device__ __forceinline__ void finish(const ProductArgs& a, const Tile& t,
                                       f32x4 (&acc)[2 * MI][16 / WN], char* lds, int wave, int lane) {
  using R = Row<DT>;
  using elem = typename R::elem;
  constexpr int kHalf = Shape<MI, WM, WN>::CJ / 2, kRows = Shape<MI, WM, WN>::kRows;   // pieces of columns in a half
  const int hi = lane / 32, wm = wave / WN, wn = wave % WN;
  Sums<16 / WN> sums(lds, wave, lane);
  constexpr bool kGate = EPI == kProductGate;
  const int n0 = t.nt * (kGate ? kKeepGroup : kProdN) + wn * kHalf * 16 + 8 * hi;   // of the lane's first eight columns
  float scale[MI][2];
  if (kGate && a.z8) {
    // the largest |g| and |u| of each row over the tile's 128 columns: over a lane's, its pair's and the waves'
    float* part = reinterpret_cast<float*>(lds + Shape<MI, WM, WN>::kWaves * Sums<16 / WN>::kBytes);
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float most = 0.f;
#pragma unroll
        for (int c = 0; c < kHalf; ++c) {
          const floatx8 v = eight_columns(acc[2 * mi][half * kHalf + c], acc[2 * mi + 1][half * kHalf + c]);
          if (n0 + 16 * c < a.N) most = most_of(v, most);
        }
        most = fmaxf(most, __shfl_xor(most, 32, kWave));
        if (hi == 0) part[(half * kRows + (wm * MI + mi) * 32 + lane) * WN + wn] = most;
      }
    __syncthreads();
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float* p = part + (half * kRows + (wm * MI + mi) * 32 + (lane & 31)) * WN;
        float most = fmaxf(p[0], p[1]);
        if constexpr (WN == 4) most = fmaxf(most, fmaxf(p[2], p[3]));
        scale[mi][half] = scale_of(most);
      }
  }
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    sums.put(acc[2 * mi], acc[2 * mi + 1]);
    const int r = (wm * MI + mi) * 32 + (lane & 31);
    if (r >= t.rows) continue;
    const int64_t row = t.row0 + r;
    if constexpr (kGate) {
      if (a.z8 && wn == 0 && hi == 0) {
        float* s = a.z_scale + row * 2 * a.groups + t.nt;
        s[0] = scale[mi][0];
        s[a.groups] = scale[mi][1];
      }
#pragma unroll 1
      for (int c = 0; c < kHalf; ++c) {
        const int n = n0 + 16 * c;
        if (n >= a.N) continue;
        const floatx8 g = sums.get(c), u = sums.get(kHalf + c);
        floatx8 h;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = act_of(g[j], a.act) * u[j];
        R::store(static_cast<elem*>(a.y) + row * a.y_stride + n, R::narrow(h));
        if (a.z8) {
          uint8_t* z = static_cast<uint8_t*>(a.z) + row * a.z_stride + n;
          *reinterpret_cast<uint2*>(z) = codes_of(g, scale[mi][0]);
          *reinterpret_cast<uint2*>(z + a.N) = codes_of(u, scale[mi][1]);
        } else if (a.z) {
          elem* z = static_cast<elem*>(a.z) + row * a.z_stride + n;
          R::store_once(z, R::narrow(g));
          R::store_once(z + a.N, R::narrow(u));
        }
      }
    } else {
#pragma unroll 1
      for (int c = 0; c < 2 * kHalf; ++c) {
        const int n = n0 + c / kHalf * 128 + c % kHalf * 16;
        if (n >= a.N) continue;
        floatx8 v = sums.get(c);
        if constexpr (EPI == kProductAct) {
          if (a.bias) v += R::wide(R::load(static_cast<const elem*>(a.bias) + (int64_t)t.e * a.N + n));
          if (a.pre) R::store_once(static_cast<elem*>(a.pre) + row * a.pre_stride + n, R::narrow(v));
          if (a.act != PW_ACT_NONE)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = act_of(v[j], a.act);
          if (a.residual) v += R::wide(R::load(static_cast<const elem*>(a.residual) + row * a.residual_stride + n));
        }
        if constexpr (EPI == kProductGateGrad) {
          floatx8 g, u, dg, du, h;
          if (a.z8) {
            const uint8_t* z = static_cast<const uint8_t*>(a.z) + row * a.z_stride + n;
            const float* s = a.z_scale + row * 2 * a.groups + n / kKeepGroup;
            g = values_of(*reinterpret_cast<const uint2*>(z), s[0]);
            u = values_of(*reinterpret_cast<const uint2*>(z + a.N), s[a.groups]);
          } else {
            const elem* z = static_cast<const elem*>(a.z) + row * a.z_stride + n;
            g = R::wide(R::load(z));
            u = R::wide(R::load(z + a.N));
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float s = act_of(g[j], a.act);
            dg[j] = v[j] * u[j] * act_slope(g[j], a.act);
            du[j] = v[j] * s;
            h[j] = s * u[j];
          }
          elem* dz = static_cast<elem*>(a.pre) + row * a.pre_stride + n;
          R::store(dz, R::narrow(dg));
          R::store(dz + a.N, R::narrow(du));
          if (a.y) R::store(static_cast<elem*>(a.y) + row * a.y_stride + n, R::narrow(h));
        } else {
          R::store(static_cast<elem*>(a.y) + row * a.y_stride + n, R::narrow(v));
        }
      }
    }
  }
}

template <int DT, int EPI, int MI, int WM, int WN>
__global__ __launch_bounds__((Shape<MI, WM, WN>::kThreads), (MI * WM == 8 && WN == 2 ? 1 : 2)) void product_kernel(ProductArgs a) {
  using S = Shape<MI, WM, WN>;
  constexpr bool kBack = EPI == kProductBack || EPI == kProductGateGrad;
  __shared__ __align__(1024) char lds[S::kLds];
  const Tile t = find_tile<S::kRows>(a.offsets, a.E, a.S, a.NT);
  if (t.rows <= 0) return;
  const int wave = uniform((int)threadIdx.x / kWave), lane = (int)threadIdx.x & (kWave - 1);
  const int wm = wave / WN, wn = wave % WN;
  const char* x = static_cast<const char*>(a.x) + (int64_t)t.row0 * a.x_stride * 2;
  const char* w = static_cast<const char*>(a.w) + (int64_t)t.e * a.w_expert * 2;

  RowsOperand<S::kRows, S::kWaves> xo;
  RowsOperand<kProdN, S::kWaves> wr;
  ColsOperand<S::kWaves> wc;
  xo.init(wave, lane, [&](int r) { return (uint32_t)min(r, t.rows - 1) * (uint32_t)(a.x_stride * 2); });
  if constexpr (kBack) {
    w += (int64_t)t.nt * kProdN * 2;
    wc.init(wave, lane, (int64_t)a.N * 2, (a.N - t.nt * kProdN + 7) / 8);
  } else {
    // gated: rows of g, then the same rows of u, which have a base of their own
    constexpr int kTile = EPI == kProductGate ? kKeepGroup : kProdN;
    const int n0 = t.nt * kTile, last = a.N - 1 - n0;
    w += (int64_t)n0 * a.K * 2;
    wr.init(wave, lane, [&](int r) { return (uint32_t)min(r & (kTile - 1), last) * (uint32_t)(a.K * 2); });
  }
  constexpr int kXCopies = RowsOperand<S::kRows, S::kWaves>::kCopies;
  constexpr int kWCopies = RowsOperand<kProdN, S::kWaves>::kCopies;
  static_assert(kWCopies == ColsOperand<S::kWaves>::kCopies, "as many copies of W by rows as by columns");
  const rsrc_t xs = copy_rsrc(x), ws = copy_rsrc(w), us = copy_rsrc(w + (int64_t)a.N * a.K * 2);
  f32x4 acc[S::RI][S::CJ];
  sum_steps<DT, S::RI, S::CJ, false, kBack, S::kXBuffers, S::kABytes, kXCopies, kWCopies>(
      acc, lds, (a.K + kProdK - 1) / kProdK, wm, wn, lane,
      [&](int i, int step, uint32_t to) { xo.copy(i, xs, to, wave, step * kProdK, a.K); },
      [&](int i, int step, uint32_t to) {
        const int k = step * kProdK;
        if constexpr (kBack) wc.copy(i, copy_rsrc(w + (int64_t)k * a.N * 2), to, wave, a.K - k);
        else wr.copy(i, EPI == kProductGate && i >= kWCopies / 2 ? us : ws, to, wave, k, a.K);
      });
  finish<DT, EPI, MI, WM, WN>(a, t, acc, lds, wave, lane);
}

template <int DT, int EPI, int MI, int WM, int WN>
hipError_t run(ProductArgs a, hipStream_t s) {
  using Sh = Shape<MI, WM, WN>;
  a.NT = EPI == kProductGate ? (a.N + kKeepGroup - 1) / kKeepGroup : (a.N + kProdN - 1) / kProdN;
  const int64_t grid = product_grid(product_row_tiles(a.offsets, a.E, a.S, Sh::kRows), a.NT);
  if (grid > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((product_kernel<DT, EPI, MI, WM, WN>), dim3((unsigned)grid), dim3(Sh::kThreads), 0, s, a);
  return hipGetLastError();
}

template <int DT, int EPI>
hipError_t pick(const ProductArgs& a, hipStream_t s) {
  const int64_t experts = a.S < a.E ? a.S : a.E, mean = a.S / (experts > 0 ? experts : 1);
  if (mean > 160) return run<DT, EPI, 4, 2, 2>(a, s);
  if (mean > 80) return run<DT, EPI, 2, 2, 4>(a, s);
  if (mean > 32) return run<DT, EPI, 2, 1, 4>(a, s);
  return run<DT, EPI, 1, 1, 4>(a, s);
}

template <int DT>
hipError_t pick_kind(const ProductArgs& a, int kind, hipStream_t s) {
  switch (kind) {
    case kProductAct: return pick<DT, kProductAct>(a, s);
    case kProductGate: return pick<DT, kProductGate>(a, s);
    case kProductBack: return pick<DT, kProductBack>(a, s);
    default: return pick<DT, kProductGateGrad>(a, s);
  }
}

}  // namespace

hipError_t launch_product(const ProductArgs& a, int dtype, int kind, hipStream_t s) {
  return dtype == PW_F16 ? pick_kind<PW_F16>(a, kind, s) : pick_kind<PW_BF16>(a, kind, s);
}

}  // namespace pw
