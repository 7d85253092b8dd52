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

// WM x WN waves, each with 32 MI rows and 64 columns.
template <int MI, int WM, int WN>
struct Shape {
  static constexpr int RI = 2 * MI, CJ = 16 / WN;   // pieces of 16 rows and of 16 columns
  static constexpr int kRows = MI * WM * 32;
  static constexpr int kWaves = WM * WN;
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int kABytes = kRows * kProdK * 2;
  static constexpr int kXBuffers = MI * WM == 2 ? 2 : 3;   // two blocks a CU with tiles of 32 and 64 rows
  static constexpr int kLds = kXBuffers * kABytes + 2 * kProdN * kProdK * 2;
  static_assert(WN == 4 && kWaves * Sums::kBytes + 2 * kRows * 16 <= kLds, "LDS of what follows the products");
};

template <int DT, int EPI, int MI, int WM, int WN>
__device__ __forceinline__ void finish(const ProductArgs& a, const Tile& t, f32x4 (&acc)[2 * MI][16 / WN], char* lds,
                                       int wave, int lane) {
  using R = Row<DT>;
  using elem = typename R::elem;
  using S = Shape<MI, WM, WN>;
  constexpr bool kGate = EPI == kProductGate;
  const int wm = wave / WN, wn = wave % WN;
  Sums sums(lds, wave, lane);
  // gated: eight lanes hold 32 columns of g and of u of two rows (four lanes each), else 64 of one row
  constexpr int kLanes = kGate ? 4 : 8;
  const int own = lane & (kLanes - 1), n = kGate ? t.nt * kKeepGroup + wn * 32 + own * 8 : t.nt * kProdN + wn * 64 + own * 8;
  // the largest |g| and |u| of each row over the tile's 128 columns: over a lane's, its pair's and the waves'
  float4* const most = reinterpret_cast<float4*>(lds + S::kWaves * Sums::kBytes);   // [2][kRows]
  if (kGate && a.z8) {
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float m = 0.f;
#pragma unroll
        for (int c = 2 * half; c < 2 * half + 2; ++c) {
          const floatx8 v = eight_columns(acc[2 * mi][c], acc[2 * mi + 1][c]);
          if (t.nt * kKeepGroup + wn * 32 + c % 2 * 16 + lane / 32 * 8 < a.N) m = most_of(v, m);
        }
        m = fmaxf(m, __shfl_xor(m, 32, kWave));
        if (lane < 32) reinterpret_cast<float*>(most + half * S::kRows + (wm * MI + mi) * 32 + lane)[wn] = m;
      }
    __syncthreads();
  }
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    sums.put(acc[2 * mi], acc[2 * mi + 1]);
#pragma unroll 1
    for (int i = lane / kLanes; i < 32; i += kWave / kLanes) {
      const int r = (wm * MI + mi) * 32 + i;
      if (r >= t.rows || n >= a.N) continue;
      const int64_t row = t.row0 + r;
      if constexpr (kGate) {
        const floatx8 g = sums.get(i, own), u = sums.get(i, 4 + own);
        floatx8 h;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = act_of(g[j], a.act) * u[j];
        R::store(static_cast<elem*>(a.y) + row * a.y_stride + n, R::narrow(h));
        if (a.z8) {
          const float4 mg = most[r], mu = most[S::kRows + r];
          const float sg = scale_of(fmaxf(fmaxf(mg.x, mg.y), fmaxf(mg.z, mg.w)));
          const float su = scale_of(fmaxf(fmaxf(mu.x, mu.y), fmaxf(mu.z, mu.w)));
          if (wn == 0 && own == 0) {
            float* s = a.z_scale + row * 2 * a.groups + t.nt;
            s[0] = sg;
            s[a.groups] = su;
          }
          uint8_t* z = static_cast<uint8_t*>(a.z) + row * a.z_stride + n;
          *reinterpret_cast<uint2*>(z) = codes_of(g, sg);
          *reinterpret_cast<uint2*>(z + a.N) = codes_of(u, su);
        } else if (a.z) {
          elem* z = static_cast<elem*>(a.z) + row * a.z_stride + n;
          R::store_once(z, R::narrow(g));
          R::store_once(z + a.N, R::narrow(u));
        }
      } else {
        floatx8 v = sums.get(i, own);
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
__global__ __launch_bounds__((Shape<MI, WM, WN>::kThreads), 2) void product_kernel(ProductArgs a) {
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
  xo.init(x, x, a.K, wave, lane, [&](int r) { return (uint32_t)min(r, t.rows - 1) * (uint32_t)(a.x_stride * 2); });
  f32x4 acc[S::RI][S::CJ];
  const int steps = (a.K + kProdK - 1) / kProdK, live = (t.rows - wm * MI * 32 + 15) / 16;
  if constexpr (kBack) {
    ColsOperand<kProdN, S::kWaves> wo;
    wo.init(w + (int64_t)t.nt * kProdN * 2, a.K, wave, lane, (int64_t)a.N * 2, (a.N - t.nt * kProdN + 7) / 8);
    sum_steps<DT, S::RI, S::CJ, S::kRows, kProdN, false, false, true, S::kXBuffers>(acc, lds, steps, live, wave, wm, wn, lane,
                                                                                   xo, wo);
  } else {
    // gated: rows of g, then the same rows of u, which have a base of their own
    constexpr int kTile = EPI == kProductGate ? kKeepGroup : kProdN;
    const int n0 = t.nt * kTile, last = a.N - 1 - n0;
    w += (int64_t)n0 * a.K * 2;
    RowsOperand<kProdN, S::kWaves, EPI == kProductGate> wo;
    wo.init(w, w + (int64_t)a.N * a.K * 2, a.K, wave, lane,
            [&](int r) { return (uint32_t)min(r & (kTile - 1), last) * (uint32_t)(a.K * 2); });
    sum_steps<DT, S::RI, S::CJ, S::kRows, kProdN, EPI == kProductGate, false, false, S::kXBuffers>(acc, lds, steps, live, wave, wm, wn, lane,
                                                                                   xo, wo);
  }
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
  if (mean > 160) return run<DT, EPI, 4, 2, 4>(a, s);
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
