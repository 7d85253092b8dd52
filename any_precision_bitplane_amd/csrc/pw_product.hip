// Products of every expert's rows with its matrix, with what follows them:
//
//   product        z = x W^T + bias,  y = act(z) + residual          W [N][K]
//   gated          [g | u] = x W^T,   h = act(g) u                   W [2N][K]
//   back           dx = dz W                                         W [K][N]
//   gated, back    dh = dy W,  dg = dh u act'(g),  du = dh act(g),  h = act(g) u
//
// in tiles of 32 to 256 rows by 256 columns (gated: 128 of g and the same 128 of
// u, so that a wave holds both for its columns).
//
// What bounds it: with many rows the matrix cores and the power they draw (8192 x
// 8192 x 8192 bf16 760 us, 1447 TFLOP/s, three quarters of the cycles busy at 1.77
// GHz; H 4096, I 14336, some 8190 rows over 8 experts, gate and up bf16 with 8-bit
// copies 1.84 ms, back to x fp16 1.52); with few rows reading the matrices (E 8, H
// 4096, I 14336, 128 rows, 2.8 GB in 488 to 515 us, 5.5 to 5.8 TB/s).
//
// h, dg and du are rounded to the rows' type: they are operands of the next
// product, and the matrix cores take 16 bits (two parts of 16 bits a value would
// be a third more products in the block, five sixths more in its gradient).  It makes the block's error
// against 64 bits sqrt 2 times as large (fp16 2.9e-4 for 2.1e-4, bf16 2.3e-3 for
// 1.7e-3), and in fp16 a value past 65504 an infinity.
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
  static constexpr int kCopied = kXBuffers * kABytes + 2 * kProdN * kProdK * 2;
  static constexpr int kAfter = kWaves * (Sums::kBytes + 8 * kWave * 16);   // what follows the products
  static constexpr int kLds = kCopied > kAfter ? kCopied : kAfter;
  static_assert(WN == 4 && 2 * kRows * 16 <= kWaves * 8 * kWave * 16, "rows' maxima fit what waits elsewhere");
};

// What eight columns from n on of a row need besides their sums: the residual, or
// gate and up (8 bits: their codes, and their scales).
struct Besides {
  uint4 first, second;
};
template <int EPI>
__device__ __forceinline__ bool wants(const ProductArgs& a) {
  return EPI == kProductGateGrad || (EPI == kProductAct && a.residual);
}
template <int DT, int EPI>
__device__ __forceinline__ Besides besides(const ProductArgs& a, int64_t row, int n) {
  Besides b{};
  if constexpr (EPI == kProductAct) {
    b.first = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.residual) + (row * a.residual_stride + n) * 2);
  } else if constexpr (EPI == kProductGateGrad) {
    if (a.z8) {
      const uint8_t* z = static_cast<const uint8_t*>(a.z) + row * a.z_stride + n;
      const float* s = a.z_scale + row * 2 * a.groups + n / kKeepGroup;
      const uint2 g = *reinterpret_cast<const uint2*>(z), u = *reinterpret_cast<const uint2*>(z + a.N);
      b.first = uint4{g.x, g.y, u.x, u.y};
      b.second.x = __float_as_uint(s[0]);
      b.second.y = __float_as_uint(s[a.groups]);
    } else {
      const char* z = static_cast<const char*>(a.z) + (row * a.z_stride + n) * 2;
      b.first = *reinterpret_cast<const uint4*>(z);
      b.second = *reinterpret_cast<const uint4*>(z + (int64_t)a.N * 2);
    }
  }
  return b;
}

// What becomes of eight columns from n on of a row's sums v (gated: of g, and u).
template <int DT, int EPI>
__device__ __forceinline__ void emit(const ProductArgs& a, int64_t row, int n, floatx8 v, floatx8 u, float sv, float su,
                                     floatx8 bias, const Besides& b) {
  using R = Row<DT>;
  using elem = typename R::elem;
  elem* const y = static_cast<elem*>(a.y) + row * a.y_stride + n;
  if constexpr (EPI == kProductGate) {
    floatx8 h;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = act_of(v[j], a.act) * u[j];
    R::store(y, R::narrow(h));
    if (a.z8) {
      uint8_t* z = static_cast<uint8_t*>(a.z) + row * a.z_stride + n;
      *reinterpret_cast<uint2*>(z) = codes_of(v, sv);
      *reinterpret_cast<uint2*>(z + a.N) = codes_of(u, su);
      if (n % kKeepGroup == 0) {
        float* s = a.z_scale + row * 2 * a.groups + n / kKeepGroup;
        s[0] = sv;
        s[a.groups] = su;
      }
    } else if (a.z) {
      elem* z = static_cast<elem*>(a.z) + row * a.z_stride + n;
      R::store_once(z, R::narrow(v));
      R::store_once(z + a.N, R::narrow(u));
    }
  } else if constexpr (EPI == kProductGateGrad) {
    floatx8 g, dg, du, h;
    if (a.z8) {
      g = values_of(uint2{b.first.x, b.first.y}, __uint_as_float(b.second.x));
      u = values_of(uint2{b.first.z, b.first.w}, __uint_as_float(b.second.y));
    } else {
      g = R::wide(__builtin_bit_cast(typename R::chunk, b.first));
      u = R::wide(__builtin_bit_cast(typename R::chunk, b.second));
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
    if (a.y) R::store(y, R::narrow(h));
  } else {
    if constexpr (EPI == kProductAct) {
      if (a.bias) v += bias;
      if (a.pre) R::store_once(static_cast<elem*>(a.pre) + row * a.pre_stride + n, R::narrow(v));
      if (a.act != PW_ACT_NONE)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = act_of(v[j], a.act);
      if (a.residual) v += R::wide(__builtin_bit_cast(typename R::chunk, b.first));
    }
    R::store(y, R::narrow(v));
  }
}

template <int DT, int EPI>
__device__ __forceinline__ floatx8 bias_of(const ProductArgs& a, int e, int n) {
  using R = Row<DT>;
  if (EPI == kProductAct && a.bias && n < a.N)
    return R::wide(R::load(static_cast<const typename R::elem*>(a.bias) + (int64_t)e * a.N + n));
  return floatx8{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
}

// A tile's sums, on their way to `part` (fp32 [kRows][256], gated g's 128 columns
// and u's) or to what becomes of them.
template <int DT, int EPI, int MI, int WM, int WN>
__device__ __forceinline__ void finish(const ProductArgs& a, const Tile& t, f32x4 (&acc)[2 * MI][16 / WN], char* lds,
                                       float* part, int wave, int lane) {
  using S = Shape<MI, WM, WN>;
  constexpr bool kGate = EPI == kProductGate;
  const int wm = wave / WN, wn = wave % WN;
  Sums sums(lds, wave, lane);
  // gated: eight lanes hold 32 columns of g and of u of two rows (four lanes each), else 64 of one row
  constexpr int kLanes = kGate ? 4 : 8;
  const int own = lane & (kLanes - 1), c = (kGate ? wn * 32 : wn * 64) + own * 8, n = t.nt * (kGate ? kKeepGroup : kProdN) + c;
  // the largest |g| and |u| of each row over the tile's 128 columns: over a lane's, its pair's and the waves'
  float4* const most = reinterpret_cast<float4*>(lds + S::kWaves * Sums::kBytes);   // [2][kRows]
  if (kGate && a.z8 && !part) {
#pragma unroll
    for (int mi = 0; mi < MI; ++mi)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float m = 0.f;
#pragma unroll
        for (int p = 2 * half; p < 2 * half + 2; ++p) {
          const floatx8 v = eight_columns(acc[2 * mi][p], acc[2 * mi + 1][p]);
          if (t.nt * kKeepGroup + wn * 32 + p % 2 * 16 + lane / 32 * 8 < a.N) m = most_of(v, m);
        }
        m = fmaxf(m, __shfl_xor(m, 32, kWave));
        if (lane < 32) reinterpret_cast<float*>(most + half * S::kRows + (wm * MI + mi) * 32 + lane)[wn] = m;
      }
    __syncthreads();
  }
  // What 32 rows need besides is requested while the 32 before are worked on, and
  // waits in LDS, each lane's own (8194 rows, 8192 x 2048 bf16 with GELU, residual
  // and pre: 387 us requested row by row, 343 so).
  constexpr bool kBesides = EPI == kProductAct || EPI == kProductGateGrad;
  const bool want = wants<EPI>(a) && !part;
  const floatx8 bias = bias_of<DT, EPI>(a, t.e, n);
  uint4* const waiting = reinterpret_cast<uint4*>(lds + S::kWaves * Sums::kBytes) + wave * (8 * kWave) + lane;
  Besides next[4];
  auto request = [&](int mi) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = (wm * MI + mi) * 32 + lane / 8 + 8 * q;
      if (r < t.rows && n < a.N) next[q] = besides<DT, EPI>(a, t.row0 + r, n);
    }
  };
  if (kBesides && want) request(0);
#pragma unroll
  for (int mi = 0; mi < MI; ++mi) {
    sums.put(acc[2 * mi], acc[2 * mi + 1]);
    if (kBesides && want) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        waiting[2 * q * kWave] = next[q].first;
        if (EPI == kProductGateGrad) waiting[(2 * q + 1) * kWave] = next[q].second;
      }
      if (mi + 1 < MI) request(mi + 1);
    }
#pragma unroll 1
    for (int i = lane / kLanes, q = 0; i < 32; i += kWave / kLanes, ++q) {
      const int r = (wm * MI + mi) * 32 + i;
      if (r >= t.rows || n >= a.N) continue;
      const floatx8 v = sums.get(i, own);
      floatx8 u = v;
      if constexpr (kGate) u = sums.get(i, 4 + own);
      if (part) {
        float* to = part + r * kProdN + c;
        *reinterpret_cast<floatx8*>(to) = v;
        if constexpr (kGate) *reinterpret_cast<floatx8*>(to + kKeepGroup) = u;
        continue;
      }
      float sv = 0.f, su = 0.f;
      if (kGate && a.z8) {
        const float4 mg = most[r], mu = most[S::kRows + r];
        sv = scale_of(fmaxf(fmaxf(mg.x, mg.y), fmaxf(mg.z, mg.w)));
        su = scale_of(fmaxf(fmaxf(mu.x, mu.y), fmaxf(mu.z, mu.w)));
      }
      Besides b{};
      if (kBesides && want) {
        b.first = waiting[2 * q * kWave];
        if (EPI == kProductGateGrad) b.second = waiting[(2 * q + 1) * kWave];
      }
      emit<DT, EPI>(a, t.row0 + r, n, v, u, sv, su, bias, b);
    }
  }
}

template <int DT, int EPI, int MI, int WM, int WN>
__global__ __launch_bounds__((Shape<MI, WM, WN>::kThreads), 2) void product_kernel(ProductArgs a) {
  using S = Shape<MI, WM, WN>;
  constexpr bool kBack = EPI == kProductBack || EPI == kProductGateGrad;
  __shared__ __align__(1024) char lds[S::kLds];
  const TileScan<S::kRows> scan(a.offsets, a.E, a.S);
  const int all_steps = (a.K + kProdK - 1) / kProdK;
  const Rounds<S::kRows> rounds((unsigned)scan.tiles * (unsigned)a.NT, all_steps, a.part != nullptr);
  unsigned id = blockIdx.x;
  int k0 = 0, k1 = a.K;
  float* part = nullptr;
  if (id < (rounds.whole + 7) / 8 * 8) {
    const unsigned each_xcd = (rounds.whole + 7) / 8, i = id / 8;
    id = (id % 8) * each_xcd + i;
    if (id >= rounds.whole) return;
  } else {
    const unsigned p = id - (rounds.whole + 7) / 8 * 8, of = p / rounds.parts, which = p - of * rounds.parts;
    if (of >= rounds.rest) return;
    id = rounds.whole + of;
    k0 = (int)(all_steps * which / rounds.parts) * kProdK;
    k1 = min((int)(all_steps * (which + 1) / rounds.parts) * kProdK, a.K);
    part = a.part + (int64_t)p * (S::kRows * kProdN);
  }
  const Tile t = scan.at(id, a.NT);
  const int wave = uniform((int)threadIdx.x / kWave), lane = (int)threadIdx.x & (kWave - 1);
  const int wm = wave / WN, wn = wave % WN;
  const char* x = static_cast<const char*>(a.x) + ((int64_t)t.row0 * a.x_stride + k0) * 2;
  const char* w = static_cast<const char*>(a.w) + (int64_t)t.e * a.w_expert * 2;

  RowsOperand<S::kRows, S::kWaves> xo;
  xo.init(x, x, k1 - k0, wave, lane, [&](int r) { return (uint32_t)min(r, t.rows - 1) * (uint32_t)(a.x_stride * 2); });
  f32x4 acc[S::RI][S::CJ];
  const int steps = (k1 - k0 + kProdK - 1) / kProdK, live = (t.rows - wm * MI * 32 + 15) / 16;
  if constexpr (kBack) {
    ColsOperand<kProdN, S::kWaves> wo;
    wo.init(w + ((int64_t)k0 * a.N + t.nt * kProdN) * 2, k1 - k0, wave, lane, (int64_t)a.N * 2, (a.N - t.nt * kProdN + 7) / 8);
    sum_steps<DT, S::RI, S::CJ, S::kRows, kProdN, false, false, true, S::kXBuffers>(acc, lds, steps, live, wave, wm, wn, lane,
                                                                                   xo, wo);
  } else {
    // gated: rows of g, then the same rows of u, which have a base of their own
    constexpr int kTile = EPI == kProductGate ? kKeepGroup : kProdN;
    const int n0 = t.nt * kTile, last = a.N - 1 - n0;
    w += ((int64_t)n0 * a.K + k0) * 2;
    RowsOperand<kProdN, S::kWaves, EPI == kProductGate> wo;
    wo.init(w, w + (int64_t)a.N * a.K * 2, k1 - k0, wave, lane,
            [&](int r) { return (uint32_t)min(r & (kTile - 1), last) * (uint32_t)(a.K * 2); });
    sum_steps<DT, S::RI, S::CJ, S::kRows, kProdN, EPI == kProductGate, false, false, S::kXBuffers>(acc, lds, steps, live, wave, wm, wn, lane,
                                                                                   xo, wo);
  }
  finish<DT, EPI, MI, WM, WN>(a, t, acc, lds, part, wave, lane);
}

// The tiles that were cut: a block has 16 rows of one, sixteen lanes a row.
template <int DT, int EPI, int ROWS>
__global__ __launch_bounds__(256) void join_kernel(ProductArgs a) {
  constexpr bool kGate = EPI == kProductGate;
  const TileScan<ROWS> scan(a.offsets, a.E, a.S);
  const Rounds<ROWS> rounds((unsigned)scan.tiles * (unsigned)a.NT, (a.K + kProdK - 1) / kProdK, true);
  const unsigned of = blockIdx.x / (ROWS / 16);
  if (of >= rounds.rest) return;
  const Tile t = scan.at(rounds.whole + of, a.NT);
  const int r = (int)(blockIdx.x % (ROWS / 16)) * 16 + (int)threadIdx.x / 16, lane = (int)threadIdx.x & 15;
  if (r >= t.rows) return;
  const float* from = a.part + (int64_t)of * rounds.parts * (ROWS * kProdN) + r * kProdN;
  floatx8 v[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const float* p = from + half * 128 + lane * 8;
    v[half] = *reinterpret_cast<const floatx8*>(p);
    for (unsigned i = 1; i < rounds.parts; ++i) v[half] += *reinterpret_cast<const floatx8*>(p + (int64_t)i * (ROWS * kProdN));
  }
  if constexpr (kGate) {
    const int n = t.nt * kKeepGroup + lane * 8;
    const bool in = n < a.N;
    float sv = 0.f, su = 0.f;
    if (a.z8) {
      sv = in ? most_of(v[0], 0.f) : 0.f;   // over the sixteen lanes of the row
      su = in ? most_of(v[1], 0.f) : 0.f;
#pragma unroll
      for (int d = 1; d < 16; d *= 2) {
        sv = fmaxf(sv, __shfl_xor(sv, d, kWave));
        su = fmaxf(su, __shfl_xor(su, d, kWave));
      }
      sv = scale_of(sv);
      su = scale_of(su);
    }
    if (in) emit<DT, EPI>(a, t.row0 + r, n, v[0], v[1], sv, su, v[0], Besides{});
  } else {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int n = t.nt * kProdN + half * 128 + lane * 8;
      if (n >= a.N) continue;
      const Besides b = wants<EPI>(a) ? besides<DT, EPI>(a, t.row0 + r, n) : Besides{};
      emit<DT, EPI>(a, t.row0 + r, n, v[half], v[half], 0.f, 0.f, bias_of<DT, EPI>(a, t.e, n), b);
    }
  }
}

template <int DT, int EPI, int MI, int WM, int WN>
hipError_t run(ProductArgs a, hipStream_t s) {
  using Sh = Shape<MI, WM, WN>;
  a.NT = product_col_tiles(EPI, a.N);
  const int64_t tiles = product_row_tiles(a.offsets != nullptr, a.E, a.S, Sh::kRows) * a.NT, most = product_blocks(Sh::kRows);
  const bool cut = a.part && product_is_cut(a.offsets != nullptr, tiles, (a.K + kProdK - 1) / kProdK, Sh::kRows);
  if (!cut) a.part = nullptr;
  const int64_t grid = (tiles + 7) / 8 * 8 + (cut ? most : 0);
  if (!launch_fits(grid, Sh::kThreads)) return hipErrorInvalidValue;
  hipLaunchKernelGGL((product_kernel<DT, EPI, MI, WM, WN>), dim3((unsigned)grid), dim3(Sh::kThreads), 0, s, a);
  if (cut) {
    const int64_t joined = tiles < most / 2 ? tiles : most / 2;
    hipLaunchKernelGGL((join_kernel<DT, EPI, Sh::kRows>), dim3((unsigned)joined * (Sh::kRows / 16)), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

template <int DT, int EPI>
hipError_t pick(const ProductArgs& a, hipStream_t s) {
  switch (product_rows(a.E, a.S, product_col_tiles(EPI, a.N))) {
    case 256: return run<DT, EPI, 4, 2, 4>(a, s);
    case 128: return run<DT, EPI, 2, 2, 4>(a, s);
    case 64: return run<DT, EPI, 2, 1, 4>(a, s);
    default: return run<DT, EPI, 1, 1, 4>(a, s);
  }
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
