// Root-mean-square norm of rows with the residual's addition, an optional
// 8-bit output, and its gradient.
//
//   r_i = x_i + residual_i            (fp32; stored rounded to the row type)
//   y_i = r_i g_i / sqrt(mean_h r_h^2 + eps)
//
// The sum of squares, the mean and y stay in fp32; y is rounded once, to the
// row type or to e4m3 after division by its scale.  The norm is taken of the
// fp32 sum, before the residual's own rounding.
//
// The work is one pass over memory: a row's chunks of eight elements stay in
// registers between the sum of squares and the output.  Above 16384 columns the
// four chunks a lane no longer all fit beside the next row's: fp32 spills 30
// registers a lane (87 to e4m3, 16-bit rows 12 to e4m3), fp32 [2048][32768]
// with the residual 274 us, 3.9 TB/s, bf16 103 us, 5.2 TB/s.
#include "pw_rows.h"

namespace pw {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kScaleMin = 7.888609052210118e-31f;   // 2^-100: scales stay divisible
constexpr unsigned kMaxGrid = 1u << 20;

// Sum and maximum over the LPR lanes that share a row (all 64 of a wave, or 8,
// 16 or 32 of them), the same bits in each.
template <int LPR>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (LPR == kWave) return wave_sum(v);
  v += dpp_row<kQuadXor1>(v);
  v += dpp_row<kQuadXor2>(v);
  v += dpp_row<kHalfRowMirror>(v);
  if constexpr (LPR >= 16) v += dpp_row<kRowMirror>(v);
  if constexpr (LPR >= 32) v += __shfl_xor(v, 16, kWave);
  return v;
}

template <int LPR>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (LPR == kWave) return wave_max(v);
  v = fmaxf(v, dpp_row<kQuadXor1>(v));
  v = fmaxf(v, dpp_row<kQuadXor2>(v));
  v = fmaxf(v, dpp_row<kHalfRowMirror>(v));
  if constexpr (LPR >= 16) v = fmaxf(v, dpp_row<kRowMirror>(v));
  if constexpr (LPR >= 32) v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return v;
}

// Sum over a row of WPR waves or LPR lanes.  `part` holds one value per wave of
// the block; callers alternate between two such arrays, so one barrier per sum
// is enough.
template <int LPR, int WPR>
__device__ __forceinline__ float row_sum(float v, float* part, int wave) {
  v = lanes_sum<LPR>(v);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & (kWave - 1)) == 0) part[wave] = v;
    __syncthreads();
    const float* p = part + wave / WPR * WPR;
    v = p[0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) v += p[i];
  }
  return v;
}

template <int LPR, int WPR>
__device__ __forceinline__ float row_max(float v, float* part, int wave) {
  v = lanes_max<LPR>(v);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & (kWave - 1)) == 0) part[wave] = v;
    __syncthreads();
    const float* p = part + wave / WPR * WPR;
    v = p[0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) v = fmaxf(v, p[i]);
  }
  return v;
}

// WPR waves (or, of one wave, LPR lanes) share a row, each lane holding NV
// chunks of it; a block has at least four waves, so it takes several rows when
// a row needs fewer.
constexpr int block_waves(int WPR) { return WPR < 4 ? 4 : WPR; }
constexpr int block_rows(int LPR, int WPR) { return block_waves(WPR) / WPR * (kWave / LPR); }

template <int DT, int LPR, int WPR, int NV, bool Q8>
__global__ __launch_bounds__(block_waves(WPR) * kWave) void rmsnorm_kernel(NormArgs a) {
  using R = Row<DT>;
  using elem = typename R::elem;
  constexpr int kRows = block_rows(LPR, WPR);
  static_assert(LPR == kWave || WPR == 1, "lanes of one wave, or whole waves");
  __shared__ float part[4][block_waves(WPR)];
  const int wave = uniform((int)threadIdx.x / kWave);
  const int lane = (int)threadIdx.x & (kWave - 1);
  const int own = wave / WPR * (kWave / LPR) + (LPR == kWave ? 0 : lane / LPR);   // the lane's row of the block
  const int first = (wave % WPR) * kWave + (lane & (LPR - 1));                    // its first chunk of that row
  const int C = a.H / 8;
  typedef typename R::chunk chunk;
  // Past the row's end the first chunk is read again, which nothing uses.
  int at[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first + i * WPR * kWave;
    at[i] = c < C ? 8 * c : 0;
  }
  chunk xc[NV], rc[NV], g[NV];
  auto fetch = [&](int64_t row) {
    if (row >= a.T) return;
    const elem* x = static_cast<const elem*>(a.x) + row * a.x_stride;
    const elem* res = static_cast<const elem*>(a.residual) + row * a.residual_stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      xc[i] = R::load(x + at[i]);
      if (a.residual) rc[i] = R::load(res + at[i]);
    }
  };
  // The weight is requested with the row, not after its sum (fp16 [16384][4096]
  // 4% faster, bf16 to e4m3 11%), and the row before the loop, ahead of what the
  // compiler moves out of it (bf16 [65536][2048] without a residual 11%).
#pragma unroll
  for (int i = 0; i < NV; ++i) g[i] = R::load(static_cast<const elem*>(a.weight) + at[i]);
  fetch((int64_t)blockIdx.x * kRows + own);
  int parity = 0;
  const int64_t step = (int64_t)gridDim.x * kRows;
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.T; base += step, parity ^= 1) {
    const int64_t row = base + own;
    const bool live = row < a.T;
    elem* out = static_cast<elem*>(a.residual_out) + row * a.residual_out_stride;
    floatx8 v[NV];
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first + i * WPR * kWave;
      v[i] = floatx8{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (!live || c >= C) continue;
      v[i] = R::wide(xc[i]);
      if (a.residual) {
        v[i] += R::wide(rc[i]);
        if (a.residual_out) R::store_once(out + 8 * c, R::narrow(v[i]));
      }
    }
    fetch(row + step);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) sq = __builtin_fmaf(v[i][j], v[i][j], sq);
    sq = row_sum<LPR, WPR>(sq, part[parity], wave);
    const float rstd = rsqrtf(sq / (float)a.H + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = v[i] * rstd * R::wide(g[i]);
    if constexpr (!Q8) {
      elem* y = static_cast<elem*>(a.y) + row * a.y_stride;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = first + i * WPR * kWave;
        if (live && c < C) R::store_once(y + 8 * c, R::narrow(v[i]));
      }
    } else {
      // A NaN or an infinity counts as infinity, so it shows in the group's maximum.  Lanes past the row's end
      // hold zeros times the first chunk's weight, which may be NaN: they count as zero.
      float m[NV], top = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        m[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float t = __builtin_fabsf(v[i][j]);
          m[i] = t < INFINITY ? fmaxf(m[i], t) : INFINITY;
        }
        if (first + i * WPR * kWave >= C) m[i] = 0.f;
        if (a.group) m[i] = lanes_max<LPR < 16 ? LPR : 16>(m[i]);   // 16 chunks of 8: one group of 128
        top = fmaxf(top, m[i]);
      }
      if (!a.group) top = row_max<LPR, WPR>(top, part[2 + parity], wave);
      uint8_t* y = static_cast<uint8_t*>(a.y) + row * a.y_stride;
      const int groups = a.group ? (a.H + kNormGroup - 1) / kNormGroup : 1;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = first + i * WPR * kWave;
        if (!live || c >= C) continue;
        const float most = a.group ? m[i] : top;
        const bool finite = most < INFINITY;
        const float scale = finite ? fmaxf(most / kE4m3Max, kScaleMin) : __builtin_nanf("");
        const float inv = 1.f / scale;
        typedef uint32_t codes_t __attribute__((ext_vector_type(2)));
        codes_t codes = {0x7F7F7F7Fu, 0x7F7F7F7Fu};
        if (finite) {
          floatx8 q;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            // y / scale to nearest: the product with the reciprocal may be a step or two off, which moves codes whose
            // quotient lies at a midpoint of e4m3; its remainder, exact in an fma, corrects it (bf16 [16384][4096]
            // 78.3 us with and without)
            const float t = v[i][j] * inv;
            q[j] = fminf(fmaxf(__builtin_fmaf(__builtin_fmaf(-t, scale, v[i][j]), inv, t), -kE4m3Max), kE4m3Max);
          }
          int p = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
          codes[0] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], p, true);
          p = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
          codes[1] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], p, true);
        }
        __builtin_nontemporal_store(codes, reinterpret_cast<codes_t*>(y + 8 * c));   // as store_once
        if (a.group ? (c % (kNormGroup / 8) == 0) : c == 0)
          a.scale[row * groups + (a.group ? c / (kNormGroup / 8) : 0)] = scale;
      }
    }
  }
}

template <int DT, int LPR, int WPR, int NV, bool Q8>
hipError_t run_norm(const NormArgs& a, hipStream_t s) {
  constexpr int kRows = block_rows(LPR, WPR);
  const unsigned want = ((unsigned)a.T + kRows - 1) / kRows;
  hipLaunchKernelGGL((rmsnorm_kernel<DT, LPR, WPR, NV, Q8>), dim3(want < kMaxGrid ? want : kMaxGrid),
                     dim3(block_waves(WPR) * kWave), 0, s, a);
  return hipGetLastError();
}

// A row over as many lanes as it has chunks for, up to sixteen waves, so each
// lane waits for one load.  Four chunks a lane and a quarter of the waves were
// slower nearly everywhere (fp16 [64][2048] 4.8 us against 3.0, [16384][4096]
// by 7%, fp32 by 11%; faster by 5% for fp16 [4096][4096], which stays in the
// caches).
// Measured with the residual: fp16 [16384][4096] 89 us, 6.0 TB/s; bf16 to e4m3
// 78 us, 6.0 TB/s; fp32 184 us, 5.8 TB/s (a large copy: 5.0).
template <int DT, bool Q8>
hipError_t pick_norm(const NormArgs& a, hipStream_t s) {
  const int C = a.H / 8;
  if (C <= 8) return run_norm<DT, 8, 1, 1, Q8>(a, s);
  if (C <= 16) return run_norm<DT, 16, 1, 1, Q8>(a, s);
  if (C <= 32) return run_norm<DT, 32, 1, 1, Q8>(a, s);
  if (C <= 64) return run_norm<DT, 64, 1, 1, Q8>(a, s);
  if (C <= 128) return run_norm<DT, 64, 2, 1, Q8>(a, s);
  if (C <= 256) return run_norm<DT, 64, 4, 1, Q8>(a, s);
  if (C <= 512) return run_norm<DT, 64, 8, 1, Q8>(a, s);
  if (C <= 1024) return run_norm<DT, 64, 16, 1, Q8>(a, s);
  if (C <= 2048) return run_norm<DT, 64, 16, 2, Q8>(a, s);
  return run_norm<DT, 64, 16, 4, Q8>(a, s);
}

// Gradient.  With s = 1 / sqrt(mean r^2 + eps) and d = sum_h g_h dy_h r_h:
//   dx_i = s (g_i dy_i - r_i s^2 d / H) + dresidual_i
//   dg_i = sum over rows of dy_i r_i s
// dx is the gradient of x and of the residual alike.  s is computed again from
// r (both sums in the same pass), so the forward keeps nothing but its
// residual output.  A block walks every gridDim-th group of rows and keeps its
// share of dg in registers; the shares meet in a second kernel, in a fixed
// order.  Measured: bf16 [16384][4096] with dresidual 95 us, 5.6 TB/s.
//
// AHEAD: the next row is requested before the current one is used (dx may be
// written over an input: the rows in flight are the block's own later ones).
// LEAN: the weight and dresidual are loaded where they are used, so that more of
// the longest rows' chunks stay in registers (above 16384 columns 17 to 21 of
// them still spill: bf16 [2048][32768] 158 us, 3.4 TB/s, fp32 254 us, 4.2 TB/s).
template <int DT, int LPR, int WPR, int NV, bool AHEAD, bool LEAN>
__global__ __launch_bounds__(block_waves(WPR) * kWave) void rmsnorm_grad_kernel(NormGradArgs a) {
  using R = Row<DT>;
  using elem = typename R::elem;
  constexpr int kRows = block_rows(LPR, WPR);
  __shared__ float part[2][2][block_waves(WPR)];
  const int wave = uniform((int)threadIdx.x / kWave);
  const int lane = (int)threadIdx.x & (kWave - 1);
  const int own = wave / WPR * (kWave / LPR) + (LPR == kWave ? 0 : lane / LPR);
  const int first = (wave % WPR) * kWave + (lane & (LPR - 1));
  const int C = a.H / 8;
  const floatx8 zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const elem* gain = static_cast<const elem*>(a.weight);
  typedef typename R::chunk chunk;
  floatx8 dg[NV];
  chunk gc[LEAN ? 1 : NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    dg[i] = zero;
    const int c = first + i * WPR * kWave;
    if constexpr (!LEAN) gc[i] = R::load(gain + 8 * (c < C ? c : 0));
  }
  const bool adds = a.dresidual != nullptr;
  // the chunks of one row of each matrix, as they lie in memory; past the row's
  // end the first chunk again, which nothing uses
  auto fetch = [&](int64_t row, chunk(&r)[NV], chunk(&d)[NV], chunk(&add)[NV]) {
    if (row >= a.T) return;
    const elem* dy = static_cast<const elem*>(a.dy) + row * a.dy_stride;
    const elem* rr = static_cast<const elem*>(a.r) + row * a.r_stride;
    const elem* dres = static_cast<const elem*>(a.dresidual) + row * a.dresidual_stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      int c = first + i * WPR * kWave;
      c = c < C ? c : 0;
      r[i] = R::load(rr + 8 * c);
      d[i] = R::load(dy + 8 * c);
      if (!LEAN && adds) add[i] = R::load(dres + 8 * c);
    }
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t base = (int64_t)blockIdx.x * kRows;
  chunk rn[NV], dn[NV], an[NV];
  if constexpr (AHEAD) fetch(base + own, rn, dn, an);
  for (int parity = 0; base < a.T; base += step, parity ^= 1) {
    const int64_t row = base + own;
    const bool live = row < a.T;
    elem* dx = static_cast<elem*>(a.dx) + row * a.dx_stride;
    const elem* dres = static_cast<const elem*>(a.dresidual) + row * a.dresidual_stride;
    chunk rc[NV], dc[NV], ac[NV];
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        rc[i] = rn[i];
        dc[i] = dn[i];
        ac[i] = an[i];
      }
      fetch(row + step, rn, dn, an);
    } else {
      fetch(row, rc, dc, ac);
    }
    float sq = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first + i * WPR * kWave;
      if (!live || c >= C) continue;
      const floatx8 r = R::wide(rc[i]), gd = R::wide(LEAN ? R::load(gain + 8 * c) : gc[LEAN ? 0 : i]) * R::wide(dc[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sq = __builtin_fmaf(r[j], r[j], sq);
        dot = __builtin_fmaf(gd[j], r[j], dot);
      }
    }
    sq = lanes_sum<LPR>(sq);
    dot = lanes_sum<LPR>(dot);
    if constexpr (WPR > 1) {
      if (lane == 0) {
        part[parity][0][wave] = sq;
        part[parity][1][wave] = dot;
      }
      __syncthreads();
      const int w0 = wave / WPR * WPR;
      sq = part[parity][0][w0];
      dot = part[parity][1][w0];
#pragma unroll
      for (int i = 1; i < WPR; ++i) {
        sq += part[parity][0][w0 + i];
        dot += part[parity][1][w0 + i];
      }
    }
    const float rstd = rsqrtf(sq / (float)a.H + a.eps);
    const float f = rstd * rstd * dot / (float)a.H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first + i * WPR * kWave;
      if (!live || c >= C) continue;
      const floatx8 r = R::wide(rc[i]), d = R::wide(dc[i]);
      floatx8 v = rstd * (R::wide(LEAN ? R::load(gain + 8 * c) : gc[LEAN ? 0 : i]) * d - r * f);
      if (adds) v += R::wide(LEAN ? R::load(dres + 8 * c) : ac[i]);
      R::store_once(dx + 8 * c, R::narrow(v));
      dg[i] += d * r * rstd;
    }
  }
  if (!a.part) return;
  float* p = a.part + (size_t)blockIdx.x * a.H;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first + i * WPR * kWave;
      if (c < C) Row<PW_F32>::store(p + 8 * c, dg[i]);
    }
  } else {
    // several rows at a time: their lanes' shares meet first
    static_assert(kRows == 1 || NV == 1, "one chunk a lane");
    constexpr int kLanes = LPR * WPR;   // of a row: thread own * kLanes + first
    __shared__ floatx8 sums[kRows * kLanes];
    sums[threadIdx.x] = dg[0];
    __syncthreads();
    if ((int)threadIdx.x < kLanes && (int)threadIdx.x < C) {
      floatx8 s = dg[0];
      for (int i = 1; i < kRows; ++i) s += sums[i * kLanes + threadIdx.x];
      Row<PW_F32>::store(p + 8 * threadIdx.x, s);
    }
  }
}

// dg = the sum of `n` partial rows: a block takes 16 columns, 64 threads of
// four lanes apiece share the rows, and LDS joins them in a fixed order.
__global__ __launch_bounds__(256) void join_rows_kernel(const float* __restrict__ part, int n, int H,
                                                        float* __restrict__ out) {
  __shared__ floatx4 sums[64][4];
  const int q = (int)threadIdx.x & 3, rg = (int)threadIdx.x >> 2;
  const int col = (int)blockIdx.x * 16 + 4 * q;
  floatx4 s = {0.f, 0.f, 0.f, 0.f};
  if (col < H)
    for (int i = rg; i < n; i += 64) s += *reinterpret_cast<const floatx4*>(part + (size_t)i * H + col);
  sums[rg][q] = s;
  __syncthreads();
  for (int w = 32; w > 0; w >>= 1) {
    if (rg < w) sums[rg][q] += sums[rg + w][q];
    __syncthreads();
  }
  if (rg == 0 && col < H) *reinterpret_cast<floatx4*>(out + col) = sums[0][q];
}

template <int DT, int LPR, int WPR, int NV>
hipError_t run_norm_grad(const NormGradArgs& a, float* dweight, hipStream_t s) {
  constexpr int kRows = block_rows(LPR, WPR);
  const unsigned want = ((unsigned)a.T + kRows - 1) / kRows;
  // Each block's share of dweight is written and read, so no more blocks than
  // keep the memory busy: one a CU, two where a row is 4 KB or less (bf16
  // [16384][4096] 98 us against 105 with two, [1024][8192] 19 against 26;
  // [16384][2048] 61 against 55).
  const unsigned most = (int64_t)a.H * (DT == PW_F32 ? 4 : 2) <= 4096 ? kNormGradBlocks : kNormGradBlocks / 2;
  const unsigned grid = want < most ? want : most;
  // registers of a lane's chunks: 4 (16-bit) or 8 (fp32) for each of three matrices, again for the row ahead
  constexpr int kChunkRegs = NV * (DT == PW_F32 ? 8 : 4);
  constexpr bool kLean = WPR == 16 && kChunkRegs >= 16, kAhead = !kLean && kChunkRegs <= 16;
  hipLaunchKernelGGL((rmsnorm_grad_kernel<DT, LPR, WPR, NV, kAhead, kLean>), dim3(grid), dim3(block_waves(WPR) * kWave),
                     0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dweight) return e;
  hipLaunchKernelGGL(join_rows_kernel, dim3((a.H + 15) / 16), dim3(256), 0, s, a.part, (int)grid, a.H, dweight);
  return hipGetLastError();
}

template <int DT>
hipError_t pick_norm_grad(const NormGradArgs& a, float* dweight, hipStream_t s) {
  const int C = a.H / 8;
  if (C <= 8) return run_norm_grad<DT, 8, 1, 1>(a, dweight, s);
  if (C <= 16) return run_norm_grad<DT, 16, 1, 1>(a, dweight, s);
  if (C <= 32) return run_norm_grad<DT, 32, 1, 1>(a, dweight, s);
  if (C <= 64) return run_norm_grad<DT, 64, 1, 1>(a, dweight, s);
  if (C <= 128) return run_norm_grad<DT, 64, 2, 1>(a, dweight, s);
  if (C <= 256) return run_norm_grad<DT, 64, 4, 1>(a, dweight, s);
  if (C <= 512) return run_norm_grad<DT, 64, 4, 2>(a, dweight, s);
  if (C <= 1024) return run_norm_grad<DT, 64, 16, 1>(a, dweight, s);
  if (C <= 2048) return run_norm_grad<DT, 64, 16, 2>(a, dweight, s);
  return run_norm_grad<DT, 64, 16, 4>(a, dweight, s);
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, int dtype, bool e4m3, hipStream_t s) {
  switch (dtype) {
    case PW_F32: return e4m3 ? pick_norm<PW_F32, true>(a, s) : pick_norm<PW_F32, false>(a, s);
    case PW_F16: return e4m3 ? pick_norm<PW_F16, true>(a, s) : pick_norm<PW_F16, false>(a, s);
    case PW_BF16: return e4m3 ? pick_norm<PW_BF16, true>(a, s) : pick_norm<PW_BF16, false>(a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_rmsnorm_grad(const NormGradArgs& a, int dtype, float* dweight, hipStream_t s) {
  switch (dtype) {
    case PW_F32: return pick_norm_grad<PW_F32>(a, dweight, s);
    case PW_F16: return pick_norm_grad<PW_F16>(a, dweight, s);
    case PW_BF16: return pick_norm_grad<PW_BF16>(a, dweight, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace pw
