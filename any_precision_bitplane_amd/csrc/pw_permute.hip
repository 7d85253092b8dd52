// Tokens sorted by expert and back, with their weights, and the gradients.
//
//   permute     xs[inv[t k + j]] = x[t]                 (a stable counting sort of the slots by expert id)
//   unpermute   y[t]  = sum_j w[t][j] rows[inv[t k + j]]        (fp32 sum in slot order, one rounding)
//   gradients   dx[t] = sum_j dxs[inv[t k + j]]                 (permute)
//               drows[inv[t k + j]] = w[t][j] dy[t],  dw[t][j] = <dy[t], rows[inv[t k + j]]>   (unpermute)
//
// A dropped slot (expert id outside [0, E)) has no place, inv = -1: nothing is
// written for it and it adds nothing.  Rows from the last expert's end on are
// left as they were.  All of it is bound by memory: every row is read and
// written once, in 16-byte accesses.
#include "pw_rows.h"

namespace pw {

namespace {

constexpr unsigned kMaxGrid = 1u << 20;
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr uint32_t kDropped = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t expert_of(int32_t id, int E) {
  return (uint32_t)id < (uint32_t)E ? (uint32_t)id : kDropped;
}

// Copies token t's row (and its scales) to the places pos[0..k), -1: none.
// `lanes` threads share the row.
__device__ __forceinline__ void scatter_row(const PermuteArgs& a, int t, const int* pos, int lane, int lanes) {
  const uint8_t* src = a.x + (int64_t)t * a.x_stride;
  constexpr int U = 4;   // chunks requested together
  const int64_t step = 16 * (int64_t)lanes;
  for (int64_t c0 = 16 * (int64_t)lane; c0 < a.row_bytes; c0 += U * step) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * step < a.row_bytes) v[u] = *reinterpret_cast<const uint4*>(src + c0 + u * step);
    for (int j = 0; j < a.k; ++j) {
      if (pos[j] < 0) continue;
      uint8_t* dst = a.xs + pos[j] * a.xs_stride + c0;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + u * step < a.row_bytes) *reinterpret_cast<uint4*>(dst + u * step) = v[u];
    }
  }
  for (int g = lane; g < a.groups; g += lanes) {
    const float v = a.x_scale[(int64_t)t * a.groups + g];
    for (int j = 0; j < a.k; ++j)
      if (pos[j] >= 0) a.xs_scale[(int64_t)pos[j] * a.groups + g] = v;
  }
}

// Few slots: one launch.  Every block takes one token and finds its slots'
// places itself, by counting the slots that sort before each (ids in LDS, one
// wave per place).  The E + 1 expert offsets are counted the same way, spread
// over the blocks.
__global__ __launch_bounds__(kThreads) void permute_small_kernel(PermuteArgs a) {
  extern __shared__ uint32_t shared[];
  uint32_t* ids = shared;                                  // [S rounded up to a wave]
  const int S = a.T * a.k;
  const int padded = (S + kWave - 1) / kWave * kWave;
  int* pos = reinterpret_cast<int*>(shared + padded);      // [k]
  const int t = blockIdx.x;
  const int wave = uniform((int)threadIdx.x / kWave), lane = (int)threadIdx.x & (kWave - 1);
  bool bad = false;
  for (int i = threadIdx.x; i < padded; i += kThreads) {
    const uint32_t e = i < S ? expert_of(a.ids[i], a.E) : kDropped;
    bad |= i < S && e == kDropped;
    ids[i] = e;
  }
  if (bad && t == 0 && a.status) raise_status(a.status, PW_DEV_BAD_EXPERT_ID);
  __syncthreads();
  const int mine = t <= a.E ? (a.E - t) / a.T + 1 : 0;     // offsets of experts t, t + T, ... <= E
  for (int item = wave; item < a.k + mine; item += kWaves) {
    const bool slot = item < a.k;
    const int s = slot ? t * a.k + item : 0;               // an offset counts the slots of lower experts only
    const uint32_t e = slot ? ids[s] : (uint32_t)(t + (item - a.k) * a.T);
    int before = 0;
    for (int i = lane; i < padded; i += kWave) {
      const uint32_t o = ids[i];
      before += __popcll(__ballot(o < e || (o == e && i < s)));
    }
    if (lane != 0) continue;
    if (slot) {
      const int p = e == kDropped ? -1 : before;
      pos[item] = p;
      a.inv[s] = p;
      if (p >= 0 && a.perm) a.perm[p] = s;
    } else {
      a.offsets[e] = before;
    }
  }
  __syncthreads();
  scatter_row(a, t, pos, threadIdx.x, kThreads);
}

// Many slots, first launch: slots per expert in each of the pieces.
__global__ __launch_bounds__(1024) void permute_count_kernel(PermuteArgs a) {
  __shared__ int count[kMaxExperts];
  for (int e = threadIdx.x; e < a.E; e += 1024) count[e] = 0;
  __syncthreads();
  const int64_t s0 = (int64_t)blockIdx.x * a.piece_tokens * a.k;
  const int64_t S = (int64_t)a.T * a.k;
  const int64_t s1 = s0 + (int64_t)a.piece_tokens * a.k < S ? s0 + (int64_t)a.piece_tokens * a.k : S;
  bool bad = false;
  for (int64_t s = s0 + threadIdx.x; s < s1; s += 1024) {
    const uint32_t e = expert_of(a.ids[s], a.E);
    if (e != kDropped) atomicAdd(&count[e], 1);
    else bad = true;
  }
  if (bad && a.status) raise_status(a.status, PW_DEV_BAD_EXPERT_ID);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += 1024) a.counts[blockIdx.x * a.E + e] = count[e];
}

// Second launch: a block takes block_tokens tokens of one piece.  An expert's
// slots of this block start at its offset plus its slots in earlier pieces and
// in earlier blocks of the piece (counted again here); inside the block a
// slot's rank is its position among the equal ids, found by ballots.
__global__ __launch_bounds__(kThreads) void permute_scatter_kernel(PermuteArgs a) {
  __shared__ int total[kWaves][kMaxExperts];
  __shared__ int before[kWaves][kMaxExperts];
  __shared__ int next[kMaxExperts];          // the expert's next place in this block
  __shared__ int wcnt[kWaves][kMaxExperts];
  extern __shared__ uint32_t shared[];
  int* pos = reinterpret_cast<int*>(shared); // [block_tokens * k]
  const int tid = threadIdx.x;
  const int wave = uniform(tid / kWave), lane = tid & (kWave - 1);
  const int64_t t0 = (int64_t)blockIdx.x * a.block_tokens;
  const int nt = (int)(a.T - t0 < a.block_tokens ? a.T - t0 : a.block_tokens);
  const int piece = (int)(t0 / a.piece_tokens);

  for (int e = lane; e < a.E; e += kWave) {
    int all = 0, prior = 0;
#pragma unroll 8
    for (int p = wave; p < a.pieces; p += kWaves) {
      const int c = a.counts[p * a.E + e];
      all += c;
      prior += p < piece ? c : 0;
    }
    total[wave][e] = all;
    before[wave][e] = prior;
  }
  for (int e = tid; e < a.E; e += kThreads) next[e] = 0;
  __syncthreads();
  for (int64_t s = (int64_t)piece * a.piece_tokens * a.k + tid; s < t0 * a.k; s += kThreads) {
    const uint32_t e = expert_of(a.ids[s], a.E);
    if (e != kDropped) atomicAdd(&next[e], 1);
  }
  __syncthreads();
  if (wave == 0) {
    int c[4], sum = 0;                        // lane l owns experts 4l .. 4l + 3
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * lane + i;
      c[i] = 0;
      if (e < a.E)
#pragma unroll
        for (int w = 0; w < kWaves; ++w) c[i] += total[w][e];
      sum += c[i];
    }
    int inclusive = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int y = __shfl_up(inclusive, d, kWave);
      if (lane >= d) inclusive += y;
    }
    int off = inclusive - sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * lane + i;
      if (e < a.E) {
        if (blockIdx.x == 0) a.offsets[e] = off;
        int start = off + next[e];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) start += before[w][e];
        next[e] = start;
      }
      off += c[i];
    }
    if (lane == kWave - 1 && blockIdx.x == 0) a.offsets[a.E] = inclusive;
  }
  __syncthreads();

  const int slots = nt * a.k;
  for (int r0 = 0; r0 < slots; r0 += kThreads) {
    for (int i = tid; i < kWaves * a.E; i += kThreads) wcnt[i / a.E][i % a.E] = 0;
    __syncthreads();
    const int s = r0 + tid;
    const uint32_t e = s < slots ? expert_of(a.ids[t0 * a.k + s], a.E) : kDropped;
    unsigned long long same = __ballot(e != kDropped);
    for (int bit = 0; (1 << bit) < a.E; ++bit) {
      const unsigned long long ones = __ballot(e != kDropped && ((e >> bit) & 1));
      same &= ((e >> bit) & 1) ? ones : ~ones;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1ull));
    if (e != kDropped && rank == 0) wcnt[wave][e] = __popcll(same);
    __syncthreads();
    for (int x = tid; x < a.E; x += kThreads) {
      int run = next[x];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const int c = wcnt[w][x];
        wcnt[w][x] = run;
        run += c;
      }
      next[x] = run;
    }
    __syncthreads();
    if (s < slots) {
      const int p = e == kDropped ? -1 : wcnt[wave][e] + rank;
      pos[s] = p;
      a.inv[t0 * a.k + s] = p;
      if (p >= 0 && a.perm) a.perm[p] = (int32_t)(t0 * a.k + s);
    }
    __syncthreads();
  }
  for (int t = wave; t < nt; t += kWaves) scatter_row(a, (int)t0 + t, pos + t * a.k, lane, kWave);
}

// y[t] = sum_j w[t][j] rows[inv[t k + j]]; w null: ones.  `lanes` threads (a
// power of two) share a token, each taking chunks of eight columns; the rows
// of four slots are requested together.
template <int DT>
__global__ __launch_bounds__(kThreads) void unpermute_kernel(UnpermuteArgs a, int shift) {
  using R = Row<DT>;
  using elem = typename R::elem;
  const int C = a.H / 8;
  const int lanes = 1 << shift;
  const int per_block = kThreads >> shift;
  const int lane = (int)threadIdx.x & (lanes - 1);
  const int64_t S = (int64_t)a.T * a.k;
  for (int64_t t = (int64_t)blockIdx.x * per_block + ((int)threadIdx.x >> shift); t < a.T;
       t += (int64_t)gridDim.x * per_block) {
    for (int c = lane; c < C; c += lanes) {
      floatx8 acc = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int j0 = 0; j0 < a.k; j0 += 4) {
        float w[4];
        bool in[4];
        typename R::chunk v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t s = t * a.k + j0 + i;
          const int32_t p = j0 + i < a.k ? a.inv[s] : -1;
          in[i] = p >= 0 && p < S;
          if (!in[i]) continue;
          w[i] = a.w ? a.w[s] : 1.f;
          v[i] = R::load(static_cast<const elem*>(a.rows) + p * a.rows_stride + 8 * c);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (in[i]) acc += w[i] * R::wide(v[i]);
      }
      R::store(static_cast<elem*>(a.y) + t * a.y_stride + 8 * c, R::narrow(acc));
    }
  }
}

// Gradient of unpermute, one slot at a time: `lanes` threads of a wave read the
// token's dy and the slot's row, write drows and sum dw.
template <int DT>
__global__ __launch_bounds__(kThreads) void unpermute_grad_kernel(UnpermuteGradArgs a, int shift) {
  using R = Row<DT>;
  using elem = typename R::elem;
  const int C = a.H / 8;
  const int lanes = 1 << shift;
  const int per_block = kThreads >> shift;
  const int lane = (int)threadIdx.x & (lanes - 1);
  const int64_t S = (int64_t)a.T * a.k;
  // whole waves stay in the loop, so the sums below see every lane
  for (int64_t base = (int64_t)blockIdx.x * per_block; base < S; base += (int64_t)gridDim.x * per_block) {
    const int64_t s = base + ((int)threadIdx.x >> shift);
    const int32_t p = s < S ? a.inv[s] : -1;
    const bool in = p >= 0 && p < S;
    float dot = 0.f;
    if (in) {
      const float w = a.w ? a.w[s] : 1.f;
      const elem* dy = static_cast<const elem*>(a.dy) + s / a.k * a.dy_stride;
      const elem* row = static_cast<const elem*>(a.rows) + p * a.rows_stride;
      elem* drow = static_cast<elem*>(a.drows) + p * a.drows_stride;
      constexpr int U = 4;   // chunks requested together
      for (int c0 = lane; c0 < C; c0 += U * lanes) {
        typename R::chunk d[U], r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u * lanes;
          if (c >= C) continue;
          d[u] = R::load(dy + 8 * c);
          if (a.dw) r[u] = R::load(row + 8 * c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u * lanes;
          if (c >= C) continue;
          const floatx8 dv = R::wide(d[u]);
          if (a.dw) {
            const floatx8 rv = R::wide(r[u]);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot = __builtin_fmaf(dv[i], rv[i], dot);
          }
          R::store(drow + 8 * c, R::narrow(w * dv));
        }
      }
    }
    if (!a.dw) continue;
    for (int d = lanes / 2; d > 0; d >>= 1) dot += __shfl_xor(dot, d, kWave);
    if (s < S && lane == 0) a.dw[s] = dot;
  }
}

// Threads that share `chunks` chunks: the next power of two, at most `most`.
int lanes_shift(int chunks, int most) {
  int shift = 0;
  while ((1 << shift) < chunks && (1 << shift) < most) ++shift;
  return shift;
}

unsigned grid_for(int64_t blocks) { return (unsigned)(blocks < (int64_t)kMaxGrid ? blocks : (int64_t)kMaxGrid); }

template <int DT>
hipError_t run_unpermute(const UnpermuteArgs& a, hipStream_t s) {
  const int shift = lanes_shift(a.H / 8, kThreads);
  const int per_block = kThreads >> shift;
  hipLaunchKernelGGL((unpermute_kernel<DT>), dim3(grid_for(((int64_t)a.T + per_block - 1) / per_block)),
                     dim3(kThreads), 0, s, a, shift);
  return hipGetLastError();
}

template <int DT>
hipError_t run_unpermute_grad(const UnpermuteGradArgs& a, hipStream_t s) {
  const int shift = lanes_shift(a.H / 8, kWave);
  const int per_block = kThreads >> shift;
  hipLaunchKernelGGL((unpermute_grad_kernel<DT>), dim3(grid_for(((int64_t)a.T * a.k + per_block - 1) / per_block)),
                     dim3(kThreads), 0, s, a, shift);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_permute(PermuteArgs a, hipStream_t s) {
  const int64_t S = (int64_t)a.T * a.k;
  if (S <= kPermuteSmallSlots) {
    const size_t lds = ((size_t)(S + kWave - 1) / kWave * kWave + a.k) * sizeof(uint32_t);
    hipLaunchKernelGGL(permute_small_kernel, dim3(a.T), dim3(kThreads), lds, s, a);
    return hipGetLastError();
  }
  // about 1024 blocks of at least two and at most 32 tokens (positions in LDS), pieces of whole blocks
  int64_t bt = ((int64_t)a.T + 1023) / 1024;
  bt = bt < 2 ? 2 : bt > 32 ? 32 : bt;
  if (bt < a.T / (int64_t)kMaxGrid) bt = a.T / (int64_t)kMaxGrid + 1;
  const int64_t blocks = (a.T + bt - 1) / bt;
  const int64_t per_piece = (blocks + kPermutePieces - 1) / kPermutePieces;
  a.block_tokens = (int)bt;
  a.piece_tokens = per_piece * bt;
  a.pieces = (int)((blocks + per_piece - 1) / per_piece);
  hipLaunchKernelGGL(permute_count_kernel, dim3(a.pieces), dim3(1024), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(permute_scatter_kernel, dim3((unsigned)blocks), dim3(kThreads), (size_t)bt * a.k * sizeof(int), s,
                     a);
  return hipGetLastError();
}

hipError_t launch_unpermute(const UnpermuteArgs& a, int dtype, hipStream_t s) {
  switch (dtype) {
    case PW_F32: return run_unpermute<PW_F32>(a, s);
    case PW_F16: return run_unpermute<PW_F16>(a, s);
    case PW_BF16: return run_unpermute<PW_BF16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_unpermute_grad(const UnpermuteGradArgs& a, int dtype, hipStream_t s) {
  switch (dtype) {
    case PW_F32: return run_unpermute_grad<PW_F32>(a, s);
    case PW_F16: return run_unpermute_grad<PW_F16>(a, s);
    case PW_BF16: return run_unpermute_grad<PW_BF16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace pw
