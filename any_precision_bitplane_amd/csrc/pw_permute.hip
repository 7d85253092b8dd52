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

// Up to here a lane per expert offset looks at all slots one by one (E = 256: T = 1, k = 8 5.2 us
// against 18, 128 slots 6.2 against 7.4; 256 slots 7.3 against 6.7).
constexpr int kLaneOffsetSlots = 128;
constexpr int kItems = 4;    // places a wave counts at a time
constexpr int kIdLoads = 8;  // ids a thread requests together

constexpr int kUnroll = 4;   // 16-byte pieces of a row requested together
typedef uint32_t piece_t __attribute__((ext_vector_type(4)));

// Up to N pieces of token t's row, `lanes` threads apart, from byte c0 on.
template <int N>
__device__ __forceinline__ void load_pieces(const PermuteArgs& a, int64_t t, int64_t c0, int lanes,
                                            piece_t (&v)[kUnroll]) {
  const uint8_t* src = a.x + t * a.x_stride + c0;
#pragma unroll
  for (int u = 0; u < N; ++u)
    v[u] = c0 + u * 16 * lanes < a.row_bytes ? *reinterpret_cast<const piece_t*>(src + u * 16 * lanes)
                                             : piece_t{0u, 0u, 0u, 0u};
}

// ... and their copies at the places pos[0..k), -1: none.  WAVE: all lanes of a
// wave have the same places.  Stored past the L2s, which hold none of it until
// its reader starts (k = 4, H = 2048, fp16: T = 1024 9.9 -> 8.7 us, 16384 78 ->
// 61; at worst 20.1 -> 20.8, at 4096).
template <int N, bool WAVE>
__device__ __forceinline__ void store_pieces(const PermuteArgs& a, const int* pos, int64_t c0, int lanes,
                                             const piece_t (&v)[kUnroll]) {
  for (int j = 0; j < a.k; ++j) {
    const int p = WAVE ? uniform(pos[j]) : pos[j];
    if (p < 0) continue;
    uint8_t* dst = a.xs + p * a.xs_stride + c0;
#pragma unroll
    for (int u = 0; u < N; ++u)
      if (c0 + u * 16 * lanes < a.row_bytes)
        __builtin_nontemporal_store(v[u], reinterpret_cast<piece_t*>(dst + u * 16 * lanes));
  }
}

__device__ __forceinline__ void scatter_scales(const PermuteArgs& a, int64_t t, const int* pos, int lane, int lanes) {
  for (int g = lane; g < a.groups; g += lanes) {
    const float v = a.x_scale[t * a.groups + g];
    for (int j = 0; j < a.k; ++j)
      if (pos[j] >= 0) a.xs_scale[(int64_t)pos[j] * a.groups + g] = v;
  }
}

// Few slots: one launch.  A block takes one to four tokens, 1 << shift threads
// each, and finds their slots' places itself, by counting the slots that sort
// before each (ids in LDS, one wave per place).  The E + 1 expert offsets are
// counted the same way, spread over the blocks; or, where there are fewer slots
// than a wave has to look at one by one, a lane per offset.  The rows are
// requested before any of that.
__global__ __launch_bounds__(kThreads) void permute_small_kernel(PermuteArgs a, int shift) {
  extern __shared__ uint32_t shared[];
  const int S = a.T * a.k;
  const int padded = (S + 4 * kWave - 1) / (4 * kWave) * (4 * kWave);
  uint32_t* ids = shared;                                  // [padded]
  int* pos = reinterpret_cast<int*>(shared + padded);      // [tokens * k]
  const int lanes = 1 << shift, tokens = kThreads >> shift;
  const int t0 = (int)blockIdx.x * tokens;
  const int nt = a.T - t0 < tokens ? a.T - t0 : tokens;
  const int wave = uniform((int)threadIdx.x / kWave), lane = (int)threadIdx.x & (kWave - 1);
  const int own = uniform((int)threadIdx.x >> shift);      // this thread's token
  const int64_t own_c = 16 * (int64_t)((int)threadIdx.x & (lanes - 1));
  piece_t v[kUnroll];
  if (own < nt) load_pieces<kUnroll>(a, t0 + own, own_c, lanes, v);
  bool bad = false;
  for (int i0 = threadIdx.x; i0 < padded; i0 += kIdLoads * kThreads) {
    int32_t id[kIdLoads];
#pragma unroll
    for (int u = 0; u < kIdLoads; ++u) {
      const int i = i0 + u * kThreads;
      id[u] = a.ids[i < S ? i : S - 1];
    }
#pragma unroll
    for (int u = 0; u < kIdLoads; ++u) {
      const int i = i0 + u * kThreads;
      const uint32_t e = i < S ? expert_of(id[u], a.E) : kDropped;
      bad |= i < S && e == kDropped;
      if (i < padded) ids[i] = e;
    }
  }
  if (bad && blockIdx.x == 0 && a.status) raise_status(a.status, PW_DEV_BAD_EXPERT_ID);
  __syncthreads();
  const bool by_lane = S <= kLaneOffsetSlots;
  const int slots = nt * a.k;
  // offsets of experts b, b + blocks, ... <= E
  const int b = blockIdx.x, blocks = gridDim.x;
  const int mine = by_lane || b > a.E ? 0 : (a.E - b) / blocks + 1;
  // kItems places or offsets at a time: ids before the block's own slots count
  // if they are at most e, those behind them if they are less
  const int lo = t0 * a.k;
  const int mixed0 = lo / (4 * kWave) * (4 * kWave);
  const int mixed1 = (lo + slots + 4 * kWave - 1) / (4 * kWave) * (4 * kWave);
  for (int item0 = wave * kItems; item0 < slots + mine; item0 += kWaves * kItems) {
    int at[kItems], before[kItems];
    uint32_t e[kItems], upto[kItems];
#pragma unroll
    for (int g = 0; g < kItems; ++g) {
      const int item = item0 + g;
      at[g] = item < slots ? lo + item : 0;
      e[g] = item < slots ? ids[at[g]] : (uint32_t)(b + (item - slots) * blocks);
      upto[g] = item < slots ? e[g] + 1 : e[g];            // an offset counts the slots of lower experts only
      before[g] = 0;
    }
    auto count = [&](int from, int to, const uint32_t(&below)[kItems]) {
#pragma unroll 2
      for (int i = from + 4 * lane; i < to; i += 4 * kWave) {
        const piece_t o = *reinterpret_cast<const piece_t*>(ids + i);
#pragma unroll
        for (int g = 0; g < kItems; ++g)
#pragma unroll
          for (int u = 0; u < 4; ++u) before[g] += o[u] < below[g] ? 1 : 0;
      }
    };
    count(0, mixed0, upto);
    for (int i = mixed0 + 4 * lane; i < mixed1; i += 4 * kWave) {
      const piece_t o = *reinterpret_cast<const piece_t*>(ids + i);
#pragma unroll
      for (int g = 0; g < kItems; ++g)
#pragma unroll
        for (int u = 0; u < 4; ++u) before[g] += o[u] < (i + u < at[g] ? upto[g] : e[g]) ? 1 : 0;
    }
    count(mixed1, padded, e);
#pragma unroll
    for (int g = 0; g < kItems; ++g) {
      const int item = item0 + g;
      const int n = wave_sum(before[g]);
      if (lane != 0 || item >= slots + mine) continue;
      if (item < slots) {
        const int p = e[g] == kDropped ? -1 : n;
        pos[item] = p;
        a.inv[at[g]] = p;
        if (p >= 0 && a.perm) a.perm[p] = at[g];
      } else {
        a.offsets[e[g]] = n;
      }
    }
  }
  if (by_lane)
    for (int e = b * kThreads + (int)threadIdx.x; e <= a.E; e += blocks * kThreads) {
      int before = 0;
      for (int i = 0; i < S; i += 4) {
        const piece_t o = *reinterpret_cast<const piece_t*>(ids + i);
#pragma unroll
        for (int u = 0; u < 4; ++u) before += o[u] < (uint32_t)e ? 1 : 0;
      }
      a.offsets[e] = before;
    }
  __syncthreads();
  if (own >= nt) return;
  const int64_t piece = (int64_t)kUnroll * lanes * 16;
  const int* mypos = pos + own * a.k;
  for (int64_t c0 = own_c; c0 < a.row_bytes; c0 += piece) {
    if (c0 >= piece) load_pieces<kUnroll>(a, t0 + own, c0, lanes, v);
    store_pieces<kUnroll, true>(a, mypos, c0, lanes, v);
  }
  scatter_scales(a, t0 + own, mypos, (int)threadIdx.x & (lanes - 1), lanes);
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
  for (int e = threadIdx.x; e < a.E; e += 1024) a.counts[(int64_t)blockIdx.x * a.E + e] = count[e];
}

// With many pieces their counts become sums in a launch of its own, a wave per
// expert: counts[p][e] turns into the expert's slots in the pieces before p, and
// one more row, counts[pieces][e], holds its slots in all of them.
__global__ __launch_bounds__(kWave) void permute_scan_kernel(PermuteArgs a) {
  const int e = blockIdx.x, lane = threadIdx.x;
  int carry = 0;
  for (int p0 = 0; p0 < a.pieces; p0 += kWave) {
    const int p = p0 + lane;
    const int c = p < a.pieces ? a.counts[(int64_t)p * a.E + e] : 0;
    int inclusive = c;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int y = __shfl_up(inclusive, d, kWave);
      if (lane >= d) inclusive += y;
    }
    if (p < a.pieces) a.counts[(int64_t)p * a.E + e] = carry + inclusive - c;
    carry += __shfl(inclusive, kWave - 1, kWave);
  }
  if (lane == 0) a.counts[(int64_t)a.pieces * a.E + e] = carry;
}

// Last launch, nearly all of a large call's time (T = 32768, H = 2048, k = 4, bf16
// 141 us, 4.8 TB/s of rows read and written, after 4.7 for the counts): a block
// takes block_tokens tokens of one piece.  An expert's slots of this block start at its offset plus
// its slots in earlier pieces and in earlier blocks of the piece (counted again
// here); inside the block a slot's rank is its position among the equal ids,
// found by ballots of one wave.  Each wave requests its first token's row before
// all that.
//
// NARROW (rows of up to 512 bytes): 1 << shift threads take a token.
template <bool SCANNED, bool NARROW>
__global__ __launch_bounds__(kThreads) void permute_scatter_kernel(PermuteArgs a, int shift) {
  __shared__ int total[kMaxExperts];         // the expert's slots
  __shared__ int next[kMaxExperts];          // its slots before this block, then its next place
  extern __shared__ uint32_t shared[];
  int* pos = reinterpret_cast<int*>(shared); // [block_tokens * k]
  const int tid = threadIdx.x;
  const int wave = uniform(tid / kWave), lane = tid & (kWave - 1);
  const int64_t t0 = (int64_t)blockIdx.x * a.block_tokens;
  const int nt = (int)(a.T - t0 < a.block_tokens ? a.T - t0 : a.block_tokens);
  const int slots = nt * a.k;
  const int64_t piece = t0 / a.piece_tokens;

  const int own = NARROW ? tid >> shift : wave, groups = NARROW ? kThreads >> shift : kWaves;
  const int lanes = NARROW ? 1 << shift : kWave, in_row = tid & (lanes - 1);
  piece_t v[kUnroll];
  if (own < nt) load_pieces<NARROW ? 1 : kUnroll>(a, t0 + own, 16 * (int64_t)in_row, lanes, v);
  for (int e = tid; e < a.E; e += kThreads) {
    total[e] = SCANNED ? a.counts[(int64_t)a.pieces * a.E + e] : 0;
    next[e] = SCANNED ? a.counts[piece * a.E + e] : 0;
  }
  __syncthreads();
  if constexpr (!SCANNED) {
    const int n = a.pieces * a.E, mine = (int)piece * a.E;   // at most 64 pieces
#pragma unroll 4
    for (int i = tid; i < n; i += kThreads) {
      const int c = a.counts[i], e = i % a.E;
      if (c == 0) continue;
      atomicAdd(&total[e], c);
      if (i < mine) atomicAdd(&next[e], c);
    }
  }
#pragma unroll 4
  for (int64_t s = piece * a.piece_tokens * a.k + tid; s < t0 * a.k; s += kThreads) {
    const uint32_t e = expert_of(a.ids[s], a.E);
    if (e != kDropped) atomicAdd(&next[e], 1);
  }
  __syncthreads();
  if (wave == 0) {
    int c[4], sum = 0;                        // lane l owns experts 4l .. 4l + 3
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * lane + i;
      c[i] = e < a.E ? total[e] : 0;
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
        next[e] += off;
      }
      off += c[i];
    }
    if (lane == kWave - 1 && blockIdx.x == 0) a.offsets[a.E] = inclusive;
    wave_lds_order();
    for (int r0 = 0; r0 < slots; r0 += kWave) {
      const int s = r0 + lane;
      const uint32_t e = s < slots ? expert_of(a.ids[t0 * a.k + s], a.E) : kDropped;
      unsigned long long same = __ballot(e != kDropped);
      for (int bit = 0; (1 << bit) < a.E; ++bit) {
        const unsigned long long ones = __ballot(e != kDropped && ((e >> bit) & 1));
        same &= ((e >> bit) & 1) ? ones : ~ones;
      }
      const int rank = __popcll(same & ((1ull << lane) - 1ull));
      const int start = e != kDropped ? next[e] : 0;
      wave_lds_order();
      if (e != kDropped && rank == 0) next[e] = start + __popcll(same);
      wave_lds_order();
      if (s < slots) {
        const int p = e == kDropped ? -1 : start + rank;
        pos[s] = p;
        a.inv[t0 * a.k + s] = p;
        if (p >= 0 && a.perm) a.perm[p] = (int32_t)(t0 * a.k + s);
      }
    }
  }
  __syncthreads();
  constexpr int64_t kPiece = (int64_t)kUnroll * kWave * 16;
  for (int t = own; t < nt; t += groups) {
    const int* mypos = pos + t * a.k;
    if constexpr (NARROW) {
      if (t != own) load_pieces<1>(a, t0 + t, 16 * (int64_t)in_row, lanes, v);
      store_pieces<1, false>(a, mypos, 16 * (int64_t)in_row, lanes, v);
    } else {
      for (int64_t c0 = 16 * (int64_t)lane; c0 - 16 * lane < a.row_bytes; c0 += kPiece) {
        if (t != own || c0 >= kPiece) load_pieces<kUnroll>(a, t0 + t, c0, kWave, v);
        store_pieces<kUnroll, true>(a, mypos, c0, kWave, v);
      }
    }
    if (a.groups) scatter_scales(a, t0 + t, mypos, in_row, lanes);
  }
}

// y[t] = sum_j w[t][j] rows[inv[t k + j]]; w null: ones.  `lanes` threads (a
// power of two) share a token, or one of the pieces of a longer row, each
// taking one chunk of eight columns; the rows of four slots are requested
// together.  Bound by memory: bf16, T = 16383, H = 4096, k = 2 68 us, 5.9 TB/s.
// STREAM: the rows are read past the L2s.
template <int DT, bool STREAM>
__global__ __launch_bounds__(kThreads) void unpermute_kernel(UnpermuteArgs a, int shift, int pieces) {
  using R = Row<DT>;
  using elem = typename R::elem;
  const int lanes = 1 << shift;
  const int per_block = kThreads >> shift;
  const int lane = (int)threadIdx.x & (lanes - 1);
  const int64_t S = (int64_t)a.T * a.k, n = (int64_t)a.T * pieces;
  for (int64_t i = (int64_t)blockIdx.x * per_block + ((int)threadIdx.x >> shift); i < n;
       i += (int64_t)gridDim.x * per_block) {
    const int64_t t = pieces == 1 ? i : i / pieces;
    const int c = (int)(i - t * pieces) * lanes + lane;
    if (8 * c >= a.H) continue;
    floatx8 acc = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < a.k; j0 += 4) {
      float w[4];
      bool in[4];
      typename R::chunk v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t s = t * a.k + j0 + u;
        const int32_t p = j0 + u < a.k ? a.inv[s] : -1;
        in[u] = p >= 0 && p < S;
        if (!in[u]) continue;
        w[u] = a.w ? a.w[s] : 1.f;
        const elem* row = static_cast<const elem*>(a.rows) + p * a.rows_stride + 8 * c;
        v[u] = STREAM ? R::load_once(row) : R::load(row);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (in[u]) acc += w[u] * R::wide(v[u]);
    }
    R::store_once(static_cast<elem*>(a.y) + t * a.y_stride + 8 * c, R::narrow(acc));
  }
}

// Gradient of unpermute, one slot at a time: `lanes` threads of a wave read the
// token's dy (k times, all but the first from the caches) and the slot's row,
// write drows and sum dw.  drows is stored past the L2s, which leaves them to dy
// (bf16, T = 4096, H = 4096, k = 2 37.6 -> 31.4 us; never slower); STREAM: the
// rows are read past them too.
// Bound by memory: fp16, T = 8191, H = 2048, k = 4 53 us, 5.7 TB/s.
template <int DT, bool STREAM>
__global__ __launch_bounds__(kThreads) void unpermute_grad_kernel(UnpermuteGradArgs a, int shift) {
  using R = Row<DT>;
  using elem = typename R::elem;
  typedef typename R::chunk chunk;
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
      // chunks requested together (fp32, T = 8192, H = 2048, k = 8: two 241 us, four 258, eight 224; fp16,
      // rows of 512 columns: four 66, eight 87)
      constexpr int U = DT == PW_F32 ? 8 : 4;
      for (int c0 = lane; c0 < C; c0 += U * lanes) {
        chunk d[U], r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u * lanes;
          if (c >= C) continue;
          d[u] = R::load(dy + 8 * c);
          if (a.dw) r[u] = STREAM ? R::load_once(row + 8 * c) : R::load(row + 8 * c);
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
          __builtin_nontemporal_store(R::narrow(w * dv), reinterpret_cast<chunk*>(drow + 8 * c));   // fp32 too
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

// Rows of 16 bits that fill half the 256 MB behind the L2s are read past the L2s
// (T = 32768, H = 2048, k = 4 119 -> 110 us, T = 8192 31.7 -> 29.9; T = 4096
// 14.2 -> 16.1; fp32, T = 16384, H = 4096, k = 2 144 -> 152).
constexpr int64_t kBehindL2 = 256 << 20;

template <int DT>
hipError_t run_unpermute(const UnpermuteArgs& a, hipStream_t s) {
  const int shift = lanes_shift(a.H / 8, kThreads);
  const int per_block = kThreads >> shift, pieces = (a.H / 8 + (1 << shift) - 1) >> shift;
  const dim3 grid(grid_for(((int64_t)a.T * pieces + per_block - 1) / per_block));
  if constexpr (DT != PW_F32)
    if ((int64_t)a.T * a.k * a.H * 2 >= kBehindL2 / 2) {
      hipLaunchKernelGGL((unpermute_kernel<DT, true>), grid, dim3(kThreads), 0, s, a, shift, pieces);
      return hipGetLastError();
    }
  hipLaunchKernelGGL((unpermute_kernel<DT, false>), grid, dim3(kThreads), 0, s, a, shift, pieces);
  return hipGetLastError();
}

// Rows of 16 bits that the 256 MB behind the L2s cannot hold beside drows and
// dy are read past the L2s (bf16, T = 8192, H = 4096, k = 2, 336 MB, 70.8 -> 59.3
// us; T = 3000, 123 MB, 20.9 -> 22.8; fp32, T = 8192, k = 2 143 -> 152).
template <int DT>
hipError_t run_unpermute_grad(const UnpermuteGradArgs& a, hipStream_t s) {
  const int shift = lanes_shift(a.H / 8, kWave);
  const int per_block = kThreads >> shift;
  const dim3 grid(grid_for(((int64_t)a.T * a.k + per_block - 1) / per_block));
  if constexpr (DT != PW_F32)
    if ((int64_t)a.T * (2 * a.k + 1) * a.H * 2 > kBehindL2) {
      hipLaunchKernelGGL((unpermute_grad_kernel<DT, true>), grid, dim3(kThreads), 0, s, a, shift);
      return hipGetLastError();
    }
  hipLaunchKernelGGL((unpermute_grad_kernel<DT, false>), grid, dim3(kThreads), 0, s, a, shift);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_permute(PermuteArgs a, hipStream_t s) {
  const int64_t S = (int64_t)a.T * a.k;
  if (S <= kPermuteSmallSlots) {
    // one, two or four tokens a block: every block reads all ids, and the blocks should fill the CUs (H = 2048,
    // k = 4: T = 256 5.4 / 5.7 / 6.9 us, 512 7.0 / 6.7 / 8.2, 1024 10.3 / 10.0 / 11.2, 1536 15.5 / 14.1 / 14.1)
    const int shift = a.T <= 256 ? 8 : a.T <= 1024 ? 7 : 6;
    const int tokens = kThreads >> shift;
    const size_t padded = (size_t)(S + 4 * kWave - 1) / (4 * kWave) * (4 * kWave);
    hipLaunchKernelGGL(permute_small_kernel, dim3((a.T + tokens - 1) / tokens), dim3(kThreads),
                       (padded + (size_t)tokens * a.k) * sizeof(uint32_t), s, a, shift);
    return hipGetLastError();
  }
  const PermutePlan p = permute_plan(a.T, a.k, a.E);
  a.block_tokens = p.block_tokens;
  a.piece_tokens = p.piece_tokens;
  a.pieces = p.pieces;
  const int64_t blocks = ((int64_t)a.T + p.block_tokens - 1) / p.block_tokens;
  hipLaunchKernelGGL(permute_count_kernel, dim3(p.pieces), dim3(1024), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const size_t lds = (size_t)p.block_tokens * a.k * sizeof(int);
  if (p.scan) {
    hipLaunchKernelGGL(permute_scan_kernel, dim3(a.E), dim3(kWave), 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const bool narrow = a.row_bytes <= 512;
  const int shift = lanes_shift((int)(a.row_bytes / 16), kWave);
  const dim3 grid((unsigned)blocks), block(kThreads);
  if (p.scan && narrow) hipLaunchKernelGGL((permute_scatter_kernel<true, true>), grid, block, lds, s, a, shift);
  else if (p.scan) hipLaunchKernelGGL((permute_scatter_kernel<true, false>), grid, block, lds, s, a, shift);
  else if (narrow) hipLaunchKernelGGL((permute_scatter_kernel<false, true>), grid, block, lds, s, a, shift);
  else hipLaunchKernelGGL((permute_scatter_kernel<false, false>), grid, block, lds, s, a, shift);
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
