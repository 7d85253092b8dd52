// 16-bit products of the rows of every expert with its matrix, on the matrix
// cores with fp32 sums: what the kernels of pw_product.hip, pw_product_grad.hip
// and pw_product_few.hip share.
//
// Tiles.  A block takes a tile of BM rows by 256 columns of one expert and walks
// the reduction in steps of 64, a cache line of every row (with steps of 32 the
// L2s serve every line twice: 8192 x 8192 x 8192 bf16 907 us against 850 when this
// was changed, 760 now).  A
// step's operands are copied from memory to LDS without passing registers, ahead
// of the products.  An operand whose reduction index is contiguous in memory lies
// in LDS as rows of 64 (eight 16-byte pieces, piece c of row r at place c ^ (r /
// 2 & 7), so that sixteen rows' pieces fall on different banks); one whose other
// index is contiguous lies as it is and is transposed by the reads.
#pragma once

#include <type_traits>

#include "pw_device.h"
#include "pw_internal.h"
#include "pw_rows.h"

namespace pw {

constexpr int kProdGroup = 8;     // row tiles that go through all columns together
constexpr uint32_t kRsrcBytes = 0x80000000u;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_void;

template <int DT>
struct Mma;
template <>
struct Mma<PW_F16> {
  typedef _Float16 frag __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ f32x4 mma(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(frag, a), __builtin_bit_cast(frag, b), c, 0, 0, 0);
  }
};
template <>
struct Mma<PW_BF16> {
  typedef __bf16 frag __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ f32x4 mma(s16x8 a, s16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(frag, a), __builtin_bit_cast(frag, b), c, 0, 0, 0);
  }
};

// Rows [first, first + count) of expert e, inside [0, S) whatever offsets holds.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e, int S, int& first, int& count) {
  if (!offsets) {
    first = 0;
    count = S;
    return;
  }
  const int a = min(max(offsets[e], 0), S), b = min(max(offsets[e + 1], 0), S);
  first = a;
  count = max(b - a, 0);
}

// Tile of a block.  Tiles are numbered expert by expert, inside one in groups of
// kProdGroup row tiles that go through the column tiles together, and dealt to
// the eight XCDs in contiguous stretches, so that what runs together on an XCD
// shares rows of x and of w in its L2.
struct Tile {
  int e, row0, rows, nt;   // rows: the expert's from row0 on; 0: no tile for this block
};

// Where every expert's row tiles of BM rows begin: lane l has experts 4 l .. 4 l + 3.
template <int BM>
struct TileScan {
  int first[4], count[4], before, upto, tiles;   // tiles: row tiles of all experts
  __device__ __forceinline__ TileScan(const int32_t* offsets, int E, int S) {
    const int lane = (int)threadIdx.x & (kWave - 1);
    int mine = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 4 * lane + j;
      first[j] = count[j] = 0;
      if (e < E) expert_rows(offsets, e, S, first[j], count[j]);
      mine += (count[j] + BM - 1) / BM;
    }
    upto = mine;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
      const int v = __shfl_up(upto, d, kWave);
      if (lane >= d) upto += v;
    }
    before = upto - mine;
    tiles = __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  // Tile `id` of tiles * NT.
  __device__ __forceinline__ Tile at(unsigned id, int NT) const {
    const int lane = (int)threadIdx.x & (kWave - 1);
    const int m = (int)(id / (unsigned)NT);
    const int owner = __builtin_ctzll(__ballot(before <= m && m < upto));
    int e = 4 * lane, from = first[0], n = count[0], done = before;
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const int t = (count[j] + BM - 1) / BM;
      if (e == 4 * lane + j && done + t <= m) {
        done += t;
        e = 4 * lane + j + 1;
        from = first[j + 1];
        n = count[j + 1];
      }
    }
    e = __builtin_amdgcn_readlane(e, owner);
    from = __builtin_amdgcn_readlane(from, owner);
    n = __builtin_amdgcn_readlane(n, owner);
    done = __builtin_amdgcn_readlane(done, owner);
    const int of_e = (n + BM - 1) / BM;
    const int local = (int)(id - (unsigned)done * (unsigned)NT);
    const int group = local / (kProdGroup * NT), rem = local - group * kProdGroup * NT;
    const int here = min(kProdGroup, of_e - group * kProdGroup);
    const int nt = rem / here, mt = group * kProdGroup + rem - nt * here;
    return {e, from + mt * BM, n - mt * BM, nt};
  }
};

template <int BM>
__device__ __forceinline__ Tile find_tile(const int32_t* offsets, int E, int S, int NT) {
  const TileScan<BM> scan(offsets, E, S);
  const unsigned total = (unsigned)scan.tiles * (unsigned)NT;
  const unsigned each = (total + 7) / 8, i = blockIdx.x / 8, id = (blockIdx.x % 8) * each + i;
  if (i >= each || id >= total) return {0, 0, 0, 0};
  return scan.at(id, NT);
}

// The tiles that do not fill a last round of the CUs are cut along the reduction,
// so that they do: each of the last `rest` tiles into `parts`, whose sums go to
// memory and are added, in their order, by a launch of their own.
template <int BM>
struct Rounds {
  static constexpr unsigned kTogether = product_blocks(BM);
  unsigned whole, rest, parts;
  __device__ __forceinline__ Rounds(unsigned total, int steps, bool cut) {
    rest = cut ? total % kTogether : 0;
    parts = product_parts(BM, rest, (unsigned)steps, kTogether);
    if (parts == 1) rest = 0;
    whole = total - rest;
  }
};

// The blocks are dealt to eight XCDs.
inline int64_t product_grid(int64_t row_tiles, int64_t NT) { return (row_tiles * NT + 7) / 8 * 8; }
// A launch has less than 2^32 threads.
inline bool launch_fits(int64_t blocks, int threads) { return blocks * threads <= 0xFFFFFFFFll; }

// ----- a tile's operands ------------------------------------------------------

// 16 bytes a lane from memory to LDS: lane l's land at `to` + 16 l.  Offsets from
// 2^31 on read as zero.  The compiler does not see that the copy writes LDS:
// what reads it stands behind a step's barrier, which waits for the copies (with
// the builtin it waits for every copy before each transposing read).
typedef uint32_t rsrc_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ rsrc_t copy_rsrc(const void* base) {
  const uint64_t p = (uint64_t)base;
  return rsrc_t{(uint32_t)p, (uint32_t)(p >> 32) & 0xFFFFu, kRsrcBytes, 0x00020000u};
}
// `to` + AWAY: the wave's place, `more`: bytes that every lane adds.  The place is
// handed over in m0, so that the compiler knows what m0 holds.
template <int AWAY>
__device__ __forceinline__ void copy16(rsrc_t rs, uint32_t to, uint32_t at, uint32_t more) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "{m0}"(to + AWAY), "v"(at), "s"(rs), "s"(more)
               : "memory");
}
__device__ __forceinline__ uint32_t lds_at(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// Where the lanes of a wave fetch their 16-byte pieces of a tile of R rows of 64
// (reduction contiguous).  at[i]: byte offset of the lane's piece of copy i.  A
// copy of a wave covers eight rows: lane l fetches row l / 8.  SPLIT: the second
// half of the rows has a base of its own.
template <int R, int WAVES, bool SPLIT = false>
struct RowsOperand {
  static constexpr int kCopies = R / 8 / WAVES, kApart = WAVES * 1024;
  uint32_t at[kCopies], more;
  int piece, K;
  rsrc_t rs, second;
  template <class RowOffset>
  __device__ __forceinline__ void init(const char* base, const char* base2, int K_, int wave, int lane, RowOffset offset_of) {
    rs = copy_rsrc(base);
    second = copy_rsrc(base2);
    K = K_;
    piece = (lane & 7) ^ (lane / 16 + 4 * (wave & 1));
#pragma unroll
    for (int i = 0; i < kCopies; ++i) at[i] = offset_of((i * WAVES + wave) * 8 + lane / 8) + (uint32_t)(piece * 16);
  }
  // The copies from now on are step t's, in rising order of t; past the end, K, reads zero.
  __device__ __forceinline__ void begin(int t) {
    const int k = t * kProdK;
    more = (uint32_t)k * 2u;
    if (k + kProdK > K)
#pragma unroll
      for (int i = 0; i < kCopies; ++i) at[i] = k + piece * 8 < K ? at[i] : kOutOfRange;
  }
  template <int I>
  __device__ __forceinline__ void copy(uint32_t to) const {
    copy16<I * kApart>(SPLIT && I >= kCopies / 2 ? second : rs, to, at[I], more);
  }
};

// The same of a tile of KS reduction rows of C contiguous columns; a copy of a
// wave covers 512 / C rows.
__device__ __forceinline__ int cols_place(int k) { return 2 * (k & 3) + (k & 8); }   // piece c of row k lies at place c ^ this
template <int C, int WAVES, int KS = kProdK>
struct ColsOperand {
  static constexpr int kCopies = KS * C / 512 / WAVES, kApart = WAVES * 1024;
  uint32_t at[kCopies];
  int first, K;
  const char* base;
  int64_t step_bytes;
  rsrc_t rs;
  // base: the first of K reduction rows.  Columns past the matrix are read from its last piece.
  __device__ __forceinline__ void init(const char* base_, int K_, int wave, int lane, int64_t row_bytes, int pieces) {
    base = base_;
    K = K_;
    step_bytes = KS * row_bytes;
    first = wave * (512 / C) + lane / (C / 8);
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int row = first + i * WAVES * (512 / C);
      at[i] = (uint32_t)(row * row_bytes) + (uint32_t)(min((lane & (C / 8 - 1)) ^ cols_place(row), pieces - 1) * 16);
    }
  }
  __device__ __forceinline__ void begin(int t) {
    const int left = K - t * KS;
    rs = copy_rsrc(base + t * step_bytes);
    if (left < KS)
#pragma unroll
      for (int i = 0; i < kCopies; ++i) at[i] = first + i * WAVES * (512 / C) < left ? at[i] : kOutOfRange;
  }
  template <int I>
  __device__ __forceinline__ void copy(uint32_t to) const {
    copy16<I * kApart>(rs, to, at[I], 0u);
  }
};

// Operand of 16 rows (or columns) from `r0` on for the 32 reduction steps from
// 32 kk on: lane l holds row l % 16, steps 8 (l / 16) .. + 7.
__device__ __forceinline__ s16x8 read_rows(const char* lds, int r0, int kk, int lane) {
  const int r = lane & 15, piece = (4 * kk + lane / 16) ^ (r / 2);
  return *reinterpret_cast<const s16x8*>(lds + (r0 + r) * 128 + piece * 16);
}
// The transposing read gives lane i of sixteen column i of four rows of sixteen
// columns, lanes 4 j .. 4 j + 3 of which hold the address of row j's.
template <int C>
__device__ __forceinline__ s16x8 read_cols(const char* lds, int c0, int kk, int lane) {
  const int k = 32 * kk + 8 * (lane / 16) + (lane & 15) / 4;
  const int c = c0 + 4 * (lane & 3);
  typedef __attribute__((address_space(3))) s16x4* p4;
  const char* p = lds + k * (C * 2) + (((c / 8) ^ cols_place(k)) * 16) + (c & 4) * 2;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((p4)(p));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((p4)(p + 4 * (C * 2)));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// All but the newest LEFT copies of every wave have landed, and every wave has
// read its operands.
template <int LEFT>
__device__ __forceinline__ void step_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(LEFT) : "memory");
}

// Sums of a wave's 16 RI rows, from 16 RI wm on, by 16 CJ columns of the tile's TN,
// from 16 CJ wn on (HALVES: by 8 CJ columns of either half, from 8 CJ wn on), over
// `steps` steps of 64.  XC, WC: the operand of
// the rows, of the columns, is read transposed.  xo, wo: their copies; past the
// last step they write zeros.  LDS holds XB steps of x (TM rows), then two of w.
//
// The products are 16 x 16 x 32 (a wave's sums are read and written half as often
// as by 32 x 32 x 16 ones, which the clock shows).  The operands of 32 reduction
// steps are read from LDS while the products of the 32 before run.  With the last
// of a step's operands in registers its buffers are free: behind the barrier the
// next step's first operands are read and the copies of w of the step after it
// are started, those of x with them (XB 2) or a part later (XB 3: a step ahead
// more, and the waves' copies do not all come at once).  Reads and copies are
// dealt out between the products, which take longer than issuing them.
template <int I, int N, class F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each<I + 1, N>(f);
  }
}

// Copies of the first two steps: LDS has to be free.
template <int TM, int XB, class XOperand, class WOperand>
__device__ __forceinline__ void start_steps(char* lds, int wave, XOperand& xo, WOperand& wo) {
  constexpr int XBYTES = TM * kProdK * 2, kWBytes = WOperand::kCopies * WOperand::kApart;
  const uint32_t base = lds_at(lds) + (uint32_t)wave * 1024u;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    xo.begin(t);
    wo.begin(t);
    each<0, XOperand::kCopies>([&](auto i) { xo.template copy<i>(base + t * XBYTES); });
    each<0, WOperand::kCopies>([&](auto i) { wo.template copy<i>(base + XB * XBYTES + t * kWBytes); });
  }
}

// LIVE: pieces of 16 rows with rows of the expert among them; the other sums stay zero.
template <int DT, int LIVE, int RI, int CJ, int TM, int TN, bool HALVES, bool XC, bool WC, int XB, class XOperand, class WOperand>
__device__ __forceinline__ void sum_live(f32x4 (&acc)[RI][CJ], char* lds, int steps, int wave, int wm, int wn, int lane,
                                         XOperand& xo, WOperand& wo) {
  constexpr int XN = XOperand::kCopies, WN = WOperand::kCopies;
  constexpr int kProducts = LIVE * CJ, kReads = LIVE ? LIVE + CJ : 0, kSlots = LIVE ? kProducts : 1, kParts = kProdK / 32;
  constexpr int XBYTES = TM * kProdK * 2, kWBytes = TN * kProdK * 2;
  static_assert(kWBytes == WOperand::kCopies * WOperand::kApart, "the copies fill a step");
  constexpr int kLast = XB == 2 ? WN + XN : WN;   // copies behind the barrier
  constexpr int kReadEvery = kSlots / (kReads + 2), kXEvery = kSlots < XN ? 1 : kSlots / XN;
  // a copy every so many products, or so many copies with each
  constexpr int kSpread = XB == 2 ? kLast : 2 * kLast, kCopyEvery = kSlots < kSpread ? 1 : kSlots / kSpread;
  constexpr int kTogether = (kLast + kSlots - 1) / kSlots, kXTogether = (XN + kSlots - 1) / kSlots;
  static_assert((kReadEvery > 0 || !LIVE) && kParts == 2, "a product for every read");
  const uint32_t base = lds_at(lds) + (uint32_t)wave * 1024u, base_w = base + XB * XBYTES;   // of the wave's copies
  // The first half of x's operands is used up early and read again into the same registers.
  constexpr int kOnce = LIVE / 2, kTwice = LIVE - kOnce;
  s16x8 xa[kOnce + 1], xb[2][kTwice + 1], w[2][CJ];
  // operand j of LIVE + CJ of part kk, in the order of their reads
  auto read = [&](const char* at_x, const char* at_w, int kk, int j) {
    if (j < CJ) {
      const int c = HALVES ? j / (CJ / 2) * (TN / 2) + (wn * (CJ / 2) + j % (CJ / 2)) * 16 : (wn * CJ + j) * 16;
      w[kk & 1][j] = WC ? read_cols<TN>(at_w, c, kk, lane) : read_rows(at_w, c, kk, lane);
    } else {
      const int i = j < CJ + kTwice ? j - CJ + kOnce : j - CJ - kTwice, r = (wm * RI + i) * 16;
      (i < kOnce ? xa[i < kOnce ? i : 0] : xb[kk & 1][i < kOnce ? 0 : i - kOnce]) =
          XC ? read_cols<TM>(at_x, r, kk, lane) : read_rows(at_x, r, kk, lane);
    }
  };
  step_barrier<XN + WN>();
#pragma unroll
  for (int j = 0; j < kReads; ++j) read(lds, lds + XB * XBYTES, 0, j);
  int bx = 0;   // x's buffer of step t
  for (int t = 0; t < steps; ++t) {
    const char* const at_x = lds + bx * XBYTES;
    const char* const at_w = lds + XB * XBYTES + (t & 1) * kWBytes;
    bx = bx == XB - 1 ? 0 : bx + 1;
    const char* const then_x = lds + bx * XBYTES;
    const char* const then_w = lds + XB * XBYTES + (~t & 1) * kWBytes;
    const uint32_t to_x = base + (uint32_t)((XB == 2 ? bx ^ 1 : bx == XB - 1 ? 0 : bx + 1) * XBYTES);   // step t + 2's
    const uint32_t to_w = base_w + (uint32_t)((t & 1) * kWBytes);
    xo.begin(t + 2);
    wo.begin(t + 2);
    each<0, kParts>([&](auto kk) {
      constexpr bool last = kk == kParts - 1;
      if constexpr (last) step_barrier<XB == 2 ? 0 : XN>();
      __builtin_amdgcn_sched_barrier(0);
      each<0, kSlots>([&](auto j) {
        constexpr int row = j / CJ;
        if constexpr (LIVE > 0)
          acc[row][j % CJ] = Mma<DT>::mma(w[kk & 1][j % CJ], row < kOnce ? xa[row < kOnce ? row : 0] : xb[kk & 1][row < kOnce ? 0 : row - kOnce],
                                          acc[row][j % CJ]);
        each<0, kReads>([&](auto i) {
          // not before the last product with what is in its registers
          constexpr int own = i - CJ - kTwice, slot = own >= 0 && (own + 1) * CJ - 1 > i * kReadEvery ? (own + 1) * CJ - 1 : i * kReadEvery;
          static_assert(slot < kSlots, "a product for every read");
          if constexpr (slot == j) {
            if constexpr (last) read(then_x, then_w, 0, i);   // behind the last step: not used
            else read(at_x, at_w, 1, i);
          }
        });
        if constexpr (last && j % kCopyEvery == 0)
          each<j / kCopyEvery * kTogether, (j / kCopyEvery + 1) * kTogether>([&](auto i) {
            if constexpr (i < WN) wo.template copy<i>(to_w);
            else if constexpr (i < kLast) xo.template copy<i - WN>(to_x);
          });
        if constexpr (XB == 3 && kk == 0 && j % kXEvery == 0)
          each<j / kXEvery * kXTogether, (j / kXEvery + 1) * kXTogether>([&](auto i) {
            if constexpr (i < XN) xo.template copy<i>(to_x);
          });
        __builtin_amdgcn_sched_barrier(0);
      });
    });
  }
}

// live: 16-row pieces of the wave that the expert has rows in (a wave may have
// none).  An expert's last tile so costs by the quarter of its rows.
template <int DT, int RI, int CJ, int TM, int TN, bool HALVES, bool XC, bool WC, int XB, class XOperand, class WOperand>
__device__ __forceinline__ void sum_steps(f32x4 (&acc)[RI][CJ], char* lds, int steps, int live, int wave, int wm, int wn,
                                          int lane, XOperand& xo, WOperand& wo) {
#pragma unroll
  for (int r = 0; r < RI; ++r)
#pragma unroll
    for (int c = 0; c < CJ; ++c) acc[r][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (steps <= 0) return;
  start_steps<TM, XB>(lds, wave, xo, wo);
  constexpr int kFew = RI / 2 < 2 ? RI : RI / 2;
  if (live > RI / 2 || (live > 0 && kFew == RI))
    sum_live<DT, RI, RI, CJ, TM, TN, HALVES, XC, WC, XB>(acc, lds, steps, wave, wm, wn, lane, xo, wo);
  else if (live > 0)
    sum_live<DT, kFew, RI, CJ, TM, TN, HALVES, XC, WC, XB>(acc, lds, steps, wave, wm, wn, lane, xo, wo);
  else
    sum_live<DT, 0, RI, CJ, TM, TN, HALVES, XC, WC, XB>(acc, lds, steps, wave, wm, wn, lane, xo, wo);
  step_barrier<0>();   // no copy is under way when LDS is used otherwise or the block ends
}

// The same for two operands that are both read transposed, over steps of 32 in
// three buffers, so that two blocks of half the size fit a CU and one's first
// copies and stores pass under the other's products.  (Lines of memory are whole
// in a step of any length here: its rows are the reduction's.)
template <int DT, int LIVE, int RI, int CJ, int TM, int TN, class XOperand, class WOperand>
__device__ __forceinline__ void sum_short_live(f32x4 (&acc)[RI][CJ], char* lds, int steps, int wave, int wm, int wn,
                                               int lane, XOperand& xo, WOperand& wo) {
  constexpr int XN = XOperand::kCopies, WN = WOperand::kCopies, kCopies = XN + WN;
  constexpr int kProducts = LIVE * CJ, kReads = LIVE ? LIVE + CJ : 0, kSlots = LIVE ? kProducts : 1;
  constexpr int kXBytes = XN * XOperand::kApart, kBytes = kXBytes + WN * WOperand::kApart;   // of a step
  constexpr int kReadEvery = kSlots / (kReads + 2), kCopyEvery = kSlots < kCopies ? 1 : kSlots / kCopies;
  constexpr int kTogether = (kCopies + kSlots - 1) / kSlots;
  const uint32_t base = lds_at(lds) + (uint32_t)wave * 1024u;
  constexpr int kOnce = LIVE / 2, kTwice = LIVE - kOnce;
  s16x8 xa[kOnce + 1], xb[2][kTwice + 1], w[2][CJ];
  auto read = [&](const char* at, int set, int j) {
    if (j < CJ) {
      w[set][j] = read_cols<TN>(at + kXBytes, (wn * CJ + j) * 16, 0, lane);
    } else {
      const int i = j < CJ + kTwice ? j - CJ + kOnce : j - CJ - kTwice, r = (wm * RI + i) * 16;
      (i < kOnce ? xa[i < kOnce ? i : 0] : xb[set][i < kOnce ? 0 : i - kOnce]) = read_cols<TM>(at, r, 0, lane);
    }
  };
  step_barrier<2 * kCopies>();
#pragma unroll
  for (int j = 0; j < kReads; ++j) read(lds, 0, j);
  int now = 0;   // buffer of the step
  for (int t = 0; t < steps; t += 2)   // a last step past the end multiplies zeros
    each<0, 2>([&](auto set) {
      const uint32_t freed = base + (uint32_t)(now * kBytes);
      now = now == 2 ? 0 : now + 1;
      const char* const then = lds + now * kBytes;
      xo.begin(t + set + 3);
      wo.begin(t + set + 3);
      step_barrier<kCopies>();
      __builtin_amdgcn_sched_barrier(0);
      each<0, kSlots>([&](auto j) {
        constexpr int row = j / CJ;
        if constexpr (LIVE > 0)
          acc[row][j % CJ] = Mma<DT>::mma(w[set][j % CJ], row < kOnce ? xa[row < kOnce ? row : 0] : xb[set][row < kOnce ? 0 : row - kOnce],
                                          acc[row][j % CJ]);
        each<0, kReads>([&](auto i) {
          constexpr int own = i - CJ - kTwice, slot = own >= 0 && (own + 1) * CJ - 1 > i * kReadEvery ? (own + 1) * CJ - 1 : i * kReadEvery;
          static_assert(slot < kSlots, "a product for every read");
          if constexpr (slot == j) read(then, 1 - set, i);
        });
        if constexpr (j % kCopyEvery == 0)
          each<j / kCopyEvery * kTogether, (j / kCopyEvery + 1) * kTogether>([&](auto i) {
            if constexpr (i < XN) xo.template copy<i>(freed);
            else if constexpr (i < kCopies) wo.template copy<i - XN>(freed + kXBytes);
          });
        __builtin_amdgcn_sched_barrier(0);
      });
    });
}

template <int DT, int RI, int CJ, int TM, int TN, class XOperand, class WOperand>
__device__ __forceinline__ void sum_short_steps(f32x4 (&acc)[RI][CJ], char* lds, int steps, int live, int wave, int wm,
                                                int wn, int lane, XOperand& xo, WOperand& wo) {
#pragma unroll
  for (int r = 0; r < RI; ++r)
#pragma unroll
    for (int c = 0; c < CJ; ++c) acc[r][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (steps <= 0) return;
  constexpr int XN = XOperand::kCopies, WN = WOperand::kCopies;
  constexpr int kXBytes = XN * XOperand::kApart, kBytes = kXBytes + WN * WOperand::kApart;
  const uint32_t base = lds_at(lds) + (uint32_t)wave * 1024u;
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    xo.begin(t);
    wo.begin(t);
    each<0, XN>([&](auto i) { xo.template copy<i>(base + t * kBytes); });
    each<0, WN>([&](auto i) { wo.template copy<i>(base + t * kBytes + kXBytes); });
  }
  if (live > RI / 2) sum_short_live<DT, RI, RI, CJ, TM, TN>(acc, lds, steps, wave, wm, wn, lane, xo, wo);
  else if (live > 0) sum_short_live<DT, RI / 2, RI, CJ, TM, TN>(acc, lds, steps, wave, wm, wn, lane, xo, wo);
  else sum_short_live<DT, 0, RI, CJ, TM, TN>(acc, lds, steps, wave, wm, wn, lane, xo, wo);
  step_barrier<0>();
}

// ----- activations ------------------------------------------------------------

// Phi(z), the normal distribution function, to some digits of itself below zero
// too: in 32 bits 1 + erf(z / sqrt 2) has lost half of its digits at z = -3.7 and
// all of them from -5.6 on, where z Phi(z) is still a number of 16 bits' range.
// With a = |z| and t = 1 / (1 + 0.3 a), Phi(-a) = exp(-a^2 / 2) t P(t); P is a
// least-maximum fit (iteratively reweighted least squares) to exp(a^2 / 2) Phi(-a) / t
// for a up to 14.5, off by 2^-22.5 of it at most.  Below -13.2, where the
// exponential leaves the normal numbers, it is zero.  (8192 x 2048 bf16, 8194
// rows over 8, with GELU, residual and kept sum: 349 us with erff, 377 with erfcf,
// 324 so.)
__device__ __forceinline__ float normal_cdf(float z) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3f, __builtin_fabsf(z), 1.f));
  float p = 0.035423707f;
  p = __builtin_fmaf(p, t, -0.15615834f);
  p = __builtin_fmaf(p, t, 0.20455663f);
  p = __builtin_fmaf(p, t, -0.052033883f);
  p = __builtin_fmaf(p, t, 0.12769172f);
  p = __builtin_fmaf(p, t, 0.10017596f);
  p = __builtin_fmaf(p, t, 0.12071213f);
  p = __builtin_fmaf(p, t, 0.11963201f);
  const float below = t * p * __expf(-0.5f * z * z);
  return z < 0.f ? below : 1.f - below;
}
__device__ __forceinline__ float act_of(float z, int act) {
  if (act == PW_ACT_SILU) return silu_f32(z);
  if (act == PW_ACT_GELU) return z * normal_cdf(z);
  return z;
}
__device__ __forceinline__ float act_slope(float z, int act) {
  if (act == PW_ACT_SILU) {
    const float q = __builtin_amdgcn_rcpf(1.f + __expf(-z));
    return q * (1.f + z * (1.f - q));
  }
  if (act == PW_ACT_GELU) return normal_cdf(z) + z * 0.39894228040143268f * __expf(-0.5f * z * z);
  return 1.f;
}

// ----- eight bits ---------------------------------------------------------------

constexpr float kE4m3Max = 448.f;
constexpr float kScaleMin = 7.888609052210118e-31f;   // 2^-100: scales stay divisible
constexpr int kKeepGroup = 128;                       // columns of gate or up that share a scale

// The largest of |v|, infinity where one is no finite number.
__device__ __forceinline__ float most_of(floatx8 v, float most) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float t = __builtin_fabsf(v[j]);
    most = t < INFINITY ? fmaxf(most, t) : INFINITY;
  }
  return most;
}
__device__ __forceinline__ float scale_of(float most) {
  return most < INFINITY ? fmaxf(most / kE4m3Max, kScaleMin) : __builtin_nanf("");
}
// Codes nearest to v / scale: the product with the reciprocal, corrected by its remainder.
__device__ __forceinline__ uint2 codes_of(floatx8 v, float scale) {
  if (!(scale < INFINITY)) return {0x7F7F7F7Fu, 0x7F7F7F7Fu};
  const float inv = 1.f / scale;
  floatx8 q;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float t = v[j] * inv;
    q[j] = fminf(fmaxf(__builtin_fmaf(__builtin_fmaf(-t, scale, v[j]), inv, t), -kE4m3Max), kE4m3Max);
  }
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false), hi;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return {(uint32_t)lo, (uint32_t)hi};
}
__device__ __forceinline__ floatx8 values_of(uint2 codes, float scale) {
  floatx8 v;
#define PW_CODE(i, word, at) v[i] = __builtin_amdgcn_cvt_f32_fp8((int)(word), at) * scale
  PW_CODE(0, codes.x, 0); PW_CODE(1, codes.x, 1); PW_CODE(2, codes.x, 2); PW_CODE(3, codes.x, 3);
  PW_CODE(4, codes.y, 0); PW_CODE(5, codes.y, 1); PW_CODE(6, codes.y, 2); PW_CODE(7, codes.y, 3);
#undef PW_CODE
  return v;
}

// Sums of 16 rows by 16 columns come with lane l holding row l % 16 and columns
// 4 (l / 16) .. + 3.  Of two such pieces, the second's rows behind the first's,
// exchanged between the sixteens of a wave, a lane holds eight neighbouring
// columns: row l % 32, columns 8 (l / 32) .. + 7.  All lanes have to be active.
__device__ __forceinline__ floatx8 eight_columns(f32x4 first, f32x4 second) {
  floatx8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(first[i]), __float_as_uint(second[i]), false, false);
    v[i] = __uint_as_float(r[0]);
    v[4 + i] = __uint_as_float(r[1]);
  }
  return v;
}

// A wave's sums of 32 rows by 64 columns on their way to rows: they come with a
// lane holding eight columns of one of 32 rows and go on with eight lanes holding
// a row's 64, so that loads and stores take whole lines of 128 bytes (stored as
// they come, 256 x 256 bf16 values a block go out at 3 TB/s).  What they become is
// written once and looped over: unrolled it would be longer than the instruction
// cache.  In LDS, the wave's own; sixteen bytes of row r lie at place c ^ (r & 15).
struct Sums {
  static constexpr int kBytes = 32 * 64 * 4;
  char* at;
  int lane;
  __device__ __forceinline__ Sums(char* lds, int wave, int lane_) : at(lds + wave * kBytes), lane(lane_) {}
  static __device__ __forceinline__ void order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  __device__ __forceinline__ float4* place(int row, int c) const {
    return reinterpret_cast<float4*>(at + row * 256 + ((c ^ (row & 15)) * 16));
  }
  __device__ __forceinline__ void put(const f32x4 (&first)[4], const f32x4 (&second)[4]) {
    order();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const floatx8 v = eight_columns(first[c], second[c]);
      *place(lane & 31, 4 * c + 2 * (lane / 32)) = float4{v[0], v[1], v[2], v[3]};
      *place(lane & 31, 4 * c + 2 * (lane / 32) + 1) = float4{v[4], v[5], v[6], v[7]};
    }
    order();
  }
  // columns 8 c .. 8 c + 7 of a row
  __device__ __forceinline__ floatx8 get(int row, int c) const {
    const float4 a = *place(row, 2 * c), b = *place(row, 2 * c + 1);
    return floatx8{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  }
};

}  // namespace pw
