// Internal interfaces between the C-ABI host layer and the kernel files.
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/pagedweight.h"

namespace pw {

constexpr int kMaxExperts = 256;
constexpr int kMinBits = 3;   // committed bitwidths with a table: 3..8
constexpr int kMaxBits = 8;
constexpr size_t kAlign = 256;

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

constexpr int kMfmaTileM = 512;   // tokens per MFMA tile
constexpr int kMaxRouterTopK = 64; // the router's top-k kernel keeps slot j in lane j
constexpr int kMaxRouterHidden = 16384;   // a multi-layer call's router keeps one token's x in LDS

inline int mtile_bound(int E, int T, int k) {
  const int slots = T * k;
  return (E < slots ? E : slots) + (slots + kMfmaTileM - 1) / kMfmaTileM;
}

constexpr int kMgTileM = 32;      // tokens per matrix-core GEMV pass

// Prefill: the tokens of an MFMA expert past its last whole 512-token tile
// go to the matrix-core GEMV when there are at most this many.  An MFMA tile
// costs the same whatever its token count (the weight decode and the products
// of all its 512 token rows); a 32-token matrix-core GEMV tile of the same
// expert costs about a quarter of it, so up to three such tiles win.
constexpr int kMfmaTailTokens = 96;

inline int mgtile_bound(int E, int T, int k) {
  const int slots = T * k;
  return (E < slots ? E : slots) + (slots + kMgTileM - 1) / kMgTileM;
}

// Parts of the down product's K range given to separate waves when a small
// batch would otherwise leave most of the chip idle.
inline int down_kparts(int H, int I, int E, int k, int T) {
  const int slots = T * k;
  if (slots > 64 || slots <= 0) return 1;
  const int bound = E < slots ? E : slots;
  const int waves = bound * (H / 16);
  const int nsl = (I / 32 + 63) / 64;
  int kp = (2048 + waves - 1) / waves;
  if (kp > nsl) kp = nsl;
  return kp < 1 ? 1 : kp;
}

// Parts of the down product's K range for the MFMA kernels when they run
// alone (prefill): the down product has few row tiles (H / 128), so with
// few token tiles its workgroups would fill the CUs only once or twice and
// the last round would run mostly empty.  Parts double until there are
// enough (token tile, row tile, part) items for two rounds, each part keeping
// at least sixteen quads of eight plane words.  Every part writes its own o
// slice, which the combine reads back: on the Mixtral-shaped prefill (512
// items) one part takes the call 3.48 -> 3.45 ms against the two that a
// four-round target gave (down kernel 1.164 -> 1.155 ms).
constexpr int kNumCUs = 256;
inline int mfma_down_kparts(int H, int I, int E, int k, int T) {
  (void)E;
  const long long slots = (long long)T * k;
  if (slots <= 0) return 1;
  const long long items = (slots + kMfmaTileM - 1) / kMfmaTileM * ((H + 127) / 128);
  const int quads = (I / 32 + 7) / 8;
  int kp = 1;
  while (kp < 4 && items * kp < 2LL * kNumCUs && quads >= 16 * 2 * kp) kp *= 2;
  return kp;
}

// Parts of the down product's K range for the matrix-core GEMV when it runs
// alone: a 32-row chunk of the down block walks all of I, and with few token
// tiles (decode batches: about one per routed expert) there are too few
// (tile, chunk) items to keep the CUs busy.  Parts double until there are
// about 2048 items, each part keeping at least eight super-chunks of eight
// plane words; every part stages the chunk's row tables again and writes its
// own o slice, so more parts cost more than they spread (Mixtral-shaped down
// product at T = 64, 1024 (tile, chunk) items: 177 / 136 / 141 / 156 us with
// 1 / 2 / 4 / 8 parts).
inline int mgemv_down_kparts(int H, int I, int E, int k, int T) {
  const long long slots = (long long)T * k;
  if (slots <= 0) return 1;
  const long long tiles = (E < slots ? E : slots) > (slots + kMgTileM - 1) / kMgTileM
                              ? (E < slots ? E : slots)
                              : (slots + kMgTileM - 1) / kMgTileM;
  const long long items = tiles * ((H + 31) / 32);
  const int supers = (I / 32 + 7) / 8;
  int kp = 1;
  while (kp < 8 && items * kp < 2048 && supers >= 8 * 2 * kp) kp *= 2;
  return kp;
}

// Workspace layout (byte offsets from the workspace base).  The first 256
// bytes are the header: status word, active-expert count.
struct WsLayout {
  size_t status = 0;        // uint32 status bits
  size_t num_active = 4;    // int32 number of experts with at least one slot
  size_t num_mtiles = 8;    // int32 number of MFMA token tiles
  size_t num_mgtiles = 12;  // int32 number of matrix-core GEMV token tiles
  size_t counts = 0;        // int32 [E]    slots per expert
  size_t offsets = 0;       // int32 [E+1]  first sorted position per expert
  size_t active = 0;        // int32 [E]    active expert ids, ascending
  size_t perm = 0;          // int32 [T*k]  sorted position -> slot (t*k + j)
  size_t inv = 0;           // int32 [T*k]  slot -> sorted position, -1 if dropped
  size_t mtiles = 0;        // int32 [2 * mtile_bound] MFMA token tiles
  size_t mgtiles = 0;       // int32 [2 * mgtile_bound] matrix-core GEMV token tiles
  size_t h = 0;             // fp16  [T*k][I] activations between the products
  size_t o = 0;             // fp32  [kparts][T*k][H] expert outputs by slot (t*k + j), before the combine
  size_t xl = 0;            // fp16  [2][T][H] layer inputs of a multi-layer call (ping-pong)
  size_t rids = 0;          // int32 [T*k]    router expert ids (routed forward)
  size_t rw = 0;            // fp32  [T*k]    router weights (routed forward)
  size_t adesc = 0;         // ActiveDesc [E] down-product work descriptors (calls routed inside gate_up)
  size_t total = 0;
};

inline WsLayout ws_layout(int H, int I, int E, int k, int T) {
  WsLayout L;
  size_t off = kAlign;
  const size_t slots = (size_t)T * (size_t)k;
  const int kpg = down_kparts(H, I, E, k, T), kpm = mfma_down_kparts(H, I, E, k, T);
  const int kpv = mgemv_down_kparts(H, I, E, k, T);
  const int kpx = kpg > kpm ? kpg : kpm;
  const size_t kp = (size_t)(kpx > kpv ? kpx : kpv);
  L.counts = off;  off = align_up(off + sizeof(int32_t) * E, kAlign);
  L.offsets = off; off = align_up(off + sizeof(int32_t) * (E + 1), kAlign);
  L.active = off;  off = align_up(off + sizeof(int32_t) * E, kAlign);
  L.perm = off;    off = align_up(off + sizeof(int32_t) * slots, kAlign);
  L.inv = off;     off = align_up(off + sizeof(int32_t) * slots, kAlign);
  L.mtiles = off;  off = align_up(off + sizeof(int32_t) * 2 * mtile_bound(E, T, k), kAlign);
  L.mgtiles = off; off = align_up(off + sizeof(int32_t) * 2 * mgtile_bound(E, T, k), kAlign);
  L.h = off;       off = align_up(off + sizeof(uint16_t) * slots * I, kAlign);
  L.o = off;       off = align_up(off + sizeof(float) * kp * slots * H, kAlign);
  L.xl = off;      off = align_up(off + sizeof(uint16_t) * 2 * (size_t)T * H, kAlign);
  L.rids = off;    off = align_up(off + sizeof(int32_t) * slots, kAlign);
  L.rw = off;      off = align_up(off + sizeof(float) * slots, kAlign);
  L.adesc = off;   off = align_up(off + 32 * (size_t)E, kAlign);
  L.total = off;
  return L;
}

// Pointers into one workspace for one call.
// What a down-product wave needs about the a-th routed expert, in one
// 32-byte record: written by the gate_up kernel that routes a small batch, so
// the down kernel reaches its planes after one dependent load.
struct ActiveDesc {
  int32_t e, n_e, off_e, q;
  const uint32_t* planes;
  const uint16_t* lut_all;
};
static_assert(sizeof(ActiveDesc) == 32, "one record per 32 bytes");

struct Route {
  uint32_t* status;
  int32_t* num_active;
  int32_t* counts;
  int32_t* offsets;
  int32_t* active;
  int32_t* perm;
  int32_t* inv;
  int32_t* mtiles;        // (expert, first sorted position) per MFMA token tile
  int32_t* num_mtiles;
  int32_t* mgtiles;       // (expert, first token) per matrix-core GEMV token tile
  int32_t* num_mgtiles;
  ActiveDesc* adesc;      // [E] down work descriptors by active index (inline routing only)
};


struct ExpertArgs {
  int H, I, E, k, T;
  const pw_block_desc* blocks;
  const uint8_t* q;
  Route rt;
  int min_tokens;   // process experts with min_tokens <= n_e < max_tokens
  int max_tokens;
  int kparts;       // parts of the down product's K range (MFMA kernels running alone)
};

// Everything the GEMV kernels need for one call.
struct GemvLaunch {
  int H, I, E, k, T;
  const pw_block_desc* blocks;
  const uint8_t* q;
  const int32_t* ids;
  Route rt;
  int inline_route;          // T*k <= 64: no route kernel, gate_up waves route by themselves
  int min_tokens, max_tokens;
  const uint16_t* x;
  uint16_t* h;
  float* o;
  int kparts;
};

// Optional start / stop events of one kernel: the library hands them to the
// launch itself, so they carry the timestamps of that kernel's execution
// rather than of the stream around it.  Null members are not recorded.
struct KernelEvents {
  hipEvent_t start = nullptr;
  hipEvent_t stop = nullptr;
};

template <typename F, typename... Args>
inline hipError_t launch_kernel(F kernel, dim3 grid, dim3 block, hipStream_t s, const KernelEvents& ev,
                                Args... args) {
  if (ev.start || ev.stop)
    hipExtLaunchKernelGGL(kernel, grid, block, 0, s, ev.start, ev.stop, 0, args...);
  else
    hipLaunchKernelGGL(kernel, grid, block, 0, s, args...);
  return hipGetLastError();
}

// Launchers (return hipSuccess or the launch error).
// mfma_tail: an MFMA expert's tokens past its last whole 512-token tile, when
// at most this many (0: never), are listed as matrix-core GEMV tiles instead
hipError_t launch_route(const int32_t* ids, int T, int k, int E, int mfma_min_tokens, int mg_min_tokens,
                        int mg_max_tokens, int mfma_tail, const Route& rt, hipStream_t s);
hipError_t launch_gemv_gate_up(const GemvLaunch& g, hipStream_t s, const KernelEvents& ev);
hipError_t launch_gemv_down(const GemvLaunch& g, hipStream_t s, const KernelEvents& ev);
hipError_t launch_mfma_gate_up(const ExpertArgs& a, const uint16_t* x, uint16_t* h, hipStream_t s,
                               const KernelEvents& ev);
hipError_t launch_mfma_down(const ExpertArgs& a, const uint16_t* h, float* o, hipStream_t s, const KernelEvents& ev);
hipError_t launch_mgemv_gate_up(const ExpertArgs& a, const uint16_t* x, uint16_t* h, hipStream_t s,
                                const KernelEvents& ev);
hipError_t launch_mgemv_down(const ExpertArgs& a, const uint16_t* h, float* o, hipStream_t s,
                             const KernelEvents& ev);
hipError_t launch_combine(const float* o, const float* w, const int32_t* inv, int T, int k, int H, int kparts,
                          uint16_t* y, hipStream_t s);
hipError_t launch_dequant(const uint32_t* planes, const uint16_t* lut_all, int N, int K, int q, int module,
                          uint16_t* out, hipStream_t s);
hipError_t launch_pack(const uint32_t* canon, int N, int K, int nplanes, int module, uint32_t* out, hipStream_t s);
hipError_t launch_fill_zero(void* p, size_t bytes, hipStream_t s);
hipError_t launch_router(const uint16_t* x, const uint16_t* wr, int T, int H, int E, int k, int32_t* ids, float* w,
                         uint32_t* count, float* mass, hipStream_t s);
// The previous layer's weighted combine (o, w_prev, inv, kparts as the
// combine kernel takes them) written to x_out, then the router on it.
hipError_t launch_combine_router(const float* o, const float* w_prev, const int32_t* inv, int kparts,
                                 uint16_t* x_out, const uint16_t* wr, int T, int H, int E, int k, int32_t* ids,
                                 float* w, uint32_t* count, float* mass, hipStream_t s);
// residual += x, the norm of it to xn, then the router on xn (fp16).
constexpr int kRouterAloneTokens = 256;   // a workgroup a token up to here
inline bool norm_router_fits(int T, int H) { return T <= kRouterAloneTokens && H <= 8192; }
hipError_t launch_norm_router(const uint16_t* x, uint16_t* residual, const uint16_t* norm_w, float eps, uint16_t* xn,
                              const uint16_t* wr, int T, int H, int E, int k, int32_t* ids, float* w, uint32_t* count,
                              float* mass, hipStream_t s);
hipError_t launch_status_clear(uint32_t* status, hipStream_t s);

// ----- operators around the layer (strides in elements unless said) --------
constexpr int kMaxNormHidden = 32768;   // a block of sixteen waves holds a row, four chunks a lane
constexpr int kNormGroup = 128;         // columns per scale of the 8-bit output
constexpr int kNormGradBlocks = 512;    // most blocks (and shares of the weight's gradient) of the norm's backward pass

struct NormArgs {
  int T, H;
  const void* x;
  int64_t x_stride;
  const void* residual;       // null: none
  int64_t residual_stride;
  void* residual_out;         // null: the sum is not stored
  int64_t residual_out_stride;
  const void* weight;
  float eps;
  void* y;
  int64_t y_stride;
  float* scale;               // e4m3 output: [T][groups]
  int group;                  // 0: one scale a row, kNormGroup: one per 128 columns
};
hipError_t launch_rmsnorm(const NormArgs& a, int dtype, bool e4m3, hipStream_t s);

struct NormGradArgs {
  int T, H;
  const void* dy;
  int64_t dy_stride;
  const void* r;
  int64_t r_stride;
  const void* weight;
  float eps;
  const void* dresidual;      // null: none
  int64_t dresidual_stride;
  void* dx;
  int64_t dx_stride;
  float* part;                // shares of dweight, null: dweight is not wanted
};
// Shares of dweight: one a block, and a block takes at least one row.
inline size_t norm_grad_parts(int T) { return T < kNormGradBlocks ? (size_t)T : (size_t)kNormGradBlocks; }
hipError_t launch_rmsnorm_grad(const NormGradArgs& a, int dtype, float* dweight, hipStream_t s);

// One launch up to here, whose blocks all read every id (5360 slots: 10.3 us
// against 17.4 of two launches; 7584: 16.4 against 14.5).
constexpr int kPermuteSmallSlots = 6144;
// Larger calls count the slots of pieces apart: at most 64 pieces, unless those
// would have more slots than the second number; then a launch of its own sums
// the counts of as many pieces as it takes.
constexpr int kPermutePieces = 64;
constexpr int64_t kPermutePieceSlots = 8192;

struct PermuteArgs {
  int T, k, E;
  const uint8_t* x;
  int64_t row_bytes, x_stride, xs_stride;   // bytes
  uint8_t* xs;
  const float* x_scale;
  float* xs_scale;
  int groups;                 // scales a row, 0: none
  const int32_t* ids;
  int32_t* offsets;
  int32_t* inv;
  int32_t* perm;              // may be null
  uint32_t* status;           // may be null
  int32_t* counts;            // [pieces][E]
  int block_tokens, pieces;
  int64_t piece_tokens;
};
// How a call of more than kPermuteSmallSlots slots is cut: blocks of 4 to 64
// tokens whose slots one wave ranks (64 of them at a time), pieces of whole
// blocks.
struct PermutePlan {
  int block_tokens, pieces;
  int64_t piece_tokens;
  bool scan;
};
inline PermutePlan permute_plan(int64_t T, int k, int E) {
  PermutePlan p;
  int64_t bt = (T + 1023) / 1024;
  const int64_t most = 64 / k > 4 ? 64 / k : 4;
  bt = bt < 4 ? 4 : bt > most ? most : bt;
  const int64_t blocks = (T + bt - 1) / bt;
  // a block reads pieces * E counts and, on average, half a piece's ids: about the least together
  int64_t want = 8;
  while (want < kPermutePieces && want * want * 2 * E < T * k) want *= 2;
  int64_t per_piece = (blocks + want - 1) / want;
  const int64_t limit = kPermutePieceSlots / (bt * k) > 1 ? kPermutePieceSlots / (bt * k) : 1;
  p.scan = per_piece > limit;
  if (p.scan) per_piece = limit;
  p.block_tokens = (int)bt;
  p.piece_tokens = per_piece * bt;
  p.pieces = (int)((blocks + per_piece - 1) / per_piece);
  return p;
}
// Ints of the counts for up to T tokens: no T' <= T has more pieces.
inline size_t permute_count_ints(int64_t T, int k, int E) {
  const int64_t bt = 64 / k > 4 ? 64 / k : 4;
  const int64_t limit = kPermutePieceSlots / (bt * k) > 1 ? kPermutePieceSlots / (bt * k) : 1;
  const int64_t scanned = (T + limit * bt - 1) / (limit * bt);
  return (size_t)((scanned > kPermutePieces ? scanned : kPermutePieces) + 1) * (size_t)E;
}
hipError_t launch_permute(PermuteArgs a, hipStream_t s);

struct UnpermuteArgs {
  int T, H, k;
  const void* rows;
  int64_t rows_stride;
  const int32_t* inv;
  const float* w;             // null: ones
  void* y;
  int64_t y_stride;
};
hipError_t launch_unpermute(const UnpermuteArgs& a, int dtype, hipStream_t s);

struct UnpermuteGradArgs {
  int T, H, k;
  const void* dy;
  int64_t dy_stride;
  const void* rows;
  int64_t rows_stride;
  const int32_t* inv;
  const float* w;             // null: ones
  void* drows;
  int64_t drows_stride;
  float* dw;                  // null: not wanted
};
hipError_t launch_unpermute_grad(const UnpermuteGradArgs& a, int dtype, hipStream_t s);

struct RouterGradArgs {
  int T, H, E, k;
  const uint16_t* x;
  const uint16_t* router_w;
  const int32_t* ids;
  const float* w;
  const float* dw;
  const uint16_t* dx_add;     // null: zero
  uint16_t* dx;
  float* drouter_w;
  float* part;                // [splits][E][H], unless there is one stretch
  int splits;
  int64_t split_slots;
  int shift;                  // log2 of the lanes that share a row (H < 512)
  int cshift;                 // log2 of a block's waves that take different columns
};
// How drouter_w is cut.  A block takes an expert, 512 << cshift columns and one
// stretch of the slots; the stretches' shares are summed apart.
// - Columns: with up to 8192 slots a block's four waves share the rows of 512
//   columns (a few-block call is as long as its longest list: skewed T = 256,
//   E = 60: 9 us against 19), above they take 512 columns each, so that the
//   ids are looked through once for 2048 (T = 16384, E = 256, top-8: 99 us
//   against 214).
// - Stretches: as many as make 4096 blocks (2048: T = 32768, E = 60 with skewed
//   routing 177 us against 146), but of at least 1024 slots (512: 10.6 us
//   against 8.2 at T = 256), and of at least 4 E tokens, since a share is E H fp32
//   values written and read (none: T = 2970, E = 155 37 us against 27).
struct RouterGradPlan {
  int splits;
  int64_t split_slots;
  int shift, cshift;
  size_t bytes;   // workspace
};
inline RouterGradPlan router_grad_plan(int H, int E, int k, int64_t T) {
  RouterGradPlan p;
  const int64_t S = T * k, by_shares = (int64_t)4 * E * k, least = by_shares > 1024 ? by_shares : 1024;
  p.shift = 0;
  while (p.shift < 6 && (8 << p.shift) < H) ++p.shift;
  p.cshift = S <= 8192 ? 0 : 2;
  while (p.cshift > 0 && (512 << p.cshift) / 2 >= H) --p.cshift;
  const int64_t blocks = (int64_t)E * ((H + (512 << p.cshift) - 1) / (512 << p.cshift));          // of one stretch
  const int64_t fill = (4095 + blocks) / blocks;
  p.split_slots = (S + fill - 1) / fill;
  p.split_slots = p.split_slots < least ? least : (p.split_slots + 255) / 256 * 256;
  p.splits = (int)((S + p.split_slots - 1) / p.split_slots);
  // no T' <= T has more stretches than this (its tiles are no wider), so a workspace for T serves them all
  const int64_t by_slots = (S + least - 1) / least;
  p.bytes = align_up(sizeof(float) * (size_t)(by_slots < fill ? by_slots : fill) * E * H + 1, kAlign);
  return p;
}
hipError_t launch_router_grad(const RouterGradArgs& a, hipStream_t s);

// Products of the experts' rows (pw_product.hip, pw_product_few.hip): what each kind reads and writes.
enum { kProductAct, kProductGate, kProductBack, kProductGateGrad };
struct ProductArgs {
  int E, S, N, K;             // columns of the result (gated: of one half), length of the reduction
  const int32_t* offsets;     // null: one expert with all rows
  const void* x;              // [S][K]
  int64_t x_stride;
  const void* w;              // [E][N][K]; gated [E][2N][K]; back [E][K][N]
  int64_t w_expert;           // elements between two experts' matrices
  const void* bias;           // [E][N] or null
  const void* residual;       // [S][N] or null
  int64_t residual_stride;
  void* pre;                  // [S][N] or null; gated, back: dz [S][2N]
  int64_t pre_stride;
  void* y;                    // [S][N]; gated, back: h, or null
  int64_t y_stride;
  int act;
  void* z;                    // gate and up [S][2N]: written by the gated product (or null), read by its way back
  int64_t z_stride;
  float* z_scale;             // [S][2 groups], of 8-bit z
  int groups;
  bool z8;
  float* part;                // product_part_bytes of scratch for tiles that are cut, or null
  int NT;                     // set by the launch: column tiles
};
// Rows of a tile: 256 from a mean of kWideRows rows an expert on, below 128, 64 or
// 32.  Where tiles of 256 would be fewer than a quarter of the CUs, 32 rows and
// the reduction cut are faster (fp16, one expert, us: S 511, N = K = 2048 22 of 36;
// S 256, N = K = 4096 26 of 34; S 128 24 of 28), up to three eighths 128 rows
// (S 1024 47 of 54).  As many blocks run together as have tiles cut into parts,
// whose sums a call needs scratch for.
constexpr int kProdN = 256;      // columns of a tile: two halves of 128
constexpr int kProdK = 64;       // reduction steps that are copied together
constexpr int kWideRows = 160, kMidRows = 56, kNarrowRows = 32;
constexpr int kProdParts = 16;   // most parts of a tile
constexpr unsigned product_blocks(int rows) { return rows <= 64 ? 2 * kNumCUs : kNumCUs; }
// Parts that a tile of the unfilled last round is cut into along its reduction of
// `steps` steps of 64, where `rest` tiles of BM rows are left for `together` blocks
// (1: it is not cut).  The launch that adds the parts takes some 5 us, a part of
// 256 rows 0.1 (256 KB written and read), a step 1.3: the number of parts that
// saves most, fewer where two save the same, in units of 1/2560 us.  In whole
// numbers, since the products and the launch that adds them work it out apart.
constexpr unsigned product_parts(unsigned BM, unsigned rest, unsigned steps, unsigned together) {
  unsigned most = rest ? together / rest : 1, parts = 1;
  if (most > steps / 2) most = steps / 2;
  if (most > kProdParts) most = kProdParts;
  int best = 5 * 2560;
  for (unsigned p = 2; p <= most; ++p) {
    const int saved = 13 * 256 * (int)(steps - (steps + p - 1) / p) - (int)(BM * rest * p);
    if (saved > best) {
      best = saved;
      parts = p;
    }
  }
  return parts;
}
inline int product_mean_rows(int E, int64_t S) {
  return S >= (int64_t)kWideRows * E ? 256 : S > (int64_t)kMidRows * E ? 128 : S > (int64_t)kNarrowRows * E ? 64 : 32;
}
inline int product_rows(int E, int64_t S, int64_t NT) {
  const int rows = product_mean_rows(E, S);
  const int64_t wide = ((S + 255) / 256 + (E > 1 ? (S < E ? S : E) : 0)) * NT;
  return wide < kNumCUs / 4 ? 32 : rows == 256 && wide < kNumCUs * 3 / 8 ? 128 : rows;
}
inline size_t product_part_bytes(int E, int64_t S) {
  // 64 MB, 32, 32 and 16: no fewer rows, and no smaller tiles, have more
  const int rows = product_mean_rows(E, S);
  return (size_t)product_blocks(rows) * rows * 256 * sizeof(float);
}
// Column tiles of a result of N columns (gated: of either half).
inline int product_col_tiles(int kind, int N) {
  const int tile = kind == kProductGate ? kProdN / 2 : kProdN;
  return (N + tile - 1) / tile;
}
// Blocks that cover every tile whatever the offsets: a row tile more per expert
// with rows than the rows fill.
inline int64_t product_row_tiles(bool ragged, int E, int64_t S, int BM) {
  if (!ragged) return (S + BM - 1) / BM;
  const int64_t with_rows = S < E ? S : E;
  return S / BM + with_rows < S ? S / BM + with_rows : S;
}
// Whether tiles may be cut: where that can save what its launch costs, with one
// round or less (the host sees no more than a bound of a ragged call's tiles), or a
// long reduction.
inline bool product_is_cut(bool ragged, int64_t tiles, int64_t steps, int rows) {
  const int64_t most = product_blocks(rows);
  return ragged ? steps >= 40 || (tiles <= most && steps >= 8) : tiles % most && steps >= 6;
}
hipError_t launch_product(const ProductArgs& a, int dtype, int kind, hipStream_t s);
// Few rows take the form without tiles: up to kFewRows an expert on average, or up
// to 64 with matrices so small that a call is as long as its launches.  Against
// tiles (us): one expert, H 2048, I 5632, 8 rows 27 of 43, 32 rows 45 of 46, 64
// rows 59 of 51; H 4096, I 14336, 8 rows 84 of 89, 16 rows 98 of 90; N = K = 1024,
// 64 rows 8 of 16; E 60, H 2048, I 1408, 256 rows 228 of 215; E 8, H 4096, I 14336,
// 128 rows 748 of 487.
constexpr int kFewRows = 2;
constexpr int64_t kFewWork = (int64_t)1 << 30;   // rows times an expert's matrix
inline bool few_rows_for(int E, int64_t S, int64_t matrix) {   // matrix: elements of an expert's
  const int64_t experts = S < E ? S : E;
  return S <= kFewRows * experts || (S <= 64 * experts && S * matrix <= kFewWork);
}
bool few_rows(const ProductArgs& a, int kind);
hipError_t launch_few(const ProductArgs& a, int dtype, int kind, hipStream_t s);

// out[e] = p^T q over the rows of expert e
struct OuterArgs {
  int E, S, M, N;
  const int32_t* offsets;
  const void* p;              // [S][M]
  int64_t p_stride;
  const void* q;              // [S][N]
  int64_t q_stride;
  void* out;                  // [E][M][N]
  float* part;                // outer_part_bytes of scratch
  int MT, NT, parts;          // set by the launch: tiles of rows and of columns, stretches of an expert's rows
};
// Small matrices have fewer tiles than fill the CUs: their experts' rows are cut
// into stretches of 256 or more, whose sums are added by a launch of their own
// (one expert, 1355 rows, 496 x 48 bf16: 55 us in one piece).
inline int64_t outer_small_tiles(int E, int64_t M, int64_t N) { return (int64_t)E * ((M + 127) / 128) * ((N + 127) / 128); }
inline bool outer_is_small(int E, int64_t M, int64_t N) { return (int64_t)E * ((M + 255) / 256) * ((N + 255) / 256) < kNumCUs; }
// Of the others, tiles of 256 x 128, two blocks a CU, take few rows an expert.  The
// two cross at some 64 rows for 60 experts of 2816 x 2048 and between 128 and 256
// for 8 of 14336 x 4096 (bf16, dx and dW, 256 x 128 against 256 x 256, us: E 60, 17
// rows 293 and 307, 64 334 and 334, 128 424 and 412, 239 500 and 493; E 8, 32 rows
// 420 and 444, 128 521 and 538, 256 657 and 655, 512 988 and 979).
inline bool outer_is_short(int E, int64_t S) { return S < 128ll * E; }
inline int outer_parts(int E, int64_t S, int64_t M, int64_t N) {
  if (!outer_is_small(E, M, N)) return 1;
  const int64_t fill = 2 * kNumCUs / outer_small_tiles(E, M, N), by_rows = S / E / 256;
  const int64_t parts = fill < by_rows ? fill : by_rows;
  return parts < 1 ? 1 : parts > 16 ? 16 : (int)parts;
}
inline size_t outer_part_bytes(int E, int64_t S, int64_t M, int64_t N) {
  const int parts = outer_parts(E, S, M, N);
  return parts > 1 ? (size_t)parts * (size_t)outer_small_tiles(E, M, N) * 128 * 128 * sizeof(float) : 0;
}
hipError_t launch_outer(const OuterArgs& a, int dtype, hipStream_t s);

struct DzArgs {
  int E, S, N, act;
  const int32_t* offsets;
  const void* dy;             // [S][N]
  int64_t dy_stride;
  const void* pre;
  int64_t pre_stride;
  void* dz;                   // [S][N] without gaps, or null
  float* part;                // column sums of stretches of rows, or null
  void* dbias;                // [E][N] or null
};
size_t dz_part_floats(int E, int64_t S, int N);
hipError_t launch_dz(const DzArgs& a, int dtype, hipStream_t s);

// The fused layer on a caller-provided scratch area (the workspace, or the
// allocation-free entry point's static array).  `status`, if non-null,
// replaces the status word of the scratch header as the place device errors
// are raised.  Arguments are checked by the caller.
pw_status forward_on(const pw_moe_shape* shape, int32_t T, const uint16_t* x, const int32_t* ids, const float* w,
                     const pw_block_desc* blocks, const uint8_t* q, uint16_t* y, uint8_t* scratch,
                     uint32_t* status, const pw_moe_options* opts, hipStream_t s, bool combine = true);

// Host checks shared by the forward entry points (everything but the scratch).
pw_status check_forward_args(const pw_moe_shape* shape, int32_t T, const uint16_t* x, const int32_t* ids,
                             const float* w, const pw_block_desc* blocks, const uint8_t* q, uint16_t* y,
                             const pw_moe_options* opts);

}  // namespace pw
