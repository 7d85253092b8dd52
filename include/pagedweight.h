/*
 * pagedweight.h -- C ABI of libpagedweight, a fused mixed-precision
 * Mixture-of-Experts expert layer for AMD Instinct MI355X (gfx950).
 *
 * What it computes.  "Technical summary: PagedWeight" (gist.science, paper
 * 2607.16184), Core components 1 (Paged Weight representation): every expert
 * linear block -- (layer, expert, gate_up | down) -- is stored as Any-Precision
 * overlaid bit planes with per-row lookup tables, and a Weight Page Table holds
 * the committed bitwidth q_i of each block.  Core components 3 (second bullet,
 * fused mixed-precision kernel): one fused operation reads the planes and the
 * tables directly and computes each block at its own q_i.  The layer is a routed
 * SwiGLU FFN:
 *     gate, up = rows [0, I) and [I, 2I) of  W_gate_up(e) x_t      (W: [2I][H])
 *     h        = SiLU(gate) * up,  SiLU(z) = z / (1 + exp(-z))
 *     o        = W_down(e) h                                       (W: [H][I])
 *     y_t      = sum_{j < k} w[t][j] * o_{ids[t][j]}(x_t)
 * with W[n][c] = LUT_{q}[n][code_q(n, c)] and code_q the value of the first q
 * planes (plane 0 = most significant bit).
 *
 * Storage of one block with N rows and K columns (K % 32 == 0, N % 16 == 0).
 * Canonical planes (what pw_pack_planes takes): uint32 [8][N][K/32],
 * plane-major; bit j (LSB = 0) of word [p][n][c] is plane p of weight
 * (n, 32c + j).  The forward and pw_dequant_block read the DEVICE layout that
 * pw_pack_planes writes from them:
 *   planes : device layout, pw_planes_bytes(N, K, nplanes) bytes.  Planes stay
 *            outermost and each takes N * K / 8 bytes, so a block committed at
 *            q needs only its first q planes resident (a shorter allocation is
 *            fine).  Inside a plane the words sit in tiles of 16 rows by 16
 *            words, tile-row-major; inside a tile the 16 rows follow each
 *            other, each holding the tile's words (16, or (K/32) mod 16 in the
 *            last column tile).  Rows of a gate_up block are interleaved: tile
 *            t holds gate rows 8t..8t+7, then up rows I+8t..I+8t+7.
 *   lut_all: fp16 bits [504 * N], the per-row tables for b = 3..8 laid one
 *            after another in canonical row order; the table of bitwidth b
 *            starts at element N * (2^b - 8) and is [N][2^b].  Only the table
 *            of q is read.
 *
 * Conventions of every entry point.
 *   - Pointers are DEVICE pointers unless the comment says host.  The caller
 *     owns every device buffer; the library allocates no device memory.  Its
 *     only state is the host-side bookkeeping of pager objects (weight pager
 *     section below); every other entry point is stateless.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *     Calls enqueue work and return; results are ready when the stream reaches
 *     that point.  Inputs (including the q table) must not change before that:
 *     a q write ordered on the stream after a forward never affects it, which
 *     is the "commit only at a safe boundary" rule (Core components 3, first
 *     bullet).
 *   - Host-detectable errors return a negative pw_status before anything is
 *     enqueued.  Device-only errors (expert id outside [0, E), committed
 *     bitwidth outside 3..8) make the offending slot / block contribute zero and
 *     set a bit in the workspace status word, read by pw_get_device_status.
 *   - No C++ exception crosses this interface.
 */
#ifndef PAGEDWEIGHT_H
#define PAGEDWEIGHT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PW_ABI_VERSION 4

typedef int32_t pw_status;
#define PW_OK                     0
#define PW_ERR_INVALID_ARG       -1  /* null pointer, negative size, bad enum  */
#define PW_ERR_UNSUPPORTED_SHAPE -2  /* H, I not multiples of 32, E > 256, k > E,
                                        2*I*H > 2^31 - 1, or T*k > 2^29 - 1      */
#define PW_ERR_BITWIDTH          -3  /* host-side bitwidth outside 3..8        */
#define PW_ERR_WORKSPACE         -4  /* workspace too small                    */
#define PW_ERR_ALIGNMENT         -5  /* pointer not 16-byte aligned            */
#define PW_ERR_HIP               -6  /* a HIP runtime call failed              */
#define PW_ERR_UNSUPPORTED       -7  /* option the library does not support     */
#define PW_ERR_OUT_OF_MEMORY     -8  /* pager: no free arena range large enough */

/* device status bits (pw_get_device_status) */
#define PW_DEV_BAD_EXPERT_ID  0x1u   /* some ids[t][j] outside [0, E)          */
#define PW_DEV_BAD_BITWIDTH   0x2u   /* some routed block has q outside 3..8   */

/* Layer shape: H = hidden size, I = expert intermediate size, E = number of
 * routed experts (1..256), k = experts per token (1..E). */
typedef struct {
  int32_t hidden;
  int32_t inter;
  int32_t num_experts;
  int32_t top_k;
} pw_moe_shape;

/* One Weight Page Table entry: where one block's planes and tables live.
 * The table is device memory [E][2] (index 2e + m, m = 0 gate_up, 1 down),
 * both pointers 16-byte aligned.  Moving a block means rewriting its entry. */
typedef struct {
  const uint32_t* planes;
  const uint16_t* lut_all;
} pw_block_desc;

/* Kernel family for the expert products. */
#define PW_PATH_AUTO  0  /* one family per call by the mean routed slots per
                            routed expert m = T*top_k / min(E, T*top_k): GEMV
                            for m < 1.6, matrix-core GEMV for 1.6 <= m <= 64,
                            MFMA above, where an expert's tokens past its last
                            whole 512-token tile take the matrix-core GEMV when
                            there are at most 96 of them (pw_path_info's
                            mfma_tail).  If either *_min_tokens option is > 0
                            and m >= 1.6, per expert by its token count n
                            instead: GEMV below mgemv_min_tokens (default 1),
                            matrix-core GEMV below mfma_min_tokens (default
                            256), MFMA from there; with m < 1.6 the GEMV still
                            takes every expert below mfma_min_tokens */
#define PW_PATH_GEMV  1  /* every expert on the bit-plane GEMV kernels            */
#define PW_PATH_MFMA  2  /* every expert on the dequant-to-LDS MFMA kernels       */
#define PW_PATH_MGEMV 3  /* every expert on the matrix-core GEMV kernels          */

/* Stage boundaries at which optional events are recorded. */
#define PW_STAGE_ROUTE   0
#define PW_STAGE_GATE_UP 1
#define PW_STAGE_DOWN    2
#define PW_STAGE_COMBINE 3
#define PW_NUM_STAGES    4

/* What the optional events of pw_moe_options record. */
#define PW_EVENTS_STAGES  0  /* stage_events[s] recorded on the stream right
                                before stage s, stage_events[PW_NUM_STAGES]
                                after the last stage (kernel time plus the
                                launch gaps between them)                      */
#define PW_EVENTS_KERNELS 1  /* stage_events[0] / [1]: start / stop of the
                                gate_up product's kernel(s), [2] / [3]: start /
                                stop of the down product's kernel(s), taken by
                                the launches themselves (the kernels' own
                                execution, no launch gap); [4] unused.  A NULL
                                entry is not recorded                          */

typedef struct {
  int32_t path;              /* PW_PATH_*                                     */
  int32_t mfma_min_tokens;   /* AUTO bands: MFMA from this many tokens per
                                expert; <= 0: per-call rule or default 256    */
  /* Optional hipEvent_t handles (as void*), used if stage_events[0] is
   * non-NULL; what they record is set by event_mode. */
  void* stage_events[PW_NUM_STAGES + 1];
  int32_t mgemv_min_tokens;  /* AUTO bands: matrix-core GEMV from this many
                                tokens per expert (below mfma_min_tokens);
                                <= 0: per-call rule or default 1              */
  int32_t event_mode;        /* PW_EVENTS_* (other values: PW_ERR_INVALID_ARG) */
} pw_moe_options;

/* ABI version of the loaded library (PW_ABI_VERSION). */
int32_t pw_abi_version(void);

/* Static, never-NULL text for a status code. */
const char* pw_status_str(pw_status status);

/* Element counts of one block's canonical storage (see the storage format above). */
size_t pw_plane_words(int32_t N, int32_t K);   /* 8 * N * K / 32, 0 if invalid */
size_t pw_lut_elems(int32_t N);                /* 504 * N                      */
size_t pw_lut_offset(int32_t N, int32_t b);    /* N * (2^b - 8)                */

/* Host-only shape check for a forward of T tokens (no device access). */
pw_status pw_check_shape(const pw_moe_shape* shape /* host */, int32_t T);

/* Workspace bytes a forward of up to T_max tokens needs (0 on a bad shape). */
size_t pw_workspace_bytes(const pw_moe_shape* shape /* host */, int32_t T_max);

/* Clear the workspace status word.  Call once on a fresh workspace before its
 * first forward (the status word is otherwise sticky; see
 * pw_get_device_status).  Enqueues one small kernel. */
pw_status pw_workspace_init(void* workspace, size_t workspace_bytes, void* stream);

/* The fused mixed-precision MoE layer (Core components 3, fused kernel).
 *   shape   host; T >= 0 tokens (T == 0 returns PW_OK and enqueues nothing)
 *   x       fp16 [T][H]                         ids  int32 [T][k]
 *   w       fp32 [T][k] routing weights, used as given (no renormalisation)
 *   blocks  device pw_block_desc [E][2]         q    device uint8 [E][2]
 *   y       fp16 [T][H], overwritten (round to nearest even from fp32)
 *   workspace, workspace_bytes: device scratch of at least
 *           pw_workspace_bytes(shape, T) bytes, 256-byte aligned; its first
 *           bytes hold the status word.  Concurrent calls need distinct
 *           workspaces.
 *   opts    host, may be NULL (AUTO path, per-call rule, no events).
 * Accumulation is fp32; h is rounded to fp16 before the down product.
 * Results are deterministic: the same inputs give the same bits. */
pw_status pw_moe_forward(const pw_moe_shape* shape, int32_t T,
                         const uint16_t* x, const int32_t* ids, const float* w,
                         const pw_block_desc* blocks, const uint8_t* q,
                         uint16_t* y, void* workspace, size_t workspace_bytes,
                         const pw_moe_options* opts, void* stream);

/* Allocation-free variant of pw_moe_forward, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation).  Same computation, kernels and results
 * as pw_moe_forward; the scratch the workspace would hold lives in a static
 * device array of PW_NOALLOC_SCRATCH_BYTES per GPU, kept until the process
 * ends.  The call allocates nothing.
 *   shape, T, x, ids, w, blocks, q, y, opts, stream: as for pw_moe_forward
 *   status  device uint32, may be NULL: device errors (PW_DEV_* bits) are OR-ed
 *           into it; the caller clears and reads it.  With NULL they are not
 *           reported.
 * Errors: those of pw_moe_forward; PW_ERR_WORKSPACE if the call needs more
 * than PW_NOALLOC_SCRATCH_BYTES (pw_workspace_bytes(shape, T) bytes);
 * PW_ERR_HIP if the scratch address cannot be found.  All calls on one GPU
 * share its scratch array: calls that overlap in time on one GPU race.  Each
 * call overwrites what it reads, so nothing needs clearing between calls. */
#define PW_NOALLOC_SCRATCH_BYTES (64u << 20)
pw_status pw_moe_forward_noalloc(const pw_moe_shape* shape, int32_t T, const uint16_t* x, const int32_t* ids,
                                 const float* w, const pw_block_desc* blocks, const uint8_t* q, uint16_t* y,
                                 uint32_t* status, const pw_moe_options* opts, void* stream);

/* The kernel families a pw_moe_forward call with this shape, T and options
 * runs (the fused kernel's dispatch between its decode, moderate-batch and
 * prefill forms, Core components 3), without touching the GPU.  Host only;
 * the result does not depend on the routing itself. */
typedef struct {
  int32_t gemv;          /* 1: the bit-plane GEMV kernels run                 */
  int32_t mgemv;         /* 1: the matrix-core GEMV kernels run (for their
                            band, or only for the MFMA experts' tails)        */
  int32_t mfma;          /* 1: the dequant-to-LDS MFMA kernels run            */
  int32_t mgemv_from;    /* experts with at least this many tokens (and below
                            mfma_from, if MFMA runs) take the matrix-core GEMV;
                            0 if it has no band                                */
  int32_t mfma_from;     /* experts with at least this many tokens take MFMA;
                            0 if it does not run                               */
  int32_t inline_route;  /* 1: no separate routing kernel (GEMV alone, at most
                            64 slots: the gate_up kernel routes)               */
  int32_t down_kparts;   /* parts of the K range of the GEMV down product    */
  int32_t launches;      /* kernels the call enqueues (T > 0)                 */
  int32_t mfma_tail;     /* an MFMA expert's tokens past its last whole
                            512-token tile, when at most this many, take the
                            matrix-core GEMV instead (the AUTO rule's prefill
                            form; the kernels of both families run); 0: never */
} pw_path_info;

/*   shape, opts  host, as for pw_moe_forward (opts may be NULL)
 *   info         host, overwritten (all zero for T == 0)
 * Errors: those pw_moe_forward reports for the shape, T and options. */
pw_status pw_moe_path_info(const pw_moe_shape* shape, int32_t T, const pw_moe_options* opts,
                           pw_path_info* info);

/* Bytes of `nplanes` planes (1..8) of an N x K block in the device layout:
 * nplanes * N * K / 8 (0 if N % 16, K % 32 or nplanes is invalid).  The
 * bitplane packing layout of Core components 1 ("Technical summary:
 * PagedWeight": overlaid Any-Precision bit planes with lookup tables). */
size_t pw_planes_bytes(int32_t N, int32_t K, int32_t nplanes);

/* Write planes 0..nplanes-1 of one block in the device layout the kernels read
 * (see the storage format above): a lossless permutation of the words of the
 * canonical planes.  module 0 (gate_up, N = 2I) interleaves gate and up rows
 * per 16-row tile, module 1 (down) keeps the row order.
 *   canon       device uint32 [nplanes][N][K/32] (4-byte aligned), not modified
 *   dev_layout  device, pw_planes_bytes(N, K, nplanes) bytes, 16-byte aligned,
 *               distinct from canon (no in-place packing); overwritten
 * Errors: PW_ERR_INVALID_ARG (null, nplanes outside 1..8, module not 0/1,
 * in place), PW_ERR_UNSUPPORTED_SHAPE (N % 16, K % 32), PW_ERR_ALIGNMENT.
 * Enqueued on `stream`; one kernel. */
pw_status pw_pack_planes(const uint32_t* canon, int32_t N, int32_t K, int32_t nplanes, int32_t module,
                         uint32_t* dev_layout, void* stream);

/* Dequantize one block at bitwidth q (host value, 3..8): w_out fp16 bits
 * [N][K] in canonical row order, = LUT_q[n][code_q(n, c)].  planes in the
 * device layout (pw_pack_planes, same module), at least q planes.  The same
 * device decode the forward uses; bit-exact by definition (a table copy).
 * Core components 1.  Errors as pw_pack_planes, PW_ERR_BITWIDTH for q. */
pw_status pw_dequant_block(const uint32_t* planes, const uint16_t* lut_all,
                           int32_t N, int32_t K, int32_t q, int32_t module,
                           uint16_t* w_out, void* stream);

/* Wait for `stream`, copy the workspace status word to *flags (host), then
 * clear it.  Returns PW_ERR_HIP if the copy or the wait fails. */
pw_status pw_get_device_status(void* workspace, uint32_t* flags /* host */, void* stream);

/* Router and online routing statistics ("Technical summary: PagedWeight",
 * Core components 2, second bullet: each expert's routing mass -- how often it
 * is selected and with what weight -- is tracked online).  The router is the
 * top-k softmax router of a routed MoE layer:
 *     logits[t][e] = sum_h x[t][h] * router_w[e][h]   (fp16 inputs, fp32 sums)
 *     ids[t][0..k)  = the k largest logits, descending; lower id first on ties
 *     w[t][j]       = exp(l_j - l_0) / sum_i exp(l_i - l_0) over the selected
 * and, if stat_count / stat_mass are non-NULL, for every slot
 *     stat_count[ids[t][j]] += 1,  stat_mass[ids[t][j]] += w[t][j]
 * (device uint32 [E] and fp32 [E], accumulated across calls; the caller
 * zeroes them to start a window; mass is an fp32 atomic sum, so its last bits
 * depend on the order the slots arrive in).
 *   x fp16 [T][H], router_w fp16 [E][H] (both 16-byte aligned);
 *   ids int32 [T][k], w fp32 [T][k] outputs; k <= 64 (else
 *   PW_ERR_UNSUPPORTED_SHAPE); workspace as for pw_moe_forward (not used by
 *   the router itself).  T == 0 returns PW_OK and enqueues nothing.  One
 *   launch. */
pw_status pw_router_topk(const pw_moe_shape* shape /* host */, int32_t T, const uint16_t* x,
                         const uint16_t* router_w, int32_t* ids, float* w, uint32_t* stat_count,
                         float* stat_mass, void* workspace, size_t workspace_bytes, void* stream);

/* Router + fused mixed-precision layer in one call: pw_router_topk into the
 * workspace (ids and weights are not returned), then pw_moe_forward on them.
 * Arguments as for those two calls. */
pw_status pw_moe_forward_routed(const pw_moe_shape* shape /* host */, int32_t T, const uint16_t* x,
                                const uint16_t* router_w, const pw_block_desc* blocks, const uint8_t* q,
                                uint16_t* y, uint32_t* stat_count, float* stat_mass, void* workspace,
                                size_t workspace_bytes, const pw_moe_options* opts, void* stream);

/* L chained layers of one decode step: layer l routes its input with its own
 * top-k softmax router (as pw_router_topk), runs the fused mixed-precision
 * layer on its own page table (as pw_moe_forward), and its output is layer
 * l + 1's input; y receives the last layer's output.  "Technical summary:
 * PagedWeight", Core components 3 (the fused kernel, which reduces overhead;
 * committed bitwidths read on the device, so a pager commit between two calls,
 * or two replays of a captured graph of one call, takes effect without new
 * launch arguments) and Core components 2 (routing statistics per layer).
 * Each layer's weighted combine is computed inside the next layer's router
 * kernel, so a layer takes the router and the expert products (three launches
 * for decode batches) and only the last layer launches a combine.  Results are
 * bit-identical to L chained pw_moe_forward_routed calls.
 *   shape        host, the same for every layer; k <= 64, H <= 16384
 *   x            fp16 [T][H], layer 0's input;  y  fp16 [T][H], overwritten
 *   router_w     host array [L] of device fp16 [E][H] router matrices
 *   blocks, q    host arrays [L] of device page tables [E][2] and bitwidths [E][2]
 *   stat_count, stat_mass  device uint32 / fp32 [L][E] or NULL: routing
 *                statistics accumulated per layer, as pw_router_topk
 *   workspace    as for pw_moe_forward with the same T (intermediate layer
 *                inputs live in it)
 *   opts         as for pw_moe_forward; events are not supported
 *                (PW_ERR_UNSUPPORTED)
 * Errors: those of pw_moe_forward and pw_router_topk; PW_ERR_INVALID_ARG for
 * L < 1 or a NULL entry. */
pw_status pw_moe_forward_layers(const pw_moe_shape* shape /* host */, int32_t L, int32_t T, const uint16_t* x,
                                const uint16_t* const* router_w /* host [L] */,
                                const pw_block_desc* const* blocks /* host [L] */,
                                const uint8_t* const* q /* host [L] */, uint16_t* y, uint32_t* stat_count,
                                float* stat_mass, void* workspace, size_t workspace_bytes,
                                const pw_moe_options* opts, void* stream);

/* ------------------------------------------------------------------------
 * Around the layer: the norm in front of it, tokens sorted by expert and back
 * with their weights, and the gradients, of the router too.
 *
 * Rows.  A matrix is T rows of H elements, its rows `*_stride` ELEMENTS apart;
 * elements are of one of the types below.  The first row and the stride are
 * 16-byte aligned (8-byte for the stride of an 8-bit output of the norm), else
 * PW_ERR_ALIGNMENT.  An input's stride may be anything from 0 on, a written
 * matrix's rows must not overlap (else PW_ERR_INVALID_ARG).  A null pointer
 * that the comment does not allow, a negative size or an unknown type is
 * PW_ERR_INVALID_ARG.  Unless a comment says that two arguments may be the
 * same, what a call writes must overlap nothing else that it reads or writes.
 *
 * Sums, means and gradients of weights are fp32; an output is rounded once, to
 * nearest even.  Every call is deterministic (but for the order of stat_mass's
 * sums in pw_moe_forward_block, see pw_router_topk), allocates nothing, can be
 * captured into a graph, and leaves what it does not write as it was.  Inputs
 * that hold NaN or infinities give what the formula gives.  A workspace is
 * 256-byte aligned and needs no initialisation; calls that may overlap in time
 * (two streams, two captured graphs) need workspaces of their own.  A call with
 * a size function of its own here writes over the status word of a workspace
 * that a forward uses too: give it another.  A shape is one that
 * pw_check_shape accepts.
 * ---------------------------------------------------------------------- */
#define PW_F32  0
#define PW_F16  1
#define PW_BF16 2
#define PW_E4M3 3   /* 8 bits: 4 of exponent, 3 of mantissa, largest 448, no infinity */

/* Root-mean-square norm with the residual's addition.
 *     r = x + residual                       (r = x if residual is NULL)
 *     y = r * weight / sqrt(mean_h r_h^2 + eps)
 *   H             a multiple of 8, at most 32768 (else PW_ERR_UNSUPPORTED_SHAPE)
 *   dtype         PW_F32, PW_F16 or PW_BF16: x, residual, residual_out, weight
 *   residual_out  receives r rounded to dtype; may be NULL (r is not stored)
 *                 and must be without residual; may be residual or x itself
 *                 (same pointer and stride).  y is computed from the fp32 sum.
 *   weight        dtype [H]
 *   eps           0 .. 1e30
 *   y_dtype       dtype, or PW_E4M3: then y holds codes and
 *                     y_value = code * scale,
 *                     scale = max(largest |y| of the group / 448, 2^-100),
 *                 scale fp32 [T][groups], groups = 1 for group 0 (one scale a
 *                 row) or ceil(H / 128) for group 128.  A group that holds a
 *                 NaN or an infinity gets the scale NaN and NaN codes.
 *                 Otherwise scale is NULL and group 0.  y may be x itself if
 *                 they have the same type and stride.
 * Range (here and in the gradient): the squares are summed in fp32, so finite
 * values follow the formula up to |r| = 2^56 (7.2e16) at any H, and where
 * mean_h r_h^2 + eps is at least 2^-100 (7.9e-31; every r then, where eps is).
 * Above, a row whose sum of squares is past fp32 gives y = 0; below, the
 * squares lose digits.  fp16 rows are always inside, with eps 0 if one value is
 * not zero.
 * One launch.  T == 0 returns PW_OK and enqueues nothing. */
pw_status pw_rmsnorm(int32_t T, int32_t H, int32_t dtype, const void* x, int64_t x_stride, const void* residual,
                     int64_t residual_stride, void* residual_out, int64_t residual_out_stride, const void* weight,
                     float eps, int32_t y_dtype, void* y, int64_t y_stride, float* scale, int32_t group, void* stream);

/* Workspace of pw_rmsnorm_backward for up to T_max rows (0 on a bad size). */
size_t pw_rmsnorm_backward_workspace_bytes(int32_t T_max, int32_t H);

/* Gradient of pw_rmsnorm (y in dtype).  With s = 1 / sqrt(mean_h r_h^2 + eps):
 *     dx      = s (weight dy - r s^2 mean_h(weight dy r)) + dresidual
 *     dweight = sum over rows of dy r s
 *   dy         dtype [T][H]: gradient of y
 *   r          dtype [T][H]: the forward's residual_out (x without a residual)
 *   dresidual  dtype [T][H] or NULL: gradient that reaches r by the residual
 *              stream
 *   dx         dtype [T][H], overwritten: the gradient of x and of residual;
 *              may be dy, r or dresidual itself (same pointer and stride)
 *   dweight    fp32 [H], 16-byte aligned, overwritten (zero for T == 0); NULL:
 *              not wanted, and then no workspace is
 * Two launches (one without dweight). */
pw_status pw_rmsnorm_backward(int32_t T, int32_t H, int32_t dtype, const void* dy, int64_t dy_stride, const void* r,
                              int64_t r_stride, const void* weight, float eps, const void* dresidual,
                              int64_t dresidual_stride, void* dx, int64_t dx_stride, float* dweight, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Workspace of pw_moe_permute for up to T_max tokens (0 on a bad shape). */
size_t pw_moe_permute_workspace_bytes(const pw_moe_shape* shape /* host */, int32_t T_max);

/* Tokens sorted by expert: slot s = t*k + j gets a place inv[s], the slots of
 * expert 0 first, then those of expert 1, ..., each expert's in slot order, and
 *     xs[inv[t*k + j]] = x[t]
 * for callers that run products of their own on an expert's tokens, send them
 * to other GPUs or collect them to measure a block's sensitivity.
 *   shape    host; hidden, num_experts and top_k are used
 *   dtype    PW_F32, PW_F16, PW_BF16 or PW_E4M3: x [T][H] and xs [T*k][H]
 *   x_scale  fp32 [T][groups], moved along to xs_scale fp32 [T*k][groups];
 *            both NULL with groups 0
 *   ids      int32 [T][k].  An id outside [0, E) drops its slot: inv -1,
 *            nothing is written for it (and PW_DEV_BAD_EXPERT_ID is raised in
 *            status).  A token may list an expert more than once.
 *   offsets  int32 [E+1]: expert e has the rows [offsets[e], offsets[e+1]);
 *            rows from offsets[E] on are left as they were
 *   inv      int32 [T*k];  perm  int32 [T*k] or NULL: perm[inv[s]] = s, from
 *            offsets[E] on left as it was
 *   status   device uint32 or NULL: PW_DEV_* bits are OR-ed into it
 * One launch for up to 6144 slots, two above, three from some hundred thousand
 * on.  T == 0 sets offsets to zero. */
pw_status pw_moe_permute(const pw_moe_shape* shape /* host */, int32_t T, int32_t dtype, const void* x,
                         int64_t x_stride, const float* x_scale, int32_t groups, const int32_t* ids, void* xs,
                         int64_t xs_stride, float* xs_scale, int32_t* offsets, int32_t* inv, int32_t* perm,
                         uint32_t* status, void* workspace, size_t workspace_bytes, void* stream);

/* Gradient of pw_moe_permute: dx[t] = sum_j dxs[inv[t*k + j]] (dropped slots
 * add nothing).  dtype PW_F32, PW_F16 or PW_BF16.  One launch. */
pw_status pw_moe_permute_backward(const pw_moe_shape* shape /* host */, int32_t T, int32_t dtype, const void* dxs,
                                  int64_t dxs_stride, const int32_t* inv, void* dx, int64_t dx_stride, void* stream);

/* Back from the experts: y[t] = sum_j w[t][j] rows[inv[t*k + j]], summed in the
 * order of j; zero for a token without a kept slot.
 *   dtype  PW_F32, PW_F16 or PW_BF16: rows [T*k][H], y [T][H]
 *   inv    as pw_moe_permute wrote it; an entry outside [0, T*k) is a dropped slot
 *   w      fp32 [T][k], used as given; NULL: ones
 * One launch; T == 0 returns PW_OK and enqueues nothing. */
pw_status pw_moe_unpermute(const pw_moe_shape* shape /* host */, int32_t T, int32_t dtype, const void* rows,
                           int64_t rows_stride, const int32_t* inv, const float* w, void* y, int64_t y_stride,
                           void* stream);

/* Gradient of pw_moe_unpermute:
 *     drows[inv[t*k + j]] = w[t][j] dy[t],   dw[t][j] = <dy[t], rows[inv[t*k + j]]>
 *   dw    fp32 [T][k], zero for dropped slots; NULL: not wanted (rows may be
 *         NULL then)
 *   drows may be rows itself (same pointer and stride); no two slots may share
 *         a place
 * One launch. */
pw_status pw_moe_unpermute_backward(const pw_moe_shape* shape /* host */, int32_t T, int32_t dtype, const void* dy,
                                    int64_t dy_stride, const void* rows, int64_t rows_stride, const int32_t* inv,
                                    const float* w, void* drows, int64_t drows_stride, float* dw, void* stream);

/* Workspace of pw_router_backward for up to T_max tokens (0 on a bad shape). */
size_t pw_router_backward_workspace_bytes(const pw_moe_shape* shape /* host */, int32_t T_max);

/* Gradient of pw_router_topk with the selection held fixed: w[t] is the
 * softmax of token t's selected logits, so
 *     dl[t][j]      = w[t][j] (dw[t][j] - sum_i w[t][i] dw[t][i])
 *     dx[t]         = dx_add[t] + sum_j dl[t][j] router_w[ids[t][j]]
 *     drouter_w[e]  = sum over the slots of expert e of dl[t][j] x[t]
 *   x, router_w, ids, w  as pw_router_topk took and wrote them (k <= 64).  A
 *              slot whose id is outside [0, E) takes no part, in the inner sum
 *              either: the gradient for weights that are a softmax over the
 *              kept slots, or of a token without any.  Where slots were masked
 *              after the router (an expert's capacity, another rank's experts)
 *              and the others kept their weights, pass the router's own ids
 *              here, with dw 0 (which pw_moe_unpermute_backward writes for a
 *              dropped slot) or the other rank's dw
 *   dw         fp32 [T][k]: gradient of w (as pw_moe_unpermute_backward writes)
 *   dx_add     fp16 [T][H] or NULL: gradient that reaches x by other ways (as
 *              pw_moe_permute_backward writes)
 *   dx         fp16 [T][H], overwritten; may be dx_add itself
 *   drouter_w  fp32 [E][H], 16-byte aligned, overwritten (zero for T == 0)
 * Two launches (one for up to max(1024, 4 E k) slots). */
pw_status pw_router_backward(const pw_moe_shape* shape /* host */, int32_t T, const uint16_t* x,
                             const uint16_t* router_w, const int32_t* ids, const float* w, const float* dw,
                             const uint16_t* dx_add, uint16_t* dx, float* drouter_w, void* workspace,
                             size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Expert products in 16 bits: what stands between pw_moe_permute and
 * pw_moe_unpermute where the experts' matrices are fp16 or bf16 ones (experts
 * that are trained or calibrated, a shared expert, projections), and the
 * gradients.  Rows, strides, alignment, overlap, determinism, graphs and
 * workspaces are as stated above; dtype is PW_F16 or PW_BF16 and holds for
 * every matrix, bias and gradient of a call but where a type is named.
 *
 *   S, offsets  S rows, of which expert e has [offsets[e], offsets[e+1])
 *               (device int32 [E+1], as pw_moe_permute wrote them; entries
 *               outside [0, S] count as the nearer end).  Rows from offsets[E]
 *               on are not read and stay as they were in every output.  NULL:
 *               one expert (E = 1) with all S rows.
 *   Matrices and biases of the experts follow each other without gaps, 16-byte
 *   aligned.  E is 1..256, sizes of rows are as each call says, and a row
 *   stride is below 2^22 elements, of a single row at most that (else
 *   PW_ERR_UNSUPPORTED_SHAPE).
 *
 * Sums are fp32; an output is rounded once.  Between two products of one call
 * (h, and gradients of gate and up or of the product's sum) values are rounded
 * to dtype, as the matrix cores take them, and past the type's largest value
 * (fp16: 65504) they are infinities there, whatever the sum that follows would
 * have made of them.
 *
 * Activations: act(z) = z, z / (1 + exp(-z)), or z Phi(z) with the normal
 * distribution function Phi(z) = erfc(-z / sqrt 2) / 2; values of act and of its
 * slope smaller than 2^-119 may come as zero.
 * ---------------------------------------------------------------------- */
#define PW_ACT_NONE 0
#define PW_ACT_SILU 1
#define PW_ACT_GELU 2

/* Workspace of pw_moe_product and of pw_moe_product_backward for up to S_max
 * rows (0 on a bad size).  From some rows on it holds 16 to 64 MB, whatever their
 * number, for the sums of products that are cut along their reduction. */
size_t pw_moe_product_workspace_bytes(int32_t E, int32_t S_max, int32_t N, int32_t K);
size_t pw_moe_product_backward_workspace_bytes(int32_t E, int32_t S_max, int32_t N, int32_t K);

/* Product with bias, activation and residual:
 *     z[s] = w[e] x[s] + bias[e],   y[s] = act(z[s]) + residual[s]
 *   S         at most 2^31 - 256, here and in the gradient
 *   N, K      multiples of 8, at most 2^22, N K at most 2^30
 *   x         [S][K];  w  [E][N][K];  bias  [E][N] or NULL
 *   act       PW_ACT_*
 *   residual  [S][N] or NULL; may be y itself (same pointer and stride)
 *   pre       [S][N] or NULL: receives z for the gradient
 *   y         [S][N], overwritten
 * One or two launches.  S == 0 returns PW_OK and enqueues nothing. */
pw_status pw_moe_product(int32_t E, int32_t S, int32_t N, int32_t K, int32_t dtype, const void* x, int64_t x_stride,
                         const int32_t* offsets, const void* w, const void* bias, int32_t act, const void* residual,
                         int64_t residual_stride, void* pre, int64_t pre_stride, void* y, int64_t y_stride,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Gradient of pw_moe_product (the residual's is dy itself):
 *     dz = dy act'(pre),  dx = dz w[e],  dw[e] = sum_s dz[s] x[s]^T,  dbias[e] = sum_s dz[s]
 *   dy     [S][N];  pre  [S][N] as the forward wrote it, NULL with PW_ACT_NONE
 *   dx     [S][K] or NULL: not wanted (w may be NULL then)
 *   dw     [E][N][K], zero for an expert without rows, or NULL: not wanted (x
 *          may be NULL then)
 *   dbias  [E][N], the same, or NULL
 * Up to six launches.  S == 0 sets dw and dbias to zero. */
pw_status pw_moe_product_backward(int32_t E, int32_t S, int32_t N, int32_t K, int32_t dtype, const void* dy,
                                  int64_t dy_stride, const void* x, int64_t x_stride, const int32_t* offsets,
                                  const void* w, int32_t act, const void* pre, int64_t pre_stride, void* dx,
                                  int64_t dx_stride, void* dw, void* dbias, void* workspace, size_t workspace_bytes,
                                  void* stream);

/* Workspace of pw_moe_ffn and of pw_moe_ffn_backward for up to S_max rows (0 on
 * a bad shape). */
size_t pw_moe_ffn_workspace_bytes(const pw_moe_shape* shape /* host */, int32_t S_max);
size_t pw_moe_ffn_backward_workspace_bytes(const pw_moe_shape* shape /* host */, int32_t S_max);

/* Gated feed-forward block of every expert over its rows:
 *     [gate | up] = w_gate_up[e] x[s],   h = act(gate) * up,   y[s] = w_down[e] h
 * (the expert product of pw_moe_forward with matrices of 16 bits and without
 * the routing weights, which pw_moe_unpermute applies).
 *   shape      host; hidden H, inter I and num_experts are used; H at most 2^22,
 *              I at most 2^21
 *   x          [S][H];  w_gate_up  [E][2I][H], gate rows first;  w_down  [E][H][I]
 *   act        PW_ACT_SILU or PW_ACT_GELU
 *   z          NULL, or the gradient's checkpoint [S][2I]: gate and up in
 *              z_dtype, which is dtype or PW_E4M3 (8 bits; the row stride and
 *              the first row are then 16-byte aligned too).  In 8 bits
 *                  value = code * scale,
 *                  scale = max(largest |value| of the group / 448, 2^-100),
 *              a group being 128 columns of gate or of up (the last of each
 *              may have fewer), and
 *   z_scale    fp32 [S][2 G], G = ceil(I / 128): the scales of gate's groups,
 *              then those of up's.  A group with a NaN or an infinity gets the
 *              scale NaN and NaN codes.  NULL otherwise.
 *              y comes from the unrounded gate and up in either case.
 *   y          [S][H], overwritten
 * Two to four launches.  S == 0 returns PW_OK and enqueues nothing. */
pw_status pw_moe_ffn(const pw_moe_shape* shape /* host */, int32_t S, int32_t dtype, const void* x, int64_t x_stride,
                     const int32_t* offsets, const void* w_gate_up, const void* w_down, int32_t act, int32_t z_dtype,
                     void* z, int64_t z_stride, float* z_scale, void* y, int64_t y_stride, void* workspace,
                     size_t workspace_bytes, void* stream);

/* Gradient of pw_moe_ffn, from the checkpoint z (its values, where it is 8-bit):
 *     dh = w_down[e]^T dy,   dgate = dh up act'(gate),   dup = dh act(gate)
 *     dx = w_gate_up[e]^T [dgate | dup]
 *     dw_gate_up[e] = sum_s [dgate | dup][s] x[s]^T,   dw_down[e] = sum_s dy[s] h[s]^T
 *   dx         [S][H] or NULL: not wanted
 *   dw_gate_up [E][2I][H], zero for an expert without rows, or NULL: not wanted
 *              (x may be NULL then)
 *   dw_down    [E][H][I], the same, or NULL
 *   w_gate_up  may be NULL without dx
 * Up to eight launches.  S == 0 sets dw_gate_up and dw_down to zero. */
pw_status pw_moe_ffn_backward(const pw_moe_shape* shape /* host */, int32_t S, int32_t dtype, const void* dy,
                              int64_t dy_stride, const void* x, int64_t x_stride, const int32_t* offsets,
                              const void* w_gate_up, const void* w_down, int32_t act, int32_t z_dtype, const void* z,
                              int64_t z_stride, const float* z_scale, void* dx, int64_t dx_stride, void* dw_gate_up,
                              void* dw_down, void* workspace, size_t workspace_bytes, void* stream);

/* The routed half of a transformer block: norm, router and layer in one call,
 *     residual += x;   y = layer(pw_rmsnorm(residual))
 * The next norm's residual addition adds y.  Equal bit for bit to pw_rmsnorm
 * (fp16, in place on residual) followed by pw_moe_forward_routed on its output;
 * the norm and the router are one launch for up to 256 tokens of H <= 8192.
 *   x         fp16 [T][H];  residual  fp16 [T][H], updated;  norm_w  fp16 [H]
 *   y         fp16 [T][H], overwritten; may be x
 *   the rest  as for pw_rmsnorm and pw_moe_forward_routed */
pw_status pw_moe_forward_block(const pw_moe_shape* shape /* host */, int32_t T, const uint16_t* x, uint16_t* residual,
                               const uint16_t* norm_w, float eps, const uint16_t* router_w,
                               const pw_block_desc* blocks, const uint8_t* q, uint16_t* y, uint32_t* stat_count,
                               float* stat_mass, void* workspace, size_t workspace_bytes, const pw_moe_options* opts,
                               void* stream);

/* ------------------------------------------------------------------------
 * Quality-aware bitwidth planner (host code; "Technical summary: PagedWeight",
 * Core components 2: offline sensitivity per block, online routing statistics
 * with hot experts protected by higher floors and damage multipliers, a
 * prompt-specific correction, and a greedy choice of the reductions with the
 * least damage per byte saved until a memory target is met).
 *
 *   D_b(q) = mu_b * (S_b(q) + R_b(q))   damage of block b at bitwidth q
 *   mu_b   = hot_multiplier for blocks of hot experts, else 1
 *   hot    = the ceil(hot_fraction * E) experts with the largest positive
 *            routing mass (equal masses: lower expert id)
 *   floor  = floor_hot for blocks of hot experts, else floor_cold; a block
 *            below its floor is raised to it first
 * If the resident plane bytes sum_b q_b * plane_bytes[b] exceed the budget,
 * one-bit reductions are taken in increasing (D_b(q-1) - D_b(q)) /
 * plane_bytes[b] (equal: lower b) until they fit or every block sits on its
 * floor.  Otherwise one-bit restorations are taken in decreasing
 * (D_b(q) - D_b(q+1)) / plane_bytes[b] (equal: lower b) among the steps that
 * still fit, up to 8 bits.  Costs are evaluated in fp64 exactly as written.
 * The result feeds pw_pager_request.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t num_blocks;          /* B                                                  */
  int32_t num_experts;         /* E                                                  */
  const int32_t* expert_of;    /* host [B]: expert of block b, in [0, E)             */
  const int64_t* plane_bytes;  /* host [B]: bytes of one bit plane of block b (> 0)  */
  const float* sensitivity;    /* host [B][6]: offline score S_b(q), column q - 3    */
  const float* correction;     /* host [B][6]: prompt correction R_b(q); NULL = 0    */
  const float* routing_mass;   /* host [E]; NULL = no expert is hot                  */
  double hot_fraction;
  int32_t floor_cold;          /* 3..8 */
  int32_t floor_hot;           /* 3..8 */
  float hot_multiplier;
  int32_t reserved;
} pw_plan_problem;

/* Plan bitwidths for a plane-byte budget.  q_cur (host [B], 3..8): current
 * desired bitwidths; q_out (host [B]) receives the plan; *plane_bytes_out
 * (may be NULL) the resident plane bytes of the plan; *fits (may be NULL) 1 if
 * they fit the budget, 0 if the floors alone exceed it (the plan then holds
 * every block at its floor).  Pure host computation; no device access. */
pw_status pw_plan_bitwidths(const pw_plan_problem* problem /* host */, const int32_t* q_cur /* host */,
                            int64_t budget_bytes, int32_t* q_out /* host */, int64_t* plane_bytes_out /* host */,
                            int32_t* fits /* host */);

/* ------------------------------------------------------------------------
 * Weight pager: the Weight Page Table kept on the host, asynchronous page
 * movement and safe-boundary commits ("Technical summary: PagedWeight",
 * Core components 1, third bullet: desired bitwidth d_i, committed bitwidth
 * q_i, pages GPU-resident, CPU-resident or in transfer; Core components 3,
 * first bullet: pages offloaded to CPU memory and reloaded asynchronously,
 * bitwidth commits only at safe boundaries).
 *
 * A page is one bit plane of one block.  The host holds all eight planes of
 * every block in pinned memory (caller-owned, never written by the library);
 * the GPU holds planes 0..q-1 of each block as one extent of a caller-owned
 * device arena.  The pager owns the device page table the forward reads
 * (`blocks` [B] and `q` [B], caller-allocated device memory, q zeroed by the
 * caller before the first commit; for a layer B = 2E and block 2e + m).
 *
 * Use:  pw_pager_request(b, d) for the blocks of a plan (host only), then
 * pw_pager_execute(copy_stream) enqueues the page movement (host-to-device
 * copies of planes the GPU lacks, device-to-device moves when an extent cannot
 * grow in place), then pw_pager_commit(stream) at a safe boundary (between
 * forwards on `stream`) enqueues one kernel that rewrites the page-table
 * entries and q bytes of every staged block together.  Forwards enqueued on
 * `stream` before the commit use the old bitwidths and storage, forwards after
 * it the new ones.  Every forward that reads the page table must run on the
 * commit stream or be ordered with it.  Arena ranges that a commit frees (a
 * lowered block's plane suffix, a moved block's old extent) are reused only
 * after `stream` has passed the commit.  The pager object is host state
 * (malloc'd bookkeeping, HIP events); it allocates no device memory.  One
 * pager is not thread-safe: calls on it must not overlap.
 * ---------------------------------------------------------------------- */
typedef struct pw_pager pw_pager;

#define PW_PAGE_CPU          0   /* no plane of the block on the GPU           */
#define PW_PAGE_GPU          1   /* planes 0..committed-1 on the GPU           */
#define PW_PAGE_IN_TRANSFER  2   /* planes for a staged increase still copying */

typedef struct {
  int32_t desired;        /* d_i (0 = never requested)                          */
  int32_t committed;      /* q_i in the device page table (0 = not committed)   */
  int32_t resident;       /* planes of the committed extent on the GPU          */
  int32_t pending;        /* bitwidth staged for the next commit, 0 if none     */
  int32_t state;          /* PW_PAGE_*                                          */
  int32_t reserved;
  uint64_t arena_offset;  /* byte offset of the committed extent, UINT64_MAX if none */
} pw_page_info;

/* Create a pager for `num_blocks` blocks of rows[b] x cols[b] weights (host
 * arrays; cols % 32 == 0).  `arena` (device, 256-byte aligned, arena_bytes
 * long) is where resident planes live.  *out receives the handle. */
pw_status pw_pager_create(int32_t num_blocks, const int32_t* rows /* host */, const int32_t* cols /* host */,
                          void* arena, size_t arena_bytes, pw_block_desc* blocks, uint8_t* q,
                          pw_pager** out /* host */);

/* Wait for the pager's outstanding copies and commits, then free it. */
pw_status pw_pager_destroy(pw_pager* pager);

/* Register block b's storage before its first commit: host_planes is pinned
 * host memory holding all 8 planes in the device layout (pw_pack_planes of the
 * block's module, pw_planes_bytes(N, K, 8) bytes; plane p starts at byte
 * p * N * K / 8, which is what the pager copies); lut_all is the device table
 * block [504 N] (fp16 bits, 16-byte aligned), which stays resident. */
pw_status pw_pager_set_block(pw_pager* pager, int32_t b, const uint32_t* host_planes /* pinned host */,
                             const uint16_t* lut_all);

/* Set the desired bitwidth d_i (3..8) of block b.  Host bookkeeping only. */
pw_status pw_pager_request(pw_pager* pager, int32_t b, int32_t desired);

/* Stage every block whose desired bitwidth differs from its committed one:
 * enqueue on copy_stream the copies of the planes it lacks.  Blocks staged
 * earlier and not yet committed are left alone.  PW_ERR_OUT_OF_MEMORY when the
 * arena has no room, PW_ERR_HIP when a copy cannot be enqueued: the blocks
 * staged before that stay staged, the rest keep their committed state
 * (commit lowered blocks first to free their planes). */
pw_status pw_pager_execute(pw_pager* pager, void* copy_stream);

/* Safe boundary: commit every staged block in one step.  If copies are still
 * in flight: with wait == 0 nothing is committed (*committed = 0); with
 * wait != 0 `stream` is made to wait for them on the device (the host does not
 * block).  *committed (host, may be NULL) receives the number of blocks whose
 * entries the enqueued commit rewrites. */
pw_status pw_pager_commit(pw_pager* pager, void* stream, int32_t wait, int32_t* committed /* host */);

/* Host view of block b's page-table entry. */
pw_status pw_pager_info(const pw_pager* pager, int32_t b, pw_page_info* info /* host */);

/* Arena bytes held by extents, including ranges freed by a commit that the
 * compute stream has not passed yet (as of the last execute/commit call). */
size_t pw_pager_arena_used(const pw_pager* pager);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDWEIGHT_H */
