/*
 * flashmask.h: C ABI of the column-wise-masked exact attention library
 * (libflashmask.so, sm_103a).
 *
 * What it computes ("FlashMask: Efficient and Rich Mask Extension of
 * FlashAttention", abstract; "FlashMask-3: ... Mask-Aware Distributed
 * Attention", abstract): exact scaled-dot-product attention, forward and
 * backward, under a mask stored column-wise as four int32 query-axis boundary
 * vectors per key column. For key column j, query row i is MASKED when
 *
 *     (causal && j > i) || (LTS[j] <= i < LTE[j]) || (UTS[j] <= i < UTE[j])
 *
 * Intervals are half-open; an interval whose start >= end masks nothing, and
 * bounds outside [0, N] act as if clamped to [0, N]. Over visible entries:
 *
 *     S = scale * Q K^T,  P = softmax_rows(S),  O = P V,  LSE = rowwise ln sum exp(S)
 *
 * A query row with no visible key gets O = 0 and LSE = -inf; it contributes
 * nothing to any gradient. The backward returns dQ, dK, dV for an upstream
 * gradient dO (the FlashAttention recomputation scheme: P is rebuilt from Q, K
 * and LSE; D = rowsum(dO * O)).
 *
 * Layouts (all row-major, contiguous, device memory owned by the caller):
 *   Q, K, V, O, dO, dQ, dK, dV : bf16  [B, H, N, d]
 *   LSE                        : fp32  [B, H, N]     (natural log)
 *   LTS, LTE, UTS, UTE         : int32 [B, Hm, N]    (head h reads mask head h / (H / Hm))
 * Supported shapes: d in {64, 128}; 1 <= N <= FM_MAX_SEQLEN (the last 128-row
 * block of a sequence whose length is not a multiple of 128 is short; its
 * missing rows and keys take no part); H % Hm == 0; B * H * Npad < 2^31 with
 * Npad = N rounded up to a multiple of 128. Other shapes return
 * FM_ERR_UNSUPPORTED.
 *
 * Workspace: the library never allocates. The caller passes one device buffer
 * of at least flashmask_workspace_bytes(...) bytes, aligned to 256 bytes. It
 * holds the tile classification (written by flashmask_classify), the backward's
 * fp32 scratch and a device status word. One workspace must not be used by two
 * calls that may run at the same time.
 *
 * The status word (the first 16 bytes of the workspace) must be zero before
 * the workspace is first passed to a call that launches kernels: allocate the
 * workspace zeroed (cudaMemset, torch.zeros) or call flashmask_check_status()
 * on it once, which reads the word and clears it. The calls themselves do not
 * clear it (a failure recorded by one call stays visible until it is checked),
 * and a kernel that finds it nonzero gives up every wait that is not already
 * satisfied, leaving its outputs undefined; flashmask_check_status() then
 * reports FM_ERR_TIMEOUT.
 *
 * Streams and errors: every call validates its arguments on the host and
 * returns an error WITHOUT launching anything if they are bad. Otherwise it
 * enqueues kernels on `stream` (a cudaStream_t, NULL for the legacy default
 * stream) and returns FM_OK without synchronising. Every wait inside a kernel
 * is bounded in time; a kernel whose wait gives up records the failure in the
 * workspace status word and exits. flashmask_check_status() reads and clears
 * that word.
 */
#ifndef FLASHMASK_H
#define FLASHMASK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FM_OK = 0,
  FM_ERR_INVALID_ARG = 1,  /* null pointer, negative size, scale not finite, ...   */
  FM_ERR_UNSUPPORTED = 2,  /* d not in {64,128}, N < 1, H % Hm != 0, ...           */
  FM_ERR_CUDA = 3,         /* a CUDA runtime call or kernel launch failed          */
  FM_ERR_TIMEOUT = 4,      /* a kernel wait gave up (see flashmask_check_status)   */
  FM_ERR_WORKSPACE = 5,    /* workspace null, misaligned or smaller than required  */
  FM_ERR_PAGE = 6          /* a page table entry, length or start on the device was
                              out of range (see flashmask_check_status)            */
} fm_status;

/* Tile edge (rows and columns) of the classification. */
#define FM_TILE 128

/* Longest supported sequence (2^21 tokens, 16384 blocks of 128). */
#define FM_MAX_SEQLEN 2097152

/* Three-way tile label ("FlashMask" abstract: skip the computation that the
 * mask makes unnecessary). */
#define FM_TILE_NONE 0    /* no entry of the tile is masked: no mask work        */
#define FM_TILE_PARTIAL 1 /* some entries masked: mask applied element by element */
#define FM_TILE_FULL 2    /* every entry masked: the tile is skipped             */

/* The column-wise mask: device pointers to int32 [B, Hm, N] vectors.
 * uts and ute may both be NULL (no upper interval). */
typedef struct {
  const int32_t* lts;
  const int32_t* lte;
  const int32_t* uts;
  const int32_t* ute;
  int Hm;     /* number of mask heads, 1 <= Hm <= H, H % Hm == 0 */
  int causal; /* nonzero: also mask j > i                         */
} fm_mask;

/* Byte offsets of the workspace regions (from the workspace base), for callers
 * that want to read the classification. Regions marked [bwd] exist only when
 * the workspace was sized with for_bwd != 0 (otherwise their offsets are 0).
 *   status    int32[4]                   device status word (0 = OK; must be zero
 *                                        before first use, see above), detail, the
 *                                        forward's work-item counter (reset by each
 *                                        call) and the dQ-zeroed tag (see flashmask_fwd)
 *   minmax    int32  [B,Hm,Tc,8]         per key block: min/max of LTS, LTE, UTS, UTE
 *   labels    uint8  [B,Hm,Tr,Tc]        tile label, query-block major
 *   labels_t  uint8  [B,Hm,Tc,Tr]        tile label, key-block major
 *   row_count int32  [B,Hm,Tr]           non-FULL tiles per query block
 *   row_list  int32  [B,Hm,Tr,Tc]        (key block << 2) | label, ascending
 *   row_order int32  [B,Hm,Tr]           query blocks by descending row_count
 *   col_count int32  [B,Hm,Tc]           non-FULL tiles per key block
 *   col_list  int32  [B,Hm,Tc,Tr]        (query block << 2) | label, ascending
 *   col_order int32  [B,Hm,Tc]           key blocks by descending col_count
 *   lse2      fp32   [B,H,Npad]   [bwd]  LSE * log2(e) (+inf for a fully masked
 *                                       row and for the padding rows n >= N)
 *   delta     fp32   [B,H,Npad]   [bwd]  rowsum(dO * O) (0 on padding rows)
 *   dq_accum  fp32   [B,H,Npad,d] [bwd]  dQ accumulator
 *   kv_part   fp32   [B,H,E,3,2,128,d] [bwd] dV, dK of the parts of a split key
 *                                        block that finish first (see flashmask_bwd)
 *   kv_sync   int32  [B,H,E,8]    [bwd]  arrivals and ready flags per split block
 * with Tr = Tc = ceil(N / 128), Npad = 128 * Tr and E = min(Tc, 16). */
typedef struct {
  size_t status, minmax, labels, labels_t, row_count, row_list, row_order, col_count, col_list,
      col_order, lse2, delta, dq_accum, kv_part, kv_sync, total;
} fm_ws_layout;

/* Workspace size in bytes for the given problem; 0 for an unsupported shape. */
size_t flashmask_workspace_bytes(int B, int H, int Hm, int N, int d, int for_bwd);

/* Fills *out with the region offsets described above. */
fm_status flashmask_workspace_layout(int B, int H, int Hm, int N, int d, int for_bwd,
                                     fm_ws_layout* out);

/* Tile classification pre-pass ("FlashMask" abstract: the column-wise
 * representation lets whole masked blocks be skipped; "FlashMask-3" abstract:
 * the four boundary vectors): reduces the boundary vectors to the
 * per-key-block min/max table, the exact three-way label of every (query
 * block, key block) tile, the compacted non-FULL lists and the
 * descending-work orders, all in the workspace. Reads 16*B*Hm*N bytes.
 * Asynchronous on `stream`. */
fm_status flashmask_classify(const fm_mask* mask, int B, int N, void* ws, size_t ws_bytes,
                             void* stream);

/* Forward ("FlashMask" abstract: exact attention under the column-wise mask,
 * masked tiles skipped; "FlashAttention-3" abstract: the block-wise matmuls
 * overlapped with the softmax): O [B,H,N,d] bf16 and LSE [B,H,N] fp32 from
 * Q, K, V, as defined at the top of this file. `scale`
 * multiplies Q K^T (pass 1/sqrt(d) for standard attention). If
 * ws_classified == 0 the call runs flashmask_classify first; pass 1 to reuse a
 * classification of the same mask already in `ws`. Asynchronous on `stream`.
 * When ws_bytes is at least flashmask_workspace_bytes(..., for_bwd = 1), the
 * forward also zeroes that layout's dQ accumulator (bulk copies issued while
 * the attention runs) and leaves a tag of the shape in the fourth status word;
 * the backward preprocess of the same shape on this workspace then skips its
 * own zeroing pass, and the backward main kernel clears the tag again. */
fm_status flashmask_fwd(const void* q, const void* k, const void* v, const fm_mask* mask, int B,
                        int H, int N, int d, float scale, void* o, float* lse, void* ws,
                        size_t ws_bytes, int ws_classified, void* stream);

/* Backward ("FlashMask" abstract: exact gradients under the same mask, masked
 * tiles skipped; the FlashAttention README's memory savings, read here as P
 * recomputed from Q, K and the saved LSE rather than stored): dQ, dK, dV
 * [B,H,N,d] bf16 from Q, K, V, the forward's O and LSE, and the upstream
 * gradient dO. The workspace must be sized with for_bwd != 0.
 * ws_classified as in flashmask_fwd. Asynchronous on `stream`. The main
 * kernel gives each (head, key block) one CTA, except that with Tc >= 512 key
 * blocks (the environment variable FM_BWD_SPLIT_MIN_BLOCKS changes 512), among
 * the E = min(Tc, 16) longest key blocks of each head one seen by n query
 * blocks is split over min(4, n / 64) CTAs when that is at least two (a
 * global prefix would otherwise keep one SM busy long after the rest); the
 * parts' fp32 dK, dV are added through the workspace. */
fm_status flashmask_bwd(const void* q, const void* k, const void* v, const void* o,
                        const float* lse, const void* dout, const fm_mask* mask, int B, int H,
                        int N, int d, float scale, void* dq, void* dk, void* dv, void* ws,
                        size_t ws_bytes, int ws_classified, void* stream);

/* The three stages flashmask_bwd runs after the (optional) classification,
 * exposed so that a caller can schedule or time them separately. They must run
 * in this order on one stream with one workspace:
 *   preprocess: D = rowsum(dO * O), lse2 = LSE * log2(e), dQ accumulator = 0
 *               (HBM-bound; reads O and dO, writes 4*(2+d)*B*H*N bytes; the
 *               accumulator's 4*d*B*H*N bytes are skipped when the preceding
 *               flashmask_fwd on this workspace, of this shape, zeroed it).
 *   main:       dK, dV and the fp32 dQ accumulator over every non-FULL tile
 *               (needs a classification of `mask` and the preprocess output).
 *   finalize:   dQ = bf16(scale * accumulator).
 * Hm is the mask's number of heads (it fixes the workspace layout). */
fm_status flashmask_bwd_preprocess(const void* o, const float* lse, const void* dout, int B, int H,
                                   int Hm, int N, int d, void* ws, size_t ws_bytes, void* stream);
fm_status flashmask_bwd_main(const void* q, const void* k, const void* v, const void* dout,
                             const fm_mask* mask, int B, int H, int N, int d, float scale,
                             void* dk, void* dv, void* ws, size_t ws_bytes, void* stream);
fm_status flashmask_bwd_finalize(int B, int H, int Hm, int N, int d, float scale, void* dq,
                                 void* ws, size_t ws_bytes, void* stream);

/* Forward without any allocation or caller workspace: the paper has no
 * counterpart; this exists for callers that cannot allocate device memory
 * (inside a memory-pool or allocator callback, in runtimes that forbid
 * cudaMalloc once started, or in plug-ins that are handed only their inputs and
 * outputs). Same arguments and results as flashmask_fwd (with ws_classified =
 * 0), but the classification tables live in a fixed scratch array of
 * FM_NOALLOC_SCRATCH_BYTES inside the library, which every GPU that loads the
 * library holds until the process exits. Shapes whose tables would not fit
 * (about B*Hm*(N/128)^2*10 bytes; N = 131072 with B*Hm = 1 fits) return
 * FM_ERR_WORKSPACE before anything is launched. The call allocates nothing:
 * no cudaMalloc, no cudaFree, no allocating library routine.
 *   - The first call on each device looks up the scratch array's device
 *     address (cudaGetSymbolAddress) with that device current; make that first
 *     call before any stream capture.
 *   - All calls share the one array and it keeps the last call's contents; each
 *     call clears the status word it needs at zero and rewrites the tables.
 *     Calls that may overlap on the GPU (other streams, other threads) race
 *     on the array and must be serialised by the caller.
 *   - A device-side wait failure is recorded in the scratch status word, which
 *     callers cannot read; callers that need that report use flashmask_fwd. */
#define FM_NOALLOC_SCRATCH_BYTES (16u << 20)
fm_status flashmask_fwd_noalloc(const void* q, const void* k, const void* v, const fm_mask* mask,
                                int B, int H, int N, int d, float scale, void* o, float* lse,
                                void* stream);

/* FP8 forward ("FlashAttention-3", abstract: block quantization for FP8
 * attention): the same inputs, mask and outputs as flashmask_fwd (bf16 Q, K, V
 * [B,H,N,d], bf16 O and fp32 LSE), with the two products of each tile taken in
 * e4m3 on the tensor cores. d must be 128 (FM_ERR_UNSUPPORTED otherwise).
 * Each call quantises into the workspace: Q and K with one scale per head and
 * 128-row block (scale = absmax / 448, values rounded to nearest even and
 * saturated), V transposed with one scale per head; P is rounded to e4m3 as
 * 28 * P before P V (the running maximum is allowed to lag the true one by
 * at most 4 in log2 units, so 28 * P <= 448). The row sums, the running
 * maximum, LSE and every
 * accumulation stay fp32, so LSE carries only the error of the quantised
 * scores. Results differ from flashmask_fwd by the e4m3 rounding (3 mantissa
 * bits, relative step 2^-4): on random data O's relative Frobenius error is a
 * few percent, not the bf16 path's 1e-3.
 *   Workspace: flashmask_fwd_fp8_workspace_bytes(B, H, Hm, N) bytes, 256-byte
 *   aligned; its first part is the forward workspace layout (for_bwd = 0) of
 *   flashmask_workspace_layout with d = 128, so ws_classified works as in
 *   flashmask_fwd and flashmask_check_status reads its status word. The rest,
 *   at the byte offsets flashmask_fwd_fp8_layout gives, holds what the call
 *   wrote last (the caller may read it back):
 *     q8, k8   e4m3   [B,H,N,128]     Q / scale_Q, K / scale_K
 *     vt8      e4m3   [B,H,128,Npad]  (V / scale_V)^T, keys >= N zero
 *     qscale   fp32   [B,H,Tr]        scale_Q of each 128-row block
 *     kscale   fp32   [B,H,Tr]        scale_K of each 128-row block
 *     vscale   fp32   [B,H]           scale_V of each head
 *   A scale is absmax / 448 computed in fp32 (1 for an all-zero block) and a
 *   value is e4m3(x * (1 / scale)), both products rounded in fp32. The size
 *   function returns 0, the layout function FM_ERR_UNSUPPORTED, for an
 *   unsupported shape. Asynchronous on `stream`. */
typedef struct {
  size_t fwd_total, q8, k8, vt8, qscale, kscale, vscale, total;
} fm_fp8_layout;
size_t flashmask_fwd_fp8_workspace_bytes(int B, int H, int Hm, int N);
fm_status flashmask_fwd_fp8_layout(int B, int H, int Hm, int N, fm_fp8_layout* out);
fm_status flashmask_fwd_fp8(const void* q, const void* k, const void* v, const fm_mask* mask,
                            int B, int H, int N, int d, float scale, void* o, float* lse, void* ws,
                            size_t ws_bytes, int ws_classified, void* stream);

/* Forward and backward between HOST buffers, for callers whose tensors live in
 * host memory (the pages have no counterpart; the computation is exactly
 * flashmask_classify + flashmask_fwd + flashmask_bwd). The heads are cut into
 * chunks of `chunk_heads` consecutive heads of one batch entry (heads are
 * independent) and three streams overlap the copy of chunk c+1 to the device,
 * the kernels of chunk c and the copy of chunk c-1 back to the host, in three
 * slots carved from the device workspace `dev_ws` (>= the size
 * flashmask_host_workspace_bytes() returns for the same shape and chunk, 256-byte
 * aligned; the function returns 0 for an unsupported shape or chunk).
 *   Host pointers: q, k, v, dout [B,H,N,d] bf16; mask->lts/lte/uts/ute
 *   [B,Hm,N] int32; outputs o, dq, dk, dv [B,H,N,d] bf16 and lse [B,H,N] fp32.
 *   Page-locked host memory (cudaHostAlloc, torch pin_memory) lets the copies
 *   run concurrently with the kernels; pageable memory works but serialises.
 *   chunk_heads must divide H and either divide H / Hm or be a multiple of it
 *   (a chunk reads whole mask heads); otherwise FM_ERR_UNSUPPORTED.
 *   The call orders its work after what is already queued on `stream` and
 *   returns only when every output is in host memory (or with the first error;
 *   a kernel wait that gave up gives FM_ERR_TIMEOUT). It allocates no device
 *   memory; three streams and a few events are created once per device and
 *   kept, and calls on one device are serialised by a lock. */
size_t flashmask_host_workspace_bytes(int B, int H, int Hm, int N, int d, int chunk_heads);
fm_status flashmask_fwd_bwd_host(const void* q, const void* k, const void* v, const void* dout,
                                 const fm_mask* mask, int B, int H, int N, int d, float scale,
                                 void* o, float* lse, void* dq, void* dk, void* dv, void* dev_ws,
                                 size_t ws_bytes, int chunk_heads, void* stream);

/* Per-rank mask localisation for context parallelism ("FlashMask-3: ... Mask-Aware
 * Distributed Attention", abstract: under any multi-chunk context-parallel
 * assignment, per-rank localisation reduces to a zero-communication
 * clip-shift-max on the boundary vectors). For a rank that holds the query rows
 * [row0, row0 + rows) of each sequence and every key, writes the boundary
 * vectors of its local problem: int32 [B, Hm, N] device arrays lts, lte, uts,
 * ute (all four written; caller-owned) in local row coordinates [0, rows),
 * with no causal flag (the local mask is non-causal):
 *   every bound b -> min(max(b - row0, 0), rows)               (clip, shift)
 *   causal: key j's masked rows [0, j) become [0, c), c = clip(j - row0), and
 *   join the upper interval as [0, max(c, end))                 (max)
 * Column j of the local mask then marks exactly the chunk's rows that the
 * global mask marks, whenever that upper interval is empty or starts at a row
 * <= c (true for every causal mask whose upper interval lies above the
 * diagonal). Otherwise the column masks more than it should and *inexact
 * (device int32, may be NULL; set to 1, never cleared) records it. A rank with
 * several chunks calls this once per chunk. Keys are not localised (the local
 * problem is rows x N). Bad arguments (row0 < 0, rows < 1, row0 + rows > N,
 * null pointers) return before any launch. Asynchronous on `stream`. */
fm_status flashmask_localize(const fm_mask* mask, int B, int N, int row0, int rows, int32_t* lts,
                             int32_t* lte, int32_t* uts, int32_t* ute, int32_t* inexact,
                             void* stream);

/* ------------------------------------------------------------------ rotary positions
 * Rotates the leading `rot_dim` elements of every head of Q and K by their
 * token's position. They form n = rot_dim / 2 pairs, (i, i + n) in the half
 * layout and (2i, 2i + 1) when `interleaved`; pair i of a token at position t
 * turns by the angle a = t * freqs[i] and is multiplied by `mscale`:
 *     (x, y) -> mscale * (x cos a - y sin a, y cos a + x sin a)
 * and the other d - rot_dim elements are copied. `inverse` turns by -a instead:
 * the map is linear, so the same call with inverse = 1 is its gradient (dX
 * from dY), and with mscale = 1 it undoes the rotation.
 *   t[0], t[1]  one or two tensors that share B, N, d, the positions and one
 *               launch (Q and K, which may differ in heads); n_tensors 1 or 2.
 *               x and y are [B, H, N, d] of `dtype` with strides in elements
 *               for batch, head and token (the last dimension is contiguous),
 *               so a slice of a fused projection is read in place. y may be x
 *               with the same strides; otherwise they must not overlap, and the
 *               rows of one y must not overlap each other.
 *   positions   int32 [B, N] with `pos_stride` elements between batches (0:
 *               one row for all), any value; NULL: token n sits at position n.
 *   freqs       fp64 [rot_dim / 2], radians per position, on the device. Any
 *               scaling for long contexts is in them and in mscale.
 * The angle is taken in turns modulo one with 64-bit integers: its error is
 * below 2^-31 turns at every position and frequency, and then 2^-26 for its
 * rounding to fp32; sums are fp32 and rounded once. A frequency that is not
 * finite, or of 2^129 or more, gives NaN. d >= 1, 0 <= rot_dim <= d and even; B * N <
 * 2^31, B * N * d <= 2^38, at most 65535 heads together. B, N or H zero is
 * FM_ERR_UNSUPPORTED. Asynchronous on `stream`; needs no workspace. */
typedef enum { FM_BF16 = 0, FM_F16 = 1, FM_F32 = 2 } fm_dtype;
typedef struct {
  const void* x;
  void* y;
  int H;
  int64_t xs[3]; /* strides of x: batch, head, token (elements) */
  int64_t ys[3]; /* strides of y                                */
} fm_heads;
fm_status flashmask_rope(const fm_heads* t, int n_tensors, const int32_t* positions,
                         int64_t pos_stride, const double* freqs, int B, int N, int d, int rot_dim,
                         int interleaved, int dtype, float mscale, int inverse, void* stream);

/* Norm of every head of Q and K and the rotation above in one pass: a head x of d
 * elements becomes x * r * w, r = 1 / sqrt(mean(x^2) + eps), and its leading
 * `rot_dim` elements are then rotated as by flashmask_rope (times mscale; the
 * others are not). rot_dim = 0 is the norm alone.
 *   t[0], t[1]  as for flashmask_rope: x, y [B, H, N, d] of `dtype` with strides in
 *               elements; y may be x with the same strides, otherwise they must not
 *               overlap. w: the weights [d] of this tensor, of `weight_dtype` (FM_F32
 *               or `dtype`); NULL: ones. dy, ds and dw are the backward's.
 * d <= 256; eps >= 1e-30; other limits, positions and freqs as for flashmask_rope. Sums and
 * everything before the one rounding at the end are fp32; a head whose squares (backward:
 * or whose sum of g * w * x) would pass fp32 is scaled first. Asynchronous on `stream`;
 * needs no workspace.
 *
 * The backward gives the gradients from dy, that of the rotated output, and x, the
 * forward's input (nothing else is kept from the forward):
 *     g = dy rotated back, times mscale where it is rotated
 *     dw = sum of g * x * r over batch, heads and tokens
 *     dx = r * (g * w - x * r * mean(g * w * x * r))
 * (a term g * w * x of the mean loses bits where it falls below fp32's normal range).
 *   x, dy       [B, H, N, d] with strides xs and ds; y: dx, which may be dy or x with the
 *               same strides and otherwise overlaps no input
 *   dw          [d] of `weight_dtype`, written; NULL where it is not wanted
 *   ws          flashmask_norm_workspace_bytes(d) bytes, 256-byte aligned, need not be
 *               zeroed; not to be shared by calls that may run at the same time. May be
 *               NULL when no dw is wanted.
 * The sums for dw have a fixed order: the same call gives the same bits. */
typedef struct {
  const void* x;
  void* y;
  const void* dy;
  const void* w;
  void* dw;
  int H;
  int64_t xs[3]; /* strides of x: batch, head, token (elements) */
  int64_t ys[3]; /* of y                                        */
  int64_t ds[3]; /* of dy                                       */
} fm_norm_heads;
fm_status flashmask_norm_rope(const fm_norm_heads* t, int n_tensors, const int32_t* positions,
                              int64_t pos_stride, const double* freqs, int B, int N, int d, int rot_dim,
                              int interleaved, int dtype, int weight_dtype, float mscale, float eps,
                              void* stream);
/* 0 for an unsupported d. */
size_t flashmask_norm_workspace_bytes(int d);
fm_status flashmask_norm_rope_bwd(const fm_norm_heads* t, int n_tensors, const int32_t* positions,
                                  int64_t pos_stride, const double* freqs, int B, int N, int d, int rot_dim,
                                  int interleaved, int dtype, int weight_dtype, float mscale, float eps, void* ws,
                                  size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ 8-bit paged cache
 * Keys and values of running sequences as e4m3 codes in pages of FM_PAGE
 * tokens, one scale for each page and head (the block scaling of the FP8
 * forward, with its 128-row block cut to a page). All arrays are the caller's:
 *   k8      e4m3 [pages, Hk, FM_PAGE, d]
 *   v8      e4m3 [pages, Hk, d, FM_PAGE]  (transposed: the tokens of one column
 *                                          lie together, as P V reads them)
 *   kscale, vscale  fp32 [pages, Hk]      a value is its code times the scale, which is
 *                                         finite and not negative
 * page_table is int32 [B, max_pages]: entry i of a row is the page holding the
 * sequence's tokens [64 i, 64 i + 64). Only the entries of pages that a call
 * needs are read; the rest may hold anything. d in {64, 128}; FM_PAGE *
 * max_pages <= FM_MAX_SEQLEN; B * H * N < 2^31 - 255, B < 2^16, and B * Hk * T * max_pages
 * < 2^31 - 256, where T = ceil(R / 128) tiles hold the R = H / Hk * N rows of a cache head
 * (T = 2 for 17 to 32 rows). Entries, lengths and starts live on the device:
 * the kernels check each one they use, leave the access out when it is out of
 * range and record it, so that flashmask_check_status() returns FM_ERR_PAGE
 * (the outputs of that sequence are then undefined). */
#define FM_PAGE 64
typedef struct {
  void* k8;
  void* v8;
  float* kscale;
  float* vscale;
  int pages, Hk, d;
} fm_cache;

/* Workspace of the two calls below for these sizes (H query heads, N new or
 * query tokens a sequence); 0 for an unsupported shape. 256-byte aligned and
 * zeroed before its first use; not to be shared by calls that may run at the
 * same time. One workspace serves these two calls in turn for all sizes that
 * it is large enough for. Zero it again after another entry point has used it
 * or after FM_ERR_TIMEOUT. Its first 16 bytes are the status word. */
size_t flashmask_cache_workspace_bytes(int B, int H, int Hk, int N, int d, int max_pages);

/* Writes N new tokens of each sequence behind the start[b] it holds: K and V
 * bf16 [B, Hk, N, d] with strides in elements for batch, head and token
 * (multiples of 8; the last dimension contiguous, 16-byte aligned). count (int32
 * [B], may be NULL: N) says how many of a sequence's N rows are real; the
 * others are not read. Codes are rounded to nearest even.
 *   Scales are powers of two: the smallest 2^k, k >= -100, with absmax <=
 *   448 * 2^k over the tokens of the page and head. While a page fills, its
 *   scale only grows; the codes already there are then rounded again to the
 *   larger scale (exact unless they fall into e4m3's subnormal range). A page
 *   whose first token is written here is begun: its old scales do not count
 *   and the slots behind the last new token are set to zero. Slots behind the
 *   last new token of a page begun earlier are left as they are.
 *   A token with a value that is not finite, in K or in V of a head, does not
 *   count for that head's scales and is stored so that every query that sees
 *   it, and no other, gets NaN: its K codes are NaN, its V codes zero.
 *   count outside [0, N] counts as the nearer bound.
 *   The pages written by one call must be distinct (a page shared by two
 *   sequences is copied by the caller before either appends to it). A start
 *   below 0 or a sequence that would outgrow max_pages is left alone and
 *   recorded. Asynchronous on `stream`; uses only the status word of `ws`. */
fm_status flashmask_cache_append(const fm_cache* cache, const int32_t* page_table, int max_pages,
                                 const void* k, const int64_t ks[3], const void* v,
                                 const int64_t vs[3], const int32_t* start, const int32_t* count,
                                 int B, int N, void* ws, size_t ws_bytes, void* stream);

/* Attention of N query tokens of each sequence over its cached keys and values:
 * one token while a sequence runs, several when drafted tokens are checked, a
 * chunk of a prompt. lens (int32 [B]) is the number of cached tokens, the query
 * tokens' own among them; q_lens (int32 [B], may be NULL: N) how many of the N
 * rows are real. Row t of sequence b sits at position i = lens[b] - q_lens[b] +
 * t; rows t >= q_lens[b] have no influence and are not written; q_lens outside
 * [0, N] counts as the nearer bound. Key j < lens[b] is
 * masked when
 *     (causal && j > i) || (LTS[j] <= i < LTE[j]) || (UTS[j] <= i < UTE[j])
 * with the vectors [B, Hm, max_pages * FM_PAGE] of `mask`, whose lts and lte
 * may both be NULL too (no lower interval); mask NULL: causal, no intervals.
 * The vectors are 16-byte aligned; entries behind a sequence's length may hold anything.
 * Head h reads mask head h / (H / Hm) and cache head h / (H / Hk); H % Hk ==
 * 0, H % Hm == 0. O, LSE and rows without a visible key are as at the top of
 * this file: O bf16 [B, H, N, d], LSE fp32 [B, H, N] (contiguous).
 * Keys and values count as their codes times their scales; scores, softmax
 * statistics and sums are fp32. For its product with V a weight P = exp(score - largest)
 * is rounded to fp16: 2^-11 of it, or 2^-32 of the row's largest P * (scale of V) where
 * that is more; LSE and the sum that O is divided by have it unrounded. What K holds
 * for masked keys, what the slots behind a sequence's end hold and what pages hold of
 * which no row sees a key has no influence, NaN included. V codes of the other slots must not be NaN, masked or not
 * (flashmask_cache_append writes none: a NaN in V becomes one in K). A query row with a
 * value that is not finite gives NaN, and so does a row that sees a key of a page whose K
 * or V scale is negative, infinite or NaN.
 *   qs, os: strides of Q and O in elements for batch, head and token (multiples
 *   of 8; the last dimension contiguous, 16-byte aligned). O may be Q itself with
 *   the same strides; otherwise O and LSE overlap neither each other nor an input.
 *   scale: positive, scale / ln 2 finite.
 * Results do not depend on the order in which CTAs run (the same call gives the
 * same bits); how a sequence's sum is split depends on the whole batch, so its
 * last bits may differ beside other sequences. Asynchronous on `stream`. */
fm_status flashmask_fwd_cache(const void* q, const int64_t qs[3], const fm_cache* cache,
                              const int32_t* page_table, int max_pages, const int32_t* lens,
                              const int32_t* q_lens, const fm_mask* mask, int B, int H, int N,
                              float scale, void* o, const int64_t os[3], float* lse, void* ws,
                              size_t ws_bytes, void* stream);

/* The attention weight that each cached key is given, for deciding which keys a cache
 * keeps: for key j of cache head hk
 *     sum over its query heads h and the query rows that see j of exp(scale q . k_j - LSE)
 * is added to weights[page][hk][slot] (fp32 [pages, Hk, FM_PAGE], laid out like the
 * scales), LSE [B, H, N] being what flashmask_fwd_cache gave for the same q, cache,
 * lens, q_lens, mask and scale. Keys from position start[b] on are new: they have had
 * nothing, so what their slots hold is replaced. start NULL: the query tokens' own
 * keys, from lens[b] - q_lens[b] on. start 0 for a prompt whose last rows alone weigh
 * all of its keys. A key that no row sees gets 0; slots from lens[b] on are left as they were.
 *   q, cache, page_table, lens, q_lens, mask, scale and their limits as for
 *   flashmask_fwd_cache; V takes no part. The pages of one call must be distinct: two
 *   sequences that share some (of a common beginning) would both add to the same slots at
 *   once, so they take a call each, one after the other, and start lies behind the shared
 *   keys in all but the first. A row whose LSE is -inf gives nothing; one whose LSE, query
 *   or visible K scale is NaN (or a K scale that is negative or infinite) gives NaN to the
 *   keys that it sees. What K holds for keys that no row sees has no influence.
 *   ws: flashmask_cache_weights_workspace_bytes(...) bytes, 256-byte aligned and zeroed
 *   before its first use; not to be shared by calls that may run at the same time; one
 *   workspace serves all sizes that it is large enough for. Zero it again after another
 *   entry point has used it and after FM_ERR_TIMEOUT or FM_ERR_CUDA. Its first 16 bytes are
 *   the status word.
 * Scores, exponentials and sums are fp32 and a key's sum has a fixed order: the same call
 * gives the same bits. Asynchronous on `stream`. */
size_t flashmask_cache_weights_workspace_bytes(int B, int H, int Hk, int N, int d, int max_pages);
fm_status flashmask_cache_weights(const void* q, const int64_t qs[3], const fm_cache* cache,
                                  const int32_t* page_table, int max_pages, const int32_t* lens,
                                  const int32_t* q_lens, const fm_mask* mask, int B, int H, int N, float scale,
                                  const float* lse, float* weights, const int32_t* start, void* ws,
                                  size_t ws_bytes, void* stream);

/* Cuts sequences down: each cache head of sequence b keeps n = min(lens[b], keep[b]) of its
 * tokens (a keep[b] below 0 counts as 0; keep NULL: `budget` for all, which is refused
 * below 0, as sink and recent are): the first min(sink, n), the last min(recent, n -
 * those), and of the others those of the largest weight (fp32 [pages, Hk, FM_PAGE], see
 * flashmask_cache_weights; any values: -0 counts as 0, NaN as less than everything else;
 * of equal ones the lower position is kept). Heads choose for themselves.
 * The kept tokens move together in their order: K, V, scales and weights go to the
 * positions 0 .. n - 1 of
 *   out_table   int32 [B, out_pages], pages that neither repeat nor occur in page_table's
 *               used entries, so that sequences which share pages can be cut down apart
 *               and the old pages stay as they are; or
 *   NULL (or page_table itself): in place, in the first ceil(n / 64) pages of page_table,
 *               which must be distinct. Pages behind them are left as they were and free.
 * new_lens (int32 [B], may be lens) gets n. index (int32 [B, Hk, index_width], may be NULL)
 * gets the old positions of each head's kept tokens (the first index_width of them; entries
 * behind n are left as they were): what a caller needs to cut down its own data for these
 * keys, such as a mask's vectors. Afterwards positions count kept tokens: causality
 * holds as before, intervals are the caller's to shorten.
 *   Scales: a page whose tokens all stay where they are is left as it was. Any other gets, for
 *   K and for V, the smallest 2^k, -100 <= k <= 127, with absmax <= 448 * 2^k over its
 *   tokens, as flashmask_cache_append would give it, and codes are rounded to nearest even
 *   for it (exact if the old scales are powers of two, unless a code falls into e4m3's
 *   subnormal range). Its slots behind the last token are set to zero. NaN codes of K stay NaN and do not
 *   count for the scale, nor does a token of a page whose K or V scale is negative, infinite
 *   or NaN: its K codes become NaN, its V codes zero.
 *   ws: flashmask_cache_evict_workspace_bytes(...) bytes, 256-byte aligned and zeroed
 *   before its first use; not to be shared by calls that may run at the same time; one
 *   workspace serves all sizes that it is large enough for. Zero it again after another
 *   entry point has used it and after FM_ERR_TIMEOUT or FM_ERR_CUDA. Its first 16 bytes are
 *   the status word.
 *   A page or length out of range, or n > 64 * out_pages, is recorded (see
 *   flashmask_check_status) and the access left out.
 * Limits as for flashmask_cache_append; out_pages <= FM_MAX_SEQLEN / FM_PAGE. The same call gives
 * the same bits. Asynchronous on `stream`. */
size_t flashmask_cache_evict_workspace_bytes(int B, int Hk, int max_pages);
fm_status flashmask_cache_evict(const fm_cache* cache, const int32_t* page_table, int max_pages,
                                const int32_t* out_table, int out_pages, const int32_t* lens, float* weights,
                                const int32_t* keep, int budget, int sink, int recent, int32_t* new_lens,
                                int32_t* index, int index_width, int B, void* ws, size_t ws_bytes, void* stream);

/* Self-test of the failure path (no counterpart in the pages). Launches `ctas`
 * (1..1024) one-warp CTAs whose mbarrier wait can never complete, bounded the
 * way every wait of the library is: CTA 0 gives up after `limit_ns` (1e6..2e9)
 * of wall time and records site 301 in the workspace status word; the other
 * CTAs use the library's own limit but leave as soon as they see that status,
 * as the CTAs of an attention kernel do when one of their waits fails. No
 * fault, no hang; the context stays usable. Returns FM_OK once queued on
 * `stream`; flashmask_check_status() then returns FM_ERR_TIMEOUT with detail
 * 301. ws: any workspace of >= 16 bytes, 256-byte aligned (only the status
 * word is used). */
fm_status flashmask_selftest_timeout(void* ws, size_t ws_bytes, long long limit_ns, int ctas,
                                     void* stream);

/* Synchronises `stream`, then reads and clears the workspace status word.
 * Returns FM_ERR_TIMEOUT if a kernel wait gave up since the last check,
 * FM_ERR_PAGE if a cache call met a page, length or start out of range,
 * FM_ERR_CUDA if the stream reports an error, FM_OK otherwise. If detail is
 * not NULL it receives the recorded failure site (0 if none). */
fm_status flashmask_check_status(void* ws, void* stream, int* detail);

/* Static description of a status code. */
const char* flashmask_status_string(fm_status s);

#ifdef __cplusplus
}
#endif
#endif /* FLASHMASK_H */
