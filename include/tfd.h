/*
 * tfd.h - C ABI of the GB300 (sm_103a) draft-head decode step library, libtfd.so.
 *
 * The library computes the per-round step of an EAGLE-style draft head in a speculative-decoding
 * server: a few-row (1..16 token rows) vocabulary-head GEMV in bf16 or FP8 fused with a
 * split-vocabulary top-1 / top-k, the two-stage head (low-rank top-cand_k then exact rescore), the
 * qk_norm + RoPE ring-window attention, the accept-prefix count, and the FP8 quantisation of the
 * weights these calls read; for requests that sample, drawing tokens from logits and the
 * rejection accept of such drafts; and, for contexts longer than a ring, a paged key-value cache: its
 * page tables, the append of new rows, and the attention of one or a few rows a request over it.
 *
 * Conventions shared by every call:
 *  - Pointers named as device buffers are caller-owned device memory on the current CUDA device.
 *    The library allocates nothing in a call and keeps no state between calls.
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream). Every call only enqueues work
 *    on it and never synchronises; results are ready when the stream reaches them.
 *  - The return value reports host-side argument checks and launch errors. A call that fails a
 *    check returns its status and enqueues nothing.
 *  - Errors that depend on device data (an out-of-range candidate id, an asked count larger than
 *    the window, a negative position) never trap: the kernel skips the offending element and, when
 *    `dev_status` is not NULL, stores TFD_ERR_DEVICE_DATA there with an atomic compare-and-swap
 *    from 0 (the first error stays). The caller zeroes *dev_status before the call.
 *  - Matrices are row-major. Every device pointer must be 16-byte aligned (8-bit and 32-bit scale
 *    arrays: 4-byte aligned), and leading dimensions keep every row 16-byte aligned.
 *  - Top-k outputs are sorted by value descending, then id ascending. Values compare as floats
 *    (-0 == +0); NaN ranks below -inf. Returned values are canonical: -0 comes back as +0 and NaN
 *    as the quiet NaN 0x7FC00000.
 *  - Workspaces: a call that needs one takes `ws`/`ws_bytes` and a `*_workspace()` query returns
 *    the bytes it needs. A workspace holds arrival counters that must start at zero: zero-fill it
 *    once before its first use; every call that completes leaves those counters at zero again.
 *    Two calls that may run at the same time need separate workspaces.
 *
 * Citations name the source page and its section:
 *  [TFE]    "dsv41 Zig: the TFE draft head (TF_DS_DRAFTER=eagle), off by default" (#42)
 *  [DSPARK] "dsv41 metal: the DSpark drafter on an FP8 head, a concurrent propose and resident
 *           buffers" (#3296)
 *  [SUBSET] "nemotron: Super's MTP drafts on the draft vocabulary's FP8 rows ..." (#1011)
 */
#ifndef TFD_H_
#define TFD_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  TFD_OK = 0,
  TFD_ERR_INVALID = 1,      /* an argument is out of range, NULL, misaligned or aliased */
  TFD_ERR_UNSUPPORTED = 2,  /* valid, but outside what this build implements (e.g. dim != 128) */
  TFD_ERR_WORKSPACE = 3,    /* ws is NULL or ws_bytes is below the *_workspace() size */
  TFD_ERR_CUDA = 4,         /* the CUDA runtime reported an error at launch */
  TFD_ERR_DEVICE_DATA = 5,  /* (device status only) bad ids, counts or positions in device data */
  TFD_ERR_TIMEOUT = 6       /* (device status only) a bounded device wait gave up */
} tfd_status;

/*
 * Weight formats. TFD_W_FP8_BLOCK32_IL holds the same codes and scales as TFD_W_FP8_BLOCK32 with
 * the codes of each row reordered in steps of 64 columns (k % 64 == 0): within step c, bytes
 * 64c + 16t + 8b + e (t = 0..3, b = 0..1, e = 0..7) hold the code of column 64c + 32b + 8t + e,
 * so the 8 codes a GEMV thread takes from each of a step's two 32-wide blocks are one 16-byte
 * load. It is this library's own layout (no counterpart on the pages); tfd_quant_fp8 writes it and
 * tfd_fp8_block32_relayout converts to and from the plain row-major layout.
 */
typedef enum {
  TFD_W_BF16 = 0,
  TFD_W_FP8_ROW = 1,
  TFD_W_FP8_BLOCK32 = 2,
  TFD_W_FP8_BLOCK32_IL = 3
} tfd_wfmt;
/*
 * Activation formats. TFD_X_BF16_E4M3 (FP8 weights only, W8A8): bf16 activations quantised per
 * row inside the call by the weights' row rule, s_r = fl32(amax_r / 448), code = e4m3_rne_sat(
 * fl32(x / s_r)) (a zero row keeps its zeros), and multiplied on the E4M3 tensor-core path; the
 * result is acc * s_r (* the weights' scales) with fp32 accumulation.
 */
typedef enum { TFD_X_BF16 = 0, TFD_X_F32 = 1, TFD_X_BF16_E4M3 = 2 } tfd_xfmt;
typedef enum { TFD_OUT_NONE = 0, TFD_OUT_F32 = 1, TFD_OUT_BF16 = 2, TFD_OUT_ADD_BF16 = 3 } tfd_out;

/* Limits from the pages' statement of the problem. */
/* [TFE] commit "pass kernels and FP8 linears": GEMV for up to 16 rows; windows of up to 32 rows
 * (rows 17-32 take k split over a thread-block cluster where one block's shared memory is too
 * small for the activation tile; fp32 activations stop at 16 rows). */
#define TFD_MAX_ROWS 32
#define TFD_MAX_TOPK 512    /* [TFE] commit "... ocabulary head": cand_k from 1 to 512 */
#define TFD_MAX_WINDOW 511  /* [TFE] commit "... ocabulary head": window up to 511 (512 keys) */
#define TFD_MAX_RANK 128     /* rank of a low-rank adapter */
#define TFD_MAX_LORA_ROWS 262144  /* rows of one tfd_lora call (every tile's search reads all ids) */
#define TFD_MAX_DRAW_COLS 1048576 /* columns of a row that a token is drawn from (exact sums) */
#define TFD_MAX_REQUESTS 8192     /* requests of one paged call */
#define TFD_MAX_PAGE 1024         /* tokens of a page */

/* A static string naming a status. Never NULL. */
const char* tfd_status_string(int status);

/* Library version (major * 10000 + minor * 100 + patch). */
int tfd_version(void);

/*
 * tfd_quant_fp8 - FP8 E4M3 codes of a bf16 weight W[n][k].
 *   mode TFD_W_FP8_ROW: per row s_n = fl32(amax_n / 448); code = e4m3_rne_sat(fl32(w / s_n)).
 *     [TFE] update "main3x heads, pass kernels, FP8 linears": "scale = row absmax / 448, round to
 *     nearest even, from the bf16 weight". A zero row gets s = 0 and keeps its (signed) zeros.
 *   mode TFD_W_FP8_BLOCK32: per 32x32 block, byte = clamp(e + 127, 0, 254) where 2^e is the
 *     smallest power of two with amax <= 448 * 2^e (an all-zero block stores 0); code =
 *     e4m3_rne_sat(w * 2^-(byte - 127)). [DSPARK] "FP8 draft head": E4M3 codes with E8M0 scales in
 *     32x32 blocks.
 *   mode TFD_W_FP8_BLOCK32_IL: the codes and scales of TFD_W_FP8_BLOCK32, codes written in the
 *     interleaved layout described at tfd_wfmt (k % 64 == 0).
 *   E4M3 is the "fn" form (bias 7, max 448, 0x7F = NaN); encoding is round-to-nearest-even with
 *   saturation to +-448. Weights must be finite.
 * Args:
 *   w_bf16  device, bf16 [n][k] (row stride k).
 *   n, k    n >= 1, k >= 16 and k % 16 == 0; BLOCK32 also needs n % 32 == 0 and k % 32 == 0.
 *   codes   device, uint8 [n][k] (written).
 *   scales  device, ROW: float [n]; BLOCK32: uint8 [n/32][k/32] (written).
 */
tfd_status tfd_quant_fp8(const void* w_bf16, int64_t n, int64_t k, int mode, uint8_t* codes,
                         void* scales, void* stream);

/*
 * tfd_head_gemv - few-row head GEMV acc[r][i] = sum_j W[i][j] * x[r][j] with fp32 accumulation,
 * optional output, and an optional fused top-k over the n outputs of each row.
 *   [TFE] commit "pass kernels and FP8 linears": GEMV over bf16 and e4m3 weights for up to 16 rows
 *   (out bf16, fp32, or added to bf16); the top-1 of a vocabulary row in parts and a join.
 *   [DSPARK] "FP8 draft head": the drafter keeps its top 64 candidates.
 *   FP8 forms keep activations in bf16/fp32 (W8A16): ROW acc = s_i * sum dec(c) x;
 *   BLOCK32 acc = sum over 32-wide k blocks of 2^(byte-127) * (sum dec(c) x).
 * Args:
 *   w        device: bf16 [n][k], or uint8 codes [n][k] for the FP8 forms.
 *   wfmt     tfd_wfmt.
 *   w_scales device: FP8_ROW float [n]; FP8_BLOCK32 uint8 [n/32][k/32]; NULL for bf16.
 *   n, k     outputs per row (>= 1) and reduction length (k >= 16, k % 16 == 0; BLOCK32 also
 *            n % 32 == 0 and k % 32 == 0).
 *   x        device: bf16 or float (xfmt) [rows][ldx], ldx >= k. Float activations are used at
 *            full fp32 precision; TFD_X_BF16_E4M3 (FP8 weights only) quantises bf16 rows to E4M3
 *            first (W8A8, see tfd_xfmt).
 *   rows     1..32 (fp32 activations 1..16). Rows 17-32 go past this page's 16: the subset
 *            page (#1011) runs decode windows of 17 to 32 rows on wider kernels.
 *   out_mode NONE: no output; F32: y float [rows][ldy] = fl32(acc); BF16: y bf16 = bf16(fl32(acc));
 *            ADD_BF16: y bf16 is read as the residual and overwritten with bf16(res + acc), which
 *            may share memory with nothing else read by the call (in place is allowed).
 *   ldy      >= n when out_mode != NONE.
 *   topk     0 = none, else 1..512 (<= n): top_vals/top_ids [rows][ldt] receive the top-k of
 *            each row's fp32 acc (the FP8_ROW scale and BLOCK32 scales applied).
 *   ldt      row stride of top_vals/top_ids (0 = topk; else >= topk), so that the top-1 of each
 *            step of a multi-step pass can land in one column of a [streams][steps] array.
 *   top1_conf device float [rows] or NULL; only with topk == 1: the top-1 "with confidence"
 *            ([TFE] "What this changes": row kernels ... top-1 with confidence), read as the
 *            softmax probability of the pick, 1 / sum_i exp(acc_i - max acc) over the row's n
 *            outputs (NaN and -inf outputs add nothing; a row of only those gives NaN).
 *   parts    the row is scanned in `parts` contiguous ranges whose partial top-k are then joined;
 *            0 = the library's choice. The result does not depend on it.
 *   id_map   device int32 [n] or NULL: the id reported (and compared on ties) for output i is
 *            id_map[i] instead of i (a candidate list or a subset vocabulary, [SUBSET]).
 *   ws       device workspace of tfd_head_gemv_workspace(rows, n, topk, parts) bytes (may be 0).
 *   dev_status device int32 or NULL. A matrix split over a cluster of two blocks (few 64-row
 *            groups, or 17-32 rows of a 4096-wide matrix) exchanges partial sums through bounded
 *            waits; one that gives up (after about a second) stores TFD_ERR_TIMEOUT there and the
 *            call's outputs are then undefined. No other device-data errors exist in this call.
 * Refused: rows outside 1..32 (1..16 for fp32 activations); topk > 512 or > n; x aliasing y; NULL or misaligned pointers;
 *   rows * k too large for the activation tile (TFD_ERR_UNSUPPORTED, see tfd_head_gemv_max_k).
 */
size_t tfd_head_gemv_workspace(int rows, int64_t n, int topk, int parts);
int64_t tfd_head_gemv_max_k(int rows, int xfmt);
tfd_status tfd_head_gemv(const void* w, int wfmt, const void* w_scales, int64_t n, int64_t k,
                         const void* x, int xfmt, int rows, int64_t ldx, int out_mode, void* y,
                         int64_t ldy, int topk, int parts, const int32_t* id_map, float* top_vals,
                         int32_t* top_ids, int64_t ldt, float* top1_conf, void* ws,
                         size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * tfd_head_gemv_noalloc - tfd_head_gemv without a caller workspace, for callers that cannot
 * allocate device memory: serving loops that keep allocator calls off the hot path because
 * cudaMalloc can block or synchronise the whole device in the middle of a decode round, and plugins
 * whose host framework owns all device memory and offers them no allocator.
 *   The pages have no counterpart of this entry point; it is an addition of this library.
 *   Same arguments and results as tfd_head_gemv, minus ws/ws_bytes. The scratch is a fixed device
 *   array of TFD_NOALLOC_SCRATCH_BYTES inside the library, held by every GPU that loads it until
 *   the process exits. A call whose tfd_head_gemv_workspace() size exceeds it returns
 *   TFD_ERR_WORKSPACE and enqueues nothing (top-1 calls always fit; a top-k > 1 call fits only when
 *   its fp32 logits and top-k lists do, i.e. for small n).
 *   The first call on a device looks the array's device address up (once per device, with that
 *   device current; a failed lookup is retried by the next call); make that first call before any
 *   stream capture. Each call clears the part of
 *   the array it uses on `stream` before the GEMV (so a call that then fails an argument check has
 *   already enqueued that clear, which touches only the library's own array). Every call shares
 *   the one array: calls whose work overlaps on the GPU (other streams, other threads) race and
 *   must be serialised by the caller. It calls no cudaMalloc, cudaFree or allocating library.
 */
#define TFD_NOALLOC_SCRATCH_BYTES 1048576
tfd_status tfd_head_gemv_noalloc(const void* w, int wfmt, const void* w_scales, int64_t n,
                                 int64_t k, const void* x, int xfmt, int rows, int64_t ldx,
                                 int out_mode, void* y, int64_t ldy, int topk, int parts,
                                 const int32_t* id_map, float* top_vals, int32_t* top_ids,
                                 int64_t ldt, float* top1_conf, int32_t* dev_status,
                                 void* stream);

/*
 * tfd_topk - top-k of given fp32 logits, ties to the lower (mapped) id; values and ids bit-exact.
 *   [TFE] commit "... ocabulary head": "the top cand_k low-rank logits (fp32, a tie at the k-th
 *   value by the lower token id)", cand_k 1 to 512; "the top-1 kernel through an id map".
 * Args:
 *   logits device float [rows][ld], ld >= n. rows >= 1, n >= 1, 1 <= k <= min(n, 512).
 *   id_map device int32 [n] or NULL (as in tfd_head_gemv).
 *   vals, ids device [rows][k] (written).
 *   ws     device workspace of tfd_topk_workspace(rows, n, k) bytes.
 */
size_t tfd_topk_workspace(int rows, int64_t n, int k);
tfd_status tfd_topk(const float* logits, int rows, int64_t n, int64_t ld, int k,
                    const int32_t* id_map, float* vals, int32_t* ids, void* ws, size_t ws_bytes,
                    void* stream);

/*
 * tfd_rescore - exact logits of each row's candidates from a dense bf16 head, and their argmax.
 *   [TFE] commit "... ocabulary head": the two_stage head drafts "the argmax of their exact logits
 *   from the target's own head, a dense bf16 copy".
 *   e[r][j] = fl32(W_exact[cand[r][j]] . x[r]) with fp32 accumulation; out_ids[r] = the candidate
 *   with the largest e (ties to the lower id). A candidate outside [0, vocab) gets e = NaN (it
 *   ranks last) and sets TFD_ERR_DEVICE_DATA.
 * Args:
 *   w_exact_bf16 device bf16 [vocab][k]; k >= 16, k % 16 == 0.
 *   x_bf16   device bf16 [rows][k]; rows 1..32.
 *   cand     device int32 [rows][cand_k]; cand_k 1..512.
 *   cand_logits device float [rows][cand_k] or NULL.
 *   out_ids  device int32 [rows]; out_vals device float [rows] or NULL.
 *   ws       device workspace of tfd_rescore_workspace(rows, cand_k) bytes.
 */
size_t tfd_rescore_workspace(int rows, int cand_k);
tfd_status tfd_rescore(const void* w_exact_bf16, int64_t vocab, int64_t k, const void* x_bf16,
                       int rows, const int32_t* cand, int cand_k, float* cand_logits,
                       int32_t* out_ids, float* out_vals, void* ws, size_t ws_bytes,
                       int32_t* dev_status, void* stream);

/*
 * tfd_window_attn - one decode position per stream: qk_norm, RoPE, ring write, window attention.
 *   [TFE] commit "... ocabulary head": qk_norm is an RMSNorm on each query and key head before
 *   RoPE; the window goes up to 511 (512 keys). Commit "pass kernels and FP8 linears": single-query
 *   attention over the window in one block. First commits: the head's rows live in a ring.
 *   Per stream s at position p = pos[s] and head h:
 *     q' = rope(rmsnorm(q) * q_gamma, p) (fp32); k' = bf16(rope(rmsnorm(k_new) * k_gamma, p));
 *     k_ring[s][p % ring][h] = k'; v_ring[s][p % ring][h] = v_new;
 *     out[s][h*dim..] = bf16(softmax_j(q' . k_j / sqrt(dim)) . v_j) over positions
 *     j = max(0, p - window) .. p read from the ring.
 *   rmsnorm(v) = v / sqrt(mean(v^2) + eps); RoPE pairs element i with i + dim/2 and turns the pair
 *   by p * rope_base^(-2i/dim). Ring slots of earlier positions must hold their keys and values.
 * Args:
 *   q, k_new, v_new device bf16 [streams][heads][dim]; q_gamma, k_gamma device bf16 [dim] or NULL
 *   (ones); pos device int32 [streams] (a negative position sets TFD_ERR_DEVICE_DATA and that
 *   stream's output is left unwritten); k_ring, v_ring device bf16 [streams][ring][heads][dim];
 *   ring >= window + 1; window 0..511; dim == 128; out device bf16 [streams][heads*dim].
 */
tfd_status tfd_window_attn(const void* q, const void* k_new, const void* v_new,
                           const void* q_gamma, const void* k_gamma, float eps, float rope_base,
                           const int32_t* pos, void* k_ring, void* v_ring, int ring, int window,
                           int streams, int heads, int dim, void* out, int32_t* dev_status,
                           void* stream);

/*
 * tfd_accept - accept-prefix count of a verify round.
 *   [TFE] commit "... rnel test TF_DS_ACCEPT_LOG=N": a draft is kept when it and every earlier
 *   draft equal the round's draws; the log counts drafts asked and kept at each window position.
 *   n_kept[s] = the largest m <= n_asked[s] with drafts[s][i] == draws[s][i] for all i < m.
 *   asked_hist[i] += (i < n_asked[s]) and kept_hist[i] += (i < n_kept[s]) over the streams.
 *   An n_asked outside [0, win] sets TFD_ERR_DEVICE_DATA; that stream keeps 0 and adds nothing.
 * Args:
 *   drafts, draws device int32 [streams][win]; n_asked device int32 [streams]; streams >= 1;
 *   win 1..512; n_kept device int32 [streams]; asked_hist, kept_hist device int64 [win] or NULL
 *   (both or neither), accumulated.
 */
tfd_status tfd_accept(const int32_t* drafts, const int32_t* n_asked, const int32_t* draws,
                      int streams, int win, int32_t* n_kept, int64_t* asked_hist,
                      int64_t* kept_hist, int32_t* dev_status, void* stream);

/*
 * tfd_fp8_block32_relayout - block-32 FP8 codes between the plain row-major layout and the
 *   interleaved layout of TFD_W_FP8_BLOCK32_IL (a permutation of bytes within each row; the
 *   scales are unchanged). No counterpart on the pages: it serves codes made elsewhere.
 * Args:
 *   in, out device uint8 [n][k], not overlapping; n >= 1; k >= 64 and k % 64 == 0; 16-byte
 *   aligned. to_interleaved: 1 plain -> interleaved, 0 interleaved -> plain.
 */
tfd_status tfd_fp8_block32_relayout(const uint8_t* in, int64_t n, int64_t k, int to_interleaved,
                                    uint8_t* out, void* stream);

/*
 * tfd_rmsnorm - RMSNorm of hidden rows.
 *   [TFE] eagle.cu's row kernels include RMSNorm; qk_norm is the same normalisation per head.
 *   out[r][i] = bf16(x[r][i] / sqrt(mean_i(x[r][i]^2) + eps) * gamma[i]), sums in fp32.
 * Args:
 *   x device bf16 [rows][ldx]; out device bf16 [rows][ldo] (may equal x: in place);
 *   gamma device bf16 [hidden] or NULL (ones); rows >= 1; hidden >= 8 and hidden % 8 == 0;
 *   ldx, ldo >= hidden and multiples of 8; eps >= 0; x, out, gamma 16-byte aligned.
 */
tfd_status tfd_rmsnorm(const void* x, int64_t ldx, const void* gamma, float eps, int rows,
                       int64_t hidden, void* out, int64_t ldo, void* stream);

/*
 * tfd_swiglu - SwiGLU of a gate and an up row, SiLU rounded to bf16 before the multiply.
 *   [TFE] the reference "rounds SiLU(g) to bf16 before the multiply", as the silu-mul row kernel
 *   does. out = bf16(bf16(SiLU(g)) * u), SiLU(g) = g / (1 + exp(-g)) in fp32.
 * Args:
 *   g, u device bf16 [rows][ld]; out device bf16 [rows][ldo] (may equal g or u); rows >= 1;
 *   cols >= 8 and cols % 8 == 0; ld, ldo >= cols and multiples of 8; 16-byte aligned.
 */
tfd_status tfd_swiglu(const void* g, const void* u, int64_t ld, int rows, int64_t cols, void* out,
                      int64_t ldo, void* stream);

/*
 * tfd_absorb - write a span of key/value rows into each stream's ring (a prompt chunk or a round).
 *   [TFE] first commits: an absorb of more rows than the ring wrote two rows to one ring row, and
 *   "absorb refuses a larger span"; commit "... ocabulary head": qk_norm before RoPE, and a prompt
 *   chunk gives the head its last ring of rows.
 *   For stream s and row i < n at position p = p0[s] + i:
 *     k_ring[s][p % ring][h] = bf16(rope(rmsnorm(k_rows[s][i][h]) * k_gamma, p));
 *     v_ring[s][p % ring][h] = v_rows[s][i][h];
 *   with the normalisation and rotation of tfd_window_attn.
 * Args:
 *   k_rows, v_rows device bf16 [streams][n][heads][dim]; k_gamma device bf16 [dim] or NULL;
 *   p0 device int32 [streams] (negative, or p0 + n past INT32_MAX: TFD_ERR_DEVICE_DATA and that
 *   stream is left unwritten); 1 <= n <= ring (a longer span is refused with TFD_ERR_INVALID);
 *   k_ring, v_ring device bf16 [streams][ring][heads][dim]; dim == 128.
 */
tfd_status tfd_absorb(const void* k_rows, const void* v_rows, const void* k_gamma, float eps,
                      float rope_base, const int32_t* p0, int n, void* k_ring, void* v_ring,
                      int ring, int streams, int heads, int dim, int32_t* dev_status,
                      void* stream);

/*
 * tfd_sample - draw one token a row from its logits, given a random number u in [0, 1).
 *   For a row with logits l and w_i = exp((l_i - max l) / temperature):
 *     1. top_k keeps the top_k largest logits (<= 0 or >= n: all), ties to the lower (mapped) id;
 *     2. top_p keeps, in that order, every column before which the mass of the kept ones is below
 *        top_p times their total; the first always stays (>= 1: all; <= 0: the first alone);
 *     3. min_p keeps columns with w_i >= min_p (<= 0: all; >= 1: those equal to the largest).
 *   The token is the first column, in column order, at which the running mass of the kept columns
 *   exceeds u times their total. temperature 0 takes the largest logit (ties to the lower id).
 *   NaN and -inf logits, and weights below 2^-44 of the largest, have no mass; where logits are
 *   +inf, those share the mass. Positive temperatures below 1e-30 count as 1e-30. A row without any
 *   mass gets id -1 and probability 0.
 *   Masses are summed as integers (multiples of 2^-43 of the largest weight), so a row's token
 *   does not depend on the other rows, the launch or the order of the sums. The pages take the
 *   round's draws as inputs; this call makes them, and has no counterpart there.
 * Args:
 *   logits   device bf16 or float (lfmt TFD_X_BF16, TFD_X_F32) [rows][ld], ld >= n; any
 *            element-aligned base and stride; rows >= 1, 1 <= n <= TFD_MAX_DRAW_COLS.
 *   temperature, top_p, min_p device float [rows], top_k device int32 [rows]; each may be NULL
 *            (1, 1, 0 and 0). u device float [rows]; mind that a double from 1 - 2^-25 on is 1 as a
 *            float.
 *   id_map   device int32 [n] or NULL: the id reported (and compared on ties) for column i. Ids
 *            differ: of columns with the same logit and the same id, top_k and top_p keep all or none.
 *   ids      device int32, row r at ids[r * ldt] (ldt 0 = 1), so that the tokens of one step can
 *            land in a column of a [streams][steps] array; prob device float or NULL, the same
 *            stride: the token's probability in the filtered distribution, to 2^-20 relative.
 *   probs    device float [rows][ldp] or NULL, ldp >= n: the filtered, normalised distribution by
 *            column (written in full, zeros where nothing is kept).
 *   The outputs' ranges (strides included) overlap no input: TFD_ERR_INVALID.
 *   A negative, infinite or NaN temperature, a NaN top_p or min_p, or a u outside [0, 1) sets
 *   TFD_ERR_DEVICE_DATA; that row gets id -1, probability 0 and a distribution of zeros.
 */
tfd_status tfd_sample(const void* logits, int lfmt, int rows, int64_t n, int64_t ld,
                      const float* temperature, const int32_t* top_k, const float* top_p,
                      const float* min_p, const float* u, const int32_t* id_map, int32_t* ids,
                      float* prob, int64_t ldt, float* probs, int64_t ldp, int32_t* dev_status,
                      void* stream);

/*
 * tfd_accept_sampled - the rejection accept of drafts that were drawn from q, and the next token.
 *   Beside tfd_accept, which keeps drafts equal to the round's draws: here draft t of stream s is
 *   kept when all before it are, t < n_asked[s] and u[s][t] * q[s][t](d) < p[s][t](d) (decided
 *   without rounding). With m drafts kept, the next token is drawn with u_next[s] from
 *   max(p[s][m] - q[s][m], 0) when a draft was turned down (from p[s][m] where that is zero
 *   everywhere), else from p[s][m], m = n_asked[s]; "drawn" as in tfd_sample: the first column at
 *   which the running mass exceeds u_next times the total. Kept drafts and next token are then
 *   distributed as if drawn from p. Probabilities are clamped to 0..1, NaN to 0, and summed as
 *   integer multiples of 2^-43; one-hot rows (temperature 0) make this the greedy accept. A
 *   stream whose p row has no mass gets next token -1 and probability 0.
 * Args:
 *   p        device float [streams][win + 1][ldp], ldp >= n: the target's distributions at the
 *            win drafts' positions and the one after; only rows 0..n_asked[s] are read.
 *   q        device float [streams][win][ldq], ldq >= nq: the distributions the drafts were drawn
 *            from. nq == n when q_map is NULL.
 *   q_map    device int32 [n] or NULL: the column of q of token i, or -1 where the draft head
 *            does not have it (q = 0): the inverse of a subset head's id map.
 *   drafts   device int32 [streams][win], token ids in [0, n); n_asked device int32 [streams];
 *   u        device float [streams][win]; u_next device float [streams]; all in [0, 1).
 *   n_kept, next_ids device int32 [streams]; next_prob device float [streams] or NULL: the next
 *            token's probability in the distribution it was drawn from.
 *   asked_hist, kept_hist device int64 [win] or NULL (both or neither), accumulated as in
 *            tfd_accept. streams >= 1; win 1..512; n, nq <= TFD_MAX_DRAW_COLS. p and q at
 *            any element-aligned base and row stride. Outputs overlap no input.
 *   An n_asked outside [0, win], an asked draft outside [0, n), or a u outside [0, 1) sets
 *   TFD_ERR_DEVICE_DATA; that stream keeps 0, gets next token -1 and adds nothing.
 */
tfd_status tfd_accept_sampled(const float* p, int64_t ldp, const float* q, int64_t ldq, int64_t n,
                              int64_t nq, const int32_t* q_map, const int32_t* drafts,
                              const int32_t* n_asked, const float* u, const float* u_next,
                              int streams, int win, int32_t* n_kept, int32_t* next_ids,
                              float* next_prob, int64_t* asked_hist, int64_t* kept_hist,
                              int32_t* dev_status, void* stream);

/*
 * tfd_lora - low-rank adapters of many requests at once, beside a projection they share.
 *   y[r] = base[r] + scales[a] * B[a] (A[a] x[r]) with a = adapter_ids[r]: the base is the shared
 *   projection's result (tfd_head_gemv's y), in place or not. Sums in fp32; h = scales[a] * A[a] x[r]
 *   in fp32 enters its product with B[a] with all its 24 bits where y is float, and to within 2^-17
 *   of its value where y is bf16 (that shows only where base nearly cancels the adapter's term);
 *   y is rounded once. An infinite activation or h gives what the formula gives; the adapters
 *   themselves are finite (else y is infinite or NaN in the outputs they reach). Rows may name adapters in any order and share them; -1 is no adapter
 *   (y[r] = base[r]). One row up to whole prompts. The pages run one set of weights for all
 *   streams; this call has no counterpart there.
 * Args:
 *   x        device bf16 [rows][ldx], ldx >= k, ldx % 8 == 0; rows 1..TFD_MAX_LORA_ROWS.
 *   a_w, b_w device bf16 [n_adapters][rank][k] and [n_adapters][n][rank]; k >= 8, k % 8 == 0;
 *            rank 8..TFD_MAX_RANK, rank % 8 == 0 (smaller ones padded with zeros); n >= 1;
 *            n_adapters 1..4096. x, a_w and b_w 16-byte aligned.
 *   adapter_ids device int32 [rows]; any other id outside [0, n_adapters) sets
 *            TFD_ERR_DEVICE_DATA and counts as -1. scales device float [n_adapters] or NULL (1).
 *   out_mode TFD_OUT_F32 or TFD_OUT_BF16: the type of base and y.
 *   base     device [rows][ldb], ldb >= n, or NULL (zeros); y device [rows][ldy], ldy >= n: any
 *            element-aligned base and stride (16-byte aligned rows are faster). y may be base
 *            itself (same stride); it overlaps nothing else the call reads.
 *   dev_status also takes TFD_ERR_TIMEOUT: tiles of many rows wait, bounded to about a second, for
 *            their own matrix products; outputs are then undefined.
 */
tfd_status tfd_lora(const void* x, int rows, int64_t k, int64_t ldx, const void* a_w,
                    const void* b_w, int n_adapters, int rank, int64_t n,
                    const int32_t* adapter_ids, const float* scales, int out_mode,
                    const void* base, int64_t ldb, void* y, int64_t ldy, int32_t* dev_status,
                    void* stream);

/*
 * A paged key-value cache: tokens stand in pages of page_size, and a request's tokens 0, 1, 2, ... in
 * the pages that its row of a page table names, in order. The pages' rings have one run of slots a
 * stream (tfd_window_attn, tfd_absorb); a paged cache has no counterpart there.
 *   k, v      device [pages][page_size][heads][dim], the same strides (in elements) for both; bf16, or
 *             E4M3 codes. Elements of a vector adjoin; the strides are multiples of 16 bytes, in any
 *             order ([page][head][token] as well), k and v 16-byte aligned.
 *   k_scales, v_scales device float [pages][heads][page_size] (E4M3 only, else NULL): a vector is its
 *             codes times its scale. Tokens have no NaN codes (0x7F, 0xFF).
 * A slot is page * page_size + the token's place in the page; pages * page_size < 2^31. page_size
 * 1..TFD_MAX_PAGE; heads 1..1024; dim 64 or 128 (others: TFD_ERR_UNSUPPORTED).
 */
typedef enum { TFD_KV_BF16 = 0, TFD_KV_E4M3 = 1 } tfd_kvfmt;
typedef struct {
  void* k;
  void* v;
  float* k_scales;
  float* v_scales;
  int64_t page_stride, token_stride, head_stride;
  int32_t pages, page_size, heads, dim, fmt;
} tfd_kv_pages;

/* What a call does to query and key vectors: RMSNorm of each head, then RoPE (see tfd_window_attn). */
#define TFD_QK_NORM 1
#define TFD_QK_ROPE 2

/*
 * tfd_page_plan - page tables and slot maps of a round, from the requests' lengths.
 *   Request r has lens[r] tokens cached and gets n_new[r] rows this round: it is given pages, or gives
 *   pages back, so that it holds ceil((lens[r] + n_new[r]) / page_size) of them. So the call that
 *   plans a round also returns what the last round's turned-down drafts took, and lens = n_new = 0
 *   returns all of a request. The free pages are a stack free_ids[0 .. *n_free): pages given back go
 *   on it, then missing ones come from its top, both in the order of requests and of their pages; of
 *   the pages given back the first ends on top, so that pages taken by one call and given back by
 *   the next leave the stack as it was. Lengths can stay on the GPU from round to round.
 *   row_start[r] = n_new[0] + .. + n_new[r - 1] (requests + 1 values); for row i = row_start[r] + j:
 *   pos[i] = lens[r] + j, slots[i] = the slot of that token. Rows from row_start[requests] to
 *   `rows` get slot and position -1.
 * Args:
 *   lens, n_new device int32 [requests]; requests 1..TFD_MAX_REQUESTS; page_size 1..TFD_MAX_PAGE.
 *   table    device int32 [requests][ldt], ldt >= max_pages >= 1, requests * max_pages < 2^31:
 *            entries up to held[r] are the request's pages; entries behind what it then holds are
 *            left as they were.
 *   held     device int32 [requests], in and out. free_ids device int32 [pages], n_free device int32,
 *            in and out; pages >= 1 is the number of the cache's pages.
 *   row_start device int32 [requests + 1]; slots, pos device int32 [rows], or both NULL (rows 0).
 *   No array overlaps another.
 *   TFD_ERR_DEVICE_DATA: a negative length or count, a held count outside [0, max_pages] or a
 *   request that needs more than max_pages (it keeps its pages, its rows get slot and position -1; a
 *   negative count counts as 0); pages that run out (a request whose missing pages, counted with
 *   those of the requests before it, exceed the free ones gets none: it keeps what it holds, the
 *   table entries of the missing pages and its rows' slots and positions become -1); an n_free
 *   outside [0, pages], or more pages given back than the stack has room for (no page moves); a page
 *   id outside [0, pages) (slot -1; one that a request gives back is left out of the stack); more rows than
 *   `rows` (those are not written).
 */
tfd_status tfd_page_plan(const int32_t* lens, const int32_t* n_new, int requests, int page_size,
                         int32_t* table, int64_t ldt, int max_pages, int32_t* held,
                         int32_t* free_ids, int pages, int32_t* n_free, int32_t* row_start,
                         int32_t* slots, int32_t* pos, int64_t rows, int32_t* dev_status,
                         void* stream);

/*
 * tfd_paged_append - write rows of keys and values into their slots of a paged cache.
 *   Beside tfd_absorb, which writes a span into each stream's ring. For row i and head h:
 *     k' = rope(rmsnorm(k_rows[i][h]) * k_gamma, pos[i]), each step as `qk` names it;
 *     bf16: the cache takes bf16(k') and v_rows[i][h]; E4M3: s = fl32(amax / 448) and
 *     e4m3_rne_sat(fl32(x / s)) of k' (not rounded to bf16 before) and of v_rows[i][h] (amax 0
 *     keeps its zeros).
 *   The normalisation is that of tfd_window_attn, and so is the rotation's angle; its sine and cosine are the
 *   hardware's, within 2^-20.5 (tfd_window_attn and tfd_absorb: fp32 functions, within 2^-23), so keys of the two
 *   may round to neighbouring values.
 * Args:
 *   k_rows, v_rows device bf16 [rows][heads][dim], row strides ldk, ldv >= heads * dim, multiples
 *            of 8, 16-byte aligned; rows >= 1, rows * heads < 2^31.
 *   slots    device int32 [rows]: -1 leaves the row out; the others differ. Any other slot outside
 *            the cache, or a negative position (with TFD_QK_ROPE), sets TFD_ERR_DEVICE_DATA and the
 *            row is left out.
 *   pos      device int32 [rows] (may be NULL without TFD_QK_ROPE); k_gamma device bf16 [dim] or NULL
 *            (ones). E4M3 wants finite rows. The cache overlaps no input.
 */
tfd_status tfd_paged_append(const void* k_rows, int64_t ldk, const void* v_rows, int64_t ldv,
                            const int32_t* slots, const int32_t* pos, int rows, int qk,
                            const void* k_gamma, float eps, float rope_base,
                            const tfd_kv_pages* cache, int32_t* dev_status, void* stream);

/*
 * tfd_paged_attn - attention of each request's new rows (1 for a decode step, up to 32 for a verify
 *   window) over its tokens in a paged cache, the new rows' own among them (append them first).
 *   Request r has rows row_start[r] .. row_start[r + 1] - 1 of q, and lens[r] tokens before them; the
 *   token of its row j is lens[r] + j. Query head h reads key head h / (q_heads / heads):
 *     q' = rope(rmsnorm(q) * q_gamma, p), each step as `qk` names it;
 *     out = softmax(scale * q' . k) . v over the tokens that the row sees; lse = ln sum exp(scale *
 *     q' . k) over them.
 *   A row sees the tokens before the new ones, and of the new ones those up to itself; with `tree`
 *   those whose bit its word has set instead (bit j: row j; bits past the rows say nothing). With
 *   window >= 0 only tokens at depth >= its own - window: a cached token's depth is its number, a new
 *   row's lens[r] + j, or with `tree` lens[r] + (bits set in its word) - 1. A row that sees nothing
 *   gets zeros and an lse of -inf. What a row does not see (pages not in use, tokens behind the
 *   last, masked ones) may hold anything, NaN too. Tokens before lens[r] - window (with `tree` before
 *   lens[r] - window - 1) are not read and need no pages: their table entries may hold anything (those of the
 *   last 127 such tokens may be read, and the E4M3 scales of a page that one names, and say nothing). Of E4M3
 *   the codes from there on are not NaN.
 *   An infinite value that a row sees makes its output infinite as the formula says (NaN where both signs
 *   meet); one whose weight is below 2^-126 of the row's largest makes it infinite or NaN.
 *   A key with infinite elements likewise: a score of -inf has no weight, and one of +inf, or NaN, makes the row
 *   and its lse NaN. A row whose scores are all -inf gets zeros and -inf.
 *   Sums and softmax statistics in fp32, sines and cosines within 2^-20.5. q' enters its products as two bf16
 *   parts (E4M3: four 8-bit parts), within 2^-16 of it; probabilities as two bf16 parts, within 2^-16. E4M3: a
 *   probability times its value's scale as f16, within 2^-11 of it or 2^-29 of the row's largest (scales below
 *   2^-96 lose more); a scale above 2^80, or NaN, makes the rows that see its token, and their lse, NaN.
 * Args:
 *   q        device bf16 [rows][q_heads][dim], row stride ldq >= q_heads * dim, a multiple of 8,
 *            16-byte aligned; q_heads a multiple of the cache's heads, at most 64 times as many.
 *   table    device int32 [requests][ldt], ldt >= max_pages; lens device int32 [requests]; row_start
 *            device int32 [requests + 1], from 0 to at most rows; max_new: no request has more rows,
 *            1..TFD_MAX_ROWS.
 *   pos      device int32 [rows] or NULL (the rows' depths): positions for TFD_QK_ROPE.
 *   tree     device int32 [rows] (32 bits) or NULL. window -1 or >= 0. scale > 0, or 0 for
 *            1 / sqrt(dim).
 *   q_gamma  device bf16 [dim] or NULL (ones).
 *   out      device bf16 [rows][ldo], ldo >= q_heads * dim, a multiple of 8, 16-byte aligned; lse
 *            device float [rows][q_heads] or NULL. Rows of no request are left as they were. Outputs
 *            overlap no input.
 *   ws       device workspace of tfd_paged_attn_workspace() bytes.
 *   dev_status also takes TFD_ERR_TIMEOUT: the parts of a block wait for each other, bounded to
 *            about a second; outputs are then undefined, and ws is zero-filled before its next use.
 *   TFD_ERR_DEVICE_DATA: a request whose length is negative, whose tokens exceed max_pages or 2^31 -
 *   1025, or whose rows are not 0..max_new rows within `rows` (its rows are left as they were); a
 *   page id outside [0, pages) where a token is read (those tokens are not seen); a negative
 *   position (counts as 0; positions that no rotation uses are not read).
 *   TFD_ERR_UNSUPPORTED: strides of the cache, or rows * q_heads, from 2^31 on; ldq or ldo above 2^30.
 */
size_t tfd_paged_attn_workspace(int max_new, int q_heads, int heads, int dim);
tfd_status tfd_paged_attn(const void* q, int64_t ldq, int rows, int q_heads,
                          const tfd_kv_pages* cache, const int32_t* table, int64_t ldt,
                          int max_pages, const int32_t* lens, const int32_t* row_start,
                          int requests, int max_new, const int32_t* pos, const int32_t* tree,
                          int window, int qk, const void* q_gamma, float eps, float rope_base,
                          float scale, void* out, int64_t ldo, float* lse, void* ws,
                          size_t ws_bytes, int32_t* dev_status, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* TFD_H_ */
