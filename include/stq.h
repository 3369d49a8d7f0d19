/*
 * stq.h -- C ABI of libstq, the STQ1_0 sparse-ternary quantized matmul for
 * AMD Instinct MI355X (gfx950).
 *
 * STQ1_0 (sources named by page title / address and section):
 *   - every group of four consecutive weights holds values in {-d, 0, +d} with
 *     exactly one zero lane: 4 zero positions x 8 sign choices = 32 patterns,
 *     five bits per group (lemmy.durstig.online post 66506, paragraph "Four
 *     weights, five bits");
 *   - the five bits are a 4-bit code plus a 1-bit table select into a
 *     32-entry codebook, one fp16 scale d is shared by 256 weights, and a block
 *     of 256 weights takes 42 bytes, 1.3125 bits per weight (alphasignal.ai,
 *     "AngelSlim Shrinks Tencent's 1.5TB Hy4-Preview ...", section "How STQ1_0
 *     works").
 *
 * Block layout (this library's definition; the pages fix only the size):
 *   bytes  0..1   d, IEEE binary16, little-endian
 *   bytes  2..33  4-bit codes: group g (0..63) in byte 2 + 4*(g>>3) + (g&3),
 *                 low nibble when bit 2 of g is clear, high nibble otherwise
 *   bytes 34..41  select bits: group g's bit is bit ((g>>2)&7) of byte
 *                 34 + 4*(g>>5) + (g&3)
 *   code c = nibble | select<<4;  zero lane z = c>>3;  m = c&7; the three
 *   other lanes in increasing order take -1 when their bit of m is set
 *   (lowest lane -> bit 0), else +1.  Decoded weight = +/-fp32(d), or +0.0
 *   in the zero lane.
 * Matrix layout (also this library's): a matrix of n rows and k columns (k a
 * multiple of 256) holds n*k/256 blocks, block b of a row covering columns
 * 256b..256b+255, n*row_bytes(k) bytes in all.  Rows are grouped in tiles of
 * 64 consecutive rows (the last tile holds the n % 64 leftover rows, if any);
 * a tile stores block 0 of each of its rows in row order, then block 1 of
 * each, and so on.  Block b of row r of a matrix starting at byte 0 is at
 *   (t*nb + b*rows_in_tile + (r - t)) * 42,   t = r - r % 64,
 *   rows_in_tile = min(64, n - t),            nb = k / 256.
 * So the 64 rows' block b of a full tile is one contiguous 2688-byte run.
 *
 * Conventions for every entry point:
 *   - array arguments are DEVICE pointers owned by the caller, unless stated;
 *   - work is enqueued on `stream` (0 = the null stream) and is asynchronous:
 *     no entry point synchronises the host;
 *   - arguments are validated on the host before any launch; a failed check
 *     returns a status and stq_last_error() holds a message (thread-local);
 *   - STQ_E_HIP means a HIP call (a launch) failed; device faults surface at
 *     the caller's next synchronisation;
 *   - the library allocates no device memory and keeps no device state: the
 *     entry points that need scratch memory (stq_gemv, stq_moe_ffn_decode,
 *     stq_layer_errors, stq_grouped_swiglu, stq_grouped_swiglu_backward,
 *     stq_token_logprobs, stq_rmsnorm_rows_backward, stq_route_tokens,
 *     stq_head_cross_entropy, stq_head_cross_entropy_backward) take a caller-owned `workspace` of `workspace_bytes`
 *     bytes, 256-byte aligned, whose required size a host-only query gives
 *     for the same shapes (stq_gemv_plan, and the call's name with _workspace
 *     behind it for the others: stq_moe_ffn_workspace for the FFN); a NULL or
 *     smaller workspace is refused with STQ_E_ARG before any launch.  The workspace is in use until the
 *     call's work on `stream` completes, so calls that run concurrently need
 *     workspaces of their own; its contents between calls are meaningless;
 *   - apart from the thread-local error text the entry points are stateless
 *     and may be called from any number of host threads.
 */
#ifndef STQ_H
#define STQ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct ihipStream_t;
typedef struct ihipStream_t* stq_stream_t; /* same object as a hipStream_t */

#define STQ_QK 256          /* weights per block */
#define STQ_BLOCK_BYTES 42  /* bytes per block   */

typedef enum {
  STQ_OK = 0,
  STQ_E_ARG = 1,   /* null pointer, bad enum, negative count               */
  STQ_E_SHAPE = 2, /* k not a multiple of 256, sizes inconsistent           */
  STQ_E_ALIGN = 3, /* pointer or stride misaligned                          */
  STQ_E_HIP = 4    /* a HIP runtime call failed                             */
} stq_status;

enum { STQ_ENC_WLS = 0, STQ_ENC_AMAX = 1 };
enum { STQ_X_F32 = 0, STQ_X_BF16 = 1 };
enum { STQ_X_I8 = 2 }; /* 8-bit rows with scales: the output head's operands only */

/* Bytes of one packed row of k weights: k/256*42, or -1 if k is not a
 * positive multiple of 256. Pure host function. */
int64_t stq_row_bytes(int64_t k);

/* Encode fp32 rows into STQ1_0 (weighted least squares scale alternating
 * with an importance-weighted choice of the zero lane; lemmy post 66506,
 * paragraph "Scale and zero position are fit together"; amax baseline from
 * the alphasignal.ai summary bullets).
 *   w        [n_rows, k] fp32, row-major, 4-byte aligned, finite values
 *   imatrix  [k] fp32 >= 0, per-column importance; NULL means all ones
 *   encoder  STQ_ENC_WLS: start from the amax pattern (zero the smallest |w|
 *              of each group, signs of w); `rounds` times fit d by weighted
 *              least squares then re-choose every group's zero lane by least
 *              added weighted error q_j*(2|w_j|-d) (lowest lane on ties);
 *              a final fit gives the stored d.
 *            STQ_ENC_AMAX: d = block max |w|, smallest |w| zeroed; `rounds`
 *              ignored.
 *   rounds   >= 0 (3 is the pages' setting)
 *   out      packed matrix, n_rows*k/256*42 bytes (layout above)
 * Sums run in fp64 in a fixed order (lanes of a group in order, then a
 * balanced tree of adjacent groups); d is stored as fp16 via fp32
 * (round-to-nearest-even both times, clamped to 65504).  These rules fix
 * every output byte: any implementation that follows them gives the same
 * bytes.  Non-finite inputs are outside the contract (output unspecified). */
stq_status stq_quantize_rows(const float* w, const float* imatrix, int64_t n_rows, int64_t k,
                             int encoder, int rounds, uint8_t* out, stq_stream_t stream);

/* Decode a packed matrix to fp32: out[r, i] = +/-fp32(d) or +0.0 (bit-exact),
 * the weights the format stands for (every weight of a group is -d, 0 or +d
 * with one zero per group of four, d the block's fp16 scale: lemmy post
 * 66506, paragraph "Four weights, five bits").
 *   q    packed matrix of n_rows rows (layout above), 2-byte aligned
 *   out  [n_rows, k] fp32, row-major */
stq_status stq_dequantize_rows(const uint8_t* q, int64_t n_rows, int64_t k, float* out,
                               stq_stream_t stream);

/* Gathered decode GEMV over (token, expert) pairs, the STQ1_0 matmul of the
 * decode path (lemmy post 66506, paragraph "Runtime": STQ1_0 kernels run the
 * expert projections; each token reaches the top 8 of 256 routed experts,
 * traictory.com "Tencent's 200GB Hy4-preview ...", section "The claim,
 * stated precisely").
 *   w_table   expert e's packed n x k matrix starts at w_table + e*expert_stride_bytes;
 *             w_table 16-byte aligned, expert_stride_bytes a multiple of 16 and
 *             >= n*row_bytes(k)
 *   x         activations [n_tokens, k] with row stride x_row_stride elements,
 *             fp32 (STQ_X_F32, 4-byte aligned) or bf16 bits (STQ_X_BF16,
 *             x_row_stride even, 4-byte aligned rows)
 *   pair_expert, pair_token  int32 [n_pairs]; pair i computes
 *             y[i, :] = W_{pair_expert[i]} x[pair_token[i], :].
 *             NULL pair_expert means expert 0 for every pair; NULL pair_token
 *             means token i for pair i.  Pairs sharing an expert are batched so
 *             the expert's weights stream once per call.  A pair whose expert
 *             is outside [0, n_experts) or whose token is outside
 *             [0, n_tokens) gets a row of NaN.
 *   y         [n_pairs, n] fp32
 *   workspace, workspace_bytes  caller-owned scratch for split outputs, at
 *             least the scratch_bytes stq_gemv_plan reports for these shapes
 *             on this stream's device (may be NULL when that is 0)
 * Accumulation is fp32 with products exact; the summation order is fixed,
 * so repeated calls give identical bits.  The k split, and the parting of an
 * expert with several tokens into up to one k range per token, are chosen
 * per call from the shapes and the CU count of the device `stream` runs on;
 * the environment variable STQ_GEMV_PLAN="s,p" (1 <= s <= k/256 splits,
 * 1 <= p <= 8 parts) replaces that choice, for tuning and tests.  Results
 * meet the same tolerance under every plan; their bits depend on the plan
 * and on the pass form (with bf16 rows and at least as many pairs as
 * experts, a pass of 3 or more tokens runs on the matrix cores), so the same
 * bits on devices of different sizes need the same plan (STQ_GEMV_PLAN). */
stq_status stq_gemv(const uint8_t* w_table, int64_t expert_stride_bytes, int64_t n_experts,
                    int64_t n, int64_t k, const void* x, int x_dtype, int64_t x_row_stride,
                    int64_t n_tokens, const int32_t* pair_expert, const int32_t* pair_token,
                    int64_t n_pairs, float* y, void* workspace, int64_t workspace_bytes,
                    stq_stream_t stream);

/* stq_gemv for callers that cannot allocate memory or pass a workspace (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation).  Same arguments, checks, plan and results as stq_gemv (bit for
 * bit), without workspace: split outputs go to a fixed scratch array that the
 * library holds on every GPU it runs on, STQ_GEMV_NOALLOC_SCRATCH_BYTES
 * bytes, from the library's load until the process ends.  Shapes whose plan
 * (stq_gemv_plan's scratch_bytes) needs more are refused with STQ_E_SHAPE
 * before any launch.  Every call on one GPU shares that GPU's array, so calls
 * that may run concurrently on one GPU (two streams, two host threads) race
 * and must not overlap; nothing in the array needs to be cleared between
 * calls (every value a call reads was written earlier in the same call).
 * Allocates nothing; the first call on a device looks up that device's copy
 * of the array (STQ_E_HIP if that fails). */
#define STQ_GEMV_NOALLOC_SCRATCH_BYTES (32ll << 20)
stq_status stq_gemv_noalloc(const uint8_t* w_table, int64_t expert_stride_bytes, int64_t n_experts,
                            int64_t n, int64_t k, const void* x, int x_dtype, int64_t x_row_stride,
                            int64_t n_tokens, const int32_t* pair_expert, const int32_t* pair_token,
                            int64_t n_pairs, float* y, stq_stream_t stream);

/* The plan stq_gemv takes for these shapes (host only: no GPU work, and no
 * GPU needed when n_cus > 0), so a caller can size its workspace or check a
 * tuning override.  The three outputs are HOST
 * pointers; all must be non-NULL (STQ_E_ARG otherwise).
 *   n_experts, n, k, n_pairs  as for stq_gemv (same checks, same errors)
 *   n_cus        compute units to plan for; 0 = the current device's (256
 *                when no device answers)
 *   splits       out: ranges the k blocks of a row are split into
 *   max_parts    out: most k parts one split is cut into for an expert with
 *                several tokens (an expert with m pairs takes min(m, max_parts))
 *   scratch_bytes  out: workspace bytes the call needs (0 when nothing is split)
 * STQ_GEMV_PLAN is honoured as in stq_gemv.  n_pairs == 0 or n == 0 gives
 * (1, 1, 0): stq_gemv launches nothing then. */
stq_status stq_gemv_plan(int64_t n_experts, int64_t n, int64_t k, int64_t n_pairs, int32_t n_cus,
                         int32_t* splits, int32_t* max_parts, int64_t* scratch_bytes);

/* Routed-expert FFN of one MoE layer for a batch of decode tokens, its
 * expert projections in STQ1_0 (lemmy post 66506, paragraph "Runtime": the
 * routed experts' projections run through STQ1_0 kernels; routing top-k of
 * the routed experts, traictory.com "Tencent's 200GB Hy4-preview ...",
 * section "The claim, stated precisely").  For token t and its pairs
 * p = t*top_k + k, k = 0..top_k-1, with e = pair_expert[p]:
 *     g, u  = rows [0, d_ff) and [d_ff, 2*d_ff) of W_gate_up[e] x_t
 *     h     = silu(g) * u,          silu(v) = v / (1 + exp(-v))   (fp32)
 *     z_p   = W_down[e] h
 *     y[t]  = sum over k, in order, of pair_weight[p] * z_p        (fp32)
 *   w_gate_up  expert e's packed [2*d_ff, d_model] matrix (gate rows, then up
 *              rows) at w_gate_up + e*gate_up_stride_bytes
 *   w_down     expert e's packed [d_model, d_ff] matrix at w_down + e*down_stride_bytes
 *              (both 16-byte aligned, strides multiples of 16 and at least
 *              the packed matrix size; d_model, d_ff multiples of 256)
 *   x          bf16 bits [n_tokens, d_model], row-major
 *   pair_expert int32, pair_weight fp32 [n_tokens*top_k], token-major
 *   y          fp32 [n_tokens, d_model]
 *   workspace, workspace_bytes  caller-owned scratch, at least what
 *              stq_moe_ffn_workspace reports for these shapes on this
 *              stream's device: the pairs' gate/up rows, activations and down
 *              rows (fp32) plus the GEMVs' split outputs
 * Both projections run through the GEMV above (pairs sharing an expert are
 * batched), with h formed once per element between them.  A pair whose
 * expert is outside [0, n_experts) makes its token's row NaN.  At most 65535
 * pairs per call. */
stq_status stq_moe_ffn_decode(const uint8_t* w_gate_up, int64_t gate_up_stride_bytes, const uint8_t* w_down,
                              int64_t down_stride_bytes, int64_t n_experts, int64_t d_model, int64_t d_ff,
                              const uint16_t* x, int64_t n_tokens, const int32_t* pair_expert,
                              const float* pair_weight, int64_t top_k, float* y, void* workspace,
                              int64_t workspace_bytes, stq_stream_t stream);

/* Workspace bytes stq_moe_ffn_decode needs for these shapes on a device with
 * n_cus compute units (0: the current device's); host only, same checks and
 * errors as the call.  workspace_bytes is a HOST pointer; 0 when n_tokens is 0. */
stq_status stq_moe_ffn_workspace(int64_t n_experts, int64_t d_model, int64_t d_ff, int64_t n_tokens,
                                 int64_t top_k, int32_t n_cus, int64_t* workspace_bytes);

/* Grouped GEMM of the prefill path: tokens routed to each expert,
 * grouped by expert, times that expert's STQ1_0 matrix (lemmy post 66506,
 * paragraph "Runtime": STQ1_0 kernels run the routed experts' projections;
 * each token reaches the top 8 of 256 routed experts, traictory.com
 * "Tencent's 200GB Hy4-preview ...", section "The claim, stated precisely",
 * so a prompt's tokens form one dense product per expert).
 *   x_sorted        [total_m, k] bf16 bits, row-major, 16-byte aligned rows
 *                   (k*2 bytes apart)
 *   expert_offsets  DEVICE int32 [n_experts+1], non-decreasing, offsets[0] = 0,
 *                   offsets[n_experts] = total_m: rows offsets[e]..offsets[e+1]-1
 *                   belong to expert e
 *   y               [total_m, n] fp32: y[r, :] = W_e x_sorted[r, :]
 * bf16 x ternary products on matrix cores (exact), fp32 accumulation, one
 * fp32 multiply by d per 256-weight block.  Offsets that break the stated
 * invariants are outside the contract, but the kernel clamps each expert's
 * rows to [0, total_m] (lo = clamp(offsets[e]), hi = clamp(offsets[e+1])
 * and at least lo), so x_sorted and y are never accessed outside their
 * total_m rows: rows in no range are left unwritten and rows in two ranges
 * get either expert's result. */
stq_status stq_grouped_gemm(const uint8_t* w_table, int64_t expert_stride_bytes, int64_t n_experts,
                            int64_t n, int64_t k, const uint16_t* x_sorted,
                            const int32_t* expert_offsets, int64_t total_m, float* y,
                            stq_stream_t stream);

/* Reconstruction error of an approximation W_hat of W under calibration
 * activations, scored with the full Hessian H = X^T X and with its diagonal
 * alone, the two layer-sensitivity measures the pages compare (lemmy post
 * 66506, paragraph "Full-Hessian scoring": off-diagonal terms carry the
 * input correlations that a diagonal-only imatrix misses).  With
 * D = W - W_hat in fp64:
 *     err_full[r] = sum_i (D_r . x_i)^2      = D_r H D_r^T
 *     err_diag[r] = sum_c H_cc D_rc^2,        H_cc = sum_i x_ic^2
 *   w, w_hat   [n_rows, k] fp32, row-major, 16-byte aligned (w_hat is
 *              typically stq_dequantize_rows or stq_q2_roundtrip of w)
 *   x_calib    [n_calib, k] fp32 calibration activations, row-major,
 *              16-byte aligned; n_calib >= 1
 *   err_full, err_diag   [n_rows] fp64, 8-byte aligned
 * Products are exact (fp32 operands in fp64); D X^T accumulates in fp64 on
 * the matrix cores, so the results agree with an fp64 reference to within
 * the fp64 rounding of sums of k and n_calib terms.  The summation order is
 * fixed: repeated calls give identical bits.  Non-finite inputs give
 * non-finite outputs.
 *   workspace, workspace_bytes  caller-owned scratch of at least
 *              stq_layer_errors_workspace bytes: 8*(k + 2*ceil(n_calib/64)*n_rows)
 *              (the diagonal of H, then per-tile partial sums) */
stq_status stq_layer_errors(const float* w, const float* w_hat, int64_t n_rows, int64_t k,
                            const float* x_calib, int64_t n_calib, double* err_full, double* err_diag,
                            void* workspace, int64_t workspace_bytes, stq_stream_t stream);

/* Workspace bytes stq_layer_errors needs (host only; same checks and errors
 * as the call; 0 when n_rows is 0).  workspace_bytes is a HOST pointer. */
stq_status stq_layer_errors_workspace(int64_t n_rows, int64_t k, int64_t n_calib, int64_t* workspace_bytes);

/* Quantize-and-reconstruct through the plain 2-bit format this library uses
 * as the larger partner format of a per-layer allocation (the pages pair
 * STQ1_0 with IQ2_XXS at 2.0625 bits per weight, lemmy post 66506,
 * paragraph "Precision follows weight sensitivity", without defining it; a
 * stand-in of the same size takes its place: 66 bytes per 256 weights).
 * Per 256-weight block: ss = sum of w^2 in fp64 (the four weights of a
 * group in order, then a balanced tree of adjacent groups), s = fp16 of
 * sqrt(ss/256)/2 (fp64 -> fp32 -> fp16, round-to-nearest-even, clamped to
 * 65504); each weight becomes s if |w| < 2s, else 3s, with the sign bit of w.
 *   w, out  [n_rows, k] fp32, row-major, 16-byte aligned (may not overlap)
 * These rules fix every output bit.  Non-finite inputs give unspecified
 * (non-finite) outputs for their block. */
stq_status stq_q2_roundtrip(const float* w, int64_t n_rows, int64_t k, float* out, stq_stream_t stream);

/* Greedy per-byte allocation of the larger format over layers (lemmy post
 * 66506, paragraph "Full-Hessian scoring": layers are taken greedily by
 * error reduction per added byte).  Visit layers by gain/extra_bytes,
 * largest first (lowest index on ties); take a layer when its gain is > 0
 * and the added bytes still fit within `budget`, else skip it.
 *   gain, extra_bytes   HOST double [n_layers]; extra_bytes > 0
 *   chosen              HOST uint8 [n_layers], 1 for a layer taken
 * Pure host function. */
stq_status stq_greedy_allocation(const double* gain, const double* extra_bytes, int64_t n_layers,
                                 double budget, uint8_t* chosen);

/* Gated feed-forward of the prefill path: the gate and up products of every
 * token with its expert, the activation and their product in one pass, for
 * rows grouped by expert as in stq_grouped_gemm (same source passages):
 *     g, u = rows [0, d_ff) and [d_ff, 2*d_ff) of W_e x_r
 *     h[r] = silu(g) * u,          silu(v) = v / (1 + exp(-v))
 *   w_gate_up, gate_up_stride_bytes   the experts' packed [2*d_ff, d_model]
 *                   matrices (gate rows, then up rows) as in
 *                   stq_moe_ffn_decode: 16-byte aligned, stride a multiple of
 *                   16, d_model and d_ff multiples of 256
 *   x_sorted        [total_m, d_model] bf16 bits, row-major, 16-byte aligned
 *   expert_offsets  DEVICE int32 [n_experts+1] as in stq_grouped_gemm,
 *                   clamped the same way: rows in no range stay unwritten
 *   h               bf16 [total_m, d_ff], the down projection's input of
 *                   stq_grouped_gemm; 16-byte aligned
 *   gate_up         bf16 [total_m, 2*d_ff] = [g | u], what the backward pass
 *                   reads, or NULL; 16-byte aligned
 * bf16 x ternary products are exact, sums fp32, and h and gate_up are each
 * rounded from the fp32 sums once.  Sums may be held in units of the current
 * block's d (the change of unit rounds them once a block), so a row of W
 * should not have a d that is 3e38 times smaller than its sums.  An infinity
 * or a NaN in x makes its row's outputs NaN, or reaches them only through
 * weights that are not 0, depending on the form taken; other rows never see
 * it.  Few rows run through stq_gemv's kernels and need scratch:
 *   workspace, workspace_bytes   at least what stq_grouped_swiglu_workspace
 *                   reports for these shapes on this stream's device (may be
 *                   NULL when that is 0)
 * d_ff * row_bytes(d_model) is below 2^31, d_model at most 2^22 and d_ff 2^21;
 * n_experts is at most 65535, total_m 2^23, and with e = min(n_experts,
 * total_m) their passes, (e + (total_m - e) / 32 + 8) * (d_ff / 128), at most
 * 2^23 (an integer division); beyond: STQ_E_SHAPE.  Repeated
 * calls give identical bits; they depend on the form taken (and, through the
 * GEMV's plan, on the device), as stq_gemv's do. */
stq_status stq_grouped_swiglu(const uint8_t* w_gate_up, int64_t gate_up_stride_bytes, int64_t n_experts,
                              int64_t d_model, int64_t d_ff, const uint16_t* x_sorted, const int32_t* expert_offsets,
                              int64_t total_m, uint16_t* h, uint16_t* gate_up, void* workspace,
                              int64_t workspace_bytes, stq_stream_t stream);

/* Workspace bytes stq_grouped_swiglu needs for these shapes on a device with
 * n_cus compute units (0: the current device's); host only, same checks and
 * errors as the call.  workspace_bytes is a HOST pointer. */
stq_status stq_grouped_swiglu_workspace(int64_t n_experts, int64_t d_model, int64_t d_ff, int64_t total_m,
                                        int32_t n_cus, int64_t* workspace_bytes);

/* The form that stq_grouped_swiglu takes for these shapes on a device with
 * n_cus compute units (0: the current device's): rows_per_pass is the most rows
 * of an expert that a workgroup multiplies at a time, or 0 where the rows run
 * through stq_gemv's kernels (and where there are none).  The choice is made
 * for rows that spread evenly over the experts, since the offsets are on the
 * device: a call whose rows go to few of its experts is right all the same,
 * but may take many times as long as with n_experts (and the offsets) of
 * those alone, up to 1,650 us instead of 50 for 300 rows of one of 256 experts
 * of 2 x 2048 x 7168.  Host only, same checks and errors as the call.  rows_per_pass
 * is a HOST pointer. */
stq_status stq_grouped_swiglu_plan(int64_t n_experts, int64_t d_model, int64_t d_ff, int64_t total_m, int32_t n_cus,
                                   int32_t* rows_per_pass);

/* Its gradients: with s = 1 / (1 + exp(-g)) and dh the gradient at h,
 *     dg = dh u s (1 + g (1 - s)),   du = dh g s,   dz = [dg | du]
 *     dx[r] = dz_r W_e                 (through the decoded, frozen weights)
 *     dw[e] = sum over e's rows of dz_r^T x_r   (the gradient with respect to
 *             the decoded weights, e.g. for the weights behind an encoder)
 *   gate_up   bf16 [total_m, 2*d_ff], from the forward call; 16-byte aligned
 *   dh        bf16 [total_m, d_ff]; 16-byte aligned
 *   dx        bf16 [total_m, d_model] or NULL (not wanted); 8-byte aligned;
 *             rows in no range stay unwritten
 *   dw        bf16 [n_experts, 2*d_ff, d_model] or NULL; 16-byte aligned;
 *             every element is written (zeros for an expert without rows)
 *   w_gate_up is read for dx only and x_sorted for dw only; either may be
 *   NULL otherwise.  The other arguments are as for stq_grouped_swiglu.
 *   workspace, workspace_bytes   at least what
 *             stq_grouped_swiglu_backward_workspace reports
 * dz is formed in fp32 and rounded for each product: for dx to fp16 (after a
 * power-of-two scaling of each row) and, times a row of W's block scale, to
 * fp16 once more, so that the weights' patterns enter exactly; for dw to bf16.
 * fp16 keeps 11 bits down to 2^-28 of a row's largest |dz| (the product: of
 * that times twice the largest |d| in the 256-column block of W); what is
 * smaller errs by at most 2^-39 of it.  Sums are fp32 in a fixed order; dx and
 * dw are rounded from them once.  The limits on a matrix, n_experts and total_m
 * are the forward call's; beside them (e + (total_m - e) / 32 + 8) *
 * (d_model / 256) is at most 2^23 where dx is wanted, and n_experts *
 * (d_ff / 64) * (d_model / 128) where dw is. */
stq_status stq_grouped_swiglu_backward(const uint8_t* w_gate_up, int64_t gate_up_stride_bytes, int64_t n_experts,
                                       int64_t d_model, int64_t d_ff, const uint16_t* x_sorted,
                                       const int32_t* expert_offsets, int64_t total_m, const uint16_t* gate_up,
                                       const uint16_t* dh, uint16_t* dx, uint16_t* dw, void* workspace,
                                       int64_t workspace_bytes, stq_stream_t stream);

/* Workspace bytes stq_grouped_swiglu_backward needs for these shapes and the
 * outputs wanted (0 or 1 each); host only.  workspace_bytes is a HOST pointer. */
stq_status stq_grouped_swiglu_backward_workspace(int64_t n_experts, int64_t d_model, int64_t d_ff, int64_t total_m,
                                                 int want_dx, int want_dw, int64_t* workspace_bytes);

/* The same of stq_grouped_swiglu_backward's dx, whose rows all go in passes. */
stq_status stq_grouped_swiglu_backward_plan(int64_t n_experts, int64_t d_model, int64_t d_ff, int64_t total_m,
                                            int32_t n_cus, int32_t* rows_per_pass);

/* Rows of 8-bit integers with one fp32 scale each, the form in which a model
 * keeps what its allocation leaves above the ternary format (attention
 * projections, the output head; lemmy post 66506, paragraph "Precision
 * follows weight sensitivity") and in which the activations meet it.  Per row
 *     scale = fp32(max |x| / 127),  q = nearest integer to x / scale
 * (the exact quotient, halves to even, held to +-127); a row of zeros, or one
 * whose scale underflows to 0, gives scale 0 and q = 0; a row that holds a
 * NaN or an infinity gives scale NaN and q = 0, so that every product with it
 * is NaN.
 *   x      [n_rows, k] fp32 (STQ_X_F32) or bf16 bits (STQ_X_BF16), rows
 *          x_row_stride elements apart, aligned to its elements; rows that
 *          start on 16 bytes load faster
 *   q      int8, row r at q + r*q_row_stride, 16-byte aligned, q_row_stride a
 *          multiple of 16 and at least k rounded up to 16; the bytes from k
 *          up to that multiple are written 0, those behind it are left
 *   scale  [n_rows] fp32
 * k >= 1; at most 2^22 rows per call. */
stq_status stq_q8_quantize_rows(const void* x, int x_dtype, int64_t x_row_stride, int64_t n_rows, int64_t k,
                                int8_t* q, int64_t q_row_stride, float* scale, stq_stream_t stream);

/* Product of two sets of such rows:
 *     y[i, j] = (sum_c a[i, c] * w[j, c]) * a_scale[i] * w_scale[j]
 * with the sum exact (int32) and the scaling in fp32.
 *   a, a_scale   [m, k] int8 and [m] fp32: the tokens
 *   w, w_scale   [n, k] int8 and [n] fp32: the output channels
 *                both 16-byte aligned with row strides (bytes) that are
 *                multiples of 16, at least k rounded up to 16 and at most
 *                2^23; a row's bytes behind k, up to that multiple, may be
 *                read and count for nothing
 *   y            [m, n] fp32 (STQ_X_F32) or bf16 (STQ_X_BF16, one rounding of
 *                the fp32 value), rows y_row_stride elements apart; rows that
 *                all start on 16 bytes store faster
 * 1 <= k <= 131071 (any sum of products of bytes then fits 32 bits); m up to
 * 2^22, n up to 2^26, m * n up to 2^38.  Integer sums do not depend on their
 * order: a result's bits do not depend on m, n, the strides or the device. */
stq_status stq_q8_matmul(const int8_t* a, int64_t a_row_stride, const float* a_scale, const int8_t* w,
                         int64_t w_row_stride, const float* w_scale, int64_t m, int64_t n, int64_t k, void* y,
                         int y_dtype, int64_t y_row_stride, stq_stream_t stream);

/* Log probabilities of given tokens under rows of logits, with each row's
 * log-sum-exp, entropy and most likely alternatives: how a compressed model
 * is scored token by token against its original.  With p = softmax(l):
 *     lse = log sum_i exp(l_i)            logprob = l_target - lse
 *     entropy = -sum_i p_i log p_i        top: the top_n largest l_i
 *   logits    [n_rows, vocab] fp32 (STQ_X_F32) or bf16 bits (STQ_X_BF16), rows
 *             row_stride elements apart, aligned to its elements.  -inf masks
 *             an entry (p = 0).
 *   targets   int32 [n_rows]; outside [0, vocab): logprob NaN
 *   logprob   fp32 [n_rows];  lse, entropy  fp32 [n_rows] or NULL
 *   top_n     0..32, at most vocab
 *   top_ids, top_logprobs  int32 / fp32 [n_rows, top_n], most likely first,
 *             equal logits by lowest id (may be NULL when top_n is 0)
 *   workspace, workspace_bytes  scratch for rows that are split, at least
 *             what stq_token_logprobs_workspace reports (may be NULL when 0)
 * A row without a distribution gives NaN log probabilities and entropy and
 * ids -1: one that is masked throughout (lse = -inf) or that holds a NaN or a
 * +inf (lse = NaN).  Sums and maxima are fp32; the order of summation is fixed
 * for a device, so repeated calls give identical bits.  At most 2^22 rows of at
 * most 2^30 entries. */
stq_status stq_token_logprobs(const void* logits, int x_dtype, int64_t row_stride, int64_t n_rows, int64_t vocab,
                              const int32_t* targets, float* logprob, float* lse, float* entropy, int64_t top_n,
                              int32_t* top_ids, float* top_logprobs, void* workspace, int64_t workspace_bytes,
                              stq_stream_t stream);

/* Workspace bytes stq_token_logprobs needs for these shapes on a device with
 * n_cus compute units (0: the current device's); host only, same checks and
 * errors as the call.  workspace_bytes is a HOST pointer. */
stq_status stq_token_logprobs_workspace(int x_dtype, int64_t n_rows, int64_t vocab, int64_t top_n, int32_t n_cus,
                                        int64_t* workspace_bytes);

/* Gradient of stq_token_logprobs with respect to the logits, for gradients
 * that arrive at logprob and entropy (the alternatives carry none):
 *     d_i = g_logprob * (1[i = target] - p_i) - g_entropy * p_i * (log p_i + entropy)
 *   logits, x_dtype, row_stride, targets   as for the call above
 *   lse, entropy   fp32 [n_rows], what the call above gave (entropy may be
 *                  NULL when grad_entropy is)
 *   grad_logprob, grad_entropy   fp32 [n_rows]; either may be NULL (zeros)
 *   d_logits       [n_rows, vocab], the logits' type, rows d_row_stride
 *                  elements apart; may be the logits themselves (same pointer
 *                  and stride), else it may not overlap them
 * A target outside [0, vocab) takes no grad_logprob; a row with lse = -inf
 * gives zeros, one with lse = NaN gives NaN.  At most 2^22 rows, and less than
 * 2^24 started pieces of 32 KB of a row in all (logits of more than 400 GB). */
stq_status stq_token_logprobs_backward(const void* logits, int x_dtype, int64_t row_stride, int64_t n_rows,
                                       int64_t vocab, const int32_t* targets, const float* lse, const float* entropy,
                                       const float* grad_logprob, const float* grad_entropy, void* d_logits,
                                       int64_t d_row_stride, stq_stream_t stream);

/* Residual addition, root-mean-square norm and 8-bit rows in one pass: what
 * stands between the residual stream and the projections that
 * stq_q8_quantize_rows and stq_q8_matmul serve, the router and the experts.
 *     h = x + residual, rounded to the residual's type (h = x without one)
 *     rstd = 1 / sqrt(mean h^2 + eps)
 *     v = h * weight (one fp32 rounding),  step = fp32(max |v| / 127)
 *     q = nearest integer to v / step (the exact quotient, halves to even),
 *     scale = step * rstd,   y = v * rstd
 * so that q * scale stands for y, and q does not depend on the order of the
 * sum.  A row of zeros, or one whose step underflows to 0, gives scale 0 and q
 * = 0; a row with a NaN or an infinity in v gives scale NaN and q = 0.  A row
 * whose sum of squares passes fp32's range has rstd 0, one whose sum is 0 there
 * rstd 1 / sqrt(eps): infinite for eps 0, and its y not finite.
 *   x          [n_rows, d] fp32 (STQ_X_F32) or bf16 bits (STQ_X_BF16), rows
 *              x_row_stride elements apart
 *   residual   [n_rows, d] likewise, or NULL
 *   h          [n_rows, d] of the residual's type; may be the residual, or x
 *              where the types are the same, with the same stride; read and
 *              written only with a residual
 *   weight     fp32 [d]
 *   rstd       fp32 [n_rows] or NULL
 *   q, scale   int8 rows as stq_q8_quantize_rows writes them (16-byte aligned,
 *              q_row_stride bytes apart, a multiple of 16 and at least d
 *              rounded up to 16; bytes from d up to that multiple are written
 *              0), and fp32 [n_rows]; both or neither
 *   y          bf16 bits [n_rows, d], rows y_row_stride elements apart, one
 *              rounding of the fp32 value, or NULL
 * Every pointer is aligned to its elements.  Sums are fp32 in a fixed order:
 * repeated calls give identical bits.  d >= 1; at most 2^22 rows and 2^26
 * columns. */
stq_status stq_rmsnorm_rows(const void* x, int x_dtype, int64_t x_row_stride, const void* residual,
                            int residual_dtype, int64_t residual_row_stride, void* h, int64_t h_row_stride,
                            const float* weight, float eps, int64_t n_rows, int64_t d, float* rstd, int8_t* q,
                            int64_t q_row_stride, float* scale, uint16_t* y, int64_t y_row_stride,
                            stq_stream_t stream);

/* Its gradients, for a gradient dy at the normed rows (the rounding to 8 bits
 * taken as the identity) and one, dh, that arrives at h by another way, such as
 * the residual stream.  With u = h * rstd and g = dy * weight:
 *     dx = dh + rstd * (g - u * mean(g * u))     (x's gradient and the residual's)
 *     dweight = sum over rows of dy * u
 *   h, rstd    what the forward call gave
 *   dy         [n_rows, d] fp32 or bf16
 *   dh         [n_rows, d] of h's type, or NULL (zeros)
 *   dx         [n_rows, d] of h's type, or NULL (not wanted); may be dh, or dy
 *              where the types are the same, with the same stride, but not h
 *   dweight    fp32 [d], or NULL (not wanted); zeros without rows
 *   workspace, workspace_bytes   at least what
 *              stq_rmsnorm_rows_backward_workspace reports (may be NULL when 0)
 * Limits as above.  Sums are fp32 in an order that is fixed for a device. */
stq_status stq_rmsnorm_rows_backward(const void* h, int h_dtype, int64_t h_row_stride, const float* weight,
                                     const float* rstd, const void* dy, int dy_dtype, int64_t dy_row_stride,
                                     const void* dh, int64_t dh_row_stride, void* dx, int64_t dx_row_stride,
                                     float* dweight, int64_t n_rows, int64_t d, void* workspace,
                                     int64_t workspace_bytes, stq_stream_t stream);

/* Workspace bytes stq_rmsnorm_rows_backward needs for these shapes on a device
 * with n_cus compute units (0: the current device's); host only.
 * workspace_bytes is a HOST pointer. */
stq_status stq_rmsnorm_rows_backward_workspace(int64_t n_rows, int64_t d, int want_dweight, int32_t n_cus,
                                               int64_t* workspace_bytes);

/* Routing (traictory.com, "The claim, stated precisely": every token goes to 8
 * of 256 experts): the top_k largest of each token's logits, their weights, and
 * the (token, expert) rows sorted by expert, stable in the tokens, as
 * stq_gemv, stq_grouped_gemm and stq_grouped_swiglu take them.  With p =
 * softmax(l) over all experts:
 *     weight of a chosen expert e:  exp(l_e) / sum of exp(l) over the chosen
 *                                   (renormalize != 0), else p_e
 *     counts[e] = tokens that chose e,    f_e = counts[e] / sum of counts
 *     balance = n_experts * sum_e f_e P_e,   P_e = mean of p_e over the tokens
 * (balance is 1 where either is even; it grows with the agreement of counts and
 * probabilities, and its gradient takes counts as given.)
 *   logits       [n_tokens, n_experts] fp32 (STQ_X_F32) or bf16 bits
 *                (STQ_X_BF16), rows row_stride elements apart, aligned to their
 *                elements.  -inf masks an expert: it is chosen last, with weight
 *                0.  Equal logits go to the lowest expert.
 *   pair_expert, pair_weight  int32 / fp32 [n_tokens * top_k], a token's pairs
 *                together, largest first
 *   counts       int32 [n_experts];   offsets  int32 [n_experts + 1]
 *   pair_row     int32 [n_tokens * top_k]: the row of each pair, -1 for none
 *   row_token, row_weight  int32 / fp32 [n_tokens * top_k]: each row's token and
 *                weight; token 0 and weight 0 from row offsets[n_experts] on
 *   balance      fp32 [1]
 * A token whose logits are all -inf (padding) goes nowhere: its pairs are expert
 * -1 with weight 0, it has no rows and counts for nothing.  One with a NaN or a
 * +inf goes nowhere either; its weights are NaN, and so is the balance.
 * 1 <= n_experts <= 1024, 1 <= top_k <= min(32, n_experts), at most 2^22 tokens.
 *   workspace, workspace_bytes   at least what stq_route_tokens_workspace
 *                reports (may be NULL when 0)
 * Sums are fp32 in a fixed order: repeated calls give identical bits. */
stq_status stq_route_tokens(const void* logits, int x_dtype, int64_t row_stride, int64_t n_tokens, int64_t n_experts,
                            int64_t top_k, int renormalize, int32_t* pair_expert, float* pair_weight, int32_t* counts,
                            int32_t* offsets, int32_t* pair_row, int32_t* row_token, float* row_weight, float* balance,
                            void* workspace, int64_t workspace_bytes, stq_stream_t stream);

/* Workspace bytes stq_route_tokens needs for these shapes; host only, same
 * checks and errors as the call.  workspace_bytes is a HOST pointer. */
stq_status stq_route_tokens_workspace(int64_t n_tokens, int64_t n_experts, int64_t top_k, int64_t* workspace_bytes);

/* Gradient of the weights and of the balance loss with respect to the logits,
 * the choice and the counts taken as given: with g the gradient at a token's
 * weights w and b the one at the balance,
 *     renormalize: d_e += w_e (g_e - sum of g w) for the chosen
 *     else:        d_e += p_e (g_e - sum of g p), g = 0 for the others
 *     and          d_e += p_e (c_e - sum of c p),  c_e = b n_experts f_e / tokens
 * (tokens: those that have rows, sum of counts / top_k).
 *   logits, renormalize, pair_expert, counts   as given to and by the call above
 *                (counts is read with grad_balance only; summed over the ranks of
 *                a job, b's share of the tokens is that of the job)
 *   grad_weight  fp32 [n_tokens * top_k] or NULL (zeros): in the order of the
 *                pairs, or, with pair_row (else NULL), of the sorted rows
 *   grad_balance fp32 [1] on the device, or NULL (zero)
 *   d_logits     [n_tokens, n_experts], the logits' type, rows d_row_stride
 *                elements apart; may be the logits themselves (same pointer and
 *                stride), else it may not overlap them
 * A token that went nowhere gives zeros, NaN where its logits hold a NaN or a
 * +inf. */
stq_status stq_route_tokens_backward(const void* logits, int x_dtype, int64_t row_stride, int64_t n_tokens,
                                     int64_t n_experts, int64_t top_k, int renormalize, const int32_t* pair_expert,
                                     const int32_t* counts, const float* grad_weight, const int32_t* pair_row,
                                     const float* grad_balance, void* d_logits, int64_t d_row_stride,
                                     stq_stream_t stream);

/* A token's expert rows added up, in routing order:
 *     y[t] = sum over j < top_k of pair_weight[t, j] * z[pair_row[t, j]]
 * With ones for weights it is also the gradient of x_sorted = x[row_token].
 *   z            [n_rows, d] fp32 (STQ_X_F32) or bf16 bits (STQ_X_BF16), rows
 *                z_row_stride elements apart: the down projection's rows
 *   pair_row     int32 [n_tokens * top_k], from stq_route_tokens; a pair whose
 *                row is outside [0, n_rows) adds nothing
 *   pair_weight  fp32 [n_tokens * top_k], or NULL (ones)
 *   y            [n_tokens, d] fp32 or bf16, rows y_row_stride elements apart;
 *                every element is written
 * Every pointer is aligned to its elements.  Sums are fp32, in order.  1 <=
 * top_k <= 32, d >= 1; at most 2^22 tokens, 2^31 - 1 rows and 2^26 columns, and less than 2^24
 * started pieces of 512 columns (2048 where d > 512) of a token in all. */
stq_status stq_combine_rows(const void* z, int z_dtype, int64_t z_row_stride, int64_t n_rows, const int32_t* pair_row,
                            const float* pair_weight, int64_t n_tokens, int64_t top_k, int64_t d, void* y, int y_dtype,
                            int64_t y_row_stride, stq_stream_t stream);

/* Its gradients, for dy [n_tokens, d] at y:
 *     dz[pair_row[t, j]] = pair_weight[t, j] * dy[t]
 *     dweight[t, j] = <dy[t], z[pair_row[t, j]]>, 0 for a pair without a row
 *   dz       [n_rows, d] fp32 or bf16, or NULL (not wanted); rows of no pair stay
 *            unwritten, and no row may have two pairs (stq_route_tokens gives none)
 *   dweight  fp32 [n_tokens * top_k], or NULL (not wanted); reads z, which may
 *            be NULL otherwise
 * The other arguments and limits are as above.  dz may be z where types and strides
 * are the same; else it may not overlap z or dy. */
stq_status stq_combine_rows_backward(const void* dy, int dy_dtype, int64_t dy_row_stride, const void* z, int z_dtype,
                                     int64_t z_row_stride, int64_t n_rows, const int32_t* pair_row,
                                     const float* pair_weight, int64_t n_tokens, int64_t top_k, int64_t d, void* dz,
                                     int dz_dtype, int64_t dz_row_stride, float* dweight, stq_stream_t stream);

/* Softmax cross entropy of an output head without keeping the logits, which for
 * a large vocabulary are many times its operands:
 *     l_i = x . w_i  (bf16), or (x . w_i) * x_scale * w_scale_i  (8-bit rows)
 *     lse = log sum_i exp(l_i)        loss = lse - l_target
 *   x         [n_rows, k] bf16 bits (x_dtype STQ_X_BF16) or int8 with x_scale
 *             fp32 [n_rows] (STQ_X_I8, as stq_q8_quantize_rows and
 *             stq_rmsnorm_rows write them)
 *   w         [vocab, k] of x's type, for int8 with w_scale fp32 [vocab]
 *             both 16-byte aligned with row strides (elements) of whole 16-byte
 *             units, at least k and at most 2^23 bytes; the bytes between one
 *             row's k elements and the next row, and behind the last row up
 *             to a whole 16-byte unit, may be read and count for nothing
 *   targets   int32 [n_rows]; a negative one leaves its row out (loss 0), one
 *             past the vocabulary gives loss NaN
 *   loss, lse fp32 [n_rows]
 *   workspace, workspace_bytes  at least what stq_head_cross_entropy_workspace
 *             reports
 * bf16 products are exact and their sums fp32; integer sums are exact and scaled
 * in fp32, as in stq_q8_matmul.  A row whose logits hold a NaN or a +inf has lse
 * and loss NaN, one whose logits are all -inf lse -inf and loss NaN.  The order
 * of every sum is fixed for a device: repeated calls give identical bits.
 * 1 <= k <= 131071, 1 <= vocab <= 2^26, n_rows at most 2^20, n_rows * vocab at
 * most 2^38. */
stq_status stq_head_cross_entropy(const void* x, int x_dtype, int64_t x_row_stride, const float* x_scale, const void* w,
                                  int64_t w_row_stride, const float* w_scale, int64_t n_rows, int64_t vocab, int64_t k,
                                  const int32_t* targets, float* loss, float* lse, void* workspace,
                                  int64_t workspace_bytes, stq_stream_t stream);

/* Workspace bytes stq_head_cross_entropy needs for these shapes on a device with
 * n_cus compute units (0: the current device's); host only, same checks and
 * errors as the call.  workspace_bytes is a HOST pointer. */
stq_status stq_head_cross_entropy_workspace(int x_dtype, int64_t n_rows, int64_t vocab, int64_t k, int32_t n_cus,
                                            int64_t* workspace_bytes);

/* Its gradients, for a gradient g at the losses; the logits are formed again, a
 * piece of the vocabulary at a time:
 *     dl_i = g (exp(l_i - lse) - 1[i = target])
 *     dx = sum_i dl_i w_i  (8-bit rows: dl_i w_scale_i w_i, the gradient at
 *          x * x_scale, the rounding to 8 bits taken as the identity)
 *     dw_i = sum over rows of dl_i x       (bf16 only)
 *   lse        fp32 [n_rows], what the forward call gave
 *   grad_loss  fp32 [n_rows]; not read where a row is left out
 *   dx         bf16 bits [n_rows, k], rows dx_row_stride elements apart, or NULL
 *              (not wanted)
 *   dw         bf16 bits [vocab, k], rows dw_row_stride elements apart, or NULL;
 *              zeros where no row is left
 *   workspace, workspace_bytes  at least what
 *              stq_head_cross_entropy_backward_workspace reports
 * The other arguments and limits are as above.  A row that is left out, whose
 * target lies past the vocabulary or whose lse is -inf has no gradient: its dx is
 * 0 and it adds nothing to dw, whatever x and w hold; another whose lse is NaN gives
 * NaN.  dl is formed in fp32 and rounded to bf16 for the two products (with 8-bit
 * rows after its w_scale, so that the integers, which bf16 holds exactly, enter as
 * they are): a term is off by at most 2^-8 of itself, half a bf16 step.  The target's
 * term, as large as all the others of its row together, is added in fp32 to dx, and
 * to dw where there are at most 32 rows; the others' roundings average out beside
 * the results' own.  dw of more rows errs by about 0.0017 of its norm from that
 * (0.0022 with 33) and as much from its own rounding.  Sums are fp32 in an order that
 * is fixed for a device.  dx and dw are rounded from them
 * once and may not overlap the operands; rows that all start on 16 bytes are
 * written faster. */
stq_status stq_head_cross_entropy_backward(const void* x, int x_dtype, int64_t x_row_stride, const float* x_scale,
                                           const void* w, int64_t w_row_stride, const float* w_scale, int64_t n_rows,
                                           int64_t vocab, int64_t k, const int32_t* targets, const float* lse,
                                           const float* grad_loss, uint16_t* dx, int64_t dx_row_stride, uint16_t* dw,
                                           int64_t dw_row_stride, void* workspace, int64_t workspace_bytes,
                                           stq_stream_t stream);

/* Workspace bytes stq_head_cross_entropy_backward needs for these shapes and the
 * outputs wanted (0 or 1 each) on a device with n_cus compute units (0: the
 * current device's); host only.  workspace_bytes is a HOST pointer. */
stq_status stq_head_cross_entropy_backward_workspace(int x_dtype, int64_t n_rows, int64_t vocab, int64_t k, int want_dx,
                                                     int want_dw, int32_t n_cus, int64_t* workspace_bytes);

/* Measurement helper, not part of the method: reads `bytes` bytes of the
 * device buffer `buf` once with 16-byte loads, the streaming-read rate this
 * GPU sustains, against which the decode GEMV's effective bandwidth is
 * compared (the HBM roofline).  `buf` 16-byte aligned, `bytes` a multiple of
 * 16; `sink` is one device uint32 that may be overwritten (its value is
 * meaningless). */
stq_status stq_stream_read_probe(const void* buf, int64_t bytes, uint32_t* sink, stq_stream_t stream);

/* Measurement helper, not part of the method: the matrix-core reference
 * beside the grouped GEMM's MFMA roofline.  Launches 4096 workgroups of 4
 * wavefronts; each wavefront runs `rounds` rounds of 8 independent
 * v_mfma_f32_16x16x32_bf16 (16,384 flops each) with no memory traffic, so a
 * launch does STQ_MFMA_PROBE_FLOP_PER_ROUND * rounds flops.  `rounds` >= 0
 * (0 launches nothing); `sink` is one device float that is never written in
 * practice (its value is meaningless). */
#define STQ_MFMA_PROBE_FLOP_PER_ROUND 2147483648.0
stq_status stq_mfma_loop_probe(int64_t rounds, float* sink, stq_stream_t stream);

/* Measurement helper, not part of the method: the LDS read rate beside the
 * grouped GEMM's operand reads.  Launches 4096 workgroups of 4 wavefronts;
 * each workgroup fills a 32 KB LDS buffer once, then each wavefront runs
 * `rounds` rounds of 8 LDS reads, each folded into a register (no other
 * memory traffic):
 *   mode 0: ds_read_b128, the 64 lanes reading one contiguous 1 KB run
 *           (conflict free), the form of the GEMM's activation reads;
 *   mode 1: ds_read2_b32 at a per-lane code 0..31 of a 32-entry table and
 *           32 words further (the form of the GEMM's pattern reads).
 * A launch issues STQ_LDS_PROBE_READS_PER_ROUND * rounds wavefront LDS
 * instructions.  `mode` 0 or 1, `rounds` >= 0; `sink` as above (uint32). */
#define STQ_LDS_PROBE_READS_PER_ROUND 131072
stq_status stq_lds_read_probe(int mode, int64_t rounds, uint32_t* sink, stq_stream_t stream);

/* Static text of a status code. */
const char* stq_status_string(stq_status s);

/* Detail of the last failure on the calling thread ("" if none). */
const char* stq_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* STQ_H */
