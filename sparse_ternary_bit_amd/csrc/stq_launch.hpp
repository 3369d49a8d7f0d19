// Host-side launchers of the libstq kernels (internal to the library).
// Arguments are validated by the C ABI layer before any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace stq {

hipError_t launch_dequantize(const uint8_t* q, int64_t n_rows, int64_t k, float* out, hipStream_t s);

hipError_t launch_quantize(const float* w, const float* imatrix, int64_t n_rows, int64_t k, int encoder,
                           int rounds, uint8_t* out, hipStream_t s);

struct GemvArgs {
  const uint8_t* w_table;
  int64_t expert_stride;
  int64_t n_experts;
  int64_t n;
  int64_t k;
  const void* x;
  int x_mode;               // 0 fp32 rows, 1 bf16 rows
  int64_t x_row_stride;     // elements
  int64_t n_tokens;
  const int32_t* pair_expert;
  const int32_t* pair_token;  // NULL: pair q uses token q / pairs_per_token
  int64_t n_pairs;
  float* y;
  int64_t pairs_per_token;  // used only without pair_token (0 means 1)
};

// Scratch needed by launch_gemv for the chosen k split (bytes, 0 if none),
// and the launch itself; with partial_bytes > 0, `partial` holds that many
// bytes (fp32 partial sums, then one int per pair).
struct GemvPlan {
  int splits;          // k split across workgroups
  int blocks_per_split;
  int max_sub;         // most parts a split's blocks are cut into for a many-token expert
  int64_t partial_floats;
  int64_t partial_bytes;
  bool mfma;           // bf16 passes of 3+ tokens on the matrix cores (kernel variant)
  bool order_units;    // more workgroups than resident slots: number units longest first
};
// cus: compute units the plan is made for (see cus_of_stream).
GemvPlan plan_gemv(const GemvArgs& a, int cus);
// Compute units of the device a stream runs on, or of the current device
// (256 when the query fails); cached per device.
int cus_of_stream(hipStream_t s);
int cus_of_current_device();
// reduce = false leaves split outputs in `partial` for the caller to add (see
// GemvPartials); the GEMV still writes y's rows that are not split and the
// NaN rows of invalid pairs.
hipError_t launch_gemv(const GemvArgs& a, const GemvPlan& plan, void* partial, hipStream_t s, bool reduce = true);

// Split outputs of a launch_gemv(..., reduce = false): valid pair p's row r
// is, when its slot count splits * (pair_sub ? pair_sub[p] : 1) exceeds 1,
// the sum over slots s in order, starting from 0.0f, of
// partial[(s * n_pairs + p) * n + r]; otherwise y's own row.  partial is
// NULL when the plan splits nothing.
struct GemvPartials {
  const float* partial;
  int splits;
  int max_slots;  // splits x the part cap: no pair has more slots
  const int32_t* pair_sub;
};
GemvPartials gemv_partials(const GemvPlan& plan, void* partial);

// h[p, c] = silu(gu[p, c]) * gu[p, d_ff + c], silu(v) = v / (1 + exp(-v)),
// for gu [n_pairs, 2*d_ff] and h [n_pairs, d_ff] fp32 (d_ff a multiple of 4),
// with gu the y of a launch_gemv(..., reduce = false) whose split rows are
// added here (pair_expert / n_experts tell valid pairs)
hipError_t launch_swiglu(const float* gu, const GemvPartials& parts, const int32_t* pair_expert, int64_t n_experts,
                         int64_t n_pairs, int64_t d_ff, float* h, hipStream_t s);

// y[t, :] = sum over k < top_k, in order, of w[t*top_k + k] * z[t*top_k + k, :],
// with z the y of a launch_gemv(..., reduce = false) over the pairs
hipError_t launch_combine(const float* z, const GemvPartials& parts, const int32_t* pair_expert, int64_t n_experts,
                          const float* w, int64_t n_tokens, int64_t top_k, int64_t n, float* y, hipStream_t s);

struct GemmArgs {
  const uint8_t* w_table;
  int64_t expert_stride;
  int64_t n_experts;
  int64_t n;
  int64_t k;
  const uint16_t* x;
  const int32_t* offsets;
  int64_t total_m;
  float* y;
};
hipError_t launch_grouped_gemm(const GemmArgs& a, hipStream_t s);

// Gated feed-forward over the packed experts, rows grouped by expert, and its
// gradients
struct SwigluArgs {
  const uint8_t* w_table;
  int64_t expert_stride;
  int64_t n_experts;
  int64_t d_model, d_ff;
  const uint16_t* x;
  const int32_t* offsets;
  int64_t total_m;
  uint16_t* h;
  uint16_t* gate_up;  // may be NULL
};
// Few rows go through the decode GEMV (one pair a row), the rest through the
// matrix cores in passes of at most max_tok rows.
struct SwigluPlan {
  int max_tok;            // 0: the GEMV
  GemvPlan plan;          // GEMV: of the gate/up product
  int64_t part, pe, gu;   // GEMV: workspace bytes of the split outputs, the rows' experts, the fp32 rows
  int64_t bytes;          // workspace bytes
};
SwigluPlan plan_swiglu(const SwigluArgs& a, int cus);
hipError_t launch_grouped_swiglu(const SwigluArgs& a, const SwigluPlan& plan, void* ws, hipStream_t s);
// Its passes of more than 32 rows (k_gated.hip)
hipError_t launch_gated(const SwigluArgs& a, int max_tok, hipStream_t s);

// The GEMV form's own kernels (k_moe.hip)
hipError_t launch_row_expert(const int32_t* offsets, int64_t n_experts, int64_t rows, int32_t* pair_expert, hipStream_t s);
hipError_t launch_swiglu_rows(const float* gu, const GemvPartials& parts, const int32_t* pair_expert, int64_t n_experts,
                              int64_t rows, int64_t d_ff, uint16_t* h, uint16_t* gate_up, hipStream_t s);

struct SwigluBwdArgs {
  const uint8_t* w_table;
  int64_t expert_stride;
  int64_t n_experts;
  int64_t d_model, d_ff;
  const uint16_t* x;         // read with dw
  const int32_t* offsets;
  int64_t total_m;
  const uint16_t* gate_up;
  const uint16_t* dh;
  uint16_t* dx;              // may be NULL
  uint16_t* dw;              // may be NULL
};
// Workspace: the scaled fp16 dz at 0 and its row scales at `inv` (dx), the
// bf16 dz at `dzb` (dw)
struct SwigluBwdLayout {
  int64_t inv, dzb, bytes;
};
SwigluBwdLayout swiglu_bwd_layout(int64_t d_ff, int64_t total_m, bool dx, bool dw);
int dx_rows_a_pass(const SwigluBwdArgs& a, int cus);
hipError_t launch_swiglu_bwd(const SwigluBwdArgs& a, void* ws, int cus, hipStream_t s);

// Layer error under calibration activations (full Hessian and diagonal);
// `scratch` holds layer_errors_scratch_bytes(...) bytes.
int64_t layer_errors_scratch_bytes(int64_t n_rows, int64_t k, int64_t n_cal);
hipError_t launch_layer_errors(const float* w, const float* w_hat, int64_t n_rows, int64_t k, const float* x,
                               int64_t n_cal, double* err_full, double* err_diag, void* scratch, hipStream_t s);

// 2-bit stand-in format: quantize and reconstruct in one pass
hipError_t launch_q2_roundtrip(const float* w, int64_t n_rows, int64_t k, float* out, hipStream_t s);

// 8-bit rows with one scale each, and their product
struct Q8QuantArgs {
  const void* x;
  int bf16;           // 0 fp32, 1 bf16
  int64_t x_stride;   // elements
  int64_t rows, k;
  int8_t* q;
  int64_t ldq;        // bytes
  float* scale;
};
hipError_t launch_q8_quantize(const Q8QuantArgs& a, hipStream_t s);

struct Q8MatmulArgs {
  const int8_t* a;
  int64_t lda;
  const float* a_scale;
  const int8_t* w;
  int64_t ldw;
  const float* w_scale;
  int64_t m, n, k;
  void* y;
  int bf16;
  int64_t ldy;
  int cus;            // compute units to plan for
};
hipError_t launch_q8_matmul(const Q8MatmulArgs& a, hipStream_t s);

// Token log probabilities, entropy and top alternatives of rows of logits
struct LogprobsArgs {
  const void* logits;
  int bf16;
  int64_t stride;     // elements
  int64_t rows, vocab;
  const int32_t* targets;
  float* logprob;
  float* lse;         // may be NULL
  float* entropy;     // may be NULL
  int32_t* top_ids;
  float* top_lp;
  int top_n;
};
struct LogprobsPlan {
  int splits;           // workgroups a row is cut into
  int64_t per;          // 16-byte chunks per split
  int64_t stats_bytes;  // offset of the splits' keys in the workspace
  int64_t bytes;        // workspace bytes (0: one workgroup a row)
};
LogprobsPlan plan_logprobs(int64_t rows, int64_t vocab, int elem_bytes, int top_n, int cus);
hipError_t launch_logprobs(const LogprobsArgs& a, const LogprobsPlan& plan, void* ws, hipStream_t s);

struct LogprobsBwdArgs {
  const void* logits;
  int bf16;
  int64_t stride;
  int64_t rows, vocab;
  const int32_t* targets;
  const float* lse;
  const float* entropy;  // read with g_ent only
  const float* g_lp;     // may be NULL
  const float* g_ent;    // may be NULL
  void* out;
  int64_t out_stride;
};
int64_t logprobs_bwd_parts(const LogprobsBwdArgs& a);  // workgroups per row, at most
hipError_t launch_logprobs_bwd(const LogprobsBwdArgs& a, hipStream_t s);

// Residual addition, root-mean-square norm and 8-bit rows; its gradients
struct NormArgs {
  const void* x;
  int x_bf16;
  int64_t x_stride;     // elements, like every stride here but q_stride
  const void* res;      // NULL: h is x
  int res_bf16;
  int64_t res_stride;
  void* h;              // the residual's type
  int64_t h_stride;
  const float* weight;
  float eps;
  int64_t rows, d;
  float* rstd;          // may be NULL
  int8_t* q;            // may be NULL
  int64_t q_stride;     // bytes
  float* scale;         // with q
  uint16_t* y;          // may be NULL
  int64_t y_stride;
};
hipError_t launch_norm(const NormArgs& a, hipStream_t s);

struct NormBwdArgs {
  const void* h;
  int h_bf16;           // h, dh and dx
  int64_t h_stride;
  const float* weight;
  const float* rstd;
  const void* dy;
  int dy_bf16;
  int64_t dy_stride;
  const void* dh;       // may be NULL
  int64_t dh_stride;
  void* dx;             // may be NULL
  int64_t dx_stride;
  float* dw;            // may be NULL
  int64_t rows, d;
};
// `part`: norm_bwd_parts(rows, cus) rows of d floats, with dw
int norm_bwd_parts(int64_t rows, int cus);
hipError_t launch_norm_bwd(const NormBwdArgs& a, float* part, int cus, hipStream_t s);

// Top-k routing, the rows sorted by expert and the balance loss; its gradient
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTop = 32;
struct RouteArgs {
  const void* logits;
  int bf16;
  int64_t stride;
  int64_t tokens;
  int experts, top_k;
  int renorm;
  int32_t* pair_expert;
  float* pair_weight;
  int32_t* counts;
  int32_t* offsets;
  int32_t* pair_row;
  int32_t* row_token;
  float* row_weight;
  float* balance;
};
// Workspace (tokens of more than one chunk): per expert and chunk the count
// (then the rows before it) at 0 and the summed probabilities at `prob`, per
// expert the summed probabilities at `prob_total`
struct RouteLayout {
  int64_t chunks, prob, prob_total, bytes;
};
RouteLayout route_layout(int64_t tokens, int64_t experts);
hipError_t launch_route(const RouteArgs& a, void* ws, hipStream_t s);

struct RouteBwdArgs {
  const void* logits;
  int bf16;
  int64_t stride;
  int64_t tokens;
  int experts, top_k;
  int renorm;
  const int32_t* pair_expert;
  const int32_t* counts;      // with g_balance
  const float* g_weight;      // may be NULL
  const int32_t* pair_row;    // g_weight is in the order of the sorted rows; NULL: of the pairs
  const float* g_balance;     // may be NULL
  void* d_logits;
  int64_t d_stride;
};
hipError_t launch_route_bwd(const RouteBwdArgs& a, hipStream_t s);

// A token's rows added up with its weights; the gradients of that
struct CombineArgs {
  const void* z;
  int z_bf16;
  int64_t z_stride, n_rows;
  const int32_t* pair_row;
  const float* weight;  // NULL: ones
  int64_t tokens;
  int top_k;
  int64_t d;
  void* y;
  int y_bf16;
  int64_t y_stride;
};
int64_t combine_col_blocks(int64_t d);  // workgroups a token
hipError_t launch_combine_rows(const CombineArgs& a, hipStream_t s);

struct CombineBwdArgs {
  const void* dy;
  int dy_bf16;
  int64_t dy_stride;
  const void* z;        // read with dw
  int z_bf16;
  int64_t z_stride, n_rows;
  const int32_t* pair_row;
  const float* weight;
  int64_t tokens;
  int top_k;
  int64_t d;
  void* dz;             // may be NULL
  int dz_bf16;
  int64_t dz_stride;
  float* dw;            // may be NULL
};
hipError_t launch_combine_rows_bwd(const CombineBwdArgs& a, hipStream_t s);

// Softmax cross entropy of an output head and its gradients
struct HeadArgs {
  const void* x;          // rows: bf16, or 8-bit integers with x_scale
  int64_t ldx;            // bytes
  const float* x_scale;
  const void* w;
  int64_t ldw;            // bytes
  const float* w_scale;
  int i8;
  int64_t rows, vocab, k;
  const int32_t* targets;
};
struct HeadLayout {
  int64_t hit, bytes;     // the targets' logits in the workspace; its size
};
HeadLayout head_layout(int64_t rows, int64_t vocab, int cus);
hipError_t launch_head(const HeadArgs& h, float* loss, float* lse, void* ws, int cus, hipStream_t s);

struct HeadBwdArgs {
  const float* lse;
  const float* g;
  uint16_t* dx;           // may be NULL
  int64_t ld_dx;          // elements
  uint16_t* dw;           // may be NULL
  int64_t ld_dw;
};
struct HeadBwdPlan {
  int64_t width, pieces;       // of the vocabulary
  int few;                     // few rows: dx from the head as it lies
  int splits, per;             // of dx's sum; stages of a split (few rows)
  int64_t rest, dlt, xt, acc;  // workspace offsets
  int64_t bytes;
};
HeadBwdPlan plan_head_bwd(bool i8, int64_t rows, int64_t vocab, int64_t k, bool dx, bool dw, int cus);
hipError_t launch_head_bwd(const HeadArgs& h, const HeadBwdArgs& b, const HeadBwdPlan& p, void* ws, int cus, hipStream_t s);
hipError_t launch_head_zero(uint16_t* dw, int64_t ld, int64_t vocab, int64_t k, hipStream_t s);

// Streaming-read reference (measurement only): reads `bytes` bytes of `buf`
hipError_t launch_stream_read(const void* buf, int64_t bytes, uint32_t* sink, hipStream_t s);

// Matrix-core and LDS references (measurement only).  Their shapes are the
// ones stq.h states, so that callers can count the work of a launch.
constexpr int kMfmaProbeGrid = 4096;  // workgroups of 4 wavefronts
constexpr int kMfmaChains = 8;        // independent MFMAs per wavefront and round
constexpr int kLdsProbeGrid = 4096;   // workgroups of 4 wavefronts
constexpr int kLdsReads = 8;          // LDS reads per wavefront and round
constexpr int kLdsProbeWords = 2048;  // 16-byte words of LDS per workgroup (32 KB)
hipError_t launch_mfma_loop(int64_t iters, float* sink, hipStream_t s);
hipError_t launch_lds_read(int mode, int64_t iters, uint32_t* sink, hipStream_t s);

}  // namespace stq
