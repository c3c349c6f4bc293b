/*
 * moe_ops.h -- C ABI of the operators next to the MoE layer, for sm_100a: matrix products
 * grouped by expert with ragged sizes, a linear layer with a fused epilogue, and the gated
 * activation, each with the products that its gradient needs.
 *
 * These are the layer's building blocks as separate calls.  moe_layer_forward() runs a whole
 * routed FFN and keeps nothing for a backward pass; with the calls below a program trains the
 * experts on the layer's own routing (moe_routing_out: `offsets` is the argument of that name
 * here, `perm` orders the rows), or runs dense FFNs and projections beside it.
 *
 * Conventions for every entry point:
 *   - tensor pointers are DEVICE pointers owned by the caller, row-major and contiguous,
 *     16-byte aligned (fp32 vectors `bias`, `row_w`, `dbias`, `d_row_w` and int32 `offsets`:
 *     4-byte aligned); the library never allocates or frees device memory;
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default stream) of the
 *     current device; work is enqueued asynchronously and the call returns without
 *     synchronising; every call can be captured into a CUDA graph;
 *   - outputs (and the workspace) must not overlap inputs or each other, except where said:
 *     such a call is refused with MOE_ERR_INVALID_ARG;
 *   - the calls keep no state between them: any number may run at the same time, on any
 *     streams (moe_linear_backward: each with a workspace of its own);
 *   - results do not depend on timing: no atomics, sums in a fixed order;
 *   - all sums are held in fp32 (bf16 products on the tensor cores, which cut off below 2^-23
 *     of the running sum, in parts of at most 16384 terms that are added in fp32: within 2^-13,
 *     and 2^-24 for each part, of the sum of the terms' magnitudes); a bf16 result is rounded once,
 *     at the end, except the gradient dz of moe_linear_backward, which is rounded to bf16 between
 *     its two products;
 *   - the return value reports argument validation and launch errors; errors found on the
 *     device (offsets out of range, a bounded wait that timed out) go to a per-device status
 *     word that moe_ops_check_status() reads and clears.
 *
 * The operators are defined by the formulas below; they have no counterpart of their own on
 * the source pages, whose layer they are parts of (llm-atlas page "Step-3.5-Flash", table
 * "Champs bruts du config.json": hidden_size 4096, moe_num_experts 288,
 * moe_intermediate_size 1280, share_expert_dim 1280, intermediate_size 11264).
 */
#ifndef MOE_OPS_H
#define MOE_OPS_H

#include "moe_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Sizes of a product: R rows, N output and K input features, E experts (1 for a linear
 * layer), dtype of all matrices (moe_dtype).
 * Supported: 0 <= R <= 2^30, 1 <= N, K <= 2^20, 1 <= E <= 1024.
 *   MOE_BF16: N and K multiples of 8 (rows of 16-byte chunks).   MOE_F32: any N and K.   */
typedef struct {
  int64_t R;
  int32_t N, K, E;
  int32_t dtype;
} moe_gemm_shape;

/* Matrix products grouped by expert.  `offsets` [E + 1] int32, on the device and
 * non-decreasing, gives the rows of each expert: offsets[e] <= r < offsets[e + 1] (none where
 * they are equal), all within [0, R].  The sizes of the groups are read on the device only.
 *   moe_grouped_gemm        y[r]  [R, N]     = x[r] W[e]^T       x [R, K], W [E, N, K]
 *   moe_grouped_gemm_dgrad  dx[r] [R, K]     = dy[r] W[e]        dy [R, N], W [E, N, K]
 *   moe_grouped_gemm_wgrad  dW[e] [E, N, K]  = sum over the rows r of e of dy[r]^T x[r]
 * Rows outside [offsets[0], offsets[E]) are neither read for a result nor written, whatever
 * they hold; dW[e] of an expert without rows is zero.  An expert whose offsets are out of
 * order or out of [0, R] counts as empty, and MOE_ERR_DEVICE_BOUNDS is recorded; what the
 * result then holds of the other experts' rows is not specified. */
MOE_API moe_status moe_grouped_gemm(const moe_gemm_shape* shape, const void* x, const void* W, const int32_t* offsets,
                                    void* y, void* stream);
MOE_API moe_status moe_grouped_gemm_dgrad(const moe_gemm_shape* shape, const void* dy, const void* W,
                                          const int32_t* offsets, void* dx, void* stream);
MOE_API moe_status moe_grouped_gemm_wgrad(const moe_gemm_shape* shape, const void* dy, const void* x,
                                          const int32_t* offsets, void* dW, void* stream);

/* Activations of the linear layer.
 *   MOE_ACT_GELU: z Phi(z) with the error function; MOE_ACT_GELU_TANH: its usual form with
 *   tanh(sqrt(2/pi) (z + 0.044715 z^3)); MOE_ACT_SILU: z / (1 + e^-z). */
enum { MOE_ACT_NONE = 0, MOE_ACT_RELU = 1, MOE_ACT_SILU = 2, MOE_ACT_GELU = 3, MOE_ACT_GELU_TANH = 4 };

/* z = x W^T + bias,  y = act(z) + residual.
 *   x [R, K], W [N, K], bias [N] fp32 or NULL, residual [R, N] or NULL (y may be the residual
 *   itself), y [R, N]; preact [R, N] or NULL receives z, which moe_linear_backward() needs
 *   unless the activation is MOE_ACT_NONE.  shape->E must be 1. */
MOE_API moe_status moe_linear(const moe_gemm_shape* shape, const void* x, const void* W, const float* bias,
                              const void* residual, int32_t activation, void* y, void* preact, void* stream);

/* Gradients of moe_linear() for the gradient dy [R, N] of y:
 *   dz = dy act'(z),  dx [R, K] = dz W,  dW [N, K] = dz^T x,  dbias [N] fp32 = sum_r dz[r]
 * (the residual's gradient is dy itself).  Any of dx, dW and dbias may be NULL and is then
 * not computed; x may be NULL without dW, and W without dx.  preact [R, N] is z (NULL with
 * MOE_ACT_NONE).  relu'(0) = 0.  For R = 0, dW and dbias are zero.
 * workspace: moe_linear_backward_workspace_bytes() bytes, 256-byte aligned, not initialised
 * (NULL if that is 0). */
MOE_API size_t moe_linear_backward_workspace_bytes(const moe_gemm_shape* shape, int32_t activation, int32_t with_dbias);
MOE_API moe_status moe_linear_backward(const moe_gemm_shape* shape, const void* dy, const void* x, const void* W,
                                       const void* preact, int32_t activation, void* dx, void* dW, float* dbias,
                                       void* workspace, size_t workspace_bytes, void* stream);

/* The gated activation between an expert's two products, on rows [gate | up] as
 * W_gate_up gives them:
 *   a = min(gate, limit), c = clamp(up, -limit, limit)   (limit > 0; 0: a = gate, c = up)
 *   h[r, i] = w[r] a sigmoid(a) c                         (row_w NULL: w = 1)
 *   gate_up [R, 2 I], row_w [R] fp32 or NULL, h [R, I].
 * Backward, for dh [R, I]:
 *   d_gate_up [R, 2 I]: w dh c (a sigmoid(a))' where gate <= limit, else 0;
 *                       w dh a sigmoid(a) where |up| <= limit, else 0
 *   d_row_w [R] fp32 = sum_i dh a sigmoid(a) c  (NULL: not computed; also without row_w)
 * 0 <= R <= 2^30, 1 <= I <= 2^20; MOE_BF16: I a multiple of 8. */
MOE_API moe_status moe_swiglu(int64_t R, int32_t I, int32_t dtype, const void* gate_up, const float* row_w, float limit,
                              void* h, void* stream);
MOE_API moe_status moe_swiglu_backward(int64_t R, int32_t I, int32_t dtype, const void* dh, const void* gate_up,
                                       const float* row_w, float limit, void* d_gate_up, float* d_row_w, void* stream);

/* Synchronises `stream`, then returns and clears the current device's status word: the first
 * error that a kernel of the calls above recorded since the last call of this function
 * (MOE_ERR_DEVICE_BOUNDS, MOE_ERR_DEVICE_TIMEOUT), MOE_OK, or MOE_ERR_CUDA if the stream
 * itself reports an error.  The word is shared by all streams of the device; it is read and
 * cleared in one step, so that what is recorded meanwhile is left for the next call. */
MOE_API moe_status moe_ops_check_status(void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_OPS_H */
