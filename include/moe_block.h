/*
 * moe_block.h - C ABI of the operators around the routing in an MoE block
 * (same library, libmoe_route.so, as moe_route.h):
 *   layer norm (forward, backward) -> [router, gating, experts, combine: the
 *   whole MoE layer for a few tokens] -> ... -> global gradient norm and
 *   clipping over the block's many weight tensors.
 *
 * The conventions of moe_route.h hold: device pointers owned by the caller,
 * no allocation, work enqueued on `stream` without a host synchronisation,
 * outputs written completely and not aliasing inputs (moe_clip_grads may
 * write in place), MOE_* return codes before anything is enqueued, MOE_STATUS_*
 * bits OR-ed into a nullable `d_status`. The current device is the one of the
 * pointers and the stream.
 * Rows passed with a stride (`*_stride`, in elements, from one row to the
 * next) are contiguous inside a row; the stride is at least the row's length
 * (any value for fewer than two rows).
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe_route.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A mixture-of-experts layer for a few tokens (a decode step):
 *   logits = x router^T                               [T, E]
 *   (top_expert, weights) = moe_topk_gating(logits)   [T, top_k]
 *   g, u   = rows [0, F) and [F, 2F) of w_gate_up[e] times x[t]
 *   h_a    = weights[a] * silu(g) * u                 a = t*top_k + k, e = top_expert[a]
 *   y[t]   = sum_a w_down[e_a] h_a
 * moe_layer is all of it; moe_experts starts from a given routing (such as
 * moe_topk_gating's), where an entry -1 is a slot without an expert: a token
 * whose slots are all -1 gets +0.0. Any other entry outside [0, E) sets
 * MOE_STATUS_BAD_EXPERT and counts as -1.
 * Sums are held in fp32 and y is rounded once. Larger bf16 layers (beyond some
 * 2^24 elements of the choices' matrices, or four choices an expert) run on the
 * tensor cores, which cut instead of rounding as they add (some 1e-5 of a sum),
 * and keep h as the sum of two bf16 numbers, 16 significant bits; both are far
 * below y's own rounding. A token's row depends on its
 * own experts only. The order of every sum is fixed: repeated calls give the
 * same bits.
 * Waits inside the kernels are bounded. One that gives up (after some two
 * seconds) sets MOE_STATUS_TIMEOUT, and what needed its data is NaN: whole rows
 * of y, or whole columns.
 *   x         [T, H] dtype, row stride x_stride; router [E, H] dtype
 *   w_gate_up [E, 2F, H] dtype, the gate rows of an expert before its up rows
 *   w_down    [E, H, F] dtype
 *   top_expert [T, top_k] int32, weights [T, top_k] fp32: outputs of
 *             moe_layer, inputs of moe_experts
 *   y         [T, H] dtype
 *   workspace >= moe_layer_workspace_size(...) bytes, 16-byte aligned, its
 *             contents need no initialisation (0 is returned for sizes that
 *             the calls refuse). Calls that may run at the same time need
 *             workspaces of their own.
 * T <= MOE_LAYER_MAX_TOKENS and T*top_k <= MOE_LAYER_MAX_CHOICES, else
 * MOE_ERR_UNSUPPORTED: with more tokens, weights are no longer what bounds
 * the layer; gather the rows with moe_padded_gather and run the experts as
 * large products. E <= MOE_GATING_MAX_EXPERTS, top_k <= min(E, MOE_MAX_TOP_K).
 */
#define MOE_LAYER_MAX_TOKENS 256
#define MOE_LAYER_MAX_CHOICES 2048
size_t moe_layer_workspace_size(int64_t num_tokens, int64_t hidden, int64_t ffn, int32_t num_experts, int32_t top_k);
int moe_layer(const void* x, int32_t dtype, int64_t x_stride, const void* router, const void* w_gate_up,
              const void* w_down, int64_t num_tokens, int64_t hidden, int64_t ffn, int32_t num_experts,
              int32_t top_k, int32_t mode, int32_t normalize, int32_t* top_expert, float* weights, void* y,
              void* workspace, size_t workspace_bytes, int32_t* d_status, moe_stream_t stream);
int moe_experts(const void* x, int32_t dtype, int64_t x_stride, const int32_t* top_expert, const float* weights,
                const void* w_gate_up, const void* w_down, int64_t num_tokens, int64_t hidden, int64_t ffn,
                int32_t num_experts, int32_t top_k, void* y, void* workspace, size_t workspace_bytes,
                int32_t* d_status, moe_stream_t stream);

/*
 * Testing only: bounded waits inside the kernels of this header give up at
 * once, as if what they wait for never came, so that a test can see how such a
 * call ends. Bits: the layer's copies of weights 1, its copies of tokens 2,
 * its products 4, the reading of their sums 8; layer norm's copies of rows 16;
 * 0 restores all. Process-wide; not for concurrent use with real calls.
 */
void moe_test_block_waits(uint32_t give_up);

/*
 * Layer norm over the last dimension:
 *   mean = sum(x) / H;  rstd = 1 / sqrt(sum((x - mean)^2) / H + eps)
 *   y    = (x - mean) * rstd * weight + bias
 * Statistics are fp32, the variance from the centred values; y is rounded once.
 * Waits inside the kernels are bounded; what needed the data of one that gave
 * up is NaN (whole rows, and the gradients' columns).
 *   x [rows, H] dtype, row stride x_stride; y [rows, H] dtype
 *   weight, bias [H] of weight_dtype, each nullable (1 and 0)
 *   mean, rstd [rows] fp32, nullable: what the backward pass takes.
 * Backward, with xhat = (x - mean) * rstd and v = dy * weight:
 *   dx      = rstd * (v - sum(v)/H - xhat * sum(v * xhat)/H)
 *   dweight = sum over rows of dy * xhat;  dbias = sum over rows of dy
 *   dy, x [rows, H] dtype with row strides; dx [rows, H] dtype;
 *   dweight, dbias [H] of weight_dtype, each nullable; zeros for rows == 0.
 *   workspace >= moe_layer_norm_bwd_workspace_size(rows, hidden) bytes, 16-byte aligned,
 *   contents need no initialisation; not needed (may be NULL) when dweight
 *   and dbias are both NULL. The sums over rows have a fixed order: repeated
 *   calls on one device give the same bits.
 */
int moe_layer_norm_fwd(const void* x, int32_t dtype, int64_t x_stride, const void* weight, const void* bias,
                       int32_t weight_dtype, int64_t rows, int64_t hidden, float eps, void* y, float* mean,
                       float* rstd, moe_stream_t stream);
size_t moe_layer_norm_bwd_workspace_size(int64_t rows, int64_t hidden);
int moe_layer_norm_bwd(const void* dy, int64_t dy_stride, const void* x, int32_t dtype, int64_t x_stride,
                       const void* weight, int32_t weight_dtype, const float* mean, const float* rstd, int64_t rows,
                       int64_t hidden, void* dx, void* dweight, void* dbias, void* workspace,
                       size_t workspace_bytes, moe_stream_t stream);

/*
 * Global norm of many gradients, and clipping:
 *   norm = sqrt(sum over all tensors and elements of g^2)
 *   out  = g * min(1, max_norm / (norm + 1e-6))       (moe_clip_grads)
 * A NaN or infinity among the gradients makes the norm NaN or infinite, and
 * the coefficient NaN or 0, as the formula says. Squares that leave fp32's
 * range do not: such a piece is summed again in 64 bits.
 * The tensors are described by a table of pieces. On the host, the caller
 * fills moe_grad_tensor entries, asks moe_grad_table_pieces for the number of
 * pieces (-1 on invalid entries), lets moe_grad_table_fill write that many
 * moe_grad_piece entries into host memory and copies them to the device; the
 * device copy (16-byte aligned) serves any number of calls for as long as the tensors stay where
 * they are. out is read by moe_clip_grads alone; out == grad clips in place
 * (then nothing is written while the coefficient is 1). Apart from that no
 * out may overlap a grad or another out.
 *   norm [1] fp32 out;
 *   workspace >= moe_grad_norm_workspace_size() bytes, 8-byte aligned,
 *   contents need no initialisation.
 * The sum has a fixed order on a device: repeated calls give the same bits.
 */
typedef struct moe_grad_tensor {
  const void* grad;
  void* out;     /* nullable: then moe_clip_grads leaves the tensor alone */
  int64_t numel;
  int32_t dtype; /* MOE_F32 or MOE_BF16, of grad and out */
  int32_t reserved;
} moe_grad_tensor;
typedef struct moe_grad_piece {
  const void* grad;
  void* out;
  int64_t numel;
  int32_t dtype;
  int32_t reserved;
} moe_grad_piece;
int64_t moe_grad_table_pieces(const moe_grad_tensor* tensors, int64_t num_tensors);
int moe_grad_table_fill(const moe_grad_tensor* tensors, int64_t num_tensors, moe_grad_piece* pieces,
                        int64_t num_pieces);
size_t moe_grad_norm_workspace_size(void);
int moe_grad_norm(const moe_grad_piece* pieces, int64_t num_pieces, float* norm, void* workspace,
                  size_t workspace_bytes, moe_stream_t stream);
int moe_clip_grads(const moe_grad_piece* pieces, int64_t num_pieces, float max_norm, float* norm, void* workspace,
                   size_t workspace_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
