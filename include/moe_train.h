/*
 * moe_train.h -- C ABI of libmoe, part two: the operators that a training step
 * of the expert layer needs next to the forward pass of moe.h.
 *
 * The conventions of moe.h hold here: device pointers owned by the caller,
 * dense row-major 16-byte aligned tensors, asynchronous on `stream`, arguments
 * checked on the host before anything is launched, nothing allocated.
 * No call here uses atomics whose order could change a result: every output is
 * the same from run to run on one GPU model.
 * The kernels are launched with programmatic stream serialization: their blocks
 * may start when those of the kernel before them on the stream are through, and
 * wait for its writes before they touch memory.
 */
#ifndef MOE_TRAIN_H
#define MOE_TRAIN_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of a tensor that may be either. */
typedef enum {
    MOE_TYPE_BF16 = 0,
    MOE_TYPE_F32 = 1
} moe_type;

/* Matrix products grouped by expert, and their gradients.  The rows are the
 * N*k expert-major rows of the layout (expert e's are the expert_counts[e]
 * rows from expert_offsets[e]; any count, zero included), W[e] is a row-major
 * [C_out, C_in] matrix (nn.Linear), whatever shape->weights says:
 *   moe_grouped_gemm              out[i, :]   = rows[i, :] W[e]^T
 *   moe_grouped_gemm_input_grad   drows[i, :] = dout[i, :] W[e]
 *   moe_grouped_gemm_weight_grad  dw[e]       = sum over the expert's rows i of
 *                                               dout[i, :]^T rows[i, :]
 * rows bf16 [N*k, C_in], dout bf16 [N*k, C_out], w bf16 [E, C_out, C_in]; out
 * [N*k, C_out], drows [N*k, C_in] and dw [E, C_out, C_in] of out_type, a
 * moe_type.  C_in and C_out are multiples of 8, N*k is less than 2^31 - 2^20
 * (MOE_ERR_UNSUPPORTED).  shape gives N, k and E; it has to be one that the calls
 * of moe.h take, but its other fields size nothing here.  Products are bf16 with
 * fp32 accumulation on the tensor cores: an output is summed from partial sums of
 * 512 terms (fp32) or 32768 (bf16), added in order and rounded to nearest.  A row's
 * values touch no other row's and no other expert's output.
 * accumulate != 0 adds to dw, which has to be fp32 then (MOE_ERR_UNSUPPORTED
 * otherwise); accumulate == 0 overwrites it, with zeros for an expert without
 * rows (and for every expert when N == 0).
 * Where there are few tiles for the device's SMs, several of them share a long
 * contraction and add up their fp32 sums in a fixed order; how many depends on N*k,
 * E, C_in and C_out (and the device) only.
 * ws: workspace of moe_workspace_bytes(shape) bytes, on a 4-byte boundary.  A layout
 * whose segments leave the N*k rows is reported there (moe_get_error) and those
 * segments are taken as empty; segments that overlap may be reported, too. */
moe_status moe_grouped_gemm(const uint16_t* rows, const moe_layout* layout,
                            const moe_shape* shape, int32_t C_in, int32_t C_out,
                            const uint16_t* w, void* out, int32_t out_type, void* ws,
                            size_t ws_bytes, void* stream);
moe_status moe_grouped_gemm_input_grad(const uint16_t* dout, const moe_layout* layout,
                                       const moe_shape* shape, int32_t C_in, int32_t C_out,
                                       const uint16_t* w, void* drows, int32_t out_type, void* ws,
                                       size_t ws_bytes, void* stream);
moe_status moe_grouped_gemm_weight_grad(const uint16_t* dout, const uint16_t* rows,
                                        const moe_layout* layout, const moe_shape* shape,
                                        int32_t C_in, int32_t C_out, void* dw, int32_t out_type,
                                        int32_t accumulate, void* ws, size_t ws_bytes,
                                        void* stream);

/* The gated activation between an expert's two products, scaled by the routing
 * weight of each expert-major row, and its gradient.  gu bf16 [N*k, 2*I] holds a
 * row's I gate columns g, then its I up columns u (the forward product of the
 * stacked [2*I, H] gate and up matrices):
 *   moe_swiglu       h[i, :]  = bf16( w_i * SiLU(g) * u )          bf16 [N*k, I]
 *   moe_swiglu_grad  dgu[i, :] = bf16( w_i * dh * u * SiLU'(g) ),
 *                                bf16( w_i * dh * SiLU(g) )        bf16 [N*k, 2*I]
 *                    dtopk_w[t, j] = sum over the columns of dh * SiLU(g) * u
 *                                                                  fp32 [N, k]
 * with w_i = topk_w[t, j] of the pair (t, j) whose pair_row is i.  With h scaled
 * here, the layer's output is the plain sum of each token's k rows of the down
 * product (moe_combine with weights of one).  topk_w may be NULL (weights of
 * one); dtopk_w may be NULL (not wanted).  shape gives N, k and I. */
moe_status moe_swiglu(const uint16_t* gu, const float* topk_w, const moe_layout* layout,
                      const moe_shape* shape, uint16_t* h, void* stream);
moe_status moe_swiglu_grad(const uint16_t* dh, const uint16_t* gu, const float* topk_w,
                           const moe_layout* layout, const moe_shape* shape, uint16_t* dgu,
                           float* dtopk_w, void* stream);

/* Gradient of the router's logits, fp32 [N, E], from that of the routing
 * weights, dtopk_w fp32 [N, k], one call per router of moe.h:
 *   moe_route_grad               of moe_route (softmax over the selected k);
 *                                topk_w as that call wrote it
 *   moe_route_full_softmax_grad  of moe_route_full_softmax
 *   moe_route_sigmoid_bias_grad  of moe_route_sigmoid_bias (its bias steers the
 *                                selection only and has no gradient)
 * The selection passes no gradient: outside the full softmax the entries of the
 * experts not selected are zero (written, not left).  Ids out of range take no
 * part.  Of the shape, which has to be one that the calls of moe.h take, N, E and k
 * are used.  The sigmoid router's gradient is finite for any finite logits, also where
 * the selected scores are all too small for fp32. */
moe_status moe_route_grad(const int32_t* topk_ids, const float* topk_w, const float* dtopk_w,
                          const moe_shape* shape, float* dlogits, void* stream);
moe_status moe_route_full_softmax_grad(const float* logits, const int32_t* topk_ids,
                                       const float* dtopk_w, const moe_shape* shape,
                                       float* dlogits, void* stream);
moe_status moe_route_sigmoid_bias_grad(const float* logits, const int32_t* topk_ids,
                                       const float* dtopk_w, const moe_shape* shape,
                                       float* dlogits, void* stream);

/* The gate on a block's output in moe_block_norm. */
typedef enum {
    MOE_GATE_NONE = 0,
    MOE_GATE_CHANNEL = 1, /* fp32 [H], learned, shared by all rows */
    MOE_GATE_TOKEN = 2    /* fp32 [N], one a row */
} moe_gate;

/* N rows (less than 2^31 - 2^20) of width H (a multiple of 8, at most 16384).
 * post, pre: whether there is an RMS norm after the block and one before the
 * next.  gate: a moe_gate.
 * stream_type: the moe_type of the residual stream and its gradients. */
typedef struct {
    int32_t N, H;
    int32_t post, pre;
    int32_t gate;
    int32_t stream_type;
    float eps;
    float residual_scale;
} moe_norm_shape;

/* The boundary between two blocks, row by row, with n(v) = v / sqrt(mean(v^2) +
 * eps):
 *   z = n(y) * w_post                        (z = y when post == 0)
 *   s = residual_scale * residual + gate * z
 *   x = n(s) * w_pre                         (when pre != 0)
 * y bf16 [N, H], the block's output (may be NULL without post and gate: the norm
 * before the first block); residual, s [N, H] of the stream type, s may be the
 * residual itself, or NULL when only x is wanted; x bf16 [N, H]; w_post, w_pre
 * fp32 [H], NULL for ones.  x is the norm of s before it is rounded to the
 * stream's type.  rstd_post, rstd_pre fp32 [N] receive 1 / sqrt(mean + eps) for
 * the gradient (NULL: not wanted). */
moe_status moe_block_norm(const uint16_t* y, const void* residual, const float* w_post,
                          const float* gate, const float* w_pre, const moe_norm_shape* shape,
                          void* s, uint16_t* x, float* rstd_post, float* rstd_pre, void* stream);

/* Bytes of device workspace of moe_block_norm_grad (partial column sums; need
 * not be cleared; 0 if the shape is invalid). */
size_t moe_norm_workspace_bytes(const moe_norm_shape* shape);

/* Its gradient, from ds [N, H] of the stream type (that of s from what follows;
 * NULL for zero when there is a norm before the next block) and dx bf16 [N, H],
 * with y, s and the rstd vectors of the forward call:
 *   dy bf16 [N, H]; dresidual [N, H] of the stream type (NULL: not wanted; may be
 *   ds itself); dw_post, dw_pre fp32 [H] and dgate fp32 [H] or [N] (each NULL: not
 *   wanted).
 * accumulate != 0 adds to dw_post, dw_pre and a per-channel dgate instead of
 * overwriting them. */
moe_status moe_block_norm_grad(const void* ds, const uint16_t* dx, const uint16_t* y,
                               const void* s, const float* w_post, const float* gate,
                               const float* w_pre, const float* rstd_post, const float* rstd_pre,
                               const moe_norm_shape* shape, uint16_t* dy, void* dresidual,
                               float* dw_post, float* dgate, float* dw_pre, int32_t accumulate,
                               void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_TRAIN_H */
