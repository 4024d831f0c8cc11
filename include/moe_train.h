/*
 * moe_train.h -- C ABI of libmoe, part two: the operators that a training step
 * of the expert layer needs next to the forward pass of moe.h.
 *
 * The conventions of moe.h hold here: device pointers owned by the caller,
 * dense row-major 16-byte aligned tensors (moe_norm_shape's and the routing
 * weights' fp32 vectors included where noted), asynchronous on `stream`,
 * arguments checked on the host before anything is launched, nothing allocated.
 * No call here uses atomics whose order could change a result: every output is
 * the same from run to run on one GPU model.
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
 * moe_type.  C_in and C_out are multiples of 8; shape gives N, k and E (its H
 * and I are not read).  Products are bf16 with fp32 accumulation on the tensor
 * cores; an fp32 output is summed from partial sums of 512 terms, added in
 * order and rounded to nearest.  A row's values touch no other row's and no
 * other expert's output.
 * accumulate != 0 adds to dw, which has to be fp32 then (MOE_ERR_UNSUPPORTED
 * otherwise); accumulate == 0 overwrites it, with zeros for an expert without
 * rows (and for every expert when N == 0).
 * ws: workspace of moe_workspace_bytes(shape) bytes.  A layout whose segments
 * leave the N*k rows is reported there (moe_get_error) and those segments are
 * taken as empty. */
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

#ifdef __cplusplus
}
#endif

#endif /* MOE_TRAIN_H */
