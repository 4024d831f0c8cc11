/*
 * moe_w4.h -- C ABI of libmoe, part three: experts with 4-bit weights, for the few rows an
 * expert of a decoding step.
 *
 * The conventions of moe.h and moe_train.h hold here: device pointers owned by the caller,
 * dense row-major 16-byte aligned tensors, asynchronous on `stream`, arguments checked on
 * the host before anything is launched, nothing allocated, the same bits every run.
 */
#ifndef MOE_W4_H
#define MOE_W4_H

#include "moe_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Matrices of 4-bit weights: weight k of row o is scale[o, k / group] * (q[o, k] - 8), q in
 * 0..15, the scales bf16.  group: 32, 64 or 128, of which C_in is a multiple; C_out is a
 * multiple of 8; both are at most 2^28.  gated: the stacked gate and up matrices
 * [2 * C_out, C_in], gate rows first; else [C_out, C_in]. */
typedef struct {
    int32_t C_out, C_in;
    int32_t group;
    int32_t gated;
} moe_w4_matrix;

/* q and scales of `rows` rows of C_in bf16 weights (finite ones), a scale for each group:
 *   scale = bf16( max |w| / 7 ),  q = w / scale + 8 rounded to nearest even, within 0..15
 * (scale 0 and q 8 where that scale is 0).  q uint8 [rows, C_in / 2], weight 2i in the low
 * four bits of byte i; scales bf16 [rows, C_in / group]. */
moe_status moe_w4_quantize(const uint16_t* w, int64_t rows, int32_t C_in, int32_t group, uint8_t* q,
                           uint16_t* scales, void* stream);

/* The order in which the products read E such matrices (q and scales as above, of any
 * origin), once for each set of weights: packed, moe_w4_packed_bytes bytes (0 if the matrix
 * is invalid), 4 bits a weight and its scales.  256 gate and up matrices of 4096 x 7168 in groups
 * of 128: 8.3 ms to quantise, 19 ms to pack (GB300). */
size_t moe_w4_packed_bytes(const moe_w4_matrix* matrix, int32_t E);
moe_status moe_w4_pack(const uint8_t* q, const uint16_t* scales, const moe_w4_matrix* matrix,
                       int32_t E, void* packed, void* stream);

/* Products of the N*k expert-major rows with their experts' packed matrices:
 *   moe_w4_gemm        out[i, :] = rows[i, :] W[e]^T                   [N*k, C_out]
 *   moe_w4_gated_gemm  [g | u] = rows[i, :] W[e]^T, h[i, :] = bf16( w_i SiLU(g) u )
 *                                                                 bf16 [N*k, C_out]
 * rows bf16 [N*k, C_in]; out of out_type, a moe_type; w_i as in moe_swiglu (topk_w NULL:
 * ones).  Products of bf16 rows with the whole numbers q - 8 are summed in fp32 over a group
 * and scaled then, in fp32.  shape gives N, k and E; rows an expert has: any number, but it
 * is few that this is made for.  An expert's rows go through in passes of 16, 32 or 64 (of 32 at
 * most with groups of 32), chosen once a call by the average of N*k rows over the experts, and
 * every pass reads and widens the expert's weights again: from some hundred rows an expert on,
 * products with bf16 weights are faster.  N*k is less than 2^31 - 2^20.
 * ws: workspace of moe_w4_workspace_bytes(shape) bytes, 16-byte aligned, zero at first.  A
 * layout whose segments leave the N*k rows is reported there (moe_get_error) and those
 * segments are taken as empty; one whose segments overlap may be reported, too, and leave rows
 * without their products.  After MOE_ERR_TIMEOUT it has to be zeroed again. */
size_t moe_w4_workspace_bytes(const moe_shape* shape);
moe_status moe_w4_gemm(const uint16_t* rows, const moe_layout* layout, const moe_shape* shape,
                       const moe_w4_matrix* matrix, const void* packed, void* out,
                       int32_t out_type, void* ws, size_t ws_bytes, void* stream);
moe_status moe_w4_gated_gemm(const uint16_t* rows, const moe_layout* layout,
                             const moe_shape* shape, const moe_w4_matrix* matrix,
                             const void* packed, const float* topk_w, uint16_t* h, void* ws,
                             size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_W4_H */
