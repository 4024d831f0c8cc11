// Gradient of the router's logits from that of the routing weights, for the
// three routers.  With the selected experts e_j, their weights w_j and
// d_j = dL/dw_j (0 for the experts not selected):
//
//   softmax over the selected k    dlogit[e_j] = w_j * (d_j - sum_i w_i d_i)
//   softmax over all E             dlogit[e]   = p_e * (d_e - sum_i p_{e_i} d_i)
//   sigmoid, renormalised          dlogit[e_j] = s_j (1 - s_j) / S
//                                                * (d_j - sum_i w_i d_i),
//     s_j = sigmoid(logit[e_j]), S = sum_i s_i, w_j = s_j / S (the selection bias
//     takes no part in the weights and has no gradient)
//
// The selection itself is piecewise constant and passes no gradient, so outside
// the full softmax the gradient is zero but for k entries a token.
//
// Memory bound: N * E fp32 written (and read, full softmax).  One warp a token:
// lane j holds choice j; the row is put together in shared memory and leaves in
// whole 16-byte vectors, so the scattered entries cost no extra global write.
// The warp's row is all zeros between tokens: only the k entries are put back.
// 32768 tokens of 256 experts, full softmax: 14 us for 69 MB (the bytes' time is 10 us,
// launch and tail the rest); 4096 of 64: 2.6 us, a launch.
#include <math.h>

#include "../../include/moe_train.h"
#include "api_checks.cuh"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;

enum Router { kSoftmax, kFullSoftmax, kSigmoid };

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// kPer: row elements a lane holds, in groups of kVec consecutive ones (4 when E
// is a multiple of 4).  in: the weights (kSoftmax) or the logits.
template <int kRouter, int kPer, int kVec>
__global__ void __launch_bounds__(32 * kWarps)
    route_grad_kernel(const float* __restrict__ in, const int32_t* __restrict__ ids,
                      const float* __restrict__ dw, int N, int E, int k,
                      float* __restrict__ dlogits) {
    extern __shared__ __align__(16) float rows[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pitch = (E + 3) & ~3;
    float* row = rows + warp * pitch;
    for (int c = lane; c < pitch; c += 32) row[c] = 0.0f;
    __syncwarp();
    for (long long t = (long long)blockIdx.x * kWarps + warp; t < N;
         t += (long long)gridDim.x * kWarps) {
        float v[kPer];
        if (kRouter == kFullSoftmax) {
#pragma unroll
            for (int i = 0; i < kPer / kVec; ++i) {
                const int c = (i * 32 + lane) * kVec;
                if (kVec == 4) {
                    float4 x = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                    if (c < E) x = __ldcs(reinterpret_cast<const float4*>(in + t * E + c));
                    v[i * kVec] = x.x;
                    v[i * kVec + 1 % kVec] = x.y;
                    v[i * kVec + 2 % kVec] = x.z;
                    v[i * kVec + 3 % kVec] = x.w;
                } else {
                    v[i] = c < E ? __ldcs(in + t * E + c) : -INFINITY;
                }
            }
        }
        // choice j of the token in lane j; an id out of range takes no part
        int id = -1;
        float d = 0.0f, x = 0.0f, rest = 0.0f;  // rest: 1 - sigmoid
        if (lane < k) {
            id = ids[t * k + lane];
            if ((unsigned)id >= (unsigned)E) id = -1;
            d = dw[t * k + lane];
            if (kRouter == kSoftmax) x = in[t * k + lane];
            if (kRouter == kSigmoid && id >= 0) {
                const float l = in[t * E + id];
                x = 1.0f / (1.0f + expf(-l));
                rest = 1.0f / (1.0f + expf(l));
            }
            if (id < 0) x = d = 0.0f;
        }
        float dot = 0.0f, inv = 0.0f;
        if (kRouter == kFullSoftmax) {
            float m = v[0];
#pragma unroll
            for (int i = 1; i < kPer; ++i) m = fmaxf(m, v[i]);
            m = warp_max(m);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                v[i] = expf(v[i] - m);
                sum += v[i];
            }
            inv = 1.0f / warp_sum(sum);
            if (id >= 0) row[id] = d;
        } else {
            if (kRouter == kSigmoid) {
                const float total = warp_sum(x);
                const float w = x / total;
                const float own = d - warp_sum(w * d);
                d = own * w * rest;
            } else {
                d = x * (d - warp_sum(x * d));
            }
            if (id >= 0) row[id] = d;
        }
        __syncwarp();
        if (kRouter == kFullSoftmax) {
            // p . d over the row: zero where nothing is selected
#pragma unroll
            for (int i = 0; i < kPer / kVec; ++i) {
                const int c = (i * 32 + lane) * kVec;
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (c < E) dot += v[i * kVec + j] * row[c + j];
            }
            dot = warp_sum(dot) * inv;
        }
#pragma unroll
        for (int i = 0; i < kPer / kVec; ++i) {
            const int c = (i * 32 + lane) * kVec;
            if (c < E) {
                float o[kVec];
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    o[j] = row[c + j];
                    if (kRouter == kFullSoftmax) o[j] = v[i * kVec + j] * inv * (o[j] - dot);
                }
                if (kVec == 4)
                    __stcs(reinterpret_cast<float4*>(dlogits + t * E + c),
                           make_float4(o[0], o[1 % kVec], o[2 % kVec], o[3 % kVec]));
                else
                    __stcs(dlogits + t * E + c, o[0]);
            }
        }
        __syncwarp();
        if (id >= 0) row[id] = 0.0f;
        __syncwarp();
    }
}

template <int kRouter, int kPer, int kVec>
cudaError_t launch_one(const float* in, const int32_t* ids, const float* dw, const moe_shape& s,
                       float* dlogits, cudaStream_t st) {
    const long long blocks = (s.N + kWarps - 1) / kWarps, most = 16LL * sm_count();
    const size_t smem = (size_t)kWarps * ((s.E + 3) & ~3) * sizeof(float);
    route_grad_kernel<kRouter, kPer, kVec>
        <<<(int)(blocks < most ? blocks : most), 32 * kWarps, smem, st>>>(in, ids, dw, s.N, s.E,
                                                                          s.k, dlogits);
    return cudaGetLastError();
}

template <int kRouter>
cudaError_t launch_router(const float* in, const int32_t* ids, const float* dw,
                          const moe_shape& s, float* dlogits, cudaStream_t st) {
    const bool vec = s.E % 4 == 0 && ((uintptr_t)dlogits & 15) == 0 &&
                     (kRouter != kFullSoftmax || ((uintptr_t)in & 15) == 0);
    if (vec) {
        if (s.E <= 128) return launch_one<kRouter, 4, 4>(in, ids, dw, s, dlogits, st);
        if (s.E <= 256) return launch_one<kRouter, 8, 4>(in, ids, dw, s, dlogits, st);
        if (s.E <= 512) return launch_one<kRouter, 16, 4>(in, ids, dw, s, dlogits, st);
        return launch_one<kRouter, 32, 4>(in, ids, dw, s, dlogits, st);
    }
    if (s.E <= 256) return launch_one<kRouter, 8, 1>(in, ids, dw, s, dlogits, st);
    return launch_one<kRouter, 32, 1>(in, ids, dw, s, dlogits, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_route_grad(const int32_t* topk_ids, const float* topk_w, const float* dtopk_w,
                          const moe_shape* shape, float* dlogits, void* stream) {
    MOE_RANGE();
    MOE_TRY(check_shape(shape));
    if (shape->N == 0) return MOE_OK;
    if (!topk_ids || !topk_w || !dtopk_w || !dlogits) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_router<kSoftmax>(topk_w, topk_ids, dtopk_w, *shape, dlogits,
                                               as_stream(stream)));
}

moe_status moe_route_full_softmax_grad(const float* logits, const int32_t* topk_ids,
                                       const float* dtopk_w, const moe_shape* shape,
                                       float* dlogits, void* stream) {
    MOE_RANGE();
    MOE_TRY(check_shape(shape));
    if (shape->N == 0) return MOE_OK;
    if (!logits || !topk_ids || !dtopk_w || !dlogits) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_router<kFullSoftmax>(logits, topk_ids, dtopk_w, *shape, dlogits,
                                                   as_stream(stream)));
}

moe_status moe_route_sigmoid_bias_grad(const float* logits, const int32_t* topk_ids,
                                       const float* dtopk_w, const moe_shape* shape,
                                       float* dlogits, void* stream) {
    MOE_RANGE();
    MOE_TRY(check_shape(shape));
    if (shape->N == 0) return MOE_OK;
    if (!logits || !topk_ids || !dtopk_w || !dlogits) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_router<kSigmoid>(logits, topk_ids, dtopk_w, *shape, dlogits,
                                               as_stream(stream)));
}

}  // extern "C"
