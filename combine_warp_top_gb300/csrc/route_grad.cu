// Gradient of the router's logits from that of the routing weights, for the
// three routers.  With the selected experts e_j, their weights w_j and
// d_j = dL/dw_j (0 for the experts not selected):
//
//   softmax over the selected k    dlogit[e_j] = w_j * (d_j - sum_i w_i d_i)
//   softmax over all E             dlogit[e]   = p_e * (d_e - sum_i p_{e_i} d_i)
//   sigmoid, renormalised          dlogit[e_j] = s_j (1 - s_j) / S
//                                                * (d_j - sum_i w_i d_i),
//     s_j = sigmoid(logit[e_j]), S = sum_i s_i, w_j = s_j / S (the selection bias
//     takes no part in the weights and has no gradient).  The scores are taken times
//     exp(-m), m = min(0, the largest selected logit), which leaves the weights as they
//     are: s_j exp(-m) = exp(l_j - m) / (1 + exp(l_j)) for l_j <= 0, so that they do not
//     all underflow where every selected logit is far below zero (fp32 scores are zero
//     from -104 on, and 0 / 0 would be the weight).
//
// The selection itself is piecewise constant and passes no gradient, so outside
// the full softmax the gradient is zero but for k entries a token.
//
// Memory bound: N * E fp32 written (and read, full softmax).  A warp, or 8 or 16 lanes of
// one, take a token: lane j holds choice j; the row is put together in shared memory and
// leaves in whole 16-byte vectors, so the scattered entries cost no extra global write.
// The row is all zeros between tokens: only the k entries are put back.  With a warp for
// every token the instructions for it (three sums over the lanes, the choices) take longer
// than a short row's bytes.  32768 tokens, full softmax: of 256 experts 12.0 us (a warp each:
// 13.4 us; the 69 MB take 10.2; back to back 10.8), of 128 7.4 us (8.1), of 64 4.2
// us (7.9); softmax over the selected, of 64 3.5 us (5.5).  4096 of 64: 1.9 us, a launch.
// Sigmoid, of 256 10.9 us, of 64 4.3: it writes as much as the softmax over the selected
// (5.8 and 2.8 us beside it) and reads k logits a token from 32-byte sectors of their own.
// The next token's loads a token ahead measured slower (15.9 us of 256).
#include <float.h>
#include <math.h>

#include "../../include/moe_train.h"
#include "api_checks.cuh"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;

enum Router { kSoftmax, kFullSoftmax, kSigmoid };

template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int kLanes>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int o = kLanes / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// kLanes lanes of a warp take a token, each kPer elements of its row, in groups of kVec
// consecutive ones (4 when E is a multiple of 4).  in: the weights (kSoftmax) or the logits.
template <int kRouter, int kLanes, int kPer, int kVec>
__global__ void __launch_bounds__(32 * kWarps)
    route_grad_kernel(const float* in, const int32_t* ids,
                      const float* dw, int N, int E, int k,
                      float* dlogits) {
    extern __shared__ __align__(16) float rows[];
    constexpr int kGroups = 32 * kWarps / kLanes;  // tokens of a block
    const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const int pitch = (E + 3) & ~3;
    float* row = rows + group * pitch;
    for (int c = lane; c < pitch; c += kLanes) row[c] = 0.0f;
    after_previous();
    __syncwarp();
    const int ahead = (threadIdx.x & 31) / kLanes;  // of the warp's first token
    for (long long t = (long long)blockIdx.x * kGroups + group; t - ahead < N;
         t += (long long)gridDim.x * kGroups) {
        const bool live = t < N;
        float v[kPer];
        if (kRouter == kFullSoftmax) {
#pragma unroll
            for (int i = 0; i < kPer / kVec; ++i) {
                const int c = (i * kLanes + lane) * kVec;
                if (kVec == 4) {
                    float4 x = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                    if (c < E && live) x = __ldcs(reinterpret_cast<const float4*>(in + t * E + c));
                    v[i * kVec] = x.x;
                    v[i * kVec + 1 % kVec] = x.y;
                    v[i * kVec + 2 % kVec] = x.z;
                    v[i * kVec + 3 % kVec] = x.w;
                } else {
                    v[i] = c < E && live ? __ldcs(in + t * E + c) : -INFINITY;
                }
            }
        }
        // choice j of the token in lane j; an id out of range takes no part
        int id = -1;
        float d = 0.0f, x = 0.0f, rest = 0.0f;  // rest: 1 - sigmoid
        if (lane < k && live) {
            id = ids[t * k + lane];
            if ((unsigned)id >= (unsigned)E) id = -1;
            d = dw[t * k + lane];
            if (kRouter == kSoftmax) x = in[t * k + lane];
            if (kRouter == kSigmoid && id >= 0) x = in[t * E + id];
            if (id < 0) x = d = 0.0f;
        }
        if (kRouter == kSigmoid) {
            // (a lane without a choice takes no part in the maximum)
            const float l = x, top = lanes_max<kLanes>(id < 0 ? -FLT_MAX : fmaxf(l, -FLT_MAX));
            const float e = expf(-fabsf(l)), inv = 1.0f / (1.0f + e);
            x = id < 0 ? 0.0f : l > 0.0f ? inv : expf(l - fminf(top, 0.0f)) * inv;
            rest = l > 0.0f ? e * inv : inv;
        }
        float inv = 0.0f;
        if (kRouter == kFullSoftmax) {
            float m = v[0];
#pragma unroll
            for (int i = 1; i < kPer; ++i) m = fmaxf(m, v[i]);
            m = lanes_max<kLanes>(m);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                v[i] = expf(v[i] - m);
                sum += v[i];
            }
            inv = 1.0f / lanes_sum<kLanes>(sum);
        } else if (kRouter == kSigmoid) {
            const float total = lanes_sum<kLanes>(x);
            const float w = total == 0.0f ? 0.0f : x / total;  // 0: no choice of the token counts
            const float own = d - lanes_sum<kLanes>(w * d);
            d = own * w * rest;
        } else {
            d = x * (d - lanes_sum<kLanes>(x * d));
        }
        if (id >= 0) row[id] = d;
        __syncwarp();
        float o[kPer];
#pragma unroll
        for (int i = 0; i < kPer / kVec; ++i) {
            const int c = (i * kLanes + lane) * kVec;
            if (kVec == 4) {
                float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (c < E) r = *reinterpret_cast<const float4*>(row + c);
                o[i * kVec] = r.x;
                o[i * kVec + 1 % kVec] = r.y;
                o[i * kVec + 2 % kVec] = r.z;
                o[i * kVec + 3 % kVec] = r.w;
            } else {
                o[i] = c < E ? row[c] : 0.0f;
            }
        }
        __syncwarp();
        if (id >= 0) row[id] = 0.0f;
        if (kRouter == kFullSoftmax) {
            // p . d over the row: zero where nothing is selected
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) dot += v[i] * o[i];
            dot = lanes_sum<kLanes>(dot) * inv;
#pragma unroll
            for (int i = 0; i < kPer; ++i) o[i] = v[i] * inv * (o[i] - dot);
        }
#pragma unroll
        for (int i = 0; i < kPer / kVec; ++i) {
            const int c = (i * kLanes + lane) * kVec;
            if (c < E && live) {
                if (kVec == 4)
                    __stcs(reinterpret_cast<float4*>(dlogits + t * E + c),
                           make_float4(o[i * kVec], o[i * kVec + 1 % kVec], o[i * kVec + 2 % kVec],
                                       o[i * kVec + 3 % kVec]));
                else
                    __stcs(dlogits + t * E + c, o[i]);
            }
        }
        __syncwarp();
    }
}

template <int kRouter, int kLanes, int kPer, int kVec>
cudaError_t launch_one(const float* in, const int32_t* ids, const float* dw, const moe_shape& s,
                       float* dlogits, cudaStream_t st) {
    constexpr int kGroups = 32 * kWarps / kLanes;
    const long long blocks = (s.N + kGroups - 1LL) / kGroups, most = 16LL * sm_count();
    const size_t smem = (size_t)kGroups * ((s.E + 3) & ~3) * sizeof(float);
    return launch_chained(route_grad_kernel<kRouter, kLanes, kPer, kVec>,
                          (int)(blocks < most ? blocks : most), 32 * kWarps, smem, st, in, ids, dw,
                          s.N, s.E, s.k, dlogits);
}

template <int kRouter>
cudaError_t launch_router(const float* in, const int32_t* ids, const float* dw,
                          const moe_shape& s, float* dlogits, cudaStream_t st) {
    const bool vec = s.E % 4 == 0 && ((uintptr_t)dlogits & 15) == 0 &&
                     (kRouter != kFullSoftmax || ((uintptr_t)in & 15) == 0);
    if (vec) {
        if (s.E <= 64 && s.k <= 8) return launch_one<kRouter, 8, 8, 4>(in, ids, dw, s, dlogits, st);
        if (s.E <= 128 && s.k <= 16)
            return launch_one<kRouter, 16, 8, 4>(in, ids, dw, s, dlogits, st);
        if (s.E <= 256 && s.k <= 16)
            return launch_one<kRouter, 16, 16, 4>(in, ids, dw, s, dlogits, st);
        if (s.E <= 256) return launch_one<kRouter, 32, 8, 4>(in, ids, dw, s, dlogits, st);
        if (s.E <= 512) return launch_one<kRouter, 32, 16, 4>(in, ids, dw, s, dlogits, st);
        return launch_one<kRouter, 32, 32, 4>(in, ids, dw, s, dlogits, st);
    }
    if (s.E <= 256) return launch_one<kRouter, 32, 8, 1>(in, ids, dw, s, dlogits, st);
    return launch_one<kRouter, 32, 32, 1>(in, ids, dw, s, dlogits, st);
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
