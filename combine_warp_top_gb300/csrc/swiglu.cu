// The gated activation between an expert's two products, scaled by each row's
// routing weight, and its gradient.  With row i of expert-major gu = [g | u]
// (I gate columns, then I up columns) and w_i the routing weight of the row's
// (token, choice) pair:
//
//   forward   h  = w_i * SiLU(g) * u,  SiLU(g) = g * s, s = 1 / (1 + exp(-g))
//   gradient  dg = w_i * dh * u * s * (1 + g * (1 - s))
//             du = w_i * dh * SiLU(g)
//             dw_i = sum over the columns of dh * SiLU(g) * u
//
// Scaling h instead of the down product's output gives the same layer output
// (the down product is linear) and makes the routing weight's gradient a sum
// over rows that the activation's gradient reads anyway.
//
// Memory bound: 3 (forward) or 5 (gradient) bf16 a column, each moved once in
// 16-byte vectors; arithmetic in fp32, one rounding to bf16 on store.
#include "../../include/moe_train.h"
#include "api_checks.cuh"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kBlock = 256;

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// exp and divide of the hardware: about 1e-6 relative, far below bf16's 4e-3
// (and the routing weight's sum of many such terms averages it further down)
__device__ __forceinline__ float sigmoid(float g) {
    return __fdividef(1.0f, 1.0f + __expf(-g));
}

// The (token, choice) pair of expert-major row i: the token from the layout,
// the choice from the lane whose pair_row names the row.  Whole warp; -1 if the
// layout names none.
__device__ __forceinline__ long long pair_of_row(const int32_t* __restrict__ row_token,
                                                 const int32_t* __restrict__ pair_row, int N,
                                                 int k, long long row) {
    const int lane = threadIdx.x & 31;
    const int t = row_token[row];
    if ((unsigned)t >= (unsigned)N) return -1;
    const bool mine = lane < k && pair_row[(long long)t * k + lane] == row;
    const unsigned hit = __ballot_sync(0xffffffffu, mine);
    return hit ? (long long)t * k + __ffs(hit) - 1 : -1;
}

// A warp takes kVecs x 32 vectors of 8 columns of a row, all their loads in flight
// at once; `parts` such pieces make a row.
template <int kVecs>
__global__ void __launch_bounds__(kBlock)
    swiglu_kernel(const uint4* __restrict__ gu, const float* __restrict__ topk_w,
                  const int32_t* __restrict__ row_token, const int32_t* __restrict__ pair_row,
                  int N, int k, long long pieces, int parts, int V, uint4* __restrict__ h) {
    const int lane = threadIdx.x & 31;
    const long long step = (long long)gridDim.x * (kBlock / 32);
    for (long long p = (long long)blockIdx.x * (kBlock / 32) + (threadIdx.x >> 5); p < pieces;
         p += step) {
        const long long row = p / parts;
        const int first = (int)(p - row * parts) * kVecs * 32 + lane;
        const uint4* g = gu + row * 2 * V;
        uint4 rg[kVecs], ru[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int c = first + i * 32;
            if (c < V) {
                rg[i] = __ldcs(g + c);
                ru[i] = __ldcs(g + V + c);
            }
        }
        float w = 1.0f;
        if (topk_w) {
            const long long q = pair_of_row(row_token, pair_row, N, k, row);
            w = q >= 0 ? topk_w[q] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int c = first + i * 32;
            if (c < V) {
                float a[8], b[8];
                unpack8(rg[i], a);
                unpack8(ru[i], b);
#pragma unroll
                for (int j = 0; j < 8; ++j) a[j] = w * (a[j] * sigmoid(a[j])) * b[j];
                __stcs(h + row * V + c, pack8(a));
            }
        }
    }
}

template <int kRowWarps>
__global__ void __launch_bounds__(kBlock)
    swiglu_grad_kernel(const uint4* __restrict__ dh, const uint4* __restrict__ gu,
                       const float* __restrict__ topk_w, const int32_t* __restrict__ row_token,
                       const int32_t* __restrict__ pair_row, int N, int k, long long R, int V,
                       uint4* __restrict__ dgu, float* __restrict__ dtopk_w) {
    __shared__ float part[kBlock / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kRows = kBlock / 32 / kRowWarps;
    const int first = (warp % kRowWarps) * 32 + lane;
    for (long long row = (long long)blockIdx.x * kRows + warp / kRowWarps; row < R;
         row += (long long)gridDim.x * kRows) {
        float w = 1.0f;
        long long p = -1;
        if (topk_w || dtopk_w) {
            p = pair_of_row(row_token, pair_row, N, k, row);
            if (topk_w) w = p >= 0 ? topk_w[p] : 0.0f;
        }
        const uint4* d = dh + row * V;
        const uint4* g = gu + row * 2 * V;
        const uint4* u = g + V;
        uint4* og = dgu + row * 2 * V;
        uint4* ou = og + V;
        float sum = 0.0f;
#pragma unroll 2
        for (int c = first; c < V; c += 32 * kRowWarps) {
            float x[8], a[8], b[8];
            unpack8(__ldcs(d + c), x);
            unpack8(__ldcs(g + c), a);
            unpack8(__ldcs(u + c), b);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float s = sigmoid(a[j]), act = a[j] * s, y = w * x[j];
                sum += x[j] * act * b[j];
                b[j] = y * b[j] * (s * (1.0f + a[j] * (1.0f - s)));
                a[j] = y * act;
            }
            __stcs(og + c, pack8(b));
            __stcs(ou + c, pack8(a));
        }
        if (dtopk_w) {
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (kRowWarps > 1) {
                if (lane == 0) part[warp] = sum;
                __syncthreads();
                sum = 0.0f;
                for (int i = 0; i < kRowWarps; ++i) sum += part[i];
                __syncthreads();
            }
            if (warp % kRowWarps == 0 && lane == 0 && p >= 0) dtopk_w[p] = sum;
        }
    }
}

// The gradient gives a warp to a row (whose sum is then its own) when that gives
// every SM at least 32 warps and a row is short; long rows leave too few warps in
// the last wave, so a block takes them.
constexpr int kWarpRowVecs = 512;
bool warp_per_row(long long R, int V) { return V <= kWarpRowVecs && R >= 32LL * sm_count(); }

int grid_for(long long blocks) {
    const long long most = 1LL << 30;
    return (int)(blocks < most ? blocks : most);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_swiglu(const uint16_t* gu, const float* topk_w, const moe_layout* layout,
                      const moe_shape* shape, uint16_t* h, void* stream) {
    MOE_RANGE();
    MOE_TRY(check_shape(shape));
    MOE_TRY(check_layout(layout, shape));
    if (shape->N == 0) return MOE_OK;
    if (!gu || !h || !aligned16(gu, h)) return MOE_ERR_INVALID_ARG;
    const long long R = (long long)shape->N * shape->k;
    const uint4* in = reinterpret_cast<const uint4*>(gu);
    uint4* out = reinterpret_cast<uint4*>(h);
    const int V = shape->I / 8;
    // the widest pieces that leave no more lanes idle than narrower ones
    const auto wide = [V](int vecs) { return (V + 32 * vecs - 1) / (32 * vecs) * vecs; };
    const int vecs = wide(4) == wide(1) ? 4 : wide(2) == wide(1) ? 2 : 1;
    const int parts = (V + 32 * vecs - 1) / (32 * vecs);
    const long long pieces = R * parts;
    const int grid = grid_for((pieces + kBlock / 32 - 1) / (kBlock / 32));
    const auto go = [&](auto kernel) {
        kernel<<<grid, kBlock, 0, as_stream(stream)>>>(in, topk_w, layout->row_token,
                                                       layout->pair_row, shape->N, shape->k,
                                                       pieces, parts, V, out);
    };
    if (vecs == 4) go(swiglu_kernel<4>);
    else if (vecs == 2) go(swiglu_kernel<2>);
    else go(swiglu_kernel<1>);
    return cuda_status(cudaGetLastError());
}

moe_status moe_swiglu_grad(const uint16_t* dh, const uint16_t* gu, const float* topk_w,
                           const moe_layout* layout, const moe_shape* shape, uint16_t* dgu,
                           float* dtopk_w, void* stream) {
    MOE_RANGE();
    MOE_TRY(check_shape(shape));
    MOE_TRY(check_layout(layout, shape));
    if (shape->N == 0) return MOE_OK;
    if (!dh || !gu || !dgu || !aligned16(dh, gu, dgu)) return MOE_ERR_INVALID_ARG;
    const long long R = (long long)shape->N * shape->k;
    const uint4* d = reinterpret_cast<const uint4*>(dh);
    const uint4* in = reinterpret_cast<const uint4*>(gu);
    uint4* out = reinterpret_cast<uint4*>(dgu);
    const int V = shape->I / 8;
    if (warp_per_row(R, V))
        swiglu_grad_kernel<1><<<grid_for((R + 7) / 8), kBlock, 0, as_stream(stream)>>>(
            d, in, topk_w, layout->row_token, layout->pair_row, shape->N, shape->k, R, V, out,
            dtopk_w);
    else
        swiglu_grad_kernel<8><<<grid_for(R), kBlock, 0, as_stream(stream)>>>(
            d, in, topk_w, layout->row_token, layout->pair_row, shape->N, shape->k, R, V, out,
            dtopk_w);
    return cuda_status(cudaGetLastError());
}

}  // extern "C"
