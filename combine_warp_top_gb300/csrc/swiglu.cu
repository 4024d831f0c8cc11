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
// 16-byte vectors; arithmetic in fp32, one rounding to bf16 on store.  16384 rows of
// 14336: forward 200 us (7.06 TB/s), gradient 332 us (7.07 TB/s); 262144 rows of 1536:
// gradient 575 us.  All of a lane's loads go out before the three dependent loads of
// the row's weight, and short rows share a warp (rows of 64 columns: 178 and 303 us
// for 2 M rows, 497 and 992 us with a warp each).
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

// exp and divide of the hardware.  The exponential is good to 2 + 1.2 |g| units of 2^-23
// (CUDA's bound): 2e-6 relative at |g| = 12, 1.2e-5 at 85, against the 4e-3 of a bf16 output.
// The routing weight's gradient is an fp32 sum of such terms, a row's, and is as good as
// the largest of them, which are those of gates near zero and above, where s is off by
// exp(-g) of that.  Below g = -87.3 the quotient is 0, which is off by less than 2^-126.
__device__ __forceinline__ float sigmoid(float g) {
    return __fdividef(1.0f, 1.0f + __expf(-g));
}

// The (token, choice) pair of an expert-major row: the token from the layout, the
// choice from the lane whose pair_row names the row.  Run by whole warps, every kLanes
// lanes for a row of their own (live: there is one); -1 if the layout names none.
template <int kLanes>
__device__ __forceinline__ long long pair_of_row(const int32_t* row_token,
                                                 const int32_t* pair_row, int N,
                                                 int k, long long row, bool live) {
    const int lane = threadIdx.x & 31, sub = lane % kLanes;
    const int t = live ? row_token[row] : -1;
    const bool token = (unsigned)t < (unsigned)N;
    long long pair = -1;
    for (int j0 = 0; j0 < k; j0 += kLanes) {
        const int j = j0 + sub;
        const bool mine = token && j < k && pair_row[(long long)t * k + j] == row;
        unsigned hit = __ballot_sync(0xffffffffu, mine);
        if (kLanes < 32) hit = (hit >> (lane - sub)) & ((1u << kLanes % 32) - 1u);
        if (hit) pair = (long long)t * k + j0 + __ffs(hit) - 1;
    }
    return pair;
}

// Pieces of a row: kLanes lanes take kVecs x kLanes vectors of 8 columns of it, all
// their loads in flight at once; `parts` pieces make a row.
template <int kLanes, int kVecs>
__global__ void __launch_bounds__(kBlock)
    swiglu_kernel(const uint4* gu, const float* topk_w,
                  const int32_t* row_token, const int32_t* pair_row,
                  int N, int k, long long pieces, int parts, int V, uint4* h) {
    constexpr int kGroups = kBlock / kLanes;
    const int sub = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int in_warp = (threadIdx.x & 31) / kLanes;  // a warp's groups leave together
    const long long step = (long long)gridDim.x * kGroups;
    after_previous();
    for (long long p = (long long)blockIdx.x * kGroups + group; p - in_warp < pieces; p += step) {
        const bool live = kLanes == 32 || p < pieces;
        const long long row = live ? p / parts : 0;
        const int first = (int)(p - row * parts) * kVecs * kLanes + sub;
        const uint4* g = gu + row * 2 * V;
        uint4 rg[kVecs], ru[kVecs];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int c = first + i * kLanes;
            if (live && c < V) {
                rg[i] = __ldcs(g + c);
                ru[i] = __ldcs(g + V + c);
            }
        }
        float w = 1.0f;
        if (topk_w) {
            const long long q = pair_of_row<kLanes>(row_token, pair_row, N, k, row, live);
            w = q >= 0 ? topk_w[q] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int c = first + i * kLanes;
            if (live && c < V) {
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

// A row for kLanes lanes of a warp (8, 16 or 32), or (kLanes = 128 or 256) for a
// block.  The first loads of a row are in flight while its pair is looked up.
template <int kLanes>
__global__ void __launch_bounds__(kLanes > 32 ? kLanes : kBlock)
    swiglu_grad_kernel(const uint4* dh, const uint4* gu,
                       const float* topk_w, const int32_t* row_token,
                       const int32_t* pair_row, int N, int k, long long R, int V,
                       uint4* dgu, float* dtopk_w) {
    constexpr bool kBlockRow = kLanes > 32;
    constexpr int kLook = kBlockRow ? 32 : kLanes;  // lanes that look up a pair
    constexpr int kVecs = 2, kGroups = kBlockRow ? 1 : kBlock / kLanes;
    __shared__ float part[8];
    const int sub = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int in_warp = kBlockRow ? 0 : (threadIdx.x & 31) / kLanes;
    const long long step = (long long)gridDim.x * kGroups;
    after_previous();
    for (long long row = (long long)blockIdx.x * kGroups + group; row - in_warp < R; row += step) {
        const bool live = kLanes >= 32 || row < R;
        const uint4* d = dh + row * V;
        const uint4* g = gu + row * 2 * V;
        uint4* og = dgu + row * 2 * V;
        uint4 rd[kVecs], rg[kVecs], ru[kVecs];
        auto load = [&](int c0) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int c = c0 + i * kLanes;
                if (live && c < V) {
                    rd[i] = __ldcs(d + c);
                    rg[i] = __ldcs(g + c);
                    ru[i] = __ldcs(g + V + c);
                }
            }
        };
        load(sub);
        float w = 1.0f;
        long long p = -1;
        if (topk_w || dtopk_w) {
            p = pair_of_row<kLook>(row_token, pair_row, N, k, row, live);
            if (topk_w) w = p >= 0 ? topk_w[p] : 0.0f;
        }
        float sum = 0.0f;
        for (int c0 = sub; c0 < V; c0 += kVecs * kLanes) {
            if (c0 != sub) load(c0);
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int c = c0 + i * kLanes;
                if (live && c < V) {
                    float x[8], a[8], b[8];
                    unpack8(rd[i], x);
                    unpack8(rg[i], a);
                    unpack8(ru[i], b);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float s = sigmoid(a[j]), act = a[j] * s, y = w * x[j];
                        sum += x[j] * act * b[j];
                        b[j] = y * b[j] * (s * (1.0f + a[j] * (1.0f - s)));
                        a[j] = y * act;
                    }
                    __stcs(og + c, pack8(b));
                    __stcs(og + V + c, pack8(a));
                }
            }
        }
        if (dtopk_w) {
#pragma unroll
            for (int o = kLook / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (kBlockRow) {
                if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
                __syncthreads();
                sum = 0.0f;
                for (int i = 0; i < kLanes / 32; ++i) sum += part[i];
                __syncthreads();
            }
            if (sub == 0 && p >= 0) dtopk_w[p] = sum;
        }
    }
}

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
    // lanes of a piece: a warp, or as many as a short row has vectors; vectors a lane:
    // the most that leave at most a fifth of the lanes idle in a row
    const int lanes = V <= 8 ? 8 : V <= 16 ? 16 : 32;
    const auto wide = [V, lanes](int vecs) {
        return (V + lanes * vecs - 1) / (lanes * vecs) * vecs;
    };
    const int vecs = wide(4) * 4 <= wide(1) * 5 ? 4 : wide(2) * 4 <= wide(1) * 5 ? 2 : 1;
    const int parts = (V + lanes * vecs - 1) / (lanes * vecs);
    const long long pieces = R * parts, groups = kBlock / lanes;
    const int grid = grid_for((pieces + groups - 1) / groups);
    const auto go = [&](auto kernel) {
        return launch_chained(kernel, grid, kBlock, 0, as_stream(stream), in, topk_w,
                              layout->row_token, layout->pair_row, shape->N, shape->k, pieces,
                              parts, V, out);
    };
    return cuda_status(lanes == 8    ? go(swiglu_kernel<8, 1>)
                       : lanes == 16 ? go(swiglu_kernel<16, 1>)
                       : vecs == 4   ? go(swiglu_kernel<32, 4>)
                       : vecs == 2   ? go(swiglu_kernel<32, 2>)
                                     : go(swiglu_kernel<32, 1>));
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
    const auto go = [&](auto kernel, int block, long long groups) {
        return launch_chained(kernel, grid_for((R + groups - 1) / groups), block, 0,
                              as_stream(stream), d, in, topk_w, layout->row_token, layout->pair_row,
                              shape->N, shape->k, R, V, out, dtopk_w);
    };
    // A warp (or the lanes of a short row) takes a row when that gives every SM at
    // least 32 warps and a row is not long; long rows leave too few warps in the last
    // wave, so a block of 4 or 8 warps takes them, whichever idles less.
    return cuda_status(
        V <= 8                                  ? go(swiglu_grad_kernel<8>, kBlock, kBlock / 8)
        : V <= 16                               ? go(swiglu_grad_kernel<16>, kBlock, kBlock / 16)
        : V <= 512 && R >= 32LL * sm_count()    ? go(swiglu_grad_kernel<32>, kBlock, kBlock / 32)
        : (V + 255) / 256 * 2 > (V + 127) / 128 ? go(swiglu_grad_kernel<128>, 128, 1)
                                                : go(swiglu_grad_kernel<256>, 256, 1));
}

}  // extern "C"
