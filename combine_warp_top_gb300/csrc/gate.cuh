// The gate of an expert's feed-forward block inside a product's epilogue: what a row needs
// beside its sums.
#pragma once

#include <stdint.h>

namespace moe {

// h = w_i SiLU(g) u, w_i the routing weight of the (token, choice) pair whose row is i.
struct Gate {
    const float* topk_w;       // [N, k], NULL: ones
    const int32_t* row_token;  // [N*k]
    const int32_t* pair_row;   // [N*k]
    int N, k;
    uint16_t* h;    // forward: [N*k, I]
    uint16_t* gu;   // forward: [N*k, 2*I] (NULL: not wanted); gradient: dgu
    const uint16_t* gu_in;  // gradient: gu
    float* parts;   // gradient: [ceil(I / 128), N*k] sums of dh SiLU(g) u (NULL: not wanted)
};

// The weight of an expert-major row; 0 for one that no pair names.
__device__ __forceinline__ float row_weight(const Gate& g, long long row) {
    if (!g.topk_w) return 1.0f;
    const int t = g.row_token[row];
    if ((unsigned)t >= (unsigned)g.N) return 0.0f;
    const long long first = (long long)t * g.k;
    int hit = -1;
#pragma unroll 4
    for (int j = 0; j < g.k; ++j)
        if (g.pair_row[first + j] == row) hit = j;
    return hit < 0 ? 0.0f : g.topk_w[first + hit];
}

// 1 / (1 + 2^(-g log2 e)) by the hardware's exponential and reciprocal, without the scaling
// that the library's functions give denormal results: a sigmoid below 2^-126 is 0.  The
// product -g log2 e is rounded to fp32, which makes the power off by |g| 2^-24 (and 2^-22 for
// ex2.approx, 2^-23 for rcp.approx): 1e-6 relative at |g| = 12, against 2^-8 of a bf16 output.
__device__ __forceinline__ float sigmoid(float g) {
    float p, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + p));
    return s;
}

}  // namespace moe
