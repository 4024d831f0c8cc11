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
    uint16_t* gu;   // forward: [N*k, 2*I] (NULL: not wanted); gradient: its gradient
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

// exp and divide of the hardware: 2 + 1.2 |g| units of 2^-23 (CUDA's bound), 2e-6 relative at
// |g| = 12, against 2^-8 of a bf16 output.  Below g = -87.3 the quotient is 0, off by less
// than 2^-126.
__device__ __forceinline__ float sigmoid(float g) {
    return __fdividef(1.0f, 1.0f + __expf(-g));
}

}  // namespace moe
