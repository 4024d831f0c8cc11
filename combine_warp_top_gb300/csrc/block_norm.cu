// RMS norms after a block and before the next one, fused with the block's gate,
// the residual scale and the residual add, and their gradient.  Row by row,
// with n(v) = v * r(v), r(v) = 1 / sqrt(mean(v^2) + eps):
//
//   z = n(y) * w_post                 (z = y without the norm after the block)
//   s = alpha * residual + gate * z   the residual stream, gate per channel, per
//                                     token or 1
//   x = n(s) * w_pre                  the next block's input
//
// and backwards, from ds (the stream's gradient from further on) and dx, with
// yh = n(y), sh = n(s), mean over the columns:
//
//   g = ds + r_pre * (dx w_pre - sh * mean(dx w_pre sh))
//   dresidual = alpha * g
//   dy = r_post * (b - yh * mean(b yh)),   b = gate * g * w_post
//   dw_pre = sum over rows of dx sh;  dw_post = sum of gate g yh
//   dgate = sum of g yh w_post over the rows (per channel) or columns (per token)
//
// Both are memory bound: forward reads y and the residual once and writes s and
// x; the gradient reads ds, dx, y and s once and writes dy and dresidual.  A row
// stays in registers between its two reductions.  All sums are fp32 in a fixed
// order: columns by shuffle trees, rows of a column by the thread that owns the
// column over its block's rows, then over the blocks' partial sums (in the
// workspace) by a second kernel.
#include "../../include/moe_train.h"
#include "api_checks.cuh"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kMaxNormH = 16384;
constexpr int kRowWarps = 4;   // rows (warps) of a block where a warp takes a row
constexpr int kWarpRowV = 64;  // up to this many vectors of 8 a row: H <= 512

struct NormArgs {
    const uint16_t* y;       // block output, bf16 (null: none)
    const void* residual;    // stream type
    const float* w_post;     // null: ones
    const float* gate;       // per channel or per token
    const float* w_pre;      // null: ones
    void* s;                 // stream out (null: not stored)
    uint16_t* x;
    float* rstd_post;
    float* rstd_pre;
    int N, V;                // V = H / 8
    int post, pre, gate_kind;
    float eps, alpha, inv_h;
};

struct NormGradArgs {
    const void* ds;          // null: zero
    const uint16_t* dx;
    const uint16_t* y;
    const void* s;
    const float* w_post;
    const float* gate;
    const float* w_pre;
    const float* rstd_post;
    const float* rstd_pre;
    uint16_t* dy;
    void* dresidual;         // null: not wanted
    float* dgate_token;
    float* partial;          // [grid][2][H]: sums of g yh (gated per token), of dx sh
    int N, V;
    int post, pre, gate_kind;
    float alpha, inv_h;
};

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

// 8 consecutive values of a stream tensor (vector index v), streamed past L1.
template <bool kF32>
__device__ __forceinline__ void load_stream(const void* p, long long v, float (&f)[8]) {
    if (kF32) {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(p) + 2 * v);
        const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 2 * v + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        unpack8(__ldcs(reinterpret_cast<const uint4*>(p) + v), f);
    }
}
template <bool kF32>
__device__ __forceinline__ void store_stream(void* p, long long v, const float (&f)[8]) {
    if (kF32) {
        float4* o = reinterpret_cast<float4*>(p) + 2 * v;
        __stcs(o, make_float4(f[0], f[1], f[2], f[3]));
        __stcs(o + 1, make_float4(f[4], f[5], f[6], f[7]));
    } else {
        __stcs(reinterpret_cast<uint4*>(p) + v, pack8(f));
    }
}
// 8 values of a per-channel vector (null: ones), kept in L1.
__device__ __forceinline__ void load_channel(const float* p, int v, float (&f)[8]) {
    if (p) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p) + 2 * v);
        const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 2 * v + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = 1.0f;
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the threads of a row: a warp, or the whole block through `part`
// (32 floats; calls in a row use different ones).
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float v, float* part) {
    v = warp_sum(v);
    if (kWarpRow) return v;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = (int)(threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.0f;
    return warp_sum(t);
}

// kV: vectors of 8 a thread holds; kWarpRow: a warp a row (a block holds
// blockDim / 32 rows), else a block a row.
template <int kV, bool kWarpRow, bool kF32>
__global__ void __launch_bounds__(kWarpRow ? 32 * kRowWarps : 1024)
    block_norm_kernel(const NormArgs a) {
    __shared__ float part[2][32];
    const int lanes = kWarpRow ? 32 : blockDim.x;
    const int tid = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
    const long long row = kWarpRow
                              ? (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)
                              : (long long)blockIdx.x;
    if (row >= a.N) return;  // a whole warp, or (one row a block) nobody
    const long long base = row * a.V;
    float z[kV][8], s[kV][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int c = tid + i * lanes;
#pragma unroll
        for (int j = 0; j < 8; ++j) z[i][j] = s[i][j] = 0.0f;
        if (c < a.V) {
            if (a.y) unpack8(__ldcs(reinterpret_cast<const uint4*>(a.y) + base + c), z[i]);
            load_stream<kF32>(a.residual, base + c, s[i]);
        }
    }
    float r_post = 1.0f;
    if (a.post) {
#pragma unroll
        for (int i = 0; i < kV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += z[i][j] * z[i][j];
        r_post = rsqrtf(row_sum<kWarpRow>(sum, part[0]) * a.inv_h + a.eps);
        if (tid == 0 && a.rstd_post) a.rstd_post[row] = r_post;
    }
    const float token_gate = a.gate_kind == MOE_GATE_TOKEN ? a.gate[row] : 1.0f;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int c = tid + i * lanes;
        if (c < a.V) {
            float w[8], g[8];
            load_channel(a.post ? a.w_post : nullptr, c, w);
            load_channel(a.gate_kind == MOE_GATE_CHANNEL ? a.gate : nullptr, c, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float t = a.post ? z[i][j] * r_post * w[j] : z[i][j];
                s[i][j] = a.alpha * s[i][j] + (a.gate_kind == MOE_GATE_TOKEN ? token_gate : g[j]) * t;
                sum += s[i][j] * s[i][j];
            }
            if (a.s) store_stream<kF32>(a.s, base + c, s[i]);
        }
    }
    if (!a.pre) return;
    const float r_pre = rsqrtf(row_sum<kWarpRow>(sum, part[1]) * a.inv_h + a.eps);
    if (tid == 0 && a.rstd_pre) a.rstd_pre[row] = r_pre;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int c = tid + i * lanes;
        if (c < a.V) {
            float w[8];
            load_channel(a.w_pre, c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = s[i][j] * r_pre * w[j];
            __stcs(reinterpret_cast<uint4*>(a.x) + base + c, pack8(w));
        }
    }
}

template <int kV, bool kWarpRow, bool kF32>
__global__ void __launch_bounds__(kWarpRow ? 32 * kRowWarps : 1024)
    block_norm_grad_kernel(const NormGradArgs a) {
    extern __shared__ float cols[];  // kWarpRow: [warps][2][H] sums of the block's warps
    __shared__ float part[2][2][32];
    const int lanes = kWarpRow ? 32 : blockDim.x;
    const int tid = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
    const int rows_at_once = kWarpRow ? (int)(blockDim.x >> 5) : 1;
    const int sub = kWarpRow ? (int)(threadIdx.x >> 5) : 0;
    float t_post[kV][8], t_pre[kV][8];
#pragma unroll
    for (int i = 0; i < kV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) t_post[i][j] = t_pre[i][j] = 0.0f;

    int buf = 0;
    for (long long row = (long long)blockIdx.x * rows_at_once + sub; row < a.N;
         row += (long long)gridDim.x * rows_at_once, buf ^= 1) {
        const long long base = row * a.V;
        float g[kV][8], b[kV][8], yh[kV][8], sh[kV][8];
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int c = tid + i * lanes;
#pragma unroll
            for (int j = 0; j < 8; ++j) g[i][j] = b[i][j] = yh[i][j] = sh[i][j] = 0.0f;
            if (c < a.V) {
                if (a.pre) {
                    unpack8(__ldcs(reinterpret_cast<const uint4*>(a.dx) + base + c), b[i]);
                    load_stream<kF32>(a.s, base + c, sh[i]);
                }
                if (a.ds) load_stream<kF32>(a.ds, base + c, g[i]);
                if (a.y) unpack8(__ldcs(reinterpret_cast<const uint4*>(a.y) + base + c), yh[i]);
            }
        }
        if (a.pre) {
            const float r = a.rstd_pre[row];
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const int c = tid + i * lanes;
                if (c < a.V) {
                    float w[8];
                    load_channel(a.w_pre, c, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        sh[i][j] *= r;
                        t_pre[i][j] += b[i][j] * sh[i][j];
                        b[i][j] *= w[j];
                        sum += b[i][j] * sh[i][j];
                    }
                }
            }
            sum = row_sum<kWarpRow>(sum, part[buf][0]) * a.inv_h;
#pragma unroll
            for (int i = 0; i < kV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) g[i][j] += r * (b[i][j] - sh[i][j] * sum);
        }
        if (a.dresidual) {
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const int c = tid + i * lanes;
                if (c < a.V) {
                    float o[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = a.alpha * g[i][j];
                    store_stream<kF32>(a.dresidual, base + c, o);
                }
            }
        }
        if (!a.y) continue;
        const float r = a.post ? a.rstd_post[row] : 1.0f;
        const float token_gate = a.gate_kind == MOE_GATE_TOKEN ? a.gate[row] : 1.0f;
        // sum: of g yh w_post (without the token's gate, which is the row's own)
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int c = tid + i * lanes;
            if (c < a.V) {
                float w[8], ch[8];
                load_channel(a.post ? a.w_post : nullptr, c, w);
                load_channel(a.gate_kind == MOE_GATE_CHANNEL ? a.gate : nullptr, c, ch);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    yh[i][j] *= r;
                    t_post[i][j] += token_gate * g[i][j] * yh[i][j];
                    b[i][j] = ch[j] * g[i][j] * w[j];
                    sum += b[i][j] * yh[i][j];
                }
            }
        }
        float mean = 0.0f;
        if (a.post || a.dgate_token) {
            sum = row_sum<kWarpRow>(sum, part[buf][1]);
            mean = a.post ? sum * a.inv_h : 0.0f;
            if (tid == 0 && a.dgate_token) a.dgate_token[row] = sum;
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int c = tid + i * lanes;
            if (c < a.V) {
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    o[j] = token_gate * r * (b[i][j] - yh[i][j] * mean);
                __stcs(reinterpret_cast<uint4*>(a.dy) + base + c, pack8(o));
            }
        }
    }

    // the block's column sums: g yh (times the token's gate), dx sh
    const int H = a.V * 8;
    float* out = a.partial + (size_t)blockIdx.x * 2 * H;
    if (kWarpRow) {
        float* mine = cols + (size_t)sub * 2 * H;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int c = tid + i * lanes;
            if (c < a.V) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    mine[c * 8 + j] = t_post[i][j];
                    mine[H + c * 8 + j] = t_pre[i][j];
                }
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * H; c += blockDim.x) {
            float v = 0.0f;
            for (int w = 0; w < rows_at_once; ++w) v += cols[(size_t)w * 2 * H + c];
            out[c] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int c = tid + i * lanes;
            if (c < a.V) {
                float4* o = reinterpret_cast<float4*>(out + c * 8);
                o[0] = make_float4(t_post[i][0], t_post[i][1], t_post[i][2], t_post[i][3]);
                o[1] = make_float4(t_post[i][4], t_post[i][5], t_post[i][6], t_post[i][7]);
                o = reinterpret_cast<float4*>(out + H + c * 8);
                o[0] = make_float4(t_pre[i][0], t_pre[i][1], t_pre[i][2], t_pre[i][3]);
                o[1] = make_float4(t_pre[i][4], t_pre[i][5], t_pre[i][6], t_pre[i][7]);
            }
        }
    }
}

// Column sums over the blocks' partial sums.  With a gate per channel both
// dw_post and dgate come from the same sum T = sum of g yh:
// dw_post = gate T, dgate = w_post T.
constexpr int kReduceRows = 32;
__global__ void __launch_bounds__(32 * kReduceRows)
    block_norm_reduce_kernel(const float* __restrict__ partial, int blocks, int H,
                             const float* __restrict__ gate, const float* __restrict__ w_post,
                             float* dw_post, float* dgate, float* dw_pre, int accumulate) {
    __shared__ float sums[kReduceRows][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), r0 = threadIdx.x >> 5;
    const int which = blockIdx.y;
    float v = 0.0f;
    if (c < H)
        for (int r = r0; r < blocks; r += kReduceRows)
            v += partial[((size_t)r * 2 + which) * H + c];
    sums[r0][threadIdx.x & 31] = v;
    __syncthreads();
    if (r0 != 0 || c >= H) return;
    v = 0.0f;
#pragma unroll
    for (int r = 0; r < kReduceRows; ++r) v += sums[r][threadIdx.x];
    if (which == 1) {
        if (dw_pre) dw_pre[c] = accumulate ? dw_pre[c] + v : v;
        return;
    }
    if (dw_post) {
        const float d = gate ? gate[c] * v : v;
        dw_post[c] = accumulate ? dw_post[c] + d : d;
    }
    if (dgate) {
        const float d = w_post ? w_post[c] * v : v;
        dgate[c] = accumulate ? dgate[c] + d : d;
    }
}

int row_threads(int V, int kv) { return ((V + kv - 1) / kv + 31) / 32 * 32; }

// Blocks of the gradient: as many as are resident at 64 registers a thread (8 at
// most, so that their partial sums stay few), or one for each row.
int grad_blocks(const moe_norm_shape& s) {
    const int V = s.H / 8;
    const bool warp_row = V <= kWarpRowV;
    const long long rows = warp_row ? (s.N + kRowWarps - 1LL) / kRowWarps : s.N;
    const int fit = warp_row ? 8 : 1024 / row_threads(V, V <= 1024 ? 1 : 2);
    const long long most = (long long)sm_count() * (fit < 8 ? fit : 8);
    return (int)(rows < most ? (rows > 0 ? rows : 1) : most);
}

moe_status check_norm(const moe_norm_shape* s) {
    if (!s) return MOE_ERR_INVALID_ARG;
    if (s->N < 0 || s->H <= 0) return MOE_ERR_INVALID_ARG;
    if (s->gate != MOE_GATE_NONE && s->gate != MOE_GATE_CHANNEL && s->gate != MOE_GATE_TOKEN)
        return MOE_ERR_INVALID_ARG;
    if (s->stream_type != MOE_TYPE_BF16 && s->stream_type != MOE_TYPE_F32)
        return MOE_ERR_INVALID_ARG;
    if (!(s->eps >= 0.0f) || !(s->eps < 1e30f)) return MOE_ERR_INVALID_ARG;
    if (s->H % 8 != 0 || s->H > kMaxNormH) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

template <bool kF32>
void run_forward(const NormArgs& a, cudaStream_t st) {
    const int V = a.V;
    if (V <= kWarpRowV) {
        const int blocks = (a.N + kRowWarps - 1) / kRowWarps, t = 32 * kRowWarps;
        if (V <= 32) block_norm_kernel<1, true, kF32><<<blocks, t, 0, st>>>(a);
        else block_norm_kernel<2, true, kF32><<<blocks, t, 0, st>>>(a);
    } else if (V <= 1024) {
        block_norm_kernel<1, false, kF32><<<a.N, row_threads(V, 1), 0, st>>>(a);
    } else {
        block_norm_kernel<2, false, kF32><<<a.N, row_threads(V, 2), 0, st>>>(a);
    }
}

template <bool kF32>
void run_grad(const NormGradArgs& a, int blocks, cudaStream_t st) {
    const int V = a.V;
    if (V <= kWarpRowV) {
        const int t = 32 * kRowWarps;
        const size_t smem = (size_t)kRowWarps * 2 * V * 8 * sizeof(float);
        if (V <= 32) block_norm_grad_kernel<1, true, kF32><<<blocks, t, smem, st>>>(a);
        else block_norm_grad_kernel<2, true, kF32><<<blocks, t, smem, st>>>(a);
    } else if (V <= 1024) {
        block_norm_grad_kernel<1, false, kF32><<<blocks, row_threads(V, 1), 0, st>>>(a);
    } else {
        block_norm_grad_kernel<2, false, kF32><<<blocks, row_threads(V, 2), 0, st>>>(a);
    }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_norm_workspace_bytes(const moe_norm_shape* shape) {
    if (check_norm(shape) != MOE_OK) return 0;
    return align256((size_t)grad_blocks(*shape) * 2 * shape->H * sizeof(float));
}

moe_status moe_block_norm(const uint16_t* y, const void* residual, const float* w_post,
                          const float* gate, const float* w_pre, const moe_norm_shape* shape,
                          void* s, uint16_t* x, float* rstd_post, float* rstd_pre, void* stream) {
    MOE_RANGE();
    MOE_TRY(check_norm(shape));
    if (shape->N == 0) return MOE_OK;
    const bool post = shape->post != 0, pre = shape->pre != 0;
    if (!residual || (pre && !x) || (!pre && !s)) return MOE_ERR_INVALID_ARG;
    if (!y && (post || shape->gate != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
    if (shape->gate != MOE_GATE_NONE && !gate) return MOE_ERR_INVALID_ARG;
    if (!aligned16(y, x, w_post, w_pre) ||
        !aligned16((const char*)residual, (const char*)s) ||
        (shape->gate == MOE_GATE_CHANNEL && !aligned16(gate)))
        return MOE_ERR_INVALID_ARG;
    const NormArgs a{y,         residual, w_post,      gate, w_pre, s,   x,
                     rstd_post, rstd_pre, shape->N,    shape->H / 8,     post, pre, shape->gate,
                     shape->eps, shape->residual_scale, 1.0f / (float)shape->H};
    if (shape->stream_type == MOE_TYPE_F32) run_forward<true>(a, as_stream(stream));
    else run_forward<false>(a, as_stream(stream));
    return cuda_status(cudaGetLastError());
}

moe_status moe_block_norm_grad(const void* ds, const uint16_t* dx, const uint16_t* y,
                               const void* s, const float* w_post, const float* gate,
                               const float* w_pre, const float* rstd_post, const float* rstd_pre,
                               const moe_norm_shape* shape, uint16_t* dy, void* dresidual,
                               float* dw_post, float* dgate, float* dw_pre, int32_t accumulate,
                               void* ws, size_t ws_bytes, void* stream) {
    MOE_RANGE();
    MOE_TRY(check_norm(shape));
    if (!ws || ws_bytes < moe_norm_workspace_bytes(shape)) return MOE_ERR_WORKSPACE;
    const bool post = shape->post != 0, pre = shape->pre != 0;
    const bool by_channel = shape->gate == MOE_GATE_CHANNEL, by_token = shape->gate == MOE_GATE_TOKEN;
    // gradients of what the block does not have
    if ((dw_post && !post) || (dw_pre && !pre) || (dgate && shape->gate == MOE_GATE_NONE))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t st = as_stream(stream);
    const size_t hb = (size_t)shape->H * sizeof(float);
    if (shape->N == 0) {
        // sums over no rows
        if (!accumulate) {
            if (dw_post && cudaMemsetAsync(dw_post, 0, hb, st) != cudaSuccess) return MOE_ERR_CUDA;
            if (dw_pre && cudaMemsetAsync(dw_pre, 0, hb, st) != cudaSuccess) return MOE_ERR_CUDA;
            if (dgate && by_channel && cudaMemsetAsync(dgate, 0, hb, st) != cudaSuccess)
                return MOE_ERR_CUDA;
        }
        return MOE_OK;
    }
    if (pre ? (!dx || !s || !rstd_pre) : !ds) return MOE_ERR_INVALID_ARG;
    if (!y && (post || shape->gate != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
    if ((y && !dy) || (post && !rstd_post)) return MOE_ERR_INVALID_ARG;
    if (shape->gate != MOE_GATE_NONE && !gate) return MOE_ERR_INVALID_ARG;
    if (!aligned16(dx, y, dy, w_post, w_pre) ||
        !aligned16((const char*)ds, (const char*)s, (const char*)dresidual, (const char*)ws) ||
        (by_channel && !aligned16(gate)))
        return MOE_ERR_INVALID_ARG;
    const NormGradArgs a{ds, dx, y, s, w_post, gate, w_pre, rstd_post, rstd_pre, dy, dresidual,
                         by_token ? dgate : nullptr, static_cast<float*>(ws), shape->N,
                         shape->H / 8, post, pre, shape->gate, shape->residual_scale,
                         1.0f / (float)shape->H};
    const int blocks = grad_blocks(*shape);
    if (shape->stream_type == MOE_TYPE_F32) run_grad<true>(a, blocks, st);
    else run_grad<false>(a, blocks, st);
    MOE_TRY(cuda_status(cudaGetLastError()));
    if (dw_post || dw_pre || (dgate && by_channel)) {
        const dim3 grid((shape->H + 31) / 32, dw_pre ? 2 : 1);
        block_norm_reduce_kernel<<<grid, 32 * kReduceRows, 0, st>>>(
            a.partial, blocks, shape->H, by_channel ? gate : nullptr, post ? w_post : nullptr,
            dw_post, by_channel ? dgate : nullptr, dw_pre, accumulate != 0);
        MOE_TRY(cuda_status(cudaGetLastError()));
    }
    return MOE_OK;
}

}  // extern "C"
