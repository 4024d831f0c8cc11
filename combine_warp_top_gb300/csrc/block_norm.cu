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
// x; the gradient reads ds, dx, y and s once and writes dy and dresidual.  A block
// keeps its columns over many rows, so per-channel vectors and column sums stay in
// registers, and the next rows' inputs are under way during a row's sums.  8192 rows of
// 4096: forward 44 us (bf16 stream, 6.1 TB/s) and 65 us (fp32, 6.1 TB/s), gradient
// 72 us (5.6 TB/s; 68 us without the column sums' kernel) and 94 us (6.4 TB/s).  What
// the bf16 gradient waits for is the latency between a row's sums and the next: two
// blocks share an SM at 4096 columns, one from 4104 on (4680 rows of 7168: 79 us for the
// same bytes), and above 8192 the 64 registers of 1024 threads spill (131 us).  All sums
// are fp32 in a fixed order: columns by shuffle trees, rows of a column by the thread
// that owns the column over its block's rows, then over the blocks' partial sums (in
// the workspace) by a second kernel.
#include "../../include/moe_train.h"
#include "api_checks.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kMaxNormH = 16384;
constexpr int kMaxRing = 216 * 1024;  // bytes of the rings of an SM's blocks
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

// Pairs of fp32 values: one instruction of the packed fp32 pipe for two elements.
using f2 = float2;
__device__ __forceinline__ unsigned long long bits2(f2 v) {
    return *reinterpret_cast<unsigned long long*>(&v);
}
__device__ __forceinline__ f2 from_bits2(unsigned long long v) {
    return *reinterpret_cast<f2*>(&v);
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return from_bits2(d);
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
    return from_bits2(d);
}
__device__ __forceinline__ f2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float across(f2 v) { return v.x + v.y; }

// 8 consecutive values of an input as they are in memory: one 16-byte word of
// bf16, or two of fp32.
template <bool kF32>
struct Raw {
    uint4 w[kF32 ? 2 : 1];
};
template <bool kF32>
__device__ __forceinline__ void unpack(const Raw<kF32>& r, f2 (&f)[4]) {
    if (kF32) {
        const uint4 a = r.w[0], b = r.w[kF32 ? 1 : 0];
        f[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
        f[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
        f[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
        f[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
    } else {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
}
__device__ __forceinline__ uint4 pack_bf16(const f2 (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[i].x, f[i].y);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The 8 columns that a thread holds of a row, as two quads of 4.  bf16 streams: 8
// consecutive columns, one 16-byte word of each bf16 tensor.  fp32 streams: the
// quads of `L` neighbouring threads lie side by side, first all their first quads, then
// the second, so that each 16-byte access of a warp to an fp32 tensor covers whole
// lines (8 consecutive fp32 columns a thread would take them by half sectors: an L2
// request for every half, and 8192 x 4096 backwards 130 us, 94 so).
struct Cols {
    uint32_t c, a, b;  // vector of 8, quads
    bool pa, pb;       // the row has them (pb implies pa)
};
template <bool kF32>
__device__ __forceinline__ Cols cols_of(uint32_t c, uint32_t L, uint32_t V) {
    if (!kF32) return {c, 2 * c, 2 * c + 1, c < V, c < V};
    const uint32_t l = c % L, a = (c - l) * 2 + l;
    return {c, a, a + L, a < 2 * V, a + L < 2 * V};
}

// A thread's columns of a tensor (kT32: fp32, else bf16) of a kernel on an fp32 stream
// (kF32) or not, past L1 (each is read or written once).
template <bool kT32, bool kF32>
__device__ __forceinline__ Raw<kT32> load_cols(const char* row, const Cols& q) {
    Raw<kT32> r;
    if (kT32) {
        const uint4* p = reinterpret_cast<const uint4*>(row);
        r.w[0] = r.w[kT32 ? 1 : 0] = make_uint4(0, 0, 0, 0);
        if (q.pa) r.w[0] = __ldcs(p + q.a);
        if (q.pb) r.w[kT32 ? 1 : 0] = __ldcs(p + q.b);
    } else if (kF32) {
        const uint2* p = reinterpret_cast<const uint2*>(row);
        uint2 x = make_uint2(0, 0), y = x;
        if (q.pa) x = __ldcs(p + q.a);
        if (q.pb) y = __ldcs(p + q.b);
        r.w[0] = make_uint4(x.x, x.y, y.x, y.y);
    } else {
        r.w[0] = __ldcs(reinterpret_cast<const uint4*>(row) + q.c);
    }
    return r;
}
template <bool kT32, bool kF32>
__device__ __forceinline__ void store_cols(char* row, const Cols& q, const f2 (&f)[4]) {
    if (kT32) {
        float4* p = reinterpret_cast<float4*>(row);
        if (q.pa) __stcs(p + q.a, make_float4(f[0].x, f[0].y, f[1].x, f[1].y));
        if (q.pb) __stcs(p + q.b, make_float4(f[2].x, f[2].y, f[3].x, f[3].y));
    } else {
        const uint4 v = pack_bf16(f);
        if (kF32) {
            uint2* p = reinterpret_cast<uint2*>(row);
            if (q.pa) __stcs(p + q.a, make_uint2(v.x, v.y));
            if (q.pb) __stcs(p + q.b, make_uint2(v.z, v.w));
        } else {
            __stcs(reinterpret_cast<uint4*>(row) + q.c, v);
        }
    }
}
// Those of a per-channel vector (null: ones).
__device__ __forceinline__ void load_channel(const float* p, const Cols& q, f2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = both(1.0f);
    if (p) {
        const float4* v = reinterpret_cast<const float4*>(p);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (q.pa) x = v[q.a];
        if (q.pb) y = v[q.b];
        f[0] = make_float2(x.x, x.y);
        f[1] = make_float2(x.z, x.w);
        f[2] = make_float2(y.x, y.y);
        f[3] = make_float2(y.z, y.w);
    }
}
// The block's scale of a channel: gate per channel times the weight after it.
__device__ __forceinline__ void load_scale(const float* gate, const float* w_post, const Cols& q,
                                           f2 (&f)[4]) {
    f2 g[4];
    load_channel(w_post, q, f);
    load_channel(gate, q, g);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], g[i]);
}

// The inputs of the next rows of a block on their way into shared memory with
// 16-byte cp.async, into slots that only the warp reads: a row in flight costs no
// registers and no block barrier.  A stage holds words of 16 bytes for every
// thread, `pitch` bytes between a thread's words (slot: the thread's first).  A bf16
// tensor's word is the thread's 8 consecutive columns, an fp32 tensor's two words
// are its quads.
template <bool kT32>
__device__ __forceinline__ void ring_copy(uint32_t slot, uint32_t pitch, const char* row,
                                          const Cols& q, uint32_t V) {
    if (kT32) {
        if (q.pa) ptx::cp_async_16(slot, row + q.a * 16u, 16);
        if (q.pb) ptx::cp_async_16(slot + pitch, row + q.b * 16u, 16);
    } else if (q.c < V) {
        ptx::cp_async_16(slot, row + q.c * 16u, 16);
    }
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
// A thread's columns from the ring.  In a kernel on an fp32 stream a bf16 tensor's
// quads are among the warp's 512 bytes.  Quads that the row does not have are zeros.
template <bool kT32, bool kF32>
__device__ __forceinline__ Raw<kT32> ring_read(uint32_t slot, uint32_t pitch, const Cols& q) {
    Raw<kT32> r;
    if (kT32) {
        r.w[0] = r.w[kT32 ? 1 : 0] = make_uint4(0, 0, 0, 0);
        if (q.pa) r.w[0] = lds16(slot);
        if (q.pb) r.w[kT32 ? 1 : 0] = lds16(slot + pitch);
    } else if (kF32) {
        const uint32_t l = threadIdx.x & 31u, at = slot - l * 16u + l * 8u;
        uint2 x = make_uint2(0, 0), y = x;
        if (q.pa) x = lds8(at);
        if (q.pb) y = lds8(at + 256u);
        r.w[0] = make_uint4(x.x, x.y, y.x, y.y);
    } else {
        r.w[0] = lds16(slot);
    }
    return r;
}
__device__ __forceinline__ void ring_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kAhead>
__device__ __forceinline__ void ring_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
    __syncwarp();  // what the warp's other lanes have copied is there too
}

// Rows are shared out to groups of kLanes threads: 8, 16 or 32 lanes of a warp
// for short rows, or (kLanes = 0) a whole block.
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
        if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over a row's threads, a block's through `part` (32 floats; calls in a row
// use different ones).
template <int kLanes>
__device__ __forceinline__ float row_sum(float v, float* part) {
    v = lanes_sum(v, kLanes ? kLanes : 32);
    if (kLanes) return v;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = (int)(threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.0f;
    return lanes_sum(t, 32);
}

// Sums of four values over a warp in 6 shuffles: the first two steps halve the
// values a lane holds as well as the lanes.  Lane 8 i ends with value i's sum
// (as do its 7 neighbours).
__device__ __forceinline__ float warp_sum4(const float (&v)[4]) {
    const int lane = threadIdx.x & 31;
    const bool hi = lane & 16, hi8 = lane & 8;
    const float x0 = (hi ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
    const float x1 = (hi ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 16);
    const float x = (hi8 ? x1 : x0) + __shfl_xor_sync(0xffffffffu, hi8 ? x0 : x1, 8);
    return lanes_sum(x, 8);
}
// Four sums over a row's threads (part: 128 floats, as for row_sum).
template <int kLanes>
__device__ __forceinline__ void row_sum4(float (&v)[4], float4* part) {
    if (kLanes == 8 || kLanes == 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lanes_sum(v[i], kLanes);
        return;
    }
    const int lane = threadIdx.x & 31;
    float x = warp_sum4(v);
    if (kLanes == 0) {
        const int warps = blockDim.x >> 5;
        if ((lane & 7) == 0) reinterpret_cast<float*>(part + (threadIdx.x >> 5))[lane >> 3] = x;
        __syncthreads();
        const float4 t = lane < warps ? part[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
        const float u[4] = {t.x, t.y, t.z, t.w};
        x = warp_sum4(u);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xffffffffu, x, 8 * i);
}

// The rows of this thread's group: its first, the step to its next, and how many
// rows ahead of the group the first of its warp (or block) is, which bounds the
// loop so that a warp's groups leave it together.
struct Rows {
    int first, step, lead;
};
template <int kLanes>
__device__ __forceinline__ Rows my_rows() {
    if (kLanes == 0) return {(int)blockIdx.x, (int)gridDim.x, 0};
    constexpr int kGroups = 32 * kRowWarps / (kLanes ? kLanes : 32);
    const int group = threadIdx.x / (kLanes ? kLanes : 32);
    const int in_warp = (threadIdx.x & 31) / (kLanes ? kLanes : 32);
    return {(int)blockIdx.x * kGroups + group, (int)gridDim.x * kGroups, in_warp};
}

// How a row's inputs reach the registers: loaded when the row begins, loaded into
// registers one row ahead, or by a ring of kRing2 or kRing3 rows in shared memory.
// One row ahead costs no traffic of shared memory but is little in flight.  It wins for
// an fp32 stream where two rows' blocks or more share an SM (8192 x 4096: 65 us, by the
// ring 70), and loses where one block has the SM (8192 x 5120: 97 us, by the ring 78)
// and for a bf16 stream, whose rows are half as many bytes (8192 x 4096: 51 and 44 us),
// but for rows of more than 8192 (2048 x 16384: 59 and 63 us).
enum Feed { kNow = 0, kAhead = 1, kRing2 = 2, kRing3 = 3 };

// kV: vectors of 8 a thread holds.  kKeep: the per-channel vectors stay in registers
// over the rows (a thread keeps its columns); else they come from L1 for every row.
// kFull: y, both norms and s are all there, so nothing is tested for.
template <int kV, int kLanes, bool kF32, Feed kFeed, bool kKeep, bool kFull, int kThreads>
__global__ void __launch_bounds__(kThreads)
    block_norm_kernel(const NormArgs a) {
    extern __shared__ uint4 ring[];
    __shared__ float part[2][2][32];
    constexpr bool kRing = kFeed >= kRing2;
    constexpr int kStages = kRing ? kFeed : 1, kPerV = kF32 ? 3 : 2;
    constexpr uint32_t kRowR = kF32 ? 32 : 16;  // bytes of a stream vector
    const uint32_t lanes = kLanes ? kLanes : blockDim.x;
    const uint32_t tid = kLanes ? threadIdx.x % lanes : threadIdx.x;
    const uint32_t V = a.V;
    const Rows rows = my_rows<kLanes>();
    const bool has_y = kFull || a.y, post = kFull || a.post, pre = kFull || a.pre;
    after_previous();

    const auto cols = [&](int i) {
        return cols_of<kF32>(tid + i * lanes, kLanes ? kLanes : 32, V);
    };
    Raw<false> ry[kV];
    Raw<kF32> rr[kV];
    auto load = [&](int row) {
        const char* y = reinterpret_cast<const char*>(a.y) + (size_t)row * V * 16;
        const char* r = reinterpret_cast<const char*>(a.residual) + (size_t)row * V * kRowR;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const Cols q = cols(i);
            if (!kFull) ry[i].w[0] = make_uint4(0, 0, 0, 0);
            if (q.pa && row < a.N) {
                if (has_y) ry[i] = load_cols<false, kF32>(y, q);
                rr[i] = load_cols<kF32, kF32>(r, q);
            }
        }
    };
    if (kFeed == kAhead) load(rows.first);

    const uint32_t pitch = blockDim.x * 16, stage_bytes = pitch * kV * kPerV;
    const uint32_t ring0 = kRing ? ptx::smem_u32(ring) : 0u;
    auto fetch = [&](int row, uint32_t stage) {
        if (row < a.N) {
            const char* y = reinterpret_cast<const char*>(a.y) + (size_t)row * V * 16;
            const char* r = reinterpret_cast<const char*>(a.residual) + (size_t)row * V * kRowR;
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const uint32_t at = stage + i * kPerV * pitch + tid * 16;
                if (has_y) ring_copy<false>(at, pitch, y, cols(i), V);
                ring_copy<kF32>(at + pitch, pitch, r, cols(i), V);
            }
        }
        ring_commit();
    };
    if (kRing)
        for (int p = 0; p < kStages - 1; ++p)
            fetch(rows.first + p * rows.step, ring0 + p * stage_bytes);

    const float* gate_c = a.gate_kind == MOE_GATE_CHANNEL ? a.gate : nullptr;
    const float* w_post = a.post ? a.w_post : nullptr;
    f2 cw[kV][4], wp[kV][4];
    auto channels = [&](int i) {
        const Cols q = cols(i);
        if (q.pa) {
            load_scale(gate_c, w_post, q, cw[i]);
            load_channel(a.w_pre, q, wp[i]);
        }
    };
    if (kKeep) {
#pragma unroll
        for (int i = 0; i < kV; ++i) channels(i);
    }

    int buf = 0, stage = 0;
    for (int row = rows.first; row - rows.lead < a.N; row += rows.step, buf ^= 1) {
        const bool live = kLanes == 0 || row < a.N;
        const float token_gate = a.gate_kind == MOE_GATE_TOKEN && live ? a.gate[row] : 1.0f;
        char* s_row = reinterpret_cast<char*>(a.s) + (size_t)row * V * kRowR;
        char* x_row = reinterpret_cast<char*>(a.x) + (size_t)row * V * 16;
        const uint32_t slot = ring0 + stage * stage_bytes + tid * 16;
        if (kFeed == kNow) load(row);
        if constexpr (kRing) {
            __syncwarp();  // every lane has read what this overwrites
            const int next = stage == 0 ? kStages - 1 : stage - 1;
            fetch(row + (kStages - 1) * rows.step, ring0 + next * stage_bytes);
            ring_wait<kStages - 1>();
            stage = stage + 1 == kStages ? 0 : stage + 1;
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                if (!kFull) ry[i].w[0] = make_uint4(0, 0, 0, 0);
                if (cols(i).pa && has_y)
                    ry[i] = ring_read<false, kF32>(slot + i * kPerV * pitch, pitch, cols(i));
            }
        }
        float r_post = 1.0f;
        if (post) {
            f2 sum = both(0.0f);
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                if (cols(i).pa && live) {
                    f2 y[4];
                    unpack(ry[i], y);
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum = fma2(y[j], y[j], sum);
                }
            }
            r_post = rsqrtf(row_sum<kLanes>(across(sum), part[buf][0]) * a.inv_h + a.eps);
            if (tid == 0 && live && a.rstd_post) a.rstd_post[row] = r_post;
        }
        f2 s[kV][4];
        f2 sum = both(0.0f);
        const f2 scale = both(r_post * token_gate), alpha = both(a.alpha);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            if (cols(i).pa && live) {
                if (!kKeep) channels(i);
                if (kRing)
                    rr[i] = ring_read<kF32, kF32>(slot + (i * kPerV + 1) * pitch, pitch, cols(i));
                f2 y[4];
                unpack(ry[i], y);
                unpack(rr[i], s[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = fma2(mul2(y[j], scale), cw[i][j], mul2(alpha, s[i][j]));
                    sum = fma2(s[i][j], s[i][j], sum);
                }
            }
        }
        // its registers are free: the next row comes in beside this row's second sum
        // and stores (s may be the residual itself: another row of it)
        if (kFeed == kAhead) load(row + rows.step);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            if (cols(i).pa && live && (kFull || a.s))
                store_cols<kF32, kF32>(s_row, cols(i), s[i]);
        }
        if (!pre) continue;
        const float r_pre = rsqrtf(row_sum<kLanes>(across(sum), part[buf][1]) * a.inv_h + a.eps);
        if (tid == 0 && live && a.rstd_pre) a.rstd_pre[row] = r_pre;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            if (cols(i).pa && live) {
                f2 x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = mul2(mul2(s[i][j], both(r_pre)), wp[i][j]);
                store_cols<false, kF32>(x_row, cols(i), x);
            }
        }
    }
}

// The gradient needs two sums over the row, of b sh (b = dx w_pre) for g and then
// of g cw yh (cw = gate per channel * w_post) for dy.  The second is linear in g:
//   sum g cw yh = sum cw yh ds + r_pre * (sum cw yh b - mean(b sh) * sum cw yh sh)
// so all four sums are taken in one pass and reduced together, with one barrier
// a row; the second pass reads the row again from the ring.  The row's factors
// r_pre, r_post and its gate are taken out of the sums over columns.
// kFull: dx, y, s, ds and dresidual are all there.
template <int kV, int kLanes, bool kF32, int kStages, bool kKeep, bool kFull>
__global__ void __launch_bounds__(kLanes ? 32 * kRowWarps : 1024)
    block_norm_grad_kernel(const NormGradArgs a) {
    extern __shared__ uint4 ring[];
    float* group_sums = reinterpret_cast<float*>(ring);  // groups of a warp: column sums
    __shared__ float4 part[2][32];
    constexpr bool kRing = kLanes == 0;
    constexpr int kWordsR = kF32 ? 2 : 1, kPerV = 2 + 2 * kWordsR;
    constexpr uint32_t kRowR = kF32 ? 32 : 16;
    const uint32_t lanes = kLanes ? kLanes : blockDim.x;
    const uint32_t tid = kLanes ? threadIdx.x % lanes : threadIdx.x;
    const uint32_t V = a.V;
    const Rows rows = my_rows<kLanes>();
    const uint32_t pitch = blockDim.x * 16, stage_bytes = pitch * kV * kPerV;
    const uint32_t ring0 = kRing ? ptx::smem_u32(ring) : 0u;
    const bool has_y = kFull || a.y, pre = kFull || a.pre, has_ds = kFull || a.ds;
    after_previous();
    f2 t_post[kV][4], t_pre[kV][4];
#pragma unroll
    for (int i = 0; i < kV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) t_post[i][j] = t_pre[i][j] = both(0.0f);

    const auto cols = [&](int i) {
        return cols_of<kF32>(tid + i * lanes, kLanes ? kLanes : 32, V);
    };
    // words of a vector in a stage: dx, y, then s and ds
    auto fetch = [&](int row, uint32_t stage) {
        if (row < a.N) {
            const size_t at16 = (size_t)row * V * 16, at_r = (size_t)row * V * kRowR;
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const Cols q = cols(i);
                const uint32_t at = stage + i * kPerV * pitch + tid * 16;
                if (pre) {
                    ring_copy<false>(at, pitch, reinterpret_cast<const char*>(a.dx) + at16, q, V);
                    ring_copy<kF32>(at + 2 * pitch, pitch,
                                    reinterpret_cast<const char*>(a.s) + at_r, q, V);
                }
                if (has_ds)
                    ring_copy<kF32>(at + (2 + kWordsR) * pitch, pitch,
                                    reinterpret_cast<const char*>(a.ds) + at_r, q, V);
                if (has_y)
                    ring_copy<false>(at + pitch, pitch,
                                     reinterpret_cast<const char*>(a.y) + at16, q, V);
            }
        }
        ring_commit();
    };
    if (kRing)
        for (int p = 0; p < kStages - 1; ++p)
            fetch(rows.first + p * rows.step, ring0 + p * stage_bytes);

    const float* gate_c = a.gate_kind == MOE_GATE_CHANNEL ? a.gate : nullptr;
    const float* w_post = a.post ? a.w_post : nullptr;
    f2 cw[kV][4], wp[kV][4];
    auto channels = [&](int i) {
        const Cols q = cols(i);
        if (q.pa) {
            load_scale(gate_c, w_post, q, cw[i]);
            load_channel(a.w_pre, q, wp[i]);
        }
    };
    if (kKeep) {
#pragma unroll
        for (int i = 0; i < kV; ++i) channels(i);
    }

    int buf = 0, stage = 0;
    for (int row = rows.first; row - rows.lead < a.N; row += rows.step, buf ^= 1) {
        const bool live = kRing || row < a.N;
        const float r_pre = pre && live ? a.rstd_pre[row] : 0.0f;
        const float r_post = a.post && live ? a.rstd_post[row] : 1.0f;
        const float token_gate = a.gate_kind == MOE_GATE_TOKEN && live ? a.gate[row] : 1.0f;
        const size_t at16 = (size_t)row * V * 16, at_r = (size_t)row * V * kRowR;
        const uint32_t slot = ring0 + stage * stage_bytes + tid * 16;
        if constexpr (kRing) {
            __syncwarp();  // every lane has read what this overwrites
            const int next = stage == 0 ? kStages - 1 : stage - 1;
            fetch(row + (kStages - 1) * rows.step, ring0 + next * stage_bytes);
            ring_wait<kStages - 1>();
            stage = stage + 1 == kStages ? 0 : stage + 1;
        }
        Raw<false> rx[kV], ry[kV];
        Raw<kF32> rs[kV], rd[kV];
        auto read = [&](int i) {
            const Cols q = cols(i);
            const uint32_t at = slot + i * kPerV * pitch;
            const char* dx = reinterpret_cast<const char*>(a.dx) + at16;
            const char* sv = reinterpret_cast<const char*>(a.s) + at_r;
            const char* ds = reinterpret_cast<const char*>(a.ds) + at_r;
            const char* y = reinterpret_cast<const char*>(a.y) + at16;
            if (!kFull) {
                rx[i].w[0] = ry[i].w[0] = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < kWordsR; ++j)
                    rs[i].w[j] = rd[i].w[j] = make_uint4(0, 0, 0, 0);
            }
            if (pre) {
                rx[i] = kRing ? ring_read<false, kF32>(at, pitch, q)
                              : load_cols<false, kF32>(dx, q);
                rs[i] = kRing ? ring_read<kF32, kF32>(at + 2 * pitch, pitch, q)
                              : load_cols<kF32, kF32>(sv, q);
            }
            if (has_ds)
                rd[i] = kRing ? ring_read<kF32, kF32>(at + (2 + kWordsR) * pitch, pitch, q)
                              : load_cols<kF32, kF32>(ds, q);
            if (has_y)
                ry[i] = kRing ? ring_read<false, kF32>(at + pitch, pitch, q)
                              : load_cols<false, kF32>(y, q);
        };
        if (!kRing) {
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (cols(i).pa && live) read(i);
        }
        f2 acc[4] = {both(0.0f), both(0.0f), both(0.0f), both(0.0f)};
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            if (cols(i).pa && live) {
                if (kRing) read(i);
                if (!kKeep) channels(i);
                f2 b[4], sv[4], y[4], d[4];
                unpack(rx[i], b);
                unpack(rs[i], sv);
                unpack(ry[i], y);
                unpack(rd[i], d);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    b[j] = mul2(b[j], both(r_pre));
                    t_pre[i][j] = fma2(b[j], sv[j], t_pre[i][j]);
                    b[j] = mul2(b[j], wp[i][j]);           // r_pre b
                    const f2 q = mul2(y[j], cw[i][j]);     // cw yh / r_post
                    acc[0] = fma2(b[j], sv[j], acc[0]);
                    acc[1] = fma2(q, d[j], acc[1]);
                    acc[2] = fma2(q, b[j], acc[2]);
                    acc[3] = fma2(q, sv[j], acc[3]);
                }
            }
        }
        float sum[4] = {across(acc[0]), across(acc[1]), across(acc[2]), across(acc[3])};
        row_sum4<kLanes>(sum, part[buf]);
        const float m = sum[0] * a.inv_h;              // mean of b sh
        const float rm = -r_pre * r_pre * m;           // g = ds + r b + rm s
        const float dot = r_post * (sum[1] + sum[2] + rm * sum[3]);
        const float mean = a.post ? dot * a.inv_h : 0.0f;
        const float tgr = token_gate * r_post, tm = -tgr * r_post * mean;
        if (tid == 0 && live && a.dgate_token) a.dgate_token[row] = dot;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            if (cols(i).pa && live) {
                if (kRing) read(i);
                if (!kKeep) channels(i);
                f2 b[4], sv[4], g[4], o[4];
                unpack(rx[i], b);
                unpack(rs[i], sv);
                unpack(rd[i], g);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    g[j] = fma2(mul2(b[j], both(r_pre)), wp[i][j], g[j]);
                    g[j] = fma2(sv[j], both(rm), g[j]);
                    o[j] = mul2(both(a.alpha), g[j]);
                }
                if (kFull || a.dresidual)
                    store_cols<kF32, kF32>(reinterpret_cast<char*>(a.dresidual) + at_r, cols(i), o);
                if (has_y) {
                    f2 y[4];
                    unpack(ry[i], y);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const f2 t = mul2(g[j], both(tgr));  // gate g r_post
                        t_post[i][j] = fma2(t, y[j], t_post[i][j]);
                        o[j] = fma2(y[j], both(tm), mul2(cw[i][j], t));
                    }
                    store_cols<false, kF32>(reinterpret_cast<char*>(a.dy) + at16, cols(i), o);
                }
            }
        }
    }

    // the block's column sums: gate g yh (the token's gate), dx sh
    const uint32_t H = V * 8;
    float* out = a.partial + (size_t)blockIdx.x * 2 * H;
    float* mine = kRing ? out : group_sums + (size_t)(threadIdx.x / lanes) * 2 * H;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const Cols q = cols(i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t at = (j < 2 ? q.a : q.b) * 4 + j % 2 * 2;
            if (j < 2 ? q.pa : q.pb) {
                *reinterpret_cast<f2*>(mine + at) = t_post[i][j];
                *reinterpret_cast<f2*>(mine + H + at) = t_pre[i][j];
            }
        }
    }
    if (!kRing) {
        __syncthreads();
        const int groups = 32 * kRowWarps / (kLanes ? kLanes : 32);
        for (uint32_t c = threadIdx.x; c < 2 * H; c += blockDim.x) {
            float v = 0.0f;
            for (int w = 0; w < groups; ++w) v += group_sums[(size_t)w * 2 * H + c];
            out[c] = v;
        }
    }
}

// Column sums over the blocks' partial sums.  With a gate per channel both
// dw_post and dgate come from the same sum T = sum of g yh:
// dw_post = gate T, dgate = w_post T.
constexpr int kReduceRows = 32;
__global__ void __launch_bounds__(32 * kReduceRows)
    block_norm_reduce_kernel(const float* partial, int blocks, int H,
                             const float* gate, const float* w_post,
                             float* dw_post, float* dgate, float* dw_pre, int accumulate) {
    __shared__ float sums[kReduceRows][33];
    after_previous();
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

// A launch of either kernel: its grid, block, lanes a row (0: the block), vectors a
// thread, ring stages and shared memory.
struct Plan {
    int grid, block, lanes, kv, stages;
    size_t smem;
};

// words: 16-byte words of a vector in the ring (0: no ring); kv: vectors a thread of
// a block's row; most_blocks: resident on an SM (few in the gradient, so that their
// partial sums stay few).  1024 threads are resident at 64 registers.
Plan plan_for(int N, int V, int words, int kv, int most_blocks) {
    Plan p;
    if (V <= kWarpRowV) {
        p.kv = V <= 32 ? 1 : 2;
        p.lanes = V <= 8 ? 8 : V <= 16 ? 16 : 32;
        p.block = 32 * kRowWarps;
        p.stages = 0;
        p.smem = 0;
        const int rows = p.block / p.lanes;
        const long long need = (N + rows - 1LL) / rows, most = 8LL * sm_count();
        p.grid = (int)(need < most ? need : most);
    } else {
        p.kv = kv;
        p.lanes = 0;
        p.block = row_threads(V, kv);
        int fit = 1024 / p.block < most_blocks ? 1024 / p.block : most_blocks;
        if (fit < 1) fit = 1;
        const size_t stage = (size_t)p.block * kv * words * 16;
        const size_t room = (size_t)kMaxRing / fit;
        p.stages = words == 0 ? 0 : stage * 3 <= room ? 3 : stage * 2 <= room ? 2 : 1;
        p.smem = stage * p.stages;
        const long long most = (long long)sm_count() * fit;
        p.grid = (int)(N < most ? N : most);
    }
    if (p.grid < 1) p.grid = 1;
    return p;
}

Plan forward_plan(const moe_norm_shape& s) {
    const bool f32 = s.stream_type == MOE_TYPE_F32;
    const int words = f32 ? (s.H > 4096 ? 3 : 0) : s.H <= 8192 ? 2 : 0;  // see Feed
    return plan_for(s.N, s.H / 8, words, s.H <= 8192 ? 1 : 2, 16);
}
Plan grad_plan(const moe_norm_shape& s) {
    Plan p = plan_for(s.N, s.H / 8, s.stream_type == MOE_TYPE_F32 ? 6 : 4, s.H <= 8192 ? 1 : 2, 8);
    if (p.lanes) p.smem = (size_t)(p.block / p.lanes) * 2 * s.H * sizeof(float);
    return p;
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
    if (s->N > INT32_MAX - (1 << 20)) return MOE_ERR_UNSUPPORTED;  // row + the next rows' steps
    return MOE_OK;
}

template <auto kKernel, typename Args>
cudaError_t run(const Args& a, const Plan& p, cudaStream_t st) {
    if (p.smem > 40 * 1024) {  // with the static arrays, past the default 48 KB
        // the attribute holds for the process and device: set once for each
        static OncePerDevice set;
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (!set.done(dev)) {
            e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kMaxRing);
            if (e != cudaSuccess) return e;
            set.finish(dev);
        }
    }
    return launch_chained(kKernel, p.grid, p.block, p.smem, st, a);
}

template <bool kF32, bool kFull>
cudaError_t run_forward(const NormArgs& a, const Plan& p, cudaStream_t st) {
    constexpr int kW = 32 * kRowWarps;
    if (p.lanes == 8) return run<block_norm_kernel<1, 8, kF32, kAhead, true, kFull, kW>>(a, p, st);
    if (p.lanes == 16)
        return run<block_norm_kernel<1, 16, kF32, kAhead, true, kFull, kW>>(a, p, st);
    if (p.lanes == 32)
        return p.kv == 1 ? run<block_norm_kernel<1, 32, kF32, kNow, true, kFull, kW>>(a, p, st)
                         : run<block_norm_kernel<2, 32, kF32, kNow, true, kFull, kW>>(a, p, st);
    // forward_plan's rings fit: 3 rows of up to 1024 vectors on an SM, 2 of more
    constexpr Feed kWide = kF32 ? kRing2 : kAhead;
    if (p.kv == 2) return run<block_norm_kernel<2, 0, kF32, kWide, false, kFull, 1024>>(a, p, st);
    if constexpr (kF32) {
        if (p.stages == 0)
            return run<block_norm_kernel<1, 0, kF32, kAhead, true, kFull, 1024>>(a, p, st);
    }
    return run<block_norm_kernel<1, 0, kF32, kRing3, true, kFull, 1024>>(a, p, st);
}

template <bool kF32, bool kFull>
cudaError_t run_grad(const NormGradArgs& a, const Plan& p, cudaStream_t st) {
    if (p.lanes == 8) return run<block_norm_grad_kernel<1, 8, kF32, 0, true, kFull>>(a, p, st);
    if (p.lanes == 16) return run<block_norm_grad_kernel<1, 16, kF32, 0, true, kFull>>(a, p, st);
    if (p.lanes == 32)
        return p.kv == 1 ? run<block_norm_grad_kernel<1, 32, kF32, 0, true, kFull>>(a, p, st)
                         : run<block_norm_grad_kernel<2, 32, kF32, 0, true, kFull>>(a, p, st);
    if (p.kv == 1) {
        if constexpr (kF32) {  // 3 rows of a bf16 stream always fit
            if (p.stages < 3)
                return run<block_norm_grad_kernel<1, 0, kF32, 2, true, kFull>>(a, p, st);
        }
        return run<block_norm_grad_kernel<1, 0, kF32, 3, true, kFull>>(a, p, st);
    }
    return p.stages >= 2 ? run<block_norm_grad_kernel<2, 0, kF32, 2, false, kFull>>(a, p, st)
                         : run<block_norm_grad_kernel<2, 0, kF32, 1, false, kFull>>(a, p, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_norm_workspace_bytes(const moe_norm_shape* shape) {
    if (check_norm(shape) != MOE_OK) return 0;
    return align256((size_t)grad_plan(*shape).grid * 2 * shape->H * sizeof(float));
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
    const Plan p = forward_plan(*shape);
    const bool f32 = shape->stream_type == MOE_TYPE_F32, full = y && post && pre && s;
    cudaStream_t st = as_stream(stream);
    return cuda_status(full ? (f32 ? run_forward<true, true>(a, p, st)
                                   : run_forward<false, true>(a, p, st))
                            : (f32 ? run_forward<true, false>(a, p, st)
                                   : run_forward<false, false>(a, p, st)));
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
    const bool by_channel = shape->gate == MOE_GATE_CHANNEL;
    const bool by_token = shape->gate == MOE_GATE_TOKEN;
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
    const Plan p = grad_plan(*shape);
    const bool f32 = shape->stream_type == MOE_TYPE_F32, full = y && pre && ds && dresidual;
    MOE_TRY(cuda_status(full ? (f32 ? run_grad<true, true>(a, p, st)
                                    : run_grad<false, true>(a, p, st))
                             : (f32 ? run_grad<true, false>(a, p, st)
                                    : run_grad<false, false>(a, p, st))));
    if (dw_post || dw_pre || (dgate && by_channel)) {
        MOE_TRY(cuda_status(launch_chained(
            block_norm_reduce_kernel, dim3((shape->H + 31) / 32, dw_pre ? 2 : 1), 32 * kReduceRows,
            0, st, a.partial, p.grid, shape->H, by_channel ? gate : nullptr,
            post ? w_post : nullptr, dw_post, by_channel ? dgate : nullptr, dw_pre,
            accumulate != 0 ? 1 : 0)));
    }
    return MOE_OK;
}

}  // extern "C"
