// Orthogonalised momentum of per-expert matrices: the update of the Muon optimiser.  With g
// the gradient and b the momentum of one [M, N] matrix:
//
//   b' = beta b + g,   u = g + beta b' (Nesterov) or b',   X = u / (|u|_F + eps)
//   steps times:  G = X X^T,  S = p1 G + p2 G^2,  X = p0 X + S X
//
// with the quintic p = (3.4445, -4.7750, 2.0315), which takes every singular value of X
// towards 1.  A tall matrix (M > N) runs on X^T X and X S instead, so that G is always the
// smaller square; nothing is transposed, the tensor maps name the operands MN-major.
//
// What is rounded.  The products' operands are fp16 (11 bits), scaled so that none of their
// numbers that matter is a denormal: X as an operand, G and S; their sums are fp32.  Every step
// multiplies small singular values by 3.4445, and what a rounding has put in their place with
// them, so X in its own place in the sum, p0 X, is kept in two fp16 halves (22 bits; the second one
// times 2^11): rounded to one, a gradient of rank 16 over noise would end 3.8e-2 of its norm from
// the 64-bit result (bf16 operands and X: 0.3).  And S, near the end some -2.7 I and little beside
// it, goes apart: its diagonal d, fp32, to p0, the rest into the product, whose roundings are then
// those of the little.  Together 4e-4 to 1.5e-3 of the result's norm (with S whole up to 2.2e-3);
// the output's own rounding to bf16 is 1.7e-3.  The largest are gradients of rank 1: 264 x 264
// 1.5e-3, 8192 x 8192 1.2e-3 (2.0e-3 with an unscaled second half, which is a denormal there).
//
// Three products a step, on 256 x 256 tiles of a CTA pair (tcgen05, two accumulators in TMEM, 5
// stages of 32 KB).  G and S are symmetric: only tiles on and above the diagonal are made, each
// stored a second time as its mirror image, so that a step is 3 m^2 n + m^3 operations instead of
// 4 m^2 n + 2 m^3 (n the longer side, m the shorter).  The epilogue does the sums, so that S and X are
// written once.  Few and small matrices: tiles of 128 or 64 columns, all of them.
//
// What bounds it (GB300): the MMAs, at the clock that the power cap leaves.  64 of 2048 x 1408:
// 4240 us, of them 650 the two passes ahead of the products (HBM: 12 bytes an element each); G
// 192 us (17700 cycles a tile, 17000 of them MMAs), S 140, X 359 (14500 cycles; 11700).  16 of
// 2048 x 7168: 5900 us, 710 ahead, G 310, S 97, X 585; all 4 m^2 n + 2 m^3 operations at a
// library product's sustained rate would be 6400 us.  8 of 512 x 128: 78 us, 17
// launches of one tile a pair, 4.6 us each.
// One kernel for all products, whose tiles wait for those that they need by counters in global
// memory, was no faster (4670 us; 125 us): a tile's end is seen by the next one 5 us later.
#include <stddef.h>

#include <cuda_fp16.h>

#include "../../include/moe_train.h"
#include "api_checks.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr float kP0 = 3.4445f, kP1 = -4.7750f, kP2 = 2.0315f;

constexpr int BT = 256;   // rows and columns of a pair's tile (columns: or 128, 64)
constexpr int BH = 128;   // rows of A and of B that a CTA of the pair holds
constexpr int BK = 64;
constexpr int UMMA_K = 16;
constexpr int kStages = 5;
constexpr int kAccs = 2;
constexpr int kTmemCols = BT * kAccs;
constexpr int OP_BYTES = BH * BK * 2;
constexpr int BOX_BYTES = OP_BYTES / 2;
constexpr int STAGE_BYTES = 2 * OP_BYTES;
// Epilogue warps, kWarps: 4 with all 256 columns of 32 rows of a CTA's half tile each, or 8 with
// 128.  Their rows come in and go out in lines of a quarter of those columns (64 or 32: 128 or
// 64 bytes) through two buffers: the next ones' inputs are on their way while these are worked on.
// Whole lines of 128 bytes are fewer rows for the copy engine, which is as busy with a tile's
// operands as the MMAs are (16 of 2048 x 7168: 5950 us with 4 warps, 6100 with 8); a tile that no
// other runs beside is done sooner by 8 (8 of 1024 x 1024: 437 and 359 us).  With one buffer 64 of
// 2048 x 1408 took 4369 us, 4195 with two.
constexpr int kMaxWarps = 8;
template <int kWarps>
constexpr int kLine = 256 / kWarps;
template <int kWarps>
constexpr int kLinesBytes = 32 * kLine<kWarps> * 2;
template <int kWarps>
constexpr int kBufferBytes = 2 * kLinesBytes<kWarps>;  // lines of two inputs or outputs
constexpr int kStagingBytes = kMaxWarps * 2 * kBufferBytes<kMaxWarps>;  // of all warps
static_assert(kStagingBytes == 4 * 2 * kBufferBytes<4>, "the same for 4 warps");
constexpr int kMaxDim = 65536;
// G and S are kept times 2^12, X times 2^p with 2^p about the root of its longer side, so
// that entries far below the largest are normal fp16 numbers.
constexpr float kSquareScale = 4096.0f;
// X's second half is kept times 2^11, which makes it the size of the first: unscaled it would be a
// denormal where X's entries are below 2^-3 (sides of hundreds), and X have fewer bits.
constexpr float kLowScale = 2048.0f;

// The three products of a step, and the last one of all.
enum Form { kGram, kSquare, kStep, kLast };

struct Ctl {
    uint64_t full[kStages];    // leader: both CTAs' operands of a stage are there
    uint64_t empty[kStages];   // each CTA: its stage may be refilled
    uint64_t tfull[kAccs];     // each CTA: accumulator ready
    uint64_t tempty[kAccs];    // leader: accumulator drained by both CTAs
    uint64_t lines[kMaxWarps];  // each CTA: a warp's lines have come in
    uint64_t done;             // leader: every issued MMA retired
    uint32_t tmem_base;
    int abort;
};
constexpr int kBarriers = 2 * kStages + 2 * kAccs + kMaxWarps + 1;
constexpr size_t kSmem = 1024 + (size_t)kStages * STAGE_BYTES +
                         (size_t)kStagingBytes + ((sizeof(Ctl) + 15) & ~size_t(15));
static_assert(kSmem <= 227 * 1024, "shared memory of one block");

struct Dims {
    int E, K, m, n;  // products: contraction, rows and columns of an output
    int wide;        // columns of a tile: BT, 128 or 64
};

__host__ __device__ __forceinline__ int blocks_of(int n, int size) { return (n + size - 1) / size; }

// Columns that the MMAs of the last column block take, where there are 128 at most.
__host__ __device__ __forceinline__ int last_columns(int n, int wide) {
    const int rest = n - (n - 1) / wide * wide;
    return rest > BH ? BT : (rest + 31) / 32 * 32;
}

struct Tile {
    int e, mb, nb;
};

// triangle: the tiles on and above the diagonal, column by column.  Else 8 row blocks by all
// column blocks at a time, so that what runs side by side shares operands in L2.
__device__ __forceinline__ Tile decode(long long tile, int per_matrix, int MB, int NB,
                                       bool triangle) {
    Tile t;
    t.e = (int)(tile / per_matrix);
    const int i = (int)(tile - (long long)t.e * per_matrix);
    if (triangle) {
        int c = (int)((sqrtf(8.0f * (float)i + 1.0f) - 1.0f) * 0.5f);
        while (c * (c + 1) / 2 > i) --c;
        while ((c + 1) * (c + 2) / 2 <= i) ++c;
        t.nb = c;
        t.mb = i - c * (c + 1) / 2;
    } else {
        const int g = i / (8 * NB), first = g * 8, rows = MB - first < 8 ? MB - first : 8;
        const int in = i - g * 8 * NB;
        t.nb = in / rows;
        t.mb = first + in - t.nb * rows;
    }
    return t;
}

__device__ __forceinline__ void umma_f16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                              uint32_t accumulate) {
    umma_bf16_pair(d, a, b, idesc, accumulate);  // kind::f16, the types are idesc's
}
// fp16 operands, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// 32 or 64 columns of an accumulator.
__device__ __forceinline__ void tmem_ld_columns(uint32_t at, uint32_t (&v)[32]) {
    tmem_ld32(at, v);
}
__device__ __forceinline__ void tmem_ld_columns(uint32_t at, uint32_t (&v)[64]) {
    tmem_ld32(at, reinterpret_cast<uint32_t(&)[32]>(v[0]));
    tmem_ld32(at + 32, reinterpret_cast<uint32_t(&)[32]>(v[32]));
}

// A line of a warp's 32 rows of an output, of the same columns of the inputs that lie in the
// buffer, and out by TMA.  v: the lane's row of the accumulator.  16-byte chunk k of row r is at
// k ^ (r % 8) of its 128 bytes or k ^ (r / 2 % 4) of its 64: TMA's swizzles; a mirror image has
// none.
//   kGram    G = acc * 2^(12 - 2p), and its mirror image
//   kSquare  S = p1 G + p2 acc * 2^-12, likewise; kSpecial: with the column `at_diag` of this row
//            taken out (into *diag), if it is one of these
//   kStep    x = (p0 + d) (hi + lo 2^-11) + acc * 2^-12, into hi and lo
//   kLast    the same times 2^-p, bf16
// with p0 + d as beta; kSpecial: with d by columns at `diag`, of which there are `left`, times
// `unscale`.
template <Form kForm, int kWarps, bool kSpecial, bool kMirrored>
__device__ __forceinline__ void combine(uint8_t* lines, const uint32_t (&v)[kLine<kWarps>],
                                        float alpha, float beta, float* diag, int at_diag, int left,
                                        float unscale) {
    constexpr int kL = kLine<kWarps>;
    const int lane = threadIdx.x & 31, flip = kL == 64 ? lane & 7 : lane >> 1 & 3;
    uint8_t* second = lines + kLinesBytes<kWarps>;
#pragma unroll
    for (int k = 0; k < kL / 8; ++k) {
        uint4* at = reinterpret_cast<uint4*>(lines + lane * (kL * 2) + ((k ^ flip) << 4));
        uint4* lo_at = at + kLinesBytes<kWarps> / 16;
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = alpha * __uint_as_float(v[k * 8 + j]);
        if (kForm != kGram) {
            const uint4 h = *at;
            const uint32_t w[4] = {h.x, h.y, h.z, h.w};
            uint32_t l[4] = {};
            if (kForm != kSquare) {
                const uint4 o = *lo_at;
                l[0] = o.x, l[1] = o.y, l[2] = o.z, l[3] = o.w;
            }
            float b[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) b[j] = beta;
            if (kForm != kSquare && kSpecial && k * 8 < left) {
                const float4 d0 = reinterpret_cast<const float4*>(diag + k * 8)[0];
                const float4 d1 = reinterpret_cast<const float4*>(diag + k * 8)[1];
                const float d[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) b[j] = fmaf(unscale, d[j], beta);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 x = unpack_half2(w[j]);
                if (kForm != kSquare) {
                    const float2 y = unpack_half2(l[j]);
                    x.x = fmaf(1.0f / kLowScale, y.x, x.x);
                    x.y = fmaf(1.0f / kLowScale, y.y, x.y);
                }
                f[2 * j] = fmaf(b[2 * j], x.x, f[2 * j]);
                f[2 * j + 1] = fmaf(b[2 * j + 1], x.y, f[2 * j + 1]);
            }
            if (kForm == kSquare && kSpecial) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (k * 8 + j == at_diag) {
                        *diag = f[j] * (1.0f / kSquareScale);
                        f[j] = 0.0f;
                    }
                }
            }
        }
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = kForm == kLast ? pack2(f[2 * j], f[2 * j + 1])
                                  : pack_half2(f[2 * j], f[2 * j + 1]);
        *at = make_uint4(o[0], o[1], o[2], o[3]);
        if (kForm == kStep) {
            uint32_t r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = unpack_half2(o[j]);
                r[j] = pack_half2(kLowScale * (f[2 * j] - x.x), kLowScale * (f[2 * j + 1] - x.y));
            }
            *lo_at = make_uint4(r[0], r[1], r[2], r[3]);
        }
        if (kMirrored) {
            // column c of the part is row c of its mirror image
            uint16_t* mirror = reinterpret_cast<uint16_t*>(second);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                mirror[(k * 8 + j) * 32 + lane] = (uint16_t)(o[j / 2] >> (j % 2 * 16));
        }
    }
}

// Behind after_previous: lets the next kernel's blocks start on SMs that this one leaves idle or
// is through with, where they set up their barriers and their TMEM and wait for this kernel's end.
// All blocks have the kernel before behind them when they say so, so a kernel's start is still
// the end of all but the one before it.  17 launches on each other's results, in a graph, on tiles
// of 256 columns: 8 of 512 x 128 117 -> 105 us, one of 1024 x 1024 176 -> 166, 8 of them 313 -> 300.  Products of many
// tiles a pair do without: 64 of 2048 x 1408 back to back 4750 -> 4830 to 4910 us with it.
__device__ __forceinline__ void start_next() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// in, in2: G, or X's two halves (kStep, kLast); out, out2: the output and its mirror image or
// X's second half.  diag: S's diagonal, fp32 [E, m]: kSquare writes it and leaves zeros in its
// place, kStep and kLast add it to p0.
template <Form kForm, bool kMnA, bool kMnB, int kWarps>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(128 + 32 * kWarps, 1)
    muon_product_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmIn,
                        const __grid_constant__ CUtensorMap tmIn2,
                        const __grid_constant__ CUtensorMap tmOut,
                        const __grid_constant__ CUtensorMap tmOut2, Dims d, float alpha,
                        float beta, float unscale, float* diag, int* err) {
    constexpr bool kSym = kForm == kGram || kForm == kSquare;
    constexpr bool kWide = kMnB;  // kStep, kLast: S X (S's rows are X's), or else X S
    constexpr int kL = kLine<kWarps>;  // columns of a line
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t* tiles = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
    const uint32_t tiles_addr = smem_u32(tiles);
    uint8_t* staging_area = tiles + (size_t)kStages * STAGE_BYTES;
    auto* ctl = reinterpret_cast<Ctl*>(staging_area + (size_t)kStagingBytes);
    volatile int* abort_flag = &ctl->abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const int wide = kWarps == 4 ? BT : d.wide;
    const bool triangle = kSym && wide == BT;
    const int MB = blocks_of(d.m, BT), NB = blocks_of(d.n, wide), KB = blocks_of(d.K, BK);
    const int per_matrix = triangle ? NB * (NB + 1) / 2 : MB * NB;
    const long long total = (long long)d.E * per_matrix;
    const int pairs = (int)(gridDim.x / 2);
    const int n_last = last_columns(d.n, wide);

    if (warp == 4) {
        if (lane < kBarriers) {
            const int tempty = 2 * kStages + kAccs;
            mbar_init(smem_u32(&ctl->full[0] + lane),
                      lane >= tempty && lane < tempty + kAccs ? 2 * kWarps : 1);
        }
        if (lane == 31) ctl->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        prefetch_map(&tmA);
        prefetch_map(&tmB);
        prefetch_map(&tmOut);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&ctl->tmem_base), kTmemCols);
        tmem_relinquish_pair();
    }
    after_previous();
    if constexpr (kWarps == 8) start_next();
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any remote signal
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    if (warp < 4) {
        if (warp == 0 && elect_one()) {
            // ---------------- TMA producer (both CTAs) ----------------
            const uint32_t full0 = mapa_shared(smem_u32(&ctl->full[0]), 0);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (long long i = blockIdx.x / 2; ok && i < total; i += pairs) {
                const Tile t = decode(i, per_matrix, MB, NB, triangle);
                const int half = (t.nb == NB - 1 ? n_last : wide) / 2;
                const int a0 = t.mb * BT + (int)rank * BH, b0 = t.nb * wide + (int)rank * half;
                const bool two = half > 64;
                const uint32_t tx = OP_BYTES + (kMnB && !two ? BOX_BYTES : OP_BYTES);
                for (int kb = 0; kb < KB; ++kb) {
                    if (!wait_bar(smem_u32(&ctl->empty[stage]), phase ^ 1u, abort_flag, err)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = full0 + (uint32_t)stage * 8u;
                    const uint32_t a_s = tiles_addr + stage * STAGE_BYTES, b_s = a_s + OP_BYTES;
                    const int k = kb * BK;
                    if (leader) mbar_expect_tx(smem_u32(&ctl->full[stage]), 2 * tx);
                    if (kMnA) {
                        tma_load_3d_pair(a_s, &tmA, full, a0, k, t.e);
                        tma_load_3d_pair(a_s + BOX_BYTES, &tmA, full, a0 + 64, k, t.e);
                    } else {
                        tma_load_3d_pair(a_s, &tmA, full, k, a0, t.e);
                    }
                    if (kMnB) {
                        tma_load_3d_pair(b_s, &tmB, full, b0, k, t.e);
                        if (two) tma_load_3d_pair(b_s + BOX_BYTES, &tmB, full, b0 + 64, k, t.e);
                    } else {
                        tma_load_3d_pair(b_s, &tmB, full, k, b0, t.e);
                    }
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // a wait has given up: let the copies in flight land before the CTA exits
            if (*abort_flag) {
                const long long t0 = clock64();
                while (clock64() - t0 < 4000000) {
                }
            }
        } else if (warp == 1 && leader && elect_one()) {
            // ---------------- MMA issuer (leader only) ----------------
            constexpr uint32_t kMajors = (kMnA ? kIdescMnA : 0u) | (kMnB ? kIdescMnB : 0u);
            constexpr uint64_t kStepA = kMnA ? 16 * 128 / 16 : 2;
            constexpr uint64_t kStepB = kMnB ? 16 * 128 / 16 : 2;
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (long long i = blockIdx.x / 2; ok && i < total; i += pairs) {
                const Tile t = decode(i, per_matrix, MB, NB, triangle);
                const uint32_t idesc = kMajors | idesc_f16(BT, t.nb == NB - 1 ? n_last : wide);
                if (!wait_bar(smem_u32(&ctl->tempty[acc]), acc_phase ^ 1u, abort_flag, err)) break;
                tc_fence_after();
                const uint32_t to = tmem + (uint32_t)(acc * BT);
                for (int kb = 0; kb < KB; ++kb) {
                    if (!wait_bar(smem_u32(&ctl->full[stage]), phase, abort_flag, err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_s = tiles_addr + stage * STAGE_BYTES, b_s = a_s + OP_BYTES;
                    const uint64_t ad = kMnA ? sw128_desc_mn(a_s, BOX_BYTES) : sw128_desc(a_s);
                    const uint64_t bd = kMnB ? sw128_desc_mn(b_s, BOX_BYTES) : sw128_desc(b_s);
#pragma unroll
                    for (int kk = 0; kk < BK / UMMA_K; ++kk)
                        umma_f16_pair(to, ad + kStepA * kk, bd + kStepB * kk, idesc,
                                      (kb | kk) != 0 ? 1u : 0u);
                    umma_commit_pair_multicast(smem_u32(&ctl->empty[stage]), 0x3);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                umma_commit_pair_multicast(smem_u32(&ctl->tfull[acc]), 0x3);
                if (++acc == kAccs) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            umma_commit_pair_multicast(smem_u32(&ctl->done), 0x1);
            wait_bar_drain(smem_u32(&ctl->done), 0);
        }
    } else {
        // ---------------- epilogue (both CTAs): own 128 rows ----------------
        const int q = warp & 3, part = (warp - 4) >> 2;  // TMEM lane quadrant, columns
        const int columns = wide / (kWarps / 4);
        uint8_t* lines = staging_area + (size_t)(warp - 4) * (kStagingBytes / kWarps);
        const uint32_t lines_addr = smem_u32(lines), bar = smem_u32(&ctl->lines[warp - 4]);
        const uint32_t tempty0 = mapa_shared(smem_u32(&ctl->tempty[0]), 0);
        int acc = 0, buf = 0;
        uint32_t acc_phase = 0, lines_phase = 0;
        for (long long i = blockIdx.x / 2; i < total; i += pairs) {
            const Tile t = decode(i, per_matrix, MB, NB, triangle);
            const int row = t.mb * BT + (int)rank * BH + q * 32, col = t.nb * wide + part * columns;
            // lines that there are
            const int left = d.n - col < columns ? d.n - col : columns;
            const int have = row >= d.m || left <= 0 ? 0 : (left + kL - 1) / kL;
            // the inputs' lines c into buffer b, once what went out from there has been read
            const auto fetch = [&](int c, int b) {
                if (kForm == kGram || lane != 0) return;
                bulk_wait_read();
                const uint32_t to = lines_addr + (uint32_t)(b * kBufferBytes<kWarps>);
                mbar_expect_tx(bar, kForm == kSquare ? kLinesBytes<kWarps> : 2 * kLinesBytes<kWarps>);
                tma_load_3d(to, &tmIn, bar, col + c * kL, row, t.e);
                if (kForm != kSquare)
                    tma_load_3d(to + kLinesBytes<kWarps>, &tmIn2, bar, col + c * kL, row, t.e);
            };
            if (have > 0) fetch(0, buf);
            float* diag_e = diag + (long long)t.e * (kForm >= kStep && !kWide ? d.n : d.m);
            float row_beta = beta;
            if (kForm >= kStep && kWide && row + lane < d.m)
                row_beta = fmaf(unscale, diag_e[row + lane], beta);
            int ok = 0;
            if (lane == 0)
                ok = wait_bar(smem_u32(&ctl->tfull[acc]), acc_phase, abort_flag, err);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            tc_fence_after();
            if (!ok) break;
            const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BT + part * columns);
            const auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(tempty0 + (uint32_t)acc * 8u);
            };
            if (have == 0) release();
#pragma unroll 1
            for (int c = 0; c < have; ++c) {
                uint32_t v[kL];
                tmem_ld_columns(at + c * kL, v);
                tmem_wait_ld();
                if (c == have - 1) release();
                if (kForm == kGram) {
                    if (lane == 0) bulk_wait_read_but_one();  // the buffer's last lines
                } else {
                    if (!wait_bar(bar, lines_phase, abort_flag, err)) ok = 0;
                    lines_phase ^= 1u;
                }
                if (!__all_sync(0xffffffffu, ok)) break;
                if (c + 1 < have) fetch(c + 1, buf ^ 1);
                uint8_t* mine = lines + buf * kBufferBytes<kWarps>;
                const int first = col + c * kL;
                const bool mirrored = triangle && t.mb != t.nb;
                if (kForm == kSquare && first < row + 32 && row < first + kL)
                    combine<kForm, kWarps, true, false>(mine, v, alpha, beta, diag_e + row + lane,
                                                        row + lane < d.m ? row + lane - first : -1,
                                                        0, 0.0f);
                else if (kForm >= kStep && !kWide)
                    combine<kForm, kWarps, true, false>(mine, v, alpha, beta, diag_e + first, 0,
                                                        d.n - first, unscale);
                else if (kSym && mirrored)
                    combine<kForm, kWarps, false, kSym>(mine, v, alpha, beta, nullptr, 0, 0, 0.0f);
                else
                    combine<kForm, kWarps, false, false>(mine, v, alpha, row_beta, nullptr, 0, 0, 0.0f);
                fence_async_shared();
                __syncwarp();
                if (lane == 0) {
                    const uint32_t from = smem_u32(mine);
                    tma_store_3d(&tmOut, from, col + c * kL, row, t.e);
                    if (kForm == kStep)
                        tma_store_3d(&tmOut2, from + kLinesBytes<kWarps>, col + c * kL, row, t.e);
                    if (mirrored)
                        tma_store_3d(&tmOut2, from + kLinesBytes<kWarps>, row, col + c * kL, t.e);
                    bulk_commit();
                }
                buf ^= 1;
            }
            if (!__all_sync(0xffffffffu, ok)) break;
            if (++acc == kAccs) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no CTA leaves while its peer may still signal it
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// ---- momentum, norm, scale ----------------------------------------------------------------

constexpr int kBlock = 256;
constexpr int kChunk = kBlock * 8 * 4;  // elements of a block's round
constexpr int kMaxParts = 256;          // blocks of a matrix
constexpr int kAhead = 2;               // vectors of a thread that are loaded together

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
// u of a matrix's 8 elements at p, from the new momentum.
template <typename G>
__device__ __forceinline__ void update8(const G* grad, const float* buf, bool nesterov, float beta,
                                        float (&u)[8]) {
    if (!buf) {
        load8(grad, u);
        return;
    }
    load8(buf, u);
    if (nesterov) {
        float g[8];
        load8(grad, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = fmaf(beta, u[j], g[j]);
    }
}

// The new momentum and the sums of squares of u, one of each block (blockIdx.y: the matrix).
// Squares of values from 2^64 on, and sums of eight of them from some 2^62 on, leave fp32: all are
// summed times 2^-132 besides, where eight squares of the largest fp32 number are below 2^127.
template <typename G>
__global__ void __launch_bounds__(kBlock)
    muon_momentum_kernel(const G* grad, const float* buf, float* new_buf, long long size,
                         bool nesterov, float beta, double2* parts) {
    after_previous();
    start_next();
    const long long at = (long long)blockIdx.y * size;
    double sum = 0.0, big = 0.0;
    const long long step = (long long)gridDim.x * kBlock * 8;
    for (long long i0 = ((long long)blockIdx.x * kBlock + threadIdx.x) * 8; i0 < size;
         i0 += kAhead * step) {
        // all loads of kAhead vectors before the first is worked on
        float g[kAhead][8], b[kAhead][8];
#pragma unroll
        for (int v = 0; v < kAhead; ++v) {
            const long long i = i0 + v * step;
            if (i < size) {
                load8(grad + at + i, g[v]);
                if (buf) load8(buf + at + i, b[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < kAhead; ++v) {
            const long long i = i0 + v * step;
            if (i >= size) break;
            float u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = g[v][j];
            if (buf) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    b[v][j] = fmaf(beta, b[v][j], g[v][j]);
                    u[j] = nesterov ? fmaf(beta, b[v][j], g[v][j]) : b[v][j];
                }
                float4* to = reinterpret_cast<float4*>(new_buf + at + i);
                to[0] = make_float4(b[v][0], b[v][1], b[v][2], b[v][3]);
                to[1] = make_float4(b[v][4], b[v][5], b[v][6], b[v][7]);
            }
            float s = 0.0f, t = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float small = u[j] * 0x1p-66f;
                s = fmaf(u[j], u[j], s);
                t = fmaf(small, small, t);
            }
            sum += s;
            big += t;
        }
    }
    __shared__ double2 warps[kBlock / 32];
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        big += __shfl_xor_sync(0xffffffffu, big, o);
    }
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = make_double2(sum, big);
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kBlock / 32; ++w) {
            sum += warps[w].x;
            big += warps[w].y;
        }
        parts[(long long)blockIdx.y * gridDim.x + blockIdx.x] = make_double2(sum, big);
    }
}

// X = u 2^p / (|u| + eps) as hi + lo 2^-11.
template <typename G>
__global__ void __launch_bounds__(kBlock)
    muon_scale_kernel(const G* grad, const float* buf, long long size, bool nesterov, float beta,
                      float eps, int p, const double2* parts, int n_parts, __half* hi, __half* lo) {
    after_previous();
    start_next();
    __shared__ float factors[2];
    const long long at = (long long)blockIdx.y * size;
    if (threadIdx.x < 32) {
        double sum = 0.0, big = 0.0;
        for (int i = threadIdx.x; i < n_parts; i += 32) {
            const double2 v = parts[(long long)blockIdx.y * n_parts + i];
            sum += v.x;
            big += v.y;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            big += __shfl_xor_sync(0xffffffffu, big, o);
        }
        // in two factors: one alone may be too small for fp32
        if (!(sum < 1e300)) sum = big * 0x1p132;
        int ex = 0;
        const double f = frexp(1.0 / (sqrt(sum) + (double)eps), &ex);
        if (threadIdx.x == 0) {
            factors[0] = (float)ldexp(f, ex / 2);
            factors[1] = (float)ldexp(1.0, ex - ex / 2 + p);
        }
    }
    __syncthreads();
    const float f0 = factors[0], f1 = factors[1];
    for (long long i = ((long long)blockIdx.x * kBlock + threadIdx.x) * 8; i < size;
         i += (long long)gridDim.x * kBlock * 8) {
        float u[8];
        update8(grad + at + i, buf ? buf + at + i : nullptr, nesterov, beta, u);
        uint32_t h[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = u[2 * j] * f0 * f1, b = u[2 * j + 1] * f0 * f1;
            h[j] = pack_half2(a, b);
            const float2 r = unpack_half2(h[j]);
            l[j] = pack_half2(kLowScale * (a - r.x), kLowScale * (b - r.y));
        }
        *reinterpret_cast<uint4*>(hi + at + i) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(lo + at + i) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

// ---- host ---------------------------------------------------------------------------------

struct Work {
    size_t parts, diag, gram, square, hi[2], lo, total;
};
Work work_of(const moe_muon_shape& s) {
    const size_t n = (size_t)s.E * s.M * s.N;
    const size_t m = s.M < s.N ? s.M : s.N, sq = (size_t)s.E * m * m;
    Work w;
    size_t o = 256;  // the error word
    w.parts = o;  o = align256(o + (size_t)s.E * kMaxParts * sizeof(double2));
    w.diag = o;   o = align256(o + (size_t)s.E * m * 4);
    w.gram = o;   o = align256(o + sq * 2);
    w.square = o; o = align256(o + sq * 2);
    for (size_t& hi : w.hi) hi = o, o = align256(o + n * 2);
    w.lo = o;     o = align256(o + n * 2);
    w.total = o;
    return w;
}

bool map_matrices(CUtensorMap* m, const void* ptr, int E, int rows, int cols, uint32_t box_cols,
                  uint32_t box_rows, MapType type, int swizzle) {
    const uint64_t sizes[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)E};
    const uint64_t strides[2] = {(uint64_t)cols * 2, (uint64_t)cols * rows * 2};
    const uint32_t box[3] = {box_cols, box_rows, 1};
    return map_typed(m, 3, ptr, sizes, strides, box, type, swizzle);
}

// The outputs' (and their inputs') maps, in lines of 64 columns and of 32: of 32 rows, and mirror
// images of 32 columns.
struct LineMaps {
    CUtensorMap g, g_mirror, s, s_mirror, hi[2], lo, out;
};

template <Form kForm, bool kMnA, bool kMnB, int kWarps>
moe_status launch_form(const CUtensorMap& a, const CUtensorMap& b, const LineMaps& l, int now,
                       const Dims& d, float alpha, float beta, float unscale, float* diag, int* err,
                       long long pairs, cudaStream_t st) {
    const auto kernel = muon_product_kernel<kForm, kMnA, kMnB, kWarps>;
    static OncePerDevice set;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    if (!set.done(dev)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)kSmem) != cudaSuccess)
            return MOE_ERR_CUDA;
        set.finish(dev);
    }
    const CUtensorMap& in = kForm <= kSquare ? l.g : l.hi[now];
    const CUtensorMap& in2 = kForm <= kSquare ? l.g : l.lo;
    const CUtensorMap& out = kForm == kGram     ? l.g
                             : kForm == kSquare ? l.s
                             : kForm == kStep   ? l.hi[1 - now]
                                                : l.out;
    const CUtensorMap& out2 = kForm == kGram     ? l.g_mirror
                              : kForm == kSquare ? l.s_mirror
                              : kForm == kStep   ? l.lo
                                                 : l.out;
    return cuda_status(launch_chained(kernel, (int)(2 * pairs), 128 + 32 * kWarps, kSmem, st, a, b,
                                      in, in2, out, out2, d, alpha, beta, unscale, diag, err));
}
template <Form kForm, bool kMnA, bool kMnB>
moe_status launch_product(const CUtensorMap& a, const CUtensorMap& b, const LineMaps (&l)[2],
                          int now, Dims d, float alpha, float beta, float unscale, float* diag,
                          int* err, cudaStream_t st) {
    constexpr bool kSym = kForm == kGram || kForm == kSquare;
    const long long MB = blocks_of(d.m, BT), most = sm_count() / 2;
    long long NB = blocks_of(d.n, BT);
    // As narrow as lets all tiles run at once: the epilogue, a line of 32 columns after the other,
    // is most of a short launch.  Symmetric products then make every tile.  With 256 columns, and
    // so: 8 of 512 x 128 105, 78 us; one of 1024 x 1024 166, 115; 4 of 256 x 4096 207, 153; one of
    // 1408 x 2048 211, 179.  Narrow tiles that run in turn gain nothing: one of 2048 x 2048 255, 281.
    for (int wide = BT / 4; wide < BT && d.wide == BT; wide *= 2)
        if (d.E * MB * blocks_of(d.n, wide) <= most) {
            d.wide = wide;
            NB = blocks_of(d.n, wide);
        }
    const long long tiles = d.E * (kSym && d.wide == BT ? NB * (NB + 1) / 2 : MB * NB);
    // 8 warps where a pair has no more than four tiles
    return tiles > 4 * most ? launch_form<kForm, kMnA, kMnB, 4>(a, b, l[0], now, d, alpha, beta,
                                                                unscale, diag, err, most, st)
                            : launch_form<kForm, kMnA, kMnB, 8>(a, b, l[1], now, d, alpha, beta,
                                                                unscale, diag, err,
                                                                tiles < most ? tiles : most, st);
}

template <typename G>
moe_status launch_prepare(const G* grad, const float* buf, float* new_buf, const moe_muon_shape& s,
                          int p, double2* parts, __half* hi, __half* lo, cudaStream_t st) {
    const long long size = (long long)s.M * s.N, rounds = (size + kChunk - 1) / kChunk;
    // some 16 blocks an SM in all, each matrix the same number
    const long long share = 16LL * sm_count() / s.E + 1;
    const long long most = share < kMaxParts ? share : kMaxParts;
    const int blocks = (int)(rounds < most ? rounds : most);
    const bool nesterov = s.nesterov != 0;
    MOE_TRY(cuda_status(launch_chained(muon_momentum_kernel<G>, dim3(blocks, s.E), kBlock, 0, st,
                                       grad, buf, new_buf, size, nesterov, s.momentum, parts)));
    return cuda_status(launch_chained(muon_scale_kernel<G>, dim3(blocks, s.E), kBlock, 0, st, grad,
                                      (const float*)new_buf, size, nesterov, s.momentum, s.eps, p,
                                      (const double2*)parts, blocks, hi, lo));
}

bool valid(const moe_muon_shape* s) {
    return s && s->E > 0 && s->M > 0 && s->N > 0 && s->steps > 0 && s->steps <= 64 &&
           s->momentum >= 0.0f && s->momentum < 1.0f && s->eps >= 1e-12f && s->eps <= 1.0f &&
           (s->grad_type == MOE_TYPE_BF16 || s->grad_type == MOE_TYPE_F32);
}
bool supported(const moe_muon_shape* s) {
    return s->M % 8 == 0 && s->N % 8 == 0 && s->M <= kMaxDim && s->N <= kMaxDim &&
           s->E <= kMaxE;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_muon_workspace_bytes(const moe_muon_shape* shape) {
    return valid(shape) && supported(shape) ? work_of(*shape).total : 0;
}

moe_status moe_muon_update(const void* grad, const float* momentum, const moe_muon_shape* shape,
                           uint16_t* update, float* new_momentum, void* ws, size_t ws_bytes,
                           void* stream) {
    MOE_RANGE();
    if (!valid(shape)) return MOE_ERR_INVALID_ARG;
    if (!supported(shape)) return MOE_ERR_UNSUPPORTED;
    const moe_muon_shape& s = *shape;
    const Work w = work_of(s);
    if (!ws || ws_bytes < w.total) return MOE_ERR_WORKSPACE;
    if (!grad || !update || (momentum == nullptr) != (new_momentum == nullptr))
        return MOE_ERR_INVALID_ARG;
    if (!aligned16(grad, momentum, update, new_momentum, ws)) return MOE_ERR_INVALID_ARG;
    const cudaStream_t st = as_stream(stream);
    const bool tall = s.M > s.N;
    const int m = tall ? s.N : s.M, longer = tall ? s.M : s.N;
    int p = 0;
    while ((1LL << (2 * p + 1)) < longer) ++p;  // 2^p about the root of the longer side
    auto* gram = ws_ptr<__half>(ws, w.gram);
    auto* square = ws_ptr<__half>(ws, w.square);
    // a step's X is an operand of all tiles of the next one: they write to the other copy
    __half* hi[2] = {ws_ptr<__half>(ws, w.hi[0]), ws_ptr<__half>(ws, w.hi[1])};
    auto* lo = ws_ptr<__half>(ws, w.lo);
    auto* parts = ws_ptr<double2>(ws, w.parts);
    float* diag = ws_ptr<float>(ws, w.diag);
    int* err = ws_ptr<int>(ws, 0);
    MOE_TRY(s.grad_type == MOE_TYPE_F32
                ? launch_prepare(static_cast<const float*>(grad), momentum, new_momentum, s, p,
                                 parts, hi[0], lo, st)
                : launch_prepare(static_cast<const __nv_bfloat16*>(grad), momentum, new_momentum,
                                 s, p, parts, hi[0], lo, st));
    // operands: rows with their contraction along them (k) or columns (mn)
    CUtensorMap x_k[2], x_mn[2], g_k, s_k;
    LineMaps l[2];
    const auto operand = [&](CUtensorMap* t, const void* ptr, int rows, int cols, uint32_t box_rows) {
        return map_matrices(t, ptr, s.E, rows, cols, BK, box_rows, kMapF16, 128);
    };
    bool ok = operand(&g_k, gram, m, m, BH) && operand(&s_k, square, m, m, BH);
    for (int i = 0; i < 2; ++i)
        ok = ok && operand(&x_k[i], hi[i], s.M, s.N, BH) && operand(&x_mn[i], hi[i], s.M, s.N, BK);
    for (int w = 0; w < 2; ++w) {
        const uint32_t cols = w == 0 ? kLine<4> : kLine<8>;
        const auto lines = [&](CUtensorMap* t, const void* ptr, int M, int N, MapType type) {
            return map_matrices(t, ptr, s.E, M, N, cols, 32, type, (int)cols * 2);
        };
        const auto mirror = [&](CUtensorMap* t, const void* ptr) {
            return map_matrices(t, ptr, s.E, m, m, 32, cols, kMapF16, 0);
        };
        ok = ok && lines(&l[w].g, gram, m, m, kMapF16) && lines(&l[w].s, square, m, m, kMapF16) &&
             mirror(&l[w].g_mirror, gram) && mirror(&l[w].s_mirror, square) &&
             lines(&l[w].hi[0], hi[0], s.M, s.N, kMapF16) &&
             lines(&l[w].hi[1], hi[1], s.M, s.N, kMapF16) &&
             lines(&l[w].lo, lo, s.M, s.N, kMapF16) &&
             lines(&l[w].out, update, s.M, s.N, kMapBF16);
    }
    if (!ok) return MOE_ERR_UNSUPPORTED;
    const float scale = ldexpf(1.0f, -2 * p) * kSquareScale, back = 1.0f / kSquareScale;
    const Dims gd = {s.E, longer, m, m, BT}, sd = {s.E, m, m, m, BT}, xd = {s.E, m, s.M, s.N, BT};
    for (int i = 0; i < s.steps; ++i) {
        const int now = i % 2;
        MOE_TRY(tall ? launch_product<kGram, true, true>(x_mn[now], x_mn[now], l, now, gd, scale,
                                                         0.0f, 1.0f, diag, err, st)
                     : launch_product<kGram, false, false>(x_k[now], x_k[now], l, now, gd, scale,
                                                           0.0f, 1.0f, diag, err, st));
        MOE_TRY(launch_product<kSquare, false, false>(g_k, g_k, l, now, sd, kP2 * back, kP1, 1.0f,
                                                      diag, err, st));
        const bool last = i == s.steps - 1;
        const float unscale = last ? ldexpf(1.0f, -p) : 1.0f;
        const CUtensorMap &a = tall ? x_k[now] : s_k, &b = tall ? s_k : x_mn[now];
        const auto step = [&](auto launch) {
            return launch(a, b, l, now, xd, back * unscale, kP0 * unscale, unscale, diag, err, st);
        };
        if (last)
            MOE_TRY(tall ? step(launch_product<kLast, false, false>)
                         : step(launch_product<kLast, false, true>));
        else
            MOE_TRY(tall ? step(launch_product<kStep, false, false>)
                         : step(launch_product<kStep, false, true>));
    }
    return MOE_OK;
}

}  // extern "C"
