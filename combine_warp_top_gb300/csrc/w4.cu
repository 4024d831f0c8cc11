// Products of few rows with matrices of 4-bit weights: the experts of a decoding step.
//
//   y[i, o] = sum over k of rows[i, k] * scale[e][o, k / group] * (q[e][o, k] - 8)
//
// with q in 0..15 and a scale for `group` weights of a matrix row; gated: the matrix holds I
// gate rows and I up rows, and h = w_i SiLU(g) u leaves instead of y.
//
// Memory bound: every weight is read once, 4 bits and its share of a scale.  So the packed
// layout (w4_pack_kernel) is the order in which the kernel reads: tiles of 256 matrix rows in
// chunks of 128 weights of each, one chunk of a tile a contiguous piece of 17 to 18 KB that one
// bulk copy brings into a ring of shared memory, the scales beside the weights.  The rows'
// chunks come by TMA boxes of 8 rows.
//
// The matrix is the MMA's A and the rows are its B (tcgen05, M = 128, N = 16 to 64).  A thread
// has one row of the matrix: it widens the row's weights to bf16 in registers (q - 8 over 64,
// exact: see widen) and stores them into TMEM, from where the MMA takes A:
// shared memory sees the 4-bit form only.  A group's sums are fp32 in TMEM; the thread reads
// its row's, scales them once and adds them to its own sums, in fp32, while the MMAs of the
// next 64 weights run.  (mma.sync on weights widened in the same way: 129 tokens of the fourth
// case below 213 us, 16 tokens of the second 379 us.)
//
// What bounds it (GB300), in a graph, and the bytes' floor:
//   1 token of 8 of 256 experts, 2048 -> 7168          22 us      8.9
//   16 tokens of the same layer, gate and up           268 us     227   (5.9 TB/s)
//   64 tokens of 6 of 64 experts, 2048 -> 2 x 1408     50 us      29
//   129 tokens of 2 of 8 experts, 14336 -> 4096        76 us      37
// In the long run the integer pipe: 5 operations (4 LOP3, a shift) for 8 weights; without the
// shift the second case would take 246 us, without the groups' sums 256, without widening 234.
// (Before widen used subnormals it had 7 operations and a subtraction for every pair: 317 us.  A
// multiplication in the shift's place 292, a byte permute the same as it.)  In short calls the
// ends: 3500 cycles until a block has found its first tile, 5400 to join a tile that blocks
// share; and an expert of more rows than a pass has its weights widened for each.
#include <stddef.h>

#include "../../include/moe_train.h"
#include "../../include/moe_w4.h"
#include "api_checks.cuh"
#include "gate.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kSlabRows = 32;  // matrix rows of a warp
constexpr int kSlabs = 8;      // warps of a tile
constexpr int kChunk = 128;    // weights of a row in a chunk
constexpr int kNibbleBytes = kSlabRows * kChunk / 2;
constexpr int kConsumers = kSlabs * 32;
constexpr int kThreads = kConsumers + 64;  // and a warp for the MMAs, one for the copies
constexpr int kMmaRows = 128;  // of an MMA: a tile has two
constexpr int kMaxBlocks = 304;

__host__ __device__ __forceinline__ int ceil_div(long long a, int b) {
    return (int)((a + b - 1) / b);
}
// A slab's chunk: nibbles, then its scales.
__host__ __device__ constexpr int record_bytes(int group) {
    return kNibbleBytes + kSlabRows * 2 * (kChunk / group);
}

// A matrix: its packed form's sizes.
struct Matrix {
    int rows, C_in, group, gated;  // rows of the output: C_out, or I of the gated
    int slabs, tiles, chunks, record;
};
Matrix matrix_of(const moe_w4_matrix& m) {
    Matrix d;
    d.rows = m.C_out;
    d.C_in = m.C_in;
    d.group = m.group;
    d.gated = m.gated != 0;
    d.slabs = ceil_div(m.C_out, d.gated ? kSlabRows / 2 : kSlabRows);
    d.tiles = ceil_div(d.slabs, kSlabs);
    d.chunks = ceil_div(m.C_in, kChunk);
    d.record = record_bytes(m.group);
    return d;
}

// The slabs of a tile's chunk lie side by side, the chunks of a tile one after the other.
__host__ __device__ __forceinline__ int tile_slabs(const Matrix& m, int tile) {
    return m.slabs - tile * kSlabs < kSlabs ? m.slabs - tile * kSlabs : kSlabs;
}
__host__ __device__ __forceinline__ long long chunk_at(const Matrix& m, int tile, int chunk) {
    return ((long long)tile * kSlabs * m.chunks + (long long)chunk * tile_slabs(m, tile)) * m.record;
}

// The output column of a slab's row r (0..31), or -1; up: whether the row is of the up matrix
// (gated: 16 gate rows, then their 16 up rows).
__device__ __forceinline__ int matrix_row(const Matrix& m, int slab, int r, bool* up) {
    *up = m.gated && r >= 16;
    const int o = m.gated ? slab * 16 + (r & 15) : slab * 32 + r;
    return o < m.rows ? o : -1;
}

// ---- the product ---------------------------------------------------------------------------

// kN: rows of a pass at most (the MMA's N, in steps of 16).
// TMEM: A's two buffers of 64 weights a row, 32 columns each, of both MMAs' rows, then the sums
// of the groups that end in one buffer or the other.
template <int kN, int kGroup>
struct Form {
    static constexpr int kHalfGroups = kGroup == 32 ? 2 : 1;  // sums of 64 weights
    static constexpr int kSumColumns = 2 * kHalfGroups * kN;  // of 128 rows
    static constexpr int kSums = 128;                         // their first column
    static constexpr int kUsed = kSums + 2 * kSumColumns;
    static constexpr int kTmem = kUsed <= 256 ? 256 : 512;
    static constexpr int kBlocks = 512 / kTmem;  // of an SM
    static constexpr int kRecord = record_bytes(kGroup);
    static constexpr int kWeightBytes = kSlabs * kRecord;
    static constexpr int kRowBytes = 2 * kN * 128;  // two halves of 64 columns
    static constexpr int kStages = kBlocks == 2 ? (kN == 16 && kGroup > 32 ? 5 : 4) : 6;
    static size_t smem(int E) {
        return 1024 + (size_t)kStages * (kWeightBytes + kRowBytes) + (size_t)(E + 1) * 4;
    }
    static_assert(kBlocks * (2048 + kStages * (kWeightBytes + kRowBytes) + (kMaxE + 1) * 4 + 1024) <=
                      228 * 1024,
                  "shared memory of an SM");
};

struct Args {
    const uint8_t* packed;
    long long expert_bytes;
    Matrix m;
    Gate gate;  // gated: h, topk_w and the pairs
    void* out;  // plain: [R, C_out]
    int out_f32;
    const int32_t* offsets;
    const int32_t* counts;
    int E, R;
    float* parts;    // partial sums: two slots a block
    int* counters;   // arrivals at a slab of a tile, one of each block's warps
    int* err;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]^T, bf16 inputs, fp32 accumulate, one CTA.
__device__ __forceinline__ void umma_bf16_ta(uint32_t d, uint32_t a, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// Eight nibbles to four pairs of (q - 8) / 64: nibble r and nibble r + 4 are the halves of
// register r.  The last eight bits of a bf16 that has no others set are its units of 2^-133
// (subnormals and the binade above them are one line), so that a nibble is a number where it
// stands, q or 16 q units, and one FMA makes it the weight, exact: no exponent to be put to it,
// and one shift for both bytes.
__device__ __forceinline__ void widen(uint32_t w, uint32_t* a) {
    const uint32_t low = 0x7f007f00u, high = 0x7d007d00u, less = 0xbe00be00u;  // 2^127, 2^123, -1/8
#pragma unroll
    for (int r = 0; r < 4; r += 2) {
        const uint32_t b = w >> (4 * r);
        a[r] = fma_bf16x2(b & 0x000f000fu, low, less);
        a[r + 1] = fma_bf16x2(b & 0x00f000f0u, high, less);
    }
}
constexpr float kWidened = 64.0f;  // the weights over what widen gives

// The unit at which block b's share starts.
__device__ __forceinline__ long long share(long long total, int b, int blocks) {
    return total * b / blocks;
}

// A run of chunks of one tile for up to kN rows of an expert.
struct Piece {
    int e, tile, first_row, rows;  // rows from first_row of the expert's on
    int chunk0, chunk1;            // of the tile's chunks
    // the blocks that share the tile (after < 0: this one has all of it), and which of its two
    // slots the first of them uses
    int owner, after, owner_slot;
};

// Units are chunks: expert by expert, tile by tile, the passes over kN rows each side by side
// (they read the same weights), chunk by chunk.  prefix: passes before each expert.
template <int kN>
__device__ __forceinline__ Piece piece_at(const Args& a, const int* prefix, long long u,
                                          long long end, long long total, int block, int blocks) {
    const long long per_pass = (long long)a.m.tiles * a.m.chunks;
    const int q = (int)(u / per_pass);
    int lo = 0, hi = a.E;  // prefix[lo] <= q < prefix[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= q) lo = mid;
        else hi = mid;
    }
    Piece p;
    p.e = lo;
    const long long local = u - prefix[lo] * per_pass;
    const int cnt = a.counts[lo], passes = prefix[lo + 1] - prefix[lo];
    const long long run = local / a.m.chunks;  // tile * passes + pass
    p.chunk0 = (int)(local - run * a.m.chunks);
    p.tile = (int)(run / passes);
    const int pass = (int)(run - (long long)p.tile * passes);
    p.first_row = pass * kN;
    p.rows = cnt - p.first_row < kN ? cnt - p.first_row : kN;
    const long long left = end - u;
    p.chunk1 = left < a.m.chunks - p.chunk0 ? p.chunk0 + (int)left : a.m.chunks;
    p.owner = p.after = -1;
    p.owner_slot = 0;
    if (p.chunk0 > 0 || p.chunk1 < a.m.chunks) {
        // a tile of several blocks: those with units of [start, start + chunks).  A block's first
        // slot is for what it starts with, its second for a tile that it starts later.
        const long long start = u - p.chunk0;
        int o = block, f = block;
        while (share(total, o, blocks) > start) --o;
        while (share(total, f + 1, blocks) < start + a.m.chunks) ++f;
        p.owner = o;
        p.after = f;
        p.owner_slot = share(total, o, blocks) != start;
    }
    return p;
}

// The sums of a tile's slab to their output.  weights: of the rows (gated).
template <int kN, bool kGated>
__device__ __forceinline__ void write_out(const Args& a, const Piece& p, int slab,
                                          const float (&s)[kN], const float* weights) {
    const int lane = threadIdx.x & 31;
    const long long row0 = (long long)a.offsets[p.e] + p.first_row;
    if (kGated) {
        // lanes l and l + 16 have the gate and the up column of the same output: the first
        // takes the even rows, the second the odd ones
        const bool upper = lane >= 16;
        const int o = slab * 16 + (lane & 15);
#pragma unroll
        for (int n = 0; n < kN; n += 2) {
            if (n >= p.rows) break;
            const float mine_of = kWidened * (upper ? s[n + 1] : s[n]);
            const float got = kWidened * __shfl_xor_sync(0xffffffffu, upper ? s[n] : s[n + 1], 16);
            const float g = upper ? got : mine_of, u = upper ? mine_of : got;
            const int mine = n + upper;
            if (mine >= p.rows || o >= a.m.rows) continue;
            const long long row = row0 + mine;
            const __nv_bfloat16 h = __float2bfloat16_rn(weights[mine] * (g * sigmoid(g)) * u);
            a.gate.h[row * a.m.rows + o] = *reinterpret_cast<const uint16_t*>(&h);
        }
        return;
    }
    const int o = slab * 32 + lane;
    if (o >= a.m.rows) return;
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        if (n >= p.rows) break;
        const long long at = (row0 + n) * a.m.rows + o;
        if (a.out_f32)
            static_cast<float*>(a.out)[at] = kWidened * s[n];
        else
            static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(kWidened * s[n]);
    }
}

// wait_bar out of line, which sleeps between its looks: a warp that polls takes issue slots
// from those that widen.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort,
                                       int* err) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        __nanosleep(20);
        if (*abort) return false;
        if (clock64() - t0 > kWaitLimit) {
            *abort = 1;
            set_error(err, MOE_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, volatile int* abort,
                                         int* err) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort, err);
}
__device__ __forceinline__ void linger() {
    const long long t0 = clock64();
    while (clock64() - t0 < 4000000) {
    }
}
// A whole warp's wait.
__device__ __forceinline__ void wait_warp(uint32_t bar, uint32_t parity, volatile int* abort,
                                          int* err) {
    if (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) wait_slow(bar, parity, abort, err);
    __syncwarp();
}

__device__ __forceinline__ uint4 ld_shared4(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
// The lane's row's bf16 scales of a chunk.
__device__ __forceinline__ void load_scales(uint32_t at, float (&s)[1]) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
    s[0] = __uint_as_float((uint32_t)v << 16);
}
__device__ __forceinline__ void load_scales(uint32_t at, float (&s)[2]) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    s[0] = __uint_as_float(v << 16);
    s[1] = __uint_as_float(v & 0xffff0000u);
}
__device__ __forceinline__ void load_scales(uint32_t at, float (&s)[4]) {
    uint32_t v, w;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                 : "=r"(v), "=r"(w)
                 : "r"(at)
                 : "memory");
    s[0] = __uint_as_float(v << 16);
    s[1] = __uint_as_float(v & 0xffff0000u);
    s[2] = __uint_as_float(w << 16);
    s[3] = __uint_as_float(w & 0xffff0000u);
}

// Each block takes an equal share of the units, whatever tiles they belong to.  A tile that
// several blocks share: each leaves its sums in a slot of the workspace, and the one that comes
// last adds them up in the order of the blocks and writes the tile out.  Nobody waits.
//
// A half is 64 weights of a row.  A warp widens half v while the MMAs of the two before it run,
// waits for those of half v - 2, whose buffer of A it takes, and reads the sums that they have
// ended: an arrival for half v says that A is there and that the place of its sums is free.
template <int kN, int kGroup, bool kGated>
__global__ void __launch_bounds__(kThreads, (Form<kN, kGroup>::kBlocks))
    w4_kernel(const __grid_constant__ CUtensorMap tmRows, const __grid_constant__ Args a) {
    using F = Form<kN, kGroup>;
    constexpr int kStages = F::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kStages], empty[kStages], a_ready[2], mma_done[2];
    __shared__ int run_sums[kThreads / 32];
    __shared__ uint32_t tmem_word;
    __shared__ int abort_word;
    // the pieces on their way and their rows' weights: those that read them are kSlots - 2 pieces
    // behind the copies at most, for a piece has a chunk at least
    constexpr int kSlots = kStages + 2;
    __shared__ Piece slots[kSlots];
    __shared__ float row_weights[kGated ? kSlots : 1][kN];
    uint8_t* rows_ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* ring = rows_ring + (size_t)kStages * F::kRowBytes;
    int* prefix = reinterpret_cast<int*>(ring + (size_t)kStages * F::kWeightBytes);
    volatile int* abort_flag = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&empty[i]), kSlabs + 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&a_ready[i]), kSlabs);
            mbar_init(smem_u32(&mma_done[i]), 1);
        }
        abort_word = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kSlabs) {
        if (lane == 0) prefetch_map(&tmRows);
        tmem_alloc(smem_u32(&tmem_word), F::kTmem);
        tmem_relinquish();
    }
    after_previous();
    // prefix[e]: passes before expert e; each thread sums a run of experts.  Only a layout whose
    // segments overlap has more of them than `most`: it gets one more and is reported, so that the
    // sums do not wrap.
    const int per = ceil_div(a.E, kThreads), e0 = threadIdx.x * per;
    const int most = a.R / kN + a.E;
    int mine = 0;
    const auto passes = [&](int e) {
        const int off = a.offsets[e], cnt = a.counts[e];
        if (off < 0 || cnt < 0 || cnt > a.R || off > a.R - cnt) {
            set_error(a.err, MOE_ERR_INVALID_ARG);
            return 0;
        }
        return ceil_div(cnt, kN);
    };
    const auto sum = [&](int x, int y) { return min(x + y, most + 1); };
    for (int e = e0; e < e0 + per && e < a.E; ++e) mine = sum(mine, passes(e));
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl = sum(incl, v);
    }
    if (lane == 31) run_sums[warp] = incl;
    int before = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 0) before = 0;
    __syncthreads();
    int all_passes = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) before = sum(before, run_sums[i]);
        all_passes = sum(all_passes, run_sums[i]);
    }
    for (int e = e0; e < e0 + per && e < a.E; ++e) {
        prefix[e] = before;
        before = sum(before, passes(e));
    }
    if (threadIdx.x == 0) {
        prefix[a.E] = all_passes;
        if (all_passes > most) set_error(a.err, MOE_ERR_INVALID_ARG);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_word;
    const long long total = (long long)all_passes * a.m.tiles * a.m.chunks;
    // no block without a unit: those of a tile are all that arrive at its counter
    const int blocks = total < (long long)gridDim.x ? (int)total : (int)gridDim.x;
    const int block = (int)blockIdx.x;
    long long first = 0, last = 0;
    if (block < blocks) {
        first = share(total, block, blocks);
        last = share(total, block + 1, blocks);
    }

    if (warp == kSlabs + 1) {
        // ---------------- copies ----------------
        Piece lp = {};
        long long lu = first;
        int load_slot = 0, boxes = 0, row = 0;
        uint32_t load_phase = 1, weights = 0;
        const uint8_t* from = nullptr;
        int pieces = 0;
        const bool one = elect_one();
        while (lu < last) {
            lp = piece_at<kN>(a, prefix, lu, last, total, block, blocks);
            boxes = ceil_div(lp.rows, 8);
            row = a.offsets[lp.e] + lp.first_row;
            weights = (uint32_t)(tile_slabs(a.m, lp.tile) * F::kRecord);
            from = a.packed + (long long)lp.e * a.expert_bytes + chunk_at(a.m, lp.tile, lp.chunk0);
            if (kGated) {
                // three loads one after the other, here in nobody's way
#pragma unroll
                for (int n = 0; n < kN; n += 32)
                    if (n + lane < lp.rows)
                        row_weights[pieces % kSlots][n + lane] =
                            row_weight(a.gate, (long long)row + n + lane);
            }
            if (lane == 0) slots[pieces % kSlots] = lp;
            __syncwarp();
            ++pieces;
            int given_up = 0;
            if (one) {
                for (int c = lp.chunk0; c < lp.chunk1; ++c) {
                    if (!wait_one(smem_u32(&empty[load_slot]), load_phase, abort_flag, a.err)) {
                        given_up = 1;
                        break;
                    }
                    const uint32_t bar = smem_u32(&full[load_slot]);
                    mbar_expect_tx(bar, weights + (uint32_t)(boxes * 2048));
                    bulk_load(smem_u32(ring) + (uint32_t)(load_slot * F::kWeightBytes), from,
                              weights, bar);
                    const uint32_t to = smem_u32(rows_ring) + (uint32_t)(load_slot * F::kRowBytes);
#pragma unroll
                    for (int b = 0; b < kN / 8; ++b) {
                        if (b >= boxes) break;
                        tma_load_2d(to + b * 1024, &tmRows, bar, c * kChunk, row + b * 8);
                        tma_load_2d(to + kN * 128 + b * 1024, &tmRows, bar, c * kChunk + 64,
                                    row + b * 8);
                    }
                    from += weights;
                    if (++load_slot == kStages) {
                        load_slot = 0;
                        load_phase ^= 1u;
                    }
                }
            }
            if (__any_sync(0xffffffffu, given_up)) break;
            lu += lp.chunk1 - lp.chunk0;
        }
        // a wait has given up: let the copies in flight land before the block ends
        if (*abort_flag) linger();
    } else if (warp == kSlabs && elect_one()) {
        // ---------------- MMAs ----------------
        bool ok = true;
        const uint64_t b0 = sw128_desc(smem_u32(rows_ring));
        uint32_t it = 0, phase = 0;
        int slot = 0;
        int pieces = 0;
        for (long long u = first; ok && u < last; ++pieces) {
            // a piece is known when its first chunk is there
            if (!wait_one(smem_u32(&full[slot]), phase, abort_flag, a.err)) break;
            const Piece p = slots[pieces % kSlots];
            const uint32_t idesc = make_idesc(kMmaRows, ceil_div(p.rows, 16) * 16);
            const bool upper = tile_slabs(a.m, p.tile) > kSlabs / 2;  // any slab of the second MMA's
            u += p.chunk1 - p.chunk0;
            for (int left = p.chunk1 - p.chunk0; left > 0; --left, ++it) {
                if (!wait_one(smem_u32(&full[slot]), phase, abort_flag, a.err)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!wait_one(smem_u32(&a_ready[h]), it & 1u, abort_flag, a.err)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t b = b0 + (uint64_t)((slot * F::kRowBytes + h * kN * 128) >> 4);
                    const uint32_t buf = kGroup == 128 ? it & 1u : (uint32_t)h;
                    const uint32_t d = tmem + F::kSums + buf * (uint32_t)(F::kHalfGroups * kN);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (t == 1 && !upper) break;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const bool starts = kGroup == 32   ? kk % 2 == 0
                                                : kGroup == 64 ? kk == 0
                                                               : kk == 0 && h == 0;
                            umma_bf16_ta(d + (uint32_t)(t * F::kSumColumns + (kGroup == 32 ? kk / 2 * kN : 0)),
                                         tmem + (uint32_t)(t * 64 + h * 32 + kk * 8), b + 2 * kk,
                                         idesc, starts ? 0u : 1u);
                        }
                    }
                    umma_commit(smem_u32(&mma_done[h]));
                }
                if (!ok) break;
                umma_commit(smem_u32(&empty[slot]));
                if (++slot == kStages) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
        }
        if (*abort_flag) linger();  // likewise the MMAs
    } else if (warp < kSlabs) {
        // ---------------- weights and sums ----------------
        // One whose wait gives up goes on with what is in memory to the piece's end (the call
        // reports it); its later waits return at once.
        constexpr int kGroups = kChunk / kGroup;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t a_at = tmem + lanes + (uint32_t)((warp >> 2) * 64);
        const uint32_t sums_at = tmem + lanes + (uint32_t)(F::kSums + (warp >> 2) * F::kSumColumns);
        // (a tile's last slabs may not be there: what the ring holds in their place gives rows of
        // sums that go nowhere)
        const uint32_t rec0 = smem_u32(ring) + (uint32_t)(warp * F::kRecord) + lane * 16;
        const uint32_t rec_scales = smem_u32(ring) + (uint32_t)(warp * F::kRecord) + kNibbleBytes +
                                    lane * (uint32_t)(kGroups * 2);
        int it = 0, slot = 0, pieces = 0;
        uint32_t phase = 0;
        for (long long u = first; u < last; ++pieces) {
            wait_warp(smem_u32(&full[slot]), phase, abort_flag, a.err);
            // (a wait that gave up may leave no piece: the block is done then)
            if (*abort_flag) break;
            const Piece p = slots[pieces % kSlots];
            const float* weights = row_weights[kGated ? pieces % kSlots : 0];
            const bool has = warp < tile_slabs(a.m, p.tile);
            const int slab = p.tile * kSlabs + warp;
            const int columns = kN == 16 ? 16 : ceil_div(p.rows, 16) * 16;
            float sums[kN];
#pragma unroll
            for (int n = 0; n < kN; ++n) sums[n] = 0.0f;
            float scale[kGroups], old[kGroups];  // the chunk's, the one's before
            // adds `by` times the sums at column `at` of the groups' sums
            const auto drain = [&](uint32_t at, float by) {
                constexpr int kPer = kN < 64 ? 16 : 32;  // read side by side
#pragma unroll
                for (int n0 = 0; n0 < kN; n0 += kPer) {
                    if (n0 >= columns) break;
                    uint32_t v[kPer / 16][16];
#pragma unroll
                    for (int j = 0; j < kPer / 16; ++j)
                        if (n0 + j * 16 < columns)
                            tmem_ld16(sums_at + at + n0 + j * 16, v[j]);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < kPer; ++j)
                        if (n0 + j / 16 * 16 < columns)
                            sums[n0 + j] = fmaf(by, __uint_as_float(v[j / 16][j % 16]), sums[n0 + j]);
                }
            };
            // the sums that half h of chunk number i has ended, s the chunk's scales
            const auto drain_half = [&](int i, int h, const float (&s)[kGroups]) {
                if constexpr (kGroup == 32) {
                    drain(h * 2 * kN, s[h * 2]);
                    drain(h * 2 * kN + kN, s[h * 2 + 1]);
                } else if constexpr (kGroup == 64) {
                    drain(h * kN, s[h]);
                } else {
                    if (h == 1) drain((i & 1) * kN, s[0]);
                }
            };
            for (int c = p.chunk0; c < p.chunk1; ++c, ++it) {
                wait_warp(smem_u32(&full[slot]), phase, abort_flag, a.err);
                const uint32_t rec = rec0 + (uint32_t)(slot * F::kWeightBytes);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // 32 weights of a row at a time
                    uint32_t x[16];
                    const auto widen_piece = [&](int piece) {
                        const uint4 v = ld_shared4(rec + (h * 2 + piece) * 512);
                        widen(v.x, x);
                        widen(v.y, x + 4);
                        widen(v.z, x + 8);
                        widen(v.w, x + 12);
                    };
                    widen_piece(0);
                    if (h == 0) {
#pragma unroll
                        for (int g = 0; g < kGroups; ++g) old[g] = scale[g];
                        load_scales(rec_scales + (uint32_t)(slot * F::kWeightBytes), scale);
                    }
                    // the buffer's MMAs of the chunk before
                    wait_warp(smem_u32(&mma_done[h]), (uint32_t)(it - 1) & 1u, abort_flag, a.err);
                    tc_fence_after();
                    tmem_st16(a_at + (uint32_t)(h * 32), x);
                    widen_piece(1);
                    tmem_st16(a_at + (uint32_t)(h * 32 + 16), x);
                    // this half's MMAs write where the sums of two halves ago are; with groups
                    // of 128, where those of two chunks ago were
                    if (kGroup < 128 && c > p.chunk0) drain_half(it - 1, h, old);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_u32(&a_ready[h]));
                        if (h == 1) mbar_arrive(smem_u32(&empty[slot]));
                    }
                    if (kGroup == 128 && c > p.chunk0) drain_half(it - 1, h, old);
                }
                if (++slot == kStages) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                wait_warp(smem_u32(&mma_done[h]), (uint32_t)(it - 1) & 1u, abort_flag, a.err);
                tc_fence_after();
                drain_half(it - 1, h, scale);
            }
            tc_fence_before();
            u += p.chunk1 - p.chunk0;
            if (!has) continue;
            if (p.after < 0) {
                write_out<kN, kGated>(a, p, slab, sums, weights);
                continue;
            }
            // this warp's slab is shared with the same warp of other blocks
            constexpr long long kSlot = (long long)kConsumers * kN;
            const auto slot_of = [&](int b) {
                return a.parts + ((long long)b * 2 + (b == p.owner ? p.owner_slot : 0)) * kSlot +
                       threadIdx.x;
            };
            float* to = slot_of(block);
#pragma unroll
            for (int n = 0; n < kN; ++n)
                if (n < p.rows) __stcg(to + n * kConsumers, sums[n]);
            __syncwarp();
            int arrived = 0;
            if (lane == 0) {
                // one lane's fences stand for the warp's accesses before and after them
                int* counter = a.counters + p.owner * kSlabs + warp;
                __threadfence();
                arrived = atomicAdd(counter, 1);
                if (arrived == p.after - p.owner) *counter = 0;  // for the next call
                __threadfence();
            }
            arrived = __shfl_sync(0xffffffffu, arrived, 0);
            if (arrived != p.after - p.owner) continue;
#pragma unroll
            for (int n = 0; n < kN; ++n) sums[n] = 0.0f;
            for (int b = p.owner; b <= p.after; ++b) {
                const float* from = slot_of(b);
#pragma unroll
                for (int n = 0; n < kN; ++n)
                    if (n < p.rows) sums[n] += __ldcg(from + n * kConsumers);
            }
            write_out<kN, kGated>(a, p, slab, sums, weights);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kSlabs) {
        tc_fence_after();
        tmem_dealloc(tmem, F::kTmem);
    }
}

// ---- quantising and packing -----------------------------------------------------------------

constexpr int kBlock = 256;

// scale = bf16(max |w| / 7) of a group, q = the nearest of w / scale + 8 in 0..15 (ties to
// even); a group of zeros has scale 0 and q 8.  8 weights a thread.
__global__ void __launch_bounds__(kBlock)
    w4_quantize_kernel(const uint4* w, long long vecs, int group, uint32_t* q, uint16_t* scales) {
    after_previous();
    const long long i = (long long)blockIdx.x * kBlock + threadIdx.x;
    const bool live = i < vecs;
    float f[8];
    float most = 0.0f;
    const uint4 v = live ? w[i] : make_uint4(0, 0, 0, 0);
    const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(words[j] << 16);
        f[2 * j + 1] = __uint_as_float(words[j] & 0xffff0000u);
        most = fmaxf(most, fmaxf(fabsf(f[2 * j]), fabsf(f[2 * j + 1])));
    }
    const int lanes = group / 8;  // 4, 8 or 16 threads a group
    for (int o = lanes / 2; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    const __nv_bfloat16 s = __float2bfloat16_rn(__fdiv_rn(most, 7.0f));
    const float scale = __bfloat162float(s);
    uint32_t out = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float x = scale > 0.0f ? rintf(__fdiv_rn(f[j], scale)) + 8.0f : 8.0f;
        out |= (uint32_t)fminf(fmaxf(x, 0.0f), 15.0f) << (4 * j);
    }
    if (!live) return;
    q[i] = out;
    if (i % lanes == 0) scales[i / lanes] = *reinterpret_cast<const uint16_t*>(&s);
}

// Once for each set of weights, so neither of these is made fast: w4_quantize_kernel reads and
// writes 2.3 TB/s, this one 0.4 TB/s (single bytes of rows); 256 matrices of 4096 x 7168 take 8.3
// and 19 ms.
// 16 bytes of the packed form a thread: 32 weights of a row (bytes' nibbles r and r + 4 of a
// word are neighbours), or 8 scales.  Rows and columns
// that the matrix does not have are weights of zero (nibble 8, scale 0).
__global__ void __launch_bounds__(kBlock)
    w4_pack_kernel(const uint8_t* q, const uint16_t* scales, Matrix m, long long pieces,
                   uint4* packed) {
    after_previous();
    const int record = m.record / 16, nibble_pieces = kNibbleBytes / 16;
    const int groups = m.C_in / m.group, all_rows = m.rows * (m.gated ? 2 : 1);
    const long long per_expert = (long long)m.slabs * m.chunks * record;
    for (long long i = (long long)blockIdx.x * kBlock + threadIdx.x; i < pieces;
         i += (long long)gridDim.x * kBlock) {
        const long long e = i / per_expert;
        const long long in = i - e * per_expert;
        const long long slab_chunk = in / record;
        const int at = (int)(in - slab_chunk * record);
        const int tile = (int)(slab_chunk / ((long long)kSlabs * m.chunks));
        const int rest = (int)(slab_chunk - (long long)tile * kSlabs * m.chunks);
        const int slabs = tile_slabs(m, tile);
        const int chunk = rest / slabs, slab = tile * kSlabs + rest % slabs;
        uint32_t o[4] = {};
        bool up;
        if (at < nibble_pieces) {
            const int r = matrix_row(m, slab, at & 31, &up);
            const uint8_t* from = q + ((e * all_rows + (up ? m.rows : 0) + r) * (long long)m.C_in) / 2;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int k = chunk * kChunk + (at >> 5) * 32 + w * 8 + j;
                    uint32_t v = 8;
                    if (r >= 0 && k < m.C_in) v = (uint32_t)(from[k >> 1] >> (k % 2 * 4)) & 15u;
                    o[w] |= v << (4 * (j / 2 + 4 * (j % 2)));
                }
            }
        } else {
            const int per_row = kChunk / m.group, first = (at - nibble_pieces) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int r = matrix_row(m, slab, (first + j) / per_row, &up);
                const int grp = chunk * per_row + (first + j) % per_row;
                uint32_t v = 0;
                if (r >= 0 && grp < groups)
                    v = scales[(e * all_rows + (up ? m.rows : 0) + r) * (long long)groups + grp];
                o[j / 2] |= v << (j % 2 * 16);
            }
        }
        packed[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// ---- host -----------------------------------------------------------------------------------

// Rows of a pass, by the experts' average: 16 take the least time for a chunk, and an expert with
// more of them than a pass has its weights widened once for each.  So the changes lie where many
// experts come to need a second pass: at the pass's own size where all have the same rows, before it
// where rows are drawn at random, and later (with less between the two) where some experts have
// several times the rows of others.  32 experts of 4096 x 2816, groups of 128, us in a graph with
// 16 and with 32 rows a pass:
//   rows an expert      8         12         14         16         20         24
//   all the same     56, 56     56, 58     56, 58     58, 58     89, 60     89, 62
//   at random        56, 56     58, 58     64, 59     72, 60     80, 61     89, 62
//   uneven           58, 58     64, 58     65, 59     70, 62     76, 64     87, 67
// and with 32 and with 64:
//   rows an expert     28         32         36         40         44         48
//   all the same     62, 72     64, 72     95, 78     95, 78     97, 80     95, 80
//   at random        68, 76     76, 78     89, 78     93, 80     96, 82     97, 82
//   uneven           72, 83     76, 87     81, 89     85, 91     89, 91     97, 93
// (uneven: shares of 1 / sqrt(i)).  8 of 14336 x 4096 and 64 of 2048 x 2 x 1408, gated: alike.
int pass_rows(long long R, int E) {
    const long long used = R < E ? R : E;
    const double mean = used > 0 ? (double)R / (double)used : 0.0;
    return mean <= 12.0 ? 16 : mean <= 33.0 ? 32 : 64;
}

struct W4Work {
    size_t counters, parts, total;
};
W4Work w4_work(const moe_shape& s) {
    W4Work w;
    w.counters = workspace_layout(s).total;
    w.parts = w.counters + align256(kMaxBlocks * kSlabs * sizeof(int));
    w.total = w.parts + (size_t)kMaxBlocks * 2 * kConsumers * sizeof(float) *
                            pass_rows((long long)s.N * s.k, s.E);
    return w;
}

bool valid(const moe_w4_matrix* m) {
    return m && m->C_out > 0 && m->C_in > 0 &&
           (m->group == 32 || m->group == 64 || m->group == 128);
}
// Rows and columns, with what the last slab and chunk add to them and a gated matrix's two halves
// as one, are 32 bits.
constexpr int kMaxSide = 1 << 28;
bool supported(const moe_w4_matrix* m) {
    return m->C_out % 8 == 0 && m->C_in % m->group == 0 && m->C_out <= kMaxSide &&
           m->C_in <= kMaxSide;
}

long long expert_bytes(const Matrix& d) { return (long long)d.slabs * d.chunks * d.record; }
// 0: more than any memory has (and, from there on, more than 64 bits).
long long packed_bytes(const moe_w4_matrix& m, int E) {
    const long long one = expert_bytes(matrix_of(m));
    return one > (1LL << 50) / E ? 0 : E * one;
}

template <int kN, int kGroup, bool kGated>
moe_status launch_as(const CUtensorMap& rows, const Args& a, long long used, cudaStream_t st) {
    using F = Form<kN, kGroup>;
    const auto kernel = w4_kernel<kN, kGroup, kGated>;
    static OncePerDevice set;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    if (!set.done(dev)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)F::smem(kMaxE)) != cudaSuccess)
            return MOE_ERR_CUDA;
        set.finish(dev);
    }
    const long long units = (used + (a.R - used) / kN) * a.m.tiles * a.m.chunks;
    long long blocks = (long long)sm_count() * F::kBlocks;
    if (blocks > kMaxBlocks) blocks = kMaxBlocks;
    if (blocks > units) blocks = units;
    return cuda_status(launch_chained(kernel, (int)blocks, kThreads, F::smem(a.E), st, rows, a));
}

// Groups of 32 in passes of 64 rows would take all of TMEM for one block: 32 rows, two blocks.
template <int kGroup, bool kGated>
moe_status launch_rows_of(int pass, const CUtensorMap& rows, const Args& a, long long used,
                          cudaStream_t st) {
    if (pass == 16) return launch_as<16, kGroup, kGated>(rows, a, used, st);
    if (pass == 32 || kGroup == 32) return launch_as<32, kGroup, kGated>(rows, a, used, st);
    return launch_as<kGroup == 32 ? 32 : 64, kGroup, kGated>(rows, a, used, st);
}

template <bool kGated>
moe_status launch_w4(int pass, const CUtensorMap& rows, const Args& a, long long used,
                     cudaStream_t st) {
    return a.m.group == 32   ? launch_rows_of<32, kGated>(pass, rows, a, used, st)
           : a.m.group == 64 ? launch_rows_of<64, kGated>(pass, rows, a, used, st)
                             : launch_rows_of<128, kGated>(pass, rows, a, used, st);
}

moe_status w4_product(const uint16_t* rows, const moe_layout* layout, const moe_shape* shape,
                      const moe_w4_matrix* matrix, const void* packed, bool gated,
                      const float* topk_w, void* out, bool out_f32, void* ws, size_t ws_bytes,
                      void* stream) {
    MOE_TRY(check_shape(shape));
    MOE_TRY(check_layout(layout, shape));
    if (!valid(matrix) || (matrix->gated != 0) != gated) return MOE_ERR_INVALID_ARG;
    if (!supported(matrix)) return MOE_ERR_UNSUPPORTED;
    const W4Work work = w4_work(*shape);
    if (!ws || ws_bytes < work.total) return MOE_ERR_WORKSPACE;
    if (!aligned16(ws)) return MOE_ERR_INVALID_ARG;
    const long long R = (long long)shape->N * shape->k;
    if (R > INT32_MAX - (1 << 20) || packed_bytes(*matrix, shape->E) == 0)
        return MOE_ERR_UNSUPPORTED;
    if (R == 0) return MOE_OK;
    if (!rows || !packed || !out || !aligned16(rows, packed, out)) return MOE_ERR_INVALID_ARG;
    const GemmGroup g = routed_group(*layout, *shape, ws);
    Args a = {};
    a.packed = static_cast<const uint8_t*>(packed);
    a.m = matrix_of(*matrix);
    a.expert_bytes = expert_bytes(a.m);
    a.gate = Gate{topk_w,  layout->row_token, layout->pair_row, shape->N, shape->k,
                  gated ? static_cast<uint16_t*>(out) : nullptr, nullptr, nullptr, nullptr};
    a.out = out;
    a.out_f32 = out_f32;
    a.offsets = g.offsets;
    a.counts = g.counts;
    a.E = g.E;
    a.R = (int)R;
    a.parts = ws_ptr<float>(ws, work.parts);
    a.counters = ws_ptr<int>(ws, work.counters);
    a.err = g.err;
    CUtensorMap map;
    const uint64_t sizes[2] = {(uint64_t)matrix->C_in, (uint64_t)R};
    const uint64_t strides[1] = {(uint64_t)matrix->C_in * 2};
    const uint32_t box[2] = {64, 8};
    if (!map_tiled(&map, 2, rows, sizes, strides, box)) return MOE_ERR_UNSUPPORTED;
    const long long used = R < g.E ? R : g.E;  // experts with rows, at most
    const int pass = pass_rows(R, g.E);
    return gated ? launch_w4<true>(pass, map, a, used, as_stream(stream))
                 : launch_w4<false>(pass, map, a, used, as_stream(stream));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_w4_packed_bytes(const moe_w4_matrix* matrix, int32_t E) {
    if (!valid(matrix) || !supported(matrix) || E <= 0 || E > kMaxE) return 0;
    return (size_t)packed_bytes(*matrix, E);
}

size_t moe_w4_workspace_bytes(const moe_shape* shape) {
    return check_shape(shape) == MOE_OK ? w4_work(*shape).total : 0;
}

moe_status moe_w4_quantize(const uint16_t* w, int64_t rows, int32_t C_in, int32_t group, uint8_t* q,
                           uint16_t* scales, void* stream) {
    MOE_RANGE();
    if (rows < 0 || C_in <= 0 || (group != 32 && group != 64 && group != 128))
        return MOE_ERR_INVALID_ARG;
    if (C_in % group != 0 || rows > (1LL << 40) / C_in) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    if (!w || !q || !scales || !aligned16(w, q, scales)) return MOE_ERR_INVALID_ARG;
    const long long vecs = rows * C_in / 8;
    return cuda_status(launch_chained(w4_quantize_kernel, (unsigned)((vecs + kBlock - 1) / kBlock),
                                      kBlock, 0, as_stream(stream),
                                      reinterpret_cast<const uint4*>(w), vecs, group,
                                      reinterpret_cast<uint32_t*>(q), scales));
}

moe_status moe_w4_pack(const uint8_t* q, const uint16_t* scales, const moe_w4_matrix* matrix,
                       int32_t E, void* packed, void* stream) {
    MOE_RANGE();
    if (!valid(matrix) || E <= 0) return MOE_ERR_INVALID_ARG;
    if (!supported(matrix) || E > kMaxE) return MOE_ERR_UNSUPPORTED;
    const long long pieces = packed_bytes(*matrix, E) / 16;
    if (pieces == 0) return MOE_ERR_UNSUPPORTED;
    if (!q || !scales || !packed || !aligned16(q, scales, packed)) return MOE_ERR_INVALID_ARG;
    const long long blocks = (pieces + kBlock - 1) / kBlock, most = 1LL << 20;
    return cuda_status(launch_chained(w4_pack_kernel, (int)(blocks < most ? blocks : most), kBlock,
                                      0, as_stream(stream), q, scales, matrix_of(*matrix), pieces,
                                      static_cast<uint4*>(packed)));
}

moe_status moe_w4_gemm(const uint16_t* rows, const moe_layout* layout, const moe_shape* shape,
                       const moe_w4_matrix* matrix, const void* packed, void* out,
                       int32_t out_type, void* ws, size_t ws_bytes, void* stream) {
    MOE_RANGE();
    if (out_type != MOE_TYPE_BF16 && out_type != MOE_TYPE_F32) return MOE_ERR_INVALID_ARG;
    return w4_product(rows, layout, shape, matrix, packed, false, nullptr, out,
                      out_type == MOE_TYPE_F32, ws, ws_bytes, stream);
}

moe_status moe_w4_gated_gemm(const uint16_t* rows, const moe_layout* layout,
                             const moe_shape* shape, const moe_w4_matrix* matrix,
                             const void* packed, const float* topk_w, uint16_t* h, void* ws,
                             size_t ws_bytes, void* stream) {
    MOE_RANGE();
    return w4_product(rows, layout, shape, matrix, packed, true, topk_w, h, false, ws, ws_bytes,
                      stream);
}

}  // extern "C"
