// Matrix products grouped by expert over ragged row segments, and their
// gradients (tcgen05 cta_group::2).  With the rows of expert e a segment of R
// expert-major rows and W[e] its [C_out, C_in] matrix:
//
//   forward          out[i, :]   = rows[i, :] W[e]^T          contracts C_in
//   rows' gradient   drows[i, :] = dout[i, :] W[e]            contracts C_out
//   weights' grad.   dW[e]       = sum_{i in e} dout[i, :]^T rows[i, :]
//                                                             contracts the rows
//
// One persistent kernel on 256 x 256 output tiles that a CTA pair shares.  All
// operands stay in their row-major layout: where a contraction runs along the
// rows of a matrix (W in the rows' gradient, both operands in the weights'
// gradient) TMA brings boxes of 64 columns x 64 rows and the matrix and
// instruction descriptors name the operand MN-major, so nothing is transposed
// or copied.  Where the matrix has whole groups of 64 columns its map has them as a
// dimension and one copy brings both boxes of an operand.
//
// The contraction of a weights' gradient ends inside a 64-row block where the
// expert's segment ends.  The MMA stops at the next 16 rows, and the rows
// between the segment's end and there (the next expert's, or anything past the
// last) are zeroed in shared memory by a warp of its own before the MMA may
// read the block: for that block the copies complete on a barrier of their
// CTA, and each CTA's warp arrives on the leader's full barrier in the
// producer's place.  Both operands are zeroed, so no value of a neighbouring
// segment, NaN included, reaches a product.  An expert with no rows gets zeros.
//
// Precision: the tensor core adds into its fp32 accumulator with truncation,
// which over a contraction of 4096 random bf16 products is a relative error of
// 4e-6 (measured; 1e-6 over 1024, 2e-7 over 256; grows with the length), all of it
// towards zero; of terms of one sign it is 1.4e-9 a term (4.4e-5 over 32768, 1.2e-2
// over 8 million).  So an accumulator takes at most kChainBlocks k-blocks, and those
// partial sums are added in fp32 registers, rounding to nearest, in a fixed order.
// fp32 outputs: 512 terms, 4e-7 whatever the length, for 6 to 11% of the time of a long
// contraction.  bf16 outputs: 32768 terms, which lose a hundredth of the output's own
// rounding (2^-8); a shorter contraction is one chain.  262144 skewed rows' weights'
// gradient with the code for it: 2064 us, without 2050.
//
// Roles per CTA (384 threads): warp 0 loads by TMA into 6 stages (9 in tiles of few rows);
// warp 1 owns TMEM (two accumulators, one filled while the other is drained) and, in the
// leader, issues the MMAs; warp 2 of the leader hands out tiles; warp 3 zeroes block ends
// (weights' gradient) or looks up rows' weights (a gate's gradient); warps 4-11 drain the accumulators, two warps to each 32 rows
// (128 columns each), with the registers that the others give up.  Every wait is
// bounded.  6 stages of 32 KB and 32 KB of outgoing lines fill the shared memory; 5 and
// 4 stages measured slower.
//
// What bounds it, and what that led to (GB300, clock cycles of an SM):
// - Long contractions run at the tensor cores' rate: 16384 x 14336 x 4096, 1021 us
//   (1885 TFLOP/s) at 2070 MHz, 1165 to 1219 us once the power cap lowers the clock
//   (cuBLAS's own rate falls from 1936 to 1715 TFLOP/s).  That takes an issuing lane that is done with a k-block (4 MMAs, a
//   commit, a wait) before the MMAs are: see the election below.
// - With few rows an expert the weights' gradient is the writing of dW.  A tile's
//   128 KB (fp32) have to leave an SM in some 5000 cycles, which takes whole 128-byte
//   lines (64-byte boxes: 22 bytes a cycle, 128-byte ones 26), by TMA (lines stored
//   by the warps: 18), and a drain with nothing in its way: an arrival at the other
//   CTA's barrier with cluster-scope release waits for every store in flight, 2000
//   to 5000 cycles a tile, so none of them is on that path; the block-end warp's
//   releases shared memory alone.  64 experts x 384 rows, 2816 x 2048, fp32: 370 us
//   with those fences and 64-byte lines, 288 us now (298 to 309 under the power cap);
//   floor 253 us.
// - A tile costs each role some 800 cycles to decode: the scheduler does it for all.
// - A decoding step streams the weights: 16 tokens of 6 of 64 experts of 2816 x 2048,
//   88 us for 586 MB, 6.7 TB/s, with the matrix as A and 64 rows as B (kFew); 97 us with
//   256 rows as A, whose MMAs take longer than the weights.
// - Few tiles leave SMs idle: with a long contraction 2 or 4 pairs of a cluster share
//   a tile's k-blocks, keep their sums in shared memory and add them up from there
//   (4096 rows of one expert, 256 x 256 fp32 weights' gradient: 29 us with one pair,
//   19 us with four; 1 row, 14336 x 3528 in tiles of few rows: 24 us with four
//   a call, 21.7 us in a graph).
// - 64 tokens of 8 experts, 128 to 512: 5.2 us, of
//   them 1.1 the experts' counts and the first tile, 0.4 the meeting of the CTAs, 0.9
//   loads, 0.6 MMAs, 0.5 stores, 0.7 the end.
#include <stddef.h>

#include "../../include/moe_train.h"
#include "api_checks.cuh"
#include "gate.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

// kGated, kGatedGrad: the products before and behind an expert's gate, with the gate (or its
// gradient) in their epilogue.  A tile of kGated is 128 gate columns and the same up columns.
enum Mode { kForward, kRowsGrad, kWeightsGrad, kGated, kGatedGrad };

constexpr int BT = 256;    // rows and columns of a pair's tile
constexpr int BH = 128;    // rows of A and of B that a CTA of the pair holds
constexpr int BK = 64;
constexpr int UMMA_K = 16;
constexpr int kAccs = 2;
constexpr int kTmemCols = BT * kAccs;
constexpr int OP_BYTES = BH * BK * 2;   // one operand of one stage in one CTA
constexpr int BOX_BYTES = OP_BYTES / 2;  // an MN-major box: 64 columns x 64 rows
constexpr int kThreads = 384;
constexpr int kEpilogueWarps = 8;
constexpr int kEpilogueCols = BT / 2;  // columns of one epilogue warp
// Registers a thread: 384 x 168 at launch = 128 x 88 + 256 x 208, or 128 x 56 + 256 x 224
// where an epilogue thread keeps 128 sums beside what it does with them.
template <int kMode>
constexpr int kRegsOther = kMode == kGatedGrad ? 56 : 88;
template <int kMode>
constexpr int kRegsEpilogue = kMode == kGatedGrad ? 224 : 208;
// A tile of few rows: their number, which is the MMA's N (see kFew).
constexpr int BF = 64;
constexpr int FEW_BYTES = BF / 2 * BK * 2;  // that operand of one stage in one CTA
template <bool kFew>
constexpr int kStageBytes = kFew ? OP_BYTES + FEW_BYTES : 2 * OP_BYTES;
template <int kMode, bool kFew>
constexpr int kStagesOf = kFew ? 9 : kMode == kGatedGrad ? 5 : 6;
constexpr int kAhead = 2;  // tiles the scheduler publishes ahead of the leader's producer
constexpr int kStagingBytes = 32 * 128;  // an epilogue warp's output: 32 lines
// kGatedGrad: 32 half lines of gate columns and 32 of up columns come in there and go out again,
// twice: the next ones come in while these are worked on
template <int kMode>
constexpr int kStagingOf = (kMode == kGatedGrad ? 2 : 1) * kStagingBytes;
// k-blocks added up in one accumulator, see "Precision" above
template <typename OutT>
constexpr int kChainBlocks = sizeof(OutT) == 4 ? 8 : 512;

// A tile: its expert (-1: no more tiles) and the expert's rows, its row and column
// block, and the k-blocks of its contraction.  Decoded once by the scheduler and
// handed to the other roles through the tile queues: the divisions and the search
// for the expert would cost each role some 800 cycles a tile.
struct __align__(16) Tile {
    int e, off, cnt, kblocks;
    int mb, nb;
    // a split contraction: this pair's first k-block of rows' products (a weights'
    // gradient's off and cnt are its own rows), and the expert's rows
    int k0, all;
};
constexpr int kQ = 6;  // slots of a tile queue
// Rows an expert, on average, up to which products take tiles of few rows: 128 rows each
// of 64 experts of 2816 x 2048 take 134 us in two of those and 136 us in one of 256 rows,
// 256 rows 209 and 146 us.
constexpr int kFewRows = 64;
constexpr int kMaxSplits = 4;    // pairs of a cluster that share a tile's contraction

struct Queues {
    Tile first;                 // each CTA: the pair's first tile, decoded by both CTAs
    Tile queue[kQ];             // each CTA: the ones after it, from the leader's scheduler
    Tile local[kQ];             // peer: the tiles its producer forwards to its other warps
    uint64_t tfull[kAccs];      // each CTA: accumulator ready
    uint64_t tempty[kAccs];     // leader: accumulator drained by both CTAs
    uint64_t done;              // leader: every issued MMA retired
    uint64_t q_full[kQ];        // each CTA: slot of queue written
    uint64_t q_empty[kQ];       // leader: slot read by every reader of both CTAs
    uint64_t q_taken[kQ];       // leader: its producer has taken the slot's tile
    uint64_t l_full[kQ];        // peer: slot of local written
    uint64_t l_empty[kQ];       // peer: slot of local read by its warps
    uint32_t tmem_base;
    int abort;
    int only;                   // no pair has more than its first tile
};
constexpr int kQueueBarriers = 2 * kAccs + 1 + 5 * kQ;
static_assert(offsetof(Queues, tmem_base) - offsetof(Queues, tfull) ==
                  kQueueBarriers * sizeof(uint64_t),
              "the queues' barriers lie side by side");
template <int kStages>
struct Barriers : Queues {
    uint64_t full[kStages];     // leader: both CTAs' operands of a stage are there
    uint64_t empty[kStages];    // each CTA: its stage may be refilled
    uint64_t land[kStages];     // each CTA: its copies of a segment's last block are there
};
template <int kMode, bool kFew>
struct Ctl : Barriers<kStagesOf<kMode, kFew>> {};
constexpr int kGateCols = 32;             // kGatedGrad: columns of a half line of 64 bytes
constexpr int kHalfLines = 32 * kGateCols * 2;  // bytes of 32 rows' half lines
constexpr int kGradChain = kChainBlocks<float>; // its k-blocks of an accumulator
constexpr int kMaxSorted = 512;  // what is left of shared memory holds
template <>
struct Ctl<kWeightsGrad, false> : Barriers<kStagesOf<kWeightsGrad, false>> {
    uint16_t order[kMaxSorted];  // experts by falling number of rows
};
template <>
struct Ctl<kGatedGrad, false> : Barriers<kStagesOf<kGatedGrad, false>> {
    uint64_t lines[kEpilogueWarps];  // each CTA: a warp's half lines have come in
    uint64_t w_full[2], w_empty[2];  // each CTA: its rows' weights are there, have been read
    float weights[2][BH];            // of two tiles in turn
};
template <int kMode, bool kFew>
constexpr size_t smem_bytes() {
    constexpr size_t n = 1024 + (size_t)kStagesOf<kMode, kFew> * kStageBytes<kFew> +
                         (size_t)kEpilogueWarps * kStagingOf<kMode> +
                         ((sizeof(Ctl<kMode, kFew>) + 15) & ~size_t(15));
    static_assert(n <= 227 * 1024, "shared memory of one block");
    return n;
}

// Blocks of `size` that n takes: widths go up to 2^31 - 8, where n + size - 1 is no int.
__host__ __device__ __forceinline__ int blocks_of(int n, int size) {
    return (int)(((unsigned)n + (unsigned)size - 1u) / (unsigned)size);
}

// Limit of a wait that lasts as long as a tile's contraction does: a k-block takes some 500
// cycles, so 4 million of them are past kWaitLimit by themselves.
__device__ __forceinline__ long long tile_limit(int kblocks) {
    return kWaitLimit + 2048LL * kblocks;
}

// Spin for about `cycles` SM clocks (lets copies in flight land on abort).
__device__ __forceinline__ void spin(long long cycles) {
    const long long t0 = clock64();
    while (clock64() - t0 < cycles) {
    }
}

__device__ __forceinline__ Tile read_slot(const Tile* p) {
    const volatile int* q = reinterpret_cast<const volatile int*>(p);
    Tile t;
    t.e = q[0];
    t.off = q[1];
    t.cnt = q[2];
    t.kblocks = q[3];
    t.mb = q[4];
    t.nb = q[5];
    t.k0 = q[6];
    t.all = q[7];
    return t;
}

// The first tile of a pair does not go through the queue: where it is the only one, as
// in most short calls, no role waits for another's decoding or for an end.
// One thread takes tile i of the queue; false when there is none or the wait gave up.
// first: the cluster's rank of the pair's leader, here and below.
// In the leader every role reads the leader's queue.  In the peer only its producer
// does and forwards each tile through the local queue, so that a tile crosses between
// the CTAs once each way.
__device__ __forceinline__ bool take(Queues* c, int i, bool leader, uint32_t first,
                                     volatile int* abort, int* err, Tile& t) {
    const int slot = i % kQ;
    const uint32_t ph = (uint32_t)(i / kQ) & 1u, full = smem_u32(&c->q_full[slot]);
    if (!(leader ? wait_bar(full, ph, abort, err) : wait_bar_cluster(full, ph, abort, err)))
        return false;
    t = read_slot(&c->queue[slot]);
    const uint32_t empty = smem_u32(&c->q_empty[slot]);
    if (leader)
        mbar_arrive(empty);
    else
        mbar_arrive_remote(mapa_shared(empty, first));
    return t.e >= 0;
}
__device__ __forceinline__ bool take_local(Queues* c, int i, volatile int* abort, int* err,
                                           Tile& t) {
    const int slot = i % kQ;
    const uint32_t ph = (uint32_t)(i / kQ) & 1u;
    if (!wait_bar(smem_u32(&c->l_full[slot]), ph, abort, err)) return false;
    t = read_slot(&c->local[slot]);
    mbar_arrive(smem_u32(&c->l_empty[slot]));
    return t.e >= 0;
}
// Peer's producer: tile i (or its end) on to the peer's other warps.
__device__ __forceinline__ bool forward(Queues* c, int i, const Tile& t, volatile int* abort,
                                        int* err) {
    const int slot = i % kQ;
    const uint32_t ph = (uint32_t)(i / kQ) & 1u;
    if (!wait_bar(smem_u32(&c->l_empty[slot]), ph ^ 1u, abort, err)) return false;
    c->local[slot] = t;
    mbar_arrive(smem_u32(&c->l_full[slot]));
    return true;
}
// Leader's scheduler: tile i (or the end) into both CTAs' queues.
__device__ __forceinline__ bool publish(Queues* c, int i, const Tile& t, uint32_t first,
                                        volatile int* abort, int* err) {
    const int slot = i % kQ;
    const uint32_t ph = (uint32_t)(i / kQ) & 1u, full = smem_u32(&c->q_full[slot]);
    if (!wait_bar(smem_u32(&c->q_empty[slot]), ph ^ 1u, abort, err)) return false;
    c->queue[slot] = t;
    mbar_arrive(full);
    const uint32_t bar = mapa_shared(full, first + 1);
    const uint32_t at = mapa_shared(smem_u32(&c->queue[slot]), first + 1);
    mbar_expect_tx_remote(bar, sizeof(Tile));
    st_async4(at, bar, t.e, t.off, t.cnt, t.kblocks);
    st_async4(at + 16, bar, t.mb, t.nb, t.k0, t.all);
    return true;
}
// The columns that the MMAs of the last column block take: where there are 128 at most,
// as few as there are, in steps of what the two CTAs' halves of them can start at (16384 x
// 1408 columns: 410 us with 256 in each, 399 us; 256 experts' 68 rows x 104: 199 and 154
// us).  With more, boxes that overlap cost what the MMAs gain.  The rows of a tile are
// the MMA's M, which is 256.
__host__ __device__ __forceinline__ int last_columns(int n_out, bool groups) {
    const int rest = n_out - (n_out - 1) / BT * BT, step = groups ? 2 * BK : 32;
    return rest > BH ? BT : (rest + step - 1) / step * step;
}
// Of a CTA's half of the columns, those that its boxes of a K-major operand or of groups of
// 64 columns bring in: all of them but where there is one column block.
__host__ __device__ __forceinline__ int box_columns(int n_out, bool groups) {
    return n_out > BT ? BH : last_columns(n_out, groups) / 2;
}

// The n-th tile of a whole warp, or of one thread with the leader's queue.
__device__ __forceinline__ bool warp_next(Queues* c, int n, bool leader, volatile int* abort,
                                          int* err, Tile& t) {
    if (n == 0) {
        t = read_slot(&c->first);
        return t.e >= 0;
    }
    if (c->only) return false;
    int more = 0;
    if ((threadIdx.x & 31) == 0)
        more = leader ? take(c, n - 1, true, 0, abort, err, t)
                      : take_local(c, n - 1, abort, err, t);
    if (!__shfl_sync(0xffffffffu, more, 0)) return false;
    t.e = __shfl_sync(0xffffffffu, t.e, 0);
    t.off = __shfl_sync(0xffffffffu, t.off, 0);
    t.cnt = __shfl_sync(0xffffffffu, t.cnt, 0);
    t.kblocks = __shfl_sync(0xffffffffu, t.kblocks, 0);
    t.mb = __shfl_sync(0xffffffffu, t.mb, 0);
    t.nb = __shfl_sync(0xffffffffu, t.nb, 0);
    return true;
}
__device__ __forceinline__ bool next(Queues* c, int n, uint32_t first, volatile int* abort,
                                     int* err, Tile& t) {
    if (n == 0) {
        t = read_slot(&c->first);
        return t.e >= 0;
    }
    return !c->only && take(c, n - 1, true, first, abort, err, t);
}

// Inclusive prefix sum over a warp.
__device__ __forceinline__ int warp_prefix(int v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Expert e's segment; one that leaves the R rows is reported and taken as empty.
__device__ __forceinline__ void segment(const int32_t* offsets, const int32_t* counts, int e,
                                        int R, int* err, int* off, int* cnt) {
    int o = offsets[e], c = counts[e];
    if (o < 0 || c < 0 || c > R || o > R - c) {
        set_error(err, MOE_ERR_INVALID_ARG);
        o = c = 0;
    }
    *off = o;
    *cnt = c;
}

// 32 or 64 columns of an accumulator.
__device__ __forceinline__ void tmem_ld_line(uint32_t at, uint32_t (&v)[32]) { tmem_ld32(at, v); }
__device__ __forceinline__ void tmem_ld_line(uint32_t at, uint32_t (&v)[64]) {
    tmem_ld32(at, reinterpret_cast<uint32_t(&)[32]>(v[0]));
    tmem_ld32(at + 32, reinterpret_cast<uint32_t(&)[32]>(v[32]));
}

// One row's 128-byte line of fp32 values (rounded to OutT) into shared memory, its
// 16-byte chunks k at k ^ (row & 7): TMA's 128-byte swizzle, and no two of 8 rows'
// stores in the same banks.
template <typename OutT>
__device__ __forceinline__ void put_line(uint8_t* staging, int row,
                                         const uint32_t (&v)[128 / sizeof(OutT)]) {
    constexpr int kChunk = 16 / (int)sizeof(OutT), kLine = kChunk * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = sizeof(OutT) == 4
                       ? v[k * kChunk + j]
                       : pack2(__uint_as_float(v[(k * kChunk + 2 * j) % kLine]),
                               __uint_as_float(v[(k * kChunk + 2 * j + 1) % kLine]));
        *reinterpret_cast<uint4*>(staging + row * 128 + ((k ^ (row & 7)) << 4)) =
            make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// The first `rows` of a warp's 32 lines in shared memory to rows of the output, n_out
// apart, 4 whole lines by each store instruction.  cols: how many the output has from p
// on (a multiple of 8).
template <typename OutT>
__device__ __forceinline__ void store_lines(const uint8_t* staging, OutT* p, int n_out, int rows,
                                            int cols) {
    constexpr int kChunk = 16 / (int)sizeof(OutT);
    const int lane = threadIdx.x & 31, ch = lane & 7;
    for (int r = lane >> 3; r < rows; r += 4) {
        if (ch * kChunk < cols)
            *reinterpret_cast<uint4*>(p + (long long)r * n_out + ch * kChunk) =
                *reinterpret_cast<const uint4*>(staging + r * 128 + ((ch ^ (r & 7)) << 4));
    }
}

// Split contractions: a pair's sums of its tile stay in the two CTAs' operand rings as
// 128 rows of 256 fp32 columns, 16-byte chunks k at k ^ (row & 7) (32 rows' stores of a
// chunk in different banks).
template <int kN>
__device__ __forceinline__ void put_part(uint8_t* ring, int row, int col, const uint32_t (&v)[kN]) {
#pragma unroll
    for (int k = 0; k < kN / 4; ++k)
        *reinterpret_cast<uint4*>(ring + row * (BT * 4) + (((col / 4 + k) ^ (row & 7)) << 4)) =
            make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
}
// Then each pair adds up all pairs' sums, in their order, of a share of the tile's
// columns, its CTAs for their rows, and writes them out (the epilogue warps).  A thread
// has 8 columns at a time of kRows rows, all their loads under way together: another
// CTA's shared memory is some 200 ns away.
template <bool kW, int kSplits, typename OutT>
__device__ __forceinline__ void join_parts(uint32_t ring, uint32_t rank, int split, const Tile& t,
                                           int m_out, int n_out, OutT* out, int accumulate) {
    constexpr int kGroups = BT / kSplits / 8, kRows = 8 / kSplits;
    constexpr int kStep = 32 * kEpilogueWarps / kGroups;  // rows of one load of the warps
    if (kW && accumulate && t.all == 0) return;  // nothing to add
    const int row0 = t.mb * BT + (int)rank * BH, left = (kW ? m_out : t.cnt) - row0;
    const int rows = left < BH ? left : BH;
    const int u = (int)threadIdx.x - 128;
    const int c = split * (BT / kSplits) + u % kGroups * 8, col = t.nb * BT + c;
    if (col >= n_out) return;
    OutT* to = out + ((kW ? (long long)t.e * m_out : (long long)t.off) + row0) * n_out + col;
    uint32_t from[kSplits];
#pragma unroll
    for (int p = 0; p < kSplits; ++p) from[p] = mapa_shared(ring, 2 * p + rank);
    for (int r0 = u / kGroups; r0 < rows; r0 += kRows * kStep) {
        float4 v[kRows][kSplits][2];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * kStep;
            const uint32_t at = (uint32_t)(r * (BT * 4)), ch = (uint32_t)c / 4, sw = r & 7;
            if (r < rows) {
#pragma unroll
                for (int p = 0; p < kSplits; ++p) {
                    v[i][p][0] = ld_cluster4(from[p] + at + ((ch ^ sw) << 4));
                    v[i][p][1] = ld_cluster4(from[p] + at + (((ch + 1) ^ sw) << 4));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * kStep;
            if (r >= rows) break;
#pragma unroll
            for (int p = 1; p < kSplits; ++p) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    v[i][0][h].x += v[i][p][h].x;
                    v[i][0][h].y += v[i][p][h].y;
                    v[i][0][h].z += v[i][p][h].z;
                    v[i][0][h].w += v[i][p][h].w;
                }
            }
            const float4 x = v[i][0][0], y = v[i][0][1];
            if constexpr (sizeof(OutT) == 4) {
                float4* line = reinterpret_cast<float4*>(to + (long long)r * n_out);
                if (accumulate) {
                    const float4 a = line[0], b = line[1];
                    line[0] = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
                    line[1] = make_float4(b.x + y.x, b.y + y.y, b.z + y.z, b.w + y.w);
                } else {
                    line[0] = x;
                    line[1] = y;
                }
            } else {
                *reinterpret_cast<uint4*>(to + (long long)r * n_out) = make_uint4(
                    pack2(x.x, x.y), pack2(x.z, x.w), pack2(y.x, y.y), pack2(y.z, y.w));
            }
        }
    }
}

// Tiles of few rows: a warp's sums are 32 columns of the output (its TMEM lanes) by 32
// rows, and leave by way of 32 lines of 128 bytes in shared memory, one a row.  One with
// its pair's share of the contraction only has its lines in the ring instead.
__device__ __forceinline__ void put_few(uint8_t* lines, int lane, const uint32_t (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 32; ++j) *reinterpret_cast<uint32_t*>(lines + j * 128 + lane * 4) = v[j];
}
template <typename OutT>
__device__ __forceinline__ void store_few(OutT* to, const float4& v) {
    if constexpr (sizeof(OutT) == 4)
        *reinterpret_cast<float4*>(to) = v;
    else
        *reinterpret_cast<uint2*>(to) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
}
// A tile of few rows of a warp: the first of its rows in the outputs, how many of its 32
// there are, its first column.
struct FewPart {
    long long row;
    int rows, col;
};
__device__ __forceinline__ FewPart few_part(const Tile& t, uint32_t rank) {
    const int warp = (int)(threadIdx.x >> 5), at = t.mb * BF + ((warp - 4) >> 2) * 32;
    return {(long long)t.off + at, t.cnt - at, t.nb * BT + (int)rank * BH + (warp & 3) * 32};
}
// The joining of a split one: the pairs take its rows in turn.
template <int kSplits, typename OutT>
__device__ __forceinline__ void join_few(uint32_t ring, uint32_t rank, int split, const Tile& t,
                                         int n_out, OutT* out) {
    const FewPart f = few_part(t, rank);
    const int lane = threadIdx.x & 31, col = f.col + (lane & 7) * 4;
    if (col >= n_out) return;
    const uint32_t at = ring + ((threadIdx.x >> 5) - 4) * kStagingBytes + (lane & 7) * 16;
    for (int r = (lane >> 3) * kSplits + split; r < 32 && r < f.rows; r += 4 * kSplits) {
        float4 v[kSplits];
#pragma unroll
        for (int p = 0; p < kSplits; ++p)
            v[p] = ld_cluster4(mapa_shared(at, 2 * p + rank) + r * 128);
#pragma unroll
        for (int p = 1; p < kSplits; ++p) {
            v[0].x += v[p].x;
            v[0].y += v[p].y;
            v[0].z += v[p].z;
            v[0].w += v[p].w;
        }
        store_few(out + (f.row + r) * n_out + col, v[0]);
    }
}

// ---- the gate in the epilogue ---------------------------------------------------------------
//
// What it saves is gu or dh going out and coming back: 8192 tokens of 2 of 8 experts, 4096 to 2 x
// 14336: 2070 us, product and activation one after the other 2180 + 218; 4099 tokens of 6 of 64,
// 2048 to 2 x 1408: 230, 220 + 37; 16 tokens of these: 91, 91 + 4.3; backwards 4099 tokens: 167,
// 138 + 61; 32768 tokens of 8 of 128 (skewed), 4096 x 1536: 2100, 1840 + 604.  A forward tile of
// 128 gate and 128 up columns costs what one of 256 does: bound by the MMAs where experts have
// many rows (tiles of 256 rows: 384 rows an expert, as in the 4099 tokens, spend those of 512).

// Lines (32 rows x 64 bf16 columns) out: by TMA where all 32 rows are the segment's, else by
// the warp's own stores.  to: the first row's first column, `pitch` apart; cols: how many there
// are from it on.
__device__ __forceinline__ void lines_out(const CUtensorMap* map, const uint8_t* lines, int c0,
                                          int c1, int c2, bool three, uint16_t* to, int pitch,
                                          int rows, int cols) {
    const int lane = threadIdx.x & 31;
    if (rows >= 32) {
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
            if (three)
                tma_store_3d(map, smem_u32(lines), c0, c1, c2);
            else
                tma_store_2d(map, smem_u32(lines), c0, c1);
            bulk_commit();
        }
    } else {
        __syncwarp();
        store_lines<__nv_bfloat16>(lines, reinterpret_cast<__nv_bfloat16*>(to), pitch, rows, cols);
        __syncwarp();
    }
}

// kGated: 32 rows of 64 gate columns at g_at and of their up columns at u_at.  h leaves as
// w SiLU(g) u of the fp32 sums, g and u rounded to bf16 where they are wanted.
template <typename Release>
__device__ __forceinline__ void gated_out(const CUtensorMap& tmGu, const CUtensorMap& tmH,
                                          const Gate& gate, uint8_t* staging, uint32_t g_at,
                                          uint32_t u_at, long long row, int rows, int col, int I,
                                          float w, Release release) {
    const int lane = threadIdx.x & 31;
    uint32_t g[64], u[64];
    tmem_ld_line(g_at, g);
    tmem_ld_line(u_at, u);
    tmem_wait_ld();
    release();
    if (rows <= 0 || col >= I) return;
    const auto put = [&](const uint32_t (&v)[64]) {
        if (lane == 0) bulk_wait_read();  // the lines before have been read
        __syncwarp();
        put_line<__nv_bfloat16>(staging, lane, v);
    };
    if (gate.gu) {
        uint16_t* to = gate.gu + row * 2 * I + col;
        put(g);
        lines_out(&tmGu, staging, col, 0, (int)row, true, to, 2 * I, rows, I - col);
        put(u);
        lines_out(&tmGu, staging, col, 1, (int)row, true, to + I, 2 * I, rows, I - col);
    }
#pragma unroll
    for (int j = 0; j < 64; ++j) {
        const float a = __uint_as_float(g[j]);
        g[j] = __float_as_uint(w * (a * sigmoid(a)) * __uint_as_float(u[j]));
    }
    put(g);
    lines_out(&tmH, staging, col, (int)row, 0, false, gate.h + row * I + col, I, rows, I - col);
}

// kGated in tiles of few rows: a warp has the sums of 32 gate or up columns (its TMEM lanes)
// by 32 rows.  The two warps of the same columns lay them down as lines of a row each, and
// take 16 of the rows each, between their two barriers of 64 threads.
__device__ __forceinline__ void named_sync(int id) {
    asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
}
__device__ __forceinline__ void named_arrive(int id) {
    asm volatile("bar.arrive %0, 64;" ::"r"(id) : "memory");
}
__device__ __forceinline__ int few_barrier(int q, int half) { return 1 + half * 2 + (q & 1); }
// A warp that takes no further tile, at the end or because a wait has given up: the other one may
// still be at these barriers with a tile of before.
__device__ __forceinline__ void gated_few_leave(int q, int half) {
    named_arrive(few_barrier(q, half));
    named_arrive(few_barrier(q, half) + 4);
}
__device__ __forceinline__ void gated_few_out(const Gate& gate, uint8_t* staging_area, int q,
                                              int half, const uint32_t (&v)[32], long long row,
                                              int rows, int col, int I, float w) {
    const int lane = threadIdx.x & 31;
    uint8_t* mine = staging_area + (size_t)(half * 4 + q) * kStagingBytes;
    put_few(mine, lane, v);
    named_sync(few_barrier(q, half));
    const uint8_t* gs = staging_area + (size_t)(half * 4 + (q & 1)) * kStagingBytes;
    const uint8_t* us = gs + 2 * kStagingBytes;
    const int c = (lane & 7) * 4;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const int r = (q >> 1) * 16 + i * 4 + (lane >> 3);
        const float wr = __shfl_sync(0xffffffffu, w, r);
        if (r >= rows || col + c >= I) continue;
        const float4 g = *reinterpret_cast<const float4*>(gs + r * 128 + c * 4);
        const float4 u = *reinterpret_cast<const float4*>(us + r * 128 + c * 4);
        const long long at = (row + r) * I + col + c;
        if (gate.gu) {
            uint16_t* to = gate.gu + at + (row + r) * I;
            *reinterpret_cast<uint2*>(to) = make_uint2(pack2(g.x, g.y), pack2(g.z, g.w));
            *reinterpret_cast<uint2*>(to + I) = make_uint2(pack2(u.x, u.y), pack2(u.z, u.w));
        }
        *reinterpret_cast<uint2*>(gate.h + at) =
            make_uint2(pack2(wr * (g.x * sigmoid(g.x)) * u.x, wr * (g.y * sigmoid(g.y)) * u.y),
                       pack2(wr * (g.z * sigmoid(g.z)) * u.z, wr * (g.w * sigmoid(g.w)) * u.w));
    }
    named_sync(few_barrier(q, half) + 4);
}

// Two fp32 numbers in one instruction.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 f2_get(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// kGatedGrad: dh's 32 columns of a lane's row in v, their g and u in the half lines; dg and du
// take their place.  16-byte chunk k of row r is at k ^ (r / 2 % 4): TMA's 64-byte swizzle.
// Returns this lane's row's sums of dh SiLU(g) u, of the even and the odd columns.
__device__ __forceinline__ F2 gated_grad_lines(uint8_t* lines, const uint32_t (&v)[32], float w) {
    const int lane = threadIdx.x & 31;
    const F2 ww = f2(w, w), one = f2(1.0f, 1.0f), minus = f2(-1.0f, -1.0f);
    F2 sum = f2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint4* g_at = reinterpret_cast<uint4*>(lines + lane * 64 + ((k ^ (lane >> 1 & 3)) << 4));
        uint4* u_at = g_at + kHalfLines / 16;
        const uint4 gv = *g_at, uv = *u_at;
        const uint32_t g[4] = {gv.x, gv.y, gv.z, gv.w}, u[4] = {uv.x, uv.y, uv.z, uv.w};
        uint32_t dg[4], du[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float g0 = __uint_as_float(g[j] << 16), g1 = __uint_as_float(g[j] & 0xffff0000u);
            const F2 gg = f2(g0, g1);
            const F2 uu = f2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u));
            const F2 x = f2(__uint_as_float(v[k * 8 + 2 * j]), __uint_as_float(v[k * 8 + 2 * j + 1]));
            const F2 s = f2(sigmoid(g0), sigmoid(g1));
            const F2 act = f2_mul(gg, s), y = f2_mul(ww, x);
            sum = f2_fma(f2_mul(x, act), uu, sum);
            // s (1 + g (1 - s)) = s + act (1 - s)
            const F2 slope = f2_fma(act, f2_fma(s, minus, one), s);
            const float2 a = f2_get(f2_mul(f2_mul(y, uu), slope)), b = f2_get(f2_mul(y, act));
            dg[j] = pack2(a.x, a.y);
            du[j] = pack2(b.x, b.y);
        }
        *g_at = make_uint4(dg[0], dg[1], dg[2], dg[3]);
        *u_at = make_uint4(du[0], du[1], du[2], du[3]);
    }
    return sum;
}
// The first `rows` of 32 half lines to rows of gu's gradient, `pitch` apart; cols: how many
// columns there are from `to` on.
__device__ __forceinline__ void store_half_lines(const uint8_t* lines, uint16_t* to, int pitch,
                                                 int rows, int cols) {
    const int lane = threadIdx.x & 31, k = lane & 3;
    for (int r = lane >> 2; r < rows; r += 8)
        if (k * 8 < cols)
            *reinterpret_cast<uint4*>(to + (long long)r * pitch + k * 8) =
                *reinterpret_cast<const uint4*>(lines + r * 64 + ((k ^ (r >> 1 & 3)) << 4));
}

// One warp's part of a tile of kGatedGrad: its 32 rows (of which the segment has `rows`), from
// column `col` on `have` half lines of 32 columns.
struct GradPart {
    long long row;
    int rows, col, have;
};
__device__ __forceinline__ GradPart grad_part(const Tile& t, uint32_t rank, int n_out) {
    const int warp = (int)(threadIdx.x >> 5), half = (warp - 4) >> 2;
    GradPart p;
    const int at = t.mb * BT + (int)rank * BH + (warp & 3) * 32;
    p.row = (long long)t.off + at;
    p.rows = t.cnt - at;
    p.col = t.nb * BT + half * kEpilogueCols;
    const int left = n_out - p.col < kEpilogueCols ? n_out - p.col : kEpilogueCols;
    p.have = p.rows <= 0 || left <= 0 ? 0 : (left + kGateCols - 1) / kGateCols;
    return p;
}
// Its epilogue warps' loop.  A half line's inputs are asked for one half line ahead, a tile's
// first ones before its products are there; its rows' weights a warp of their own has looked up
// (three loads one after the other, 3600 cycles).  What this does for a tile has to fit the two
// chains that the MMAs are ahead, 8500 cycles: half of them the exponentials and reciprocals.
template <typename Take, typename Ready, typename Release, typename Weight>
__device__ __forceinline__ void gated_grad_tiles(const CUtensorMap& tmGu, const CUtensorMap& tmOut,
                                                 const Gate& gate, uint8_t* staging, uint32_t bar,
                                                 uint32_t rank, int R, int n_out, int kblocks,
                                                 volatile int* abort, int* err, Take take_tile,
                                                 Ready ready, Release release, Weight weight) {
    const int lane = threadIdx.x & 31;
    const uint32_t staging_at = smem_u32(staging);
    uint32_t phase = 0;
    int buf = 0;
    GradPart p;
    {
        Tile t = {};
        if (!take_tile(0, t)) return;
        p = grad_part(t, rank, n_out);
    }
    const auto fetch = [&](const GradPart& q, int c, int b) {
        if (lane != 0) return;
        bulk_wait_read();  // what went out from there has been read
        const uint32_t to = staging_at + (uint32_t)(b * 2 * kHalfLines);
        mbar_expect_tx(bar, 2 * kHalfLines);
        tma_load_3d(to, &tmGu, bar, q.col + c * kGateCols, 0, (int)q.row);
        tma_load_3d(to + kHalfLines, &tmGu, bar, q.col + c * kGateCols, 1, (int)q.row);
    };
    if (p.have > 0) fetch(p, 0, 0);
    for (int i = 1;; ++i) {
        // dh, the chains' partial sums added up in fp32 registers (the sums over a row of dh
        // times what the gate gives are fp32 outputs), which frees the accumulators
        uint32_t dh[kEpilogueCols / 32][32];
#pragma unroll
        for (int c = 0; c < kEpilogueCols; ++c) dh[c / 32][c % 32] = 0u;
#pragma unroll 1
        for (int k = 0; k < kblocks; k += kGradChain) {
            uint32_t at;
            if (!ready(&at)) return;
#pragma unroll
            for (int c = 0; c < kEpilogueCols / 32; ++c) {
                uint32_t v[32];
                tmem_ld32(at + c * 32, v);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    dh[c][j] = __float_as_uint(__uint_as_float(dh[c][j]) + __uint_as_float(v[j]));
            }
            release();
        }
        float w;
        if (!weight(i - 1, &w)) return;
        F2 sum = f2(0.0f, 0.0f);
        const F2 one = f2(1.0f, 1.0f);
#pragma unroll
        for (int c = 0; c < kEpilogueCols / kGateCols; ++c) {
            if (c >= p.have) break;
            const bool in = wait_bar(bar, phase, abort, err);
            phase ^= 1u;
            if (!__all_sync(0xffffffffu, in)) return;
            if (c + 1 < p.have) fetch(p, c + 1, buf ^ 1);
            uint8_t* lines = staging + buf * 2 * kHalfLines;
            sum = f2_fma(gated_grad_lines(lines, dh[c], w), one, sum);
            const int col = p.col + c * kGateCols;
            fence_async_shared();
            __syncwarp();
            if (p.rows >= 32) {
                if (lane == 0) {
                    const uint32_t from = staging_at + (uint32_t)(buf * 2 * kHalfLines);
                    tma_store_3d(&tmOut, from, col, 0, (int)p.row);
                    tma_store_3d(&tmOut, from + kHalfLines, col, 1, (int)p.row);
                    bulk_commit();
                }
            } else {
                // the segment ends inside these rows: the ones after it are another expert's
                uint16_t* to = gate.gu + p.row * 2 * n_out + col;
                store_half_lines(lines, to, 2 * n_out, p.rows, n_out - col);
                store_half_lines(lines + kHalfLines, to + n_out, 2 * n_out, p.rows, n_out - col);
                fence_async_shared();
                __syncwarp();
            }
            buf ^= 1;
        }
        if (gate.parts && lane < p.rows && p.have > 0)
            gate.parts[(long long)(p.col / kEpilogueCols) * R + p.row + lane] =
                f2_get(sum).x + f2_get(sum).y;
        // the next tile's first inputs while its products run
        Tile t = {};
        if (!take_tile(i, t)) return;
        p = grad_part(t, rank, n_out);
        if (p.have > 0) fetch(p, 0, buf);
    }
}

// kFew (products over rows): tiles of 256 columns of the output and BF rows, the matrix
// being A and the rows B.  An MMA takes the same time for 1 row and for 128 of A, and 512
// cycles a k-block for 256 of B, which is longer than the 32 KB of the matrix need to come
// in; so it is a quarter of that, and the stages are 9.  64 experts of 2816 x 2048: 111 us
// for 1 row each and 121 us for 64 (256 rows as A: 118 and 128 us); 512 x 512, 16 rows
// each: 13.5 us (14.6 us).
// kSplit: a cluster of several pairs has one tile, each pair a share of its
// contraction, and the pairs' sums are joined at the end.
// kWeightsGrad: K unused, m_out x n_out = C_out x C_in; otherwise K the contraction and
// n_out the columns of out.  a_groups, b_groups: the map of an MN-major operand has its
// groups of 64 columns as a dimension.
// kLong (bf16 outputs in tiles of 256 rows): a contraction may take more than one chain.
template <int kMode, typename OutT, bool kFew, bool kSplit, bool kLong>
__device__ __forceinline__ void grouped_product(
    const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmOut,
    const int32_t* expert_offsets, const int32_t* expert_counts, int E,
    int R, int K, int m_out, int n_out, OutT* out, int accumulate, int a_groups,
    int b_groups, int* err, int* tile_counter, const CUtensorMap& tmGu, const Gate& gate) {
    constexpr bool kW = kMode == kWeightsGrad;
    constexpr bool kGate = kMode == kGated || kMode == kGatedGrad;
    static_assert(!kGate || (!kSplit && !kLong && sizeof(OutT) == 2), "the gate's forms");
    static_assert(kMode != kGatedGrad || !kFew, "a gate's gradient has no tiles of few rows");
    static_assert(!kW || !kFew, "a weights' gradient has no tiles of few rows");
    constexpr int kStages = kStagesOf<kMode, kFew>, STAGE_BYTES = kStageBytes<kFew>;
    constexpr int kTileRows = kFew ? BF : BT;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t* tiles = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
    const uint32_t tiles_addr = smem_u32(tiles);
    uint8_t* staging_area = tiles + (size_t)kStages * STAGE_BYTES;
    auto* ctl = reinterpret_cast<Ctl<kMode, kFew>*>(staging_area +
                                                    (size_t)kEpilogueWarps * kStagingOf<kMode>);
    volatile int* abort_flag = &ctl->abort;

    constexpr int kChain = kMode == kGatedGrad ? kGradChain : kChainBlocks<OutT>;
    // the partial sums before the last are added to it in registers; else (kLong) in TMEM:
    // beside a line of 64 bf16 columns 128 sums would not fit the registers
    constexpr bool kSums = sizeof(OutT) == 4 || kFew;
    static_assert(!kSums || !kLong, "these take any length");
    constexpr bool kMnA = kW;                 // the contraction runs along tmA's rows
    constexpr bool kMnB = kMode != kForward && kMode != kGated;  // and along tmB's
    // readers of a slot of the leader's queue: its producer, MMA thread,
    // epilogue warps (and block-end warp, or the one for rows' weights), and the peer's producer
    constexpr int kLocalReaders = kEpilogueWarps + (kW || kMode == kGatedGrad ? 1 : 0);
    constexpr int kQueueReaders = kLocalReaders + 3;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the pair's leader is the even one of its two CTAs of the cluster
    const uint32_t in_cluster = cluster_rank(), rank = in_cluster & 1u;
    const uint32_t first = kSplit ? in_cluster & ~1u : 0u;
    const int split = kSplit ? (int)(in_cluster >> 1) : 0;
    const int splits = kSplit ? (int)(cluster_ctas() >> 1) : 1;
    const uint16_t pair_mask = (uint16_t)(0x3u << first), leader_mask = (uint16_t)(0x1u << first);
    const bool leader = rank == 0;
    const int MB = blocks_of(m_out, BT);
    const int NB = blocks_of(n_out, kMode == kGated ? BT / 2 : BT);
    const int KB = blocks_of(K, BK);
    const int n_last = kFew || kMode == kGated ? BT : last_columns(n_out, kMnB && b_groups);

    // one or two barriers a thread, not 63 and more of them one after the other
    static_assert(3 * kStages <= 64 && kQueueBarriers <= 64, "barriers of 64 threads");
    if (warp == 4 || warp == 5) {
        const int i = threadIdx.x - 128, q = i - (2 * kAccs + 1);
        int count = 1;
        if (i >= kAccs && i < 2 * kAccs) count = 2 * kEpilogueWarps;  // tempty
        if (q >= kQ && q < 2 * kQ) count = kQueueReaders;             // q_empty
        if (q >= 4 * kQ) count = kLocalReaders;                       // l_empty
        if (i < kQueueBarriers) mbar_init(smem_u32(&ctl->tfull[0] + i), count);
        if (i < 3 * kStages) mbar_init(smem_u32(&ctl->full[0] + i), kW && i < kStages ? 2 : 1);
        if (i == 63) ctl->abort = 0;
        if constexpr (kMode == kGatedGrad) {
            if (i < kEpilogueWarps) mbar_init(smem_u32(&ctl->lines[i]), 1);
            if (i < 2) mbar_init(smem_u32(&ctl->w_full[i]), 1);
            if (i < 2) mbar_init(smem_u32(&ctl->w_empty[i]), kEpilogueWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        prefetch_map(&tmA);
        prefetch_map(&tmB);
        if (!kFew) prefetch_map(&tmOut);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&ctl->tmem_base), kTmemCols);
        tmem_relinquish_pair();
    }
    after_previous();
    // A weights' gradient hands out the experts with the most rows first: their tiles
    // take the longest, and the short ones fill the pairs up at the end (Zipf-skewed
    // case of 262144 rows in 128 experts: 2190 us in the experts' order, 2040 so).
    bool sorted = false;
    if constexpr (kW && !kSplit) {
        sorted = E <= kMaxSorted && E * MB * NB > (int)(gridDim.x / 2);
        if (sorted) {
            int* cnts = reinterpret_cast<int*>(tiles);  // the operand ring, not in use yet
            for (int i = threadIdx.x; i < E; i += blockDim.x) cnts[i] = expert_counts[i];
            __syncthreads();
            for (int i = threadIdx.x; i < E; i += blockDim.x) {
                const int mine = cnts[i];
                int before = 0;
                for (int j = 0; j < E; ++j)
                    before += cnts[j] > mine || (cnts[j] == mine && j < i) ? 1 : 0;
                ctl->order[before] = (uint16_t)i;
            }
            fence_async_shared();  // before TMA writes there
            __syncthreads();
        }
    }
    // Products over rows: lane l of the scheduler holds the row blocks in its run of
    // experts [l * per, (l + 1) * per) and up to its end.
    const int per = (E + 31) / 32;
    int blocks_end = 0, blocks_in = 0, total = E * MB * NB;
    int run_off = 0, run_cnt = 0;  // the run's last expert: the lane's own where per = 1
    int last_e = -1, last_off = 0, last_cnt = 0;  // the last tile's (weights' gradient)
    // A tile by its number, decoded by a whole warp.
    const auto decode = [&](int tile) {
        Tile t = {};
        t.e = -1;
        if (tile >= total) return t;
        if constexpr (kW) {
            t.e = tile / (MB * NB);
            const int local = tile - t.e * MB * NB;
            t.mb = local / NB;
            t.nb = local - t.mb * NB;
            if constexpr (!kSplit) {
                if (sorted) t.e = ctl->order[t.e];
            }
            if (t.e != last_e)
                segment(expert_offsets, expert_counts, t.e, R, err, &last_off, &last_cnt);
            last_e = t.e;
            t.off = last_off;
            t.cnt = last_cnt;
            t.kblocks = blocks_of(t.cnt, BK);
        } else {
            // the run of experts that holds row block q, then the expert
            const int q = tile / NB;
            int run = 0, before = 0, o = run_off, c = run_cnt;
            if (per > 1) {
                run = __ffs(__ballot_sync(0xffffffffu, blocks_end > q)) - 1;
                before = __shfl_sync(0xffffffffu, blocks_end - blocks_in, run);
                const int mine = run * per + lane;
                o = c = 0;
                if (lane < per && mine < E)
                    segment(expert_offsets, expert_counts, mine, R, err, &o, &c);
            }
            const int b = blocks_of(c, kTileRows), end = before + warp_prefix(b);
            const int k = __ffs(__ballot_sync(0xffffffffu, end > q)) - 1;
            const int MBe = __shfl_sync(0xffffffffu, b, k);
            const int local = tile - NB * (__shfl_sync(0xffffffffu, end, k) - MBe);
            t.e = run * per + k;
            t.off = __shfl_sync(0xffffffffu, o, k);
            t.cnt = __shfl_sync(0xffffffffu, c, k);
            t.kblocks = KB;
            // the expert's smaller operand is the one read again: its row blocks side by
            // side when they are fewer than its columns'
            if (MBe > NB) {
                t.mb = local / NB;
                t.nb = local - t.mb * NB;
            } else {
                t.nb = local / MBe;
                t.mb = local - t.nb * MBe;
            }
        }
        if (kSplit) {
            const int all = t.kblocks;
            t.k0 = (int)((long long)all * split / splits);
            t.kblocks = (int)((long long)all * (split + 1) / splits) - t.k0;
            t.all = t.cnt;
            if (kW) {
                const int end = (t.k0 + t.kblocks) * BK;
                t.off += t.k0 * BK;
                t.cnt = (t.cnt < end ? t.cnt : end) - t.k0 * BK;
            }
        }
        return t;
    };
    if (warp == 2) {
        if (!kW) {
            for (int j = 0; j < per; ++j) {
                if (lane * per + j < E) {
                    segment(expert_offsets, expert_counts, lane * per + j, R, err, &run_off,
                            &run_cnt);
                    blocks_in += blocks_of(run_cnt, kTileRows);
                }
            }
            // Only a layout whose segments overlap has more blocks than R rows can fill: it
            // gets no more, nor sums that wrap, and is reported where tiles are launched one
            // by one.
            if (blocks_in > 1 << 25) blocks_in = 1 << 25;
            blocks_end = warp_prefix(blocks_in);
            const int blocks = __shfl_sync(0xffffffffu, blocks_end, 31), most = R / kTileRows + E;
            total = (blocks < most ? blocks : most) * NB;
            if (kSplit && blockIdx.x == 0 && lane == 0 && total > (int)gridDim.x / (2 * splits))
                set_error(err, MOE_ERR_INVALID_ARG);
        }
        // the pair's first tile is its own index (its cluster's, in split contractions)
        const Tile t = decode((int)blockIdx.x / (2 * splits));
        if (lane == 0) {
            ctl->first = t;
            ctl->only = kSplit || total <= (int)gridDim.x / 2;
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before any remote signal
    tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    Tile joined = {};  // the tile of a split contraction (epilogue warps)
    joined.e = -1;
    if (warp < 4) {
        regs_shrink<kRegsOther<kMode>>();
        // One lane each of the producer and the MMA issuer, elected rather than lane 0: the
        // compiler then knows that the lane is alone and keeps the operands of copies and
        // MMAs in uniform registers (tiles of few rows: a k-block in 0.19 us,
        // 0.27 us otherwise).
        if (warp == 0 && elect_one()) {
            // ---------------- TMA producer (both CTAs) ----------------
            const uint32_t full0 = mapa_shared(smem_u32(&ctl->full[0]), first);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int i = 0; ok; ++i) {
                Tile t = {};
                t.e = -1;
                bool more;
                if (i == 0) {
                    t = read_slot(&ctl->first);
                    more = t.e >= 0;
                } else {
                    if (ctl->only) break;
                    more = take(ctl, i - 1, leader, first, abort_flag, err, t);
                    if (leader && more) mbar_arrive(smem_u32(&ctl->q_taken[(i - 1) % kQ]));
                    if (!leader && !forward(ctl, i - 1, t, abort_flag, err)) more = false;
                }
                if (!more) break;
                const int off = t.off;
                const bool ragged = kW && (t.cnt % UMMA_K) != 0;
                // this CTA's half of A's rows and of B's
                const int a0 = t.mb * BT + (int)rank * BH;
                const int half = (t.nb == NB - 1 ? n_last : BT) / 2;
                const int b0 = t.nb * BT + (int)rank * half;
                // boxes of 64 columns where those come one by one
                const bool two = half > 64;
                const uint32_t stage_tx =
                    kFew || kMode == kGated ? STAGE_BYTES
                         : OP_BYTES + (kMnB && !b_groups ? (two ? 2 : 1) * BOX_BYTES
                                                         : box_columns(n_out, kMnB) * BK * 2);
                for (int kb = 0; kb < t.kblocks; ++kb) {
                    if (!wait_bar(smem_u32(&ctl->empty[stage]), phase ^ 1u, abort_flag, err)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full_local = smem_u32(&ctl->full[stage]);
                    const uint32_t a_s = tiles_addr + stage * STAGE_BYTES;
                    const uint32_t b_s = a_s + OP_BYTES;
                    if (kW) {
                        const int row = off + kb * BK;
                        if (ragged && kb == t.kblocks - 1) {
                            const uint32_t land = smem_u32(&ctl->land[stage]);
                            mbar_expect_tx(land, stage_tx);
                            if (a_groups) {
                                tma_load_3d(a_s, &tmA, land, 0, row, a0 / 64);
                            } else {
                                tma_load_2d(a_s, &tmA, land, a0, row);
                                tma_load_2d(a_s + BOX_BYTES, &tmA, land, a0 + 64, row);
                            }
                            if (b_groups) {
                                tma_load_3d(b_s, &tmB, land, 0, row, b0 / 64);
                            } else {
                                tma_load_2d(b_s, &tmB, land, b0, row);
                                if (two) tma_load_2d(b_s + BOX_BYTES, &tmB, land, b0 + 64, row);
                            }
                        } else {
                            const uint32_t full = full0 + (uint32_t)stage * 8u;
                            if (leader) {
                                mbar_arrive(full_local);
                                mbar_expect_tx(full_local, 2 * stage_tx);
                            }
                            if (a_groups) {
                                tma_load_3d_pair(a_s, &tmA, full, 0, row, a0 / 64);
                            } else {
                                tma_load_2d_pair(a_s, &tmA, full, a0, row);
                                tma_load_2d_pair(a_s + BOX_BYTES, &tmA, full, a0 + 64, row);
                            }
                            if (b_groups) {
                                tma_load_3d_pair(b_s, &tmB, full, 0, row, b0 / 64);
                            } else {
                                tma_load_2d_pair(b_s, &tmB, full, b0, row);
                                if (two)
                                    tma_load_2d_pair(b_s + BOX_BYTES, &tmB, full, b0 + 64, row);
                            }
                        }
                    } else {
                        const uint32_t full = full0 + (uint32_t)stage * 8u;
                        const int k = (kSplit ? t.k0 + kb : kb) * BK;
                        // the matrix is B, or A of a tile of few rows
                        const uint32_t w_s = kFew ? a_s : b_s, r_s = kFew ? b_s : a_s;
                        if (leader) mbar_expect_tx(full_local, 2 * stage_tx);
                        tma_load_2d_pair(r_s, &tmA, full, k,
                                         off + (kFew ? t.mb * BF + (int)rank * (BF / 2) : a0));
                        if (kMode == kGated && kFew) {
                            // each CTA has 64 gate columns and their up columns
                            const int c0 = t.nb * BH + (int)rank * 64;
                            tma_load_4d_pair(w_s, &tmB, full, k, c0, 0, t.e);
                            tma_load_4d_pair(w_s + BOX_BYTES, &tmB, full, k, c0, 1, t.e);
                        } else if (kMode == kGated) {
                            // one CTA brings the gate columns, one the up columns
                            tma_load_4d_pair(w_s, &tmB, full, k, t.nb * BH, (int)rank, t.e);
                        } else if (kMnB && b_groups) {
                            tma_load_4d_pair(w_s, &tmB, full, 0, k, b0 / 64, t.e);
                        } else if (kMnB) {
                            tma_load_3d_pair(w_s, &tmB, full, b0, k, t.e);
                            if (kFew || two)
                                tma_load_3d_pair(w_s + BOX_BYTES, &tmB, full, b0 + 64, k, t.e);
                        } else {
                            tma_load_3d_pair(w_s, &tmB, full, k, b0, t.e);
                        }
                    }
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // a wait has given up: let the copies in flight land before the CTA exits
            if (*abort_flag) spin(4000000);
        } else if (warp == 1 && leader && elect_one()) {
            // ---------------- MMA issuer (leader only) ----------------
            constexpr bool kMajA = kFew ? kMnB : kMnA, kMajB = kFew ? kMnA : kMnB;
            constexpr uint32_t kMajors = (kMajA ? kIdescMnA : 0u) | (kMajB ? kIdescMnB : 0u);
            // a K step of 16 inside a stage: 32 bytes of a K-major row, or 16 rows
            constexpr uint64_t kStepA = kMajA ? 16 * 128 / 16 : 2;
            constexpr uint64_t kStepB = kMajB ? 16 * 128 / 16 : 2;
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            for (int i = 0; ok; ++i) {
                Tile t = {};
                if (!next(ctl, i, first, abort_flag, err, t)) break;
                // K steps of the last block (a segment's end)
                const int last_steps =
                    kW ? (t.cnt - (t.kblocks - 1) * BK + UMMA_K - 1) / UMMA_K
                       : BK / UMMA_K;
                const uint32_t idesc =
                    kMajors |
                    (kFew ? make_idesc(BT, BF) : make_idesc(BT, t.nb == NB - 1 ? n_last : BT));
                int in_chain = 0;
                for (int kb = 0; kb < t.kblocks; ++kb) {
                    if (in_chain == 0) {
                        if (!wait_bar(smem_u32(&ctl->tempty[acc]), acc_phase ^ 1u, abort_flag,
                                      err)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                    }
                    // the peer's block-end warp arrives at cluster scope
                    const uint32_t full = smem_u32(&ctl->full[stage]);
                    if (!(kW ? wait_bar_cluster(full, phase, abort_flag, err)
                             : wait_bar(full, phase, abort_flag, err))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + (uint32_t)(acc * BT);
                    const uint32_t a_s = tiles_addr + stage * STAGE_BYTES;
                    const uint32_t b_s = a_s + OP_BYTES;
                    const uint64_t ad = kMajA ? sw128_desc_mn(a_s, BOX_BYTES) : sw128_desc(a_s);
                    const uint64_t bd = kMajB ? sw128_desc_mn(b_s, BOX_BYTES) : sw128_desc(b_s);
                    const int steps = kW && kb == t.kblocks - 1 ? last_steps : BK / UMMA_K;
#pragma unroll
                    for (int kk = 0; kk < BK / UMMA_K; ++kk) {
                        if (!kW || kk < steps)
                            umma_bf16_pair(d, ad + kStepA * kk, bd + kStepB * kk, idesc,
                                           (in_chain | kk) != 0 ? 1u : 0u);
                    }
                    umma_commit_pair_multicast(smem_u32(&ctl->empty[stage]), pair_mask);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    ++in_chain;
                    if (((kSums || kLong || kMode == kGatedGrad) && in_chain == kChain) ||
                        kb == t.kblocks - 1) {
                        umma_commit_pair_multicast(smem_u32(&ctl->tfull[acc]), pair_mask);
                        in_chain = 0;
                        if (++acc == kAccs) {
                            acc = 0;
                            acc_phase ^= 1u;
                        }
                    }
                }
            }
            umma_commit_pair_multicast(smem_u32(&ctl->done), leader_mask);
            wait_bar_drain(smem_u32(&ctl->done), 0);
        } else if (warp == 2 && leader && !ctl->only) {
            // ---------------- tile scheduler (leader) ----------------
            // The counter hands out the tiles after the pairs' first ones.  Tile i of the
            // queue is published once the producer has taken tile i - kAhead.
            const int pairs = (int)(gridDim.x / 2);
            int longest = ctl->first.kblocks;  // of the tiles handed out
            for (int i = 0;; ++i) {
                int tile = -1;
                if (lane == 0) {
                    bool ok = true;
                    if (i >= kAhead) {
                        const int j = i - kAhead;
                        ok = wait_bar(smem_u32(&ctl->q_taken[j % kQ]), (uint32_t)(j / kQ) & 1u,
                                      abort_flag, err, tile_limit(longest));
                    }
                    if (ok) tile = pairs + atomicAdd(tile_counter, 1);
                }
                tile = __shfl_sync(0xffffffffu, tile, 0);
                if (tile < 0) break;
                const Tile t = decode(tile);
                longest = t.kblocks > longest ? t.kblocks : longest;
                int more = 0;
                if (lane == 0) more = publish(ctl, i, t, first, abort_flag, err) && t.e >= 0;
                if (!__shfl_sync(0xffffffffu, more, 0)) break;
            }
        } else if (kMode == kGatedGrad && warp == 3) {
            if constexpr (kMode == kGatedGrad) {
                // ---------------- rows' weights (both CTAs) ----------------
                for (int i = 0;; ++i) {
                    Tile t = {};
                    if (!warp_next(ctl, i, leader, abort_flag, err, t)) break;
                    const int b = i & 1, left = t.cnt - t.mb * BT - (int)rank * BH;
                    const long long row = (long long)t.off + t.mb * BT + (int)rank * BH;
                    float w[BH / 32];
#pragma unroll
                    for (int r = 0; r < BH / 32; ++r)
                        w[r] = r * 32 + lane < left ? row_weight(gate, row + r * 32 + lane) : 0.0f;
                    const bool free = wait_bar(smem_u32(&ctl->w_empty[b]),
                                               ((uint32_t)(i >> 1) & 1u) ^ 1u, abort_flag, err,
                                               tile_limit(t.kblocks));
                    if (!__all_sync(0xffffffffu, free)) break;
#pragma unroll
                    for (int r = 0; r < BH / 32; ++r) ctl->weights[b][r * 32 + lane] = w[r];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&ctl->w_full[b]));
                }
            }
        } else if (kW && warp == 3) {
            // ---------------- block ends (both CTAs) ----------------
            const uint32_t full0 = mapa_shared(smem_u32(&ctl->full[0]), first);
            int stage = 0;
            uint32_t land_phase = 0;
            for (int i = 0;; ++i) {
                Tile t = {};
                if (!warp_next(ctl, i, leader, abort_flag, err, t)) break;
                const int cnt = t.cnt;
                if (t.kblocks == 0) continue;
                const int last = (stage + t.kblocks - 1) % kStages;
                stage = (stage + t.kblocks) % kStages;
                if (cnt % UMMA_K == 0) continue;
                int landed = 0;
                if (lane == 0)
                    landed = wait_bar(smem_u32(&ctl->land[last]), (land_phase >> last) & 1u,
                                      abort_flag, err, tile_limit(t.kblocks));
                landed = __shfl_sync(0xffffffffu, landed, 0);
                if (!landed) break;
                land_phase ^= 1u << last;
                // rows [r0, r1) of the 4 boxes of the stage, 8 chunks of 16 bytes each
                const int r0 = cnt % BK, r1 = (r0 + UMMA_K - 1) / UMMA_K * UMMA_K;
                uint8_t* st = tiles + (size_t)last * STAGE_BYTES;
                for (int c = lane; c < (r1 - r0) * 32; c += 32) {
                    const int box = c & 3, chunk = (c >> 2) & 7, r = r0 + (c >> 5);
                    *reinterpret_cast<uint4*>(st + box * BOX_BYTES + r * 128 + chunk * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote_shared(full0 + (uint32_t)last * 8u);
            }
        }
    } else {
        // ---------------- epilogue (both CTAs): own 128 rows ----------------
        regs_grow<kRegsEpilogue<kMode>>();
        const int q = warp & 3;               // TMEM lane quadrant
        const int half = (warp - 4) >> 2;     // 128 columns of the tile, or 32 of its few rows
        constexpr int kCols = kFew ? BF / 2 : kEpilogueCols;  // of the accumulator
        uint8_t* staging = staging_area + (size_t)(warp - 4) * kStagingOf<kMode>;
        const uint32_t tempty0 = mapa_shared(smem_u32(&ctl->tempty[0]), first);
        int acc = 0;
        uint32_t acc_phase = 0;
        if constexpr (kMode == kGatedGrad) {
            const auto take_tile = [&](int i, Tile& t) {
                return warp_next(ctl, i, leader, abort_flag, err, t);
            };
            // this warp's columns of the next accumulator, once it is ready
            const auto ready = [&](uint32_t* at) {
                int ok = 0;
                if (lane == 0)
                    ok = wait_bar(smem_u32(&ctl->tfull[acc]), acc_phase, abort_flag, err);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                tc_fence_after();
                *at = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BT + half * kCols);
                return ok != 0;
            };
            const auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(tempty0 + (uint32_t)acc * 8u);
                if (++acc == kAccs) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            };
            // this lane's row's weight in tile i
            const auto weight = [&](int i, float* w) {
                const int b = i & 1;
                const bool ok = wait_bar(smem_u32(&ctl->w_full[b]), (uint32_t)(i >> 1) & 1u,
                                         abort_flag, err);
                *w = ctl->weights[b][q * 32 + lane];
                const bool all = __all_sync(0xffffffffu, ok);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->w_empty[b]));
                return all;
            };
            gated_grad_tiles(tmGu, tmOut, gate, staging, smem_u32(&ctl->lines[warp - 4]), rank, R,
                             n_out, KB, abort_flag, err, take_tile, ready, release, weight);
        } else
        for (int i = 0;; ++i) {
            Tile t = {};
            if (!warp_next(ctl, i, leader, abort_flag, err, t)) {
                if constexpr (kMode == kGated && kFew) gated_few_leave(q, half);
                break;
            }
            if (!kSplit && kW && t.kblocks == 0 && accumulate) continue;  // nothing to add
            if (kSplit) joined = t;

            // this warp's part of the next accumulator, once it is ready
            const auto ready = [&]() {
                int ok = 0;
                if (lane == 0)
                    ok = wait_bar(smem_u32(&ctl->tfull[acc]), acc_phase, abort_flag, err);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                tc_fence_after();
                return ok != 0;
            };
            const auto part = [&]() {
                return tmem + ((uint32_t)(q * 32) << 16) +
                       (uint32_t)(acc * BT + half * kCols);
            };
            // the accumulator has been read
            const auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(tempty0 + (uint32_t)acc * 8u);
                if (++acc == kAccs) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            };
            if constexpr (kMode == kGated && kFew) {
                const int left = t.cnt - t.mb * BF - half * 32, rows = left < 32 ? left : 32;
                const long long row = (long long)t.off + t.mb * BF + half * 32;
                const float w = lane < rows ? row_weight(gate, row + lane) : 0.0f;
                if (!ready() || *abort_flag) {
                    gated_few_leave(q, half);
                    break;
                }
                uint32_t v[32];
                tmem_ld32(part(), v);
                tmem_wait_ld();
                release();
                gated_few_out(gate, staging_area, q, half, v, row, rows,
                              t.nb * BH + (int)rank * 64 + (q & 1) * 32, n_out, w);
                continue;
            } else if constexpr (kMode == kGated) {
                const int at_row = t.mb * BT + (int)rank * BH + q * 32, rows = t.cnt - at_row;
                const long long row = (long long)t.off + at_row;
                const float w = lane < rows ? row_weight(gate, row + lane) : 0.0f;
                if (!ready()) break;
                const uint32_t g_at = tmem + ((uint32_t)(q * 32) << 16) +
                                      (uint32_t)(acc * BT + half * 64);
                gated_out(tmGu, tmOut, gate, staging, g_at, g_at + BT / 2, row, rows,
                          t.nb * BH + half * 64, n_out, w, release);
                continue;
            }

            const int chains = kSums ? (t.kblocks + kChain - 1) / kChain
                                     : (t.kblocks > 0 ? 1 : 0);
            uint32_t sum[kSums ? kCols / 32 : 1][32];
            bool ok = true;
            if (kSums && chains > 1) {
#pragma unroll
                for (int c = 0; c < kCols; ++c) sum[c / 32][c % 32] = 0u;
                for (int n = 0; ok && n < chains - 1; ++n) {
                    if (!ready()) {
                        ok = false;
                        break;
                    }
                    const uint32_t at = part();
#pragma unroll
                    for (int c = 0; c < kCols / 32; ++c) {
                        uint32_t v[32];
                        tmem_ld32(at + c * 32, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            sum[c][j] = __float_as_uint(__uint_as_float(sum[c][j]) +
                                                        __uint_as_float(v[j]));
                    }
                    release();
                }
            }
            if (!ok || (chains > 0 && !ready())) break;
            if constexpr (kLong) {
                // adds the chains before the last to it, where the lines below read it
                if (t.kblocks > kChain) {
                    uint32_t before[kCols / 32][32] = {};
                    for (int k = t.kblocks; ok && k > kChain; k -= kChain) {
                        const uint32_t from = part();
#pragma unroll
                        for (int c = 0; c < kCols / 32; ++c) {
                            uint32_t v[32];
                            tmem_ld32(from + c * 32, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                before[c][j] = __float_as_uint(__uint_as_float(before[c][j]) +
                                                               __uint_as_float(v[j]));
                        }
                        release();
                        ok = ready();
                    }
                    if (!ok) break;
                    const uint32_t last = part();
#pragma unroll
                    for (int c = 0; c < kCols / 32; ++c) {
                        uint32_t v[32];
                        tmem_ld32(last + c * 32, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[j] = __float_as_uint(__uint_as_float(before[c][j]) +
                                                   __uint_as_float(v[j]));
                        tmem_st32(last + c * 32, v);
                    }
                    tmem_wait_st();
                }
            }
            if constexpr (kFew) {
                uint32_t v[32];
                tmem_ld32(part(), v);
                tmem_wait_ld();
                release();
                if (kSums && chains > 1) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = __float_as_uint(__uint_as_float(sum[0][j]) + __uint_as_float(v[j]));
                }
                const FewPart f = few_part(t, rank);
                const int c = f.col + (lane & 7) * 4;
                if (f.rows <= 0 || f.col >= n_out) continue;
                if (kSplit) {
                    put_few(tiles + (warp - 4) * kStagingBytes, lane, v);
                    continue;
                }
                put_few(staging, lane, v);
                __syncwarp();
                for (int r = lane >> 3; r < 32 && r < f.rows; r += 4)
                    if (c < n_out)
                        store_few(out + (f.row + r) * n_out + c,
                                  *reinterpret_cast<const float4*>(staging + r * 128 +
                                                                   (lane & 7) * 16));
                __syncwarp();
                continue;
            }

            // the last one (or zeros), stored line by line: the reads of a line from
            // TMEM go on beside the stores of the one before
            const int row = t.mb * BT + (int)rank * BH + q * 32;
            const int rows = (kW ? m_out : t.cnt) - row;
            const int col = t.nb * BT + half * kEpilogueCols;
            constexpr int kLine = 128 / (int)sizeof(OutT);
            const uint32_t at = part();
            const auto put = [&](int c, const uint32_t (&v)[kLine]) {
                if (rows <= 0 || col + c >= n_out) return;
                if constexpr (kSplit) {
                    put_part<kLine>(tiles, q * 32 + lane, half * kEpilogueCols + c, v);
                    return;
                }
                if (lane == 0) bulk_wait_read();  // the line before has been read
                __syncwarp();
                put_line<OutT>(staging, lane, v);
                if (kW || rows >= 32) {
                    // columns (and rows of dW) past the matrix are clipped by its map
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        if (!kW)
                            tma_store_2d(&tmOut, smem_u32(staging), col + c, t.off + row);
                        else if (accumulate)
                            tma_reduce_add_3d(&tmOut, smem_u32(staging), col + c, row, t.e);
                        else
                            tma_store_3d(&tmOut, smem_u32(staging), col + c, row, t.e);
                        bulk_commit();
                    }
                } else {
                    // the segment ends inside these rows: the ones after it are another
                    // expert's
                    __syncwarp();
                    store_lines<OutT>(staging, out + ((long long)t.off + row) * n_out + col + c,
                                      n_out, rows, n_out - col - c);
                }
            };
            if (kSums && chains > 1) {
#pragma unroll
                for (int c = 0; c < kEpilogueCols; c += kLine) {
                    uint32_t v[kLine];
                    tmem_ld_line(at + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < kLine; ++j)
                        v[j] = __float_as_uint(
                            __uint_as_float(sum[kSums ? c / 32 : 0][j % 32]) +
                            __uint_as_float(v[j]));
                    if (c == kEpilogueCols - kLine) release();
                    put(c, v);
                }
            } else {
                // not unrolled: in a short call most of this is the fetch of its code
#pragma unroll 1
                for (int c = 0; c < kEpilogueCols; c += kLine) {
                    uint32_t v[kLine];
                    if (!kW || chains > 0) {
                        tmem_ld_line(at + c, v);
                        tmem_wait_ld();
                        if (c == kEpilogueCols - kLine) release();
                    } else {
#pragma unroll
                        for (int j = 0; j < kLine; ++j) v[j] = 0u;
                    }
                    put(c, v);
                }
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();  // no CTA leaves while its peer may still signal it
    if constexpr (kSplit) {
        if (kFew && joined.e >= 0 && splits == 2)
            join_few<2>(tiles_addr, rank, split, joined, n_out, out);
        else if (kFew && joined.e >= 0)
            join_few<kMaxSplits>(tiles_addr, rank, split, joined, n_out, out);
        else if (joined.e >= 0 && splits == 2)
            join_parts<kW, 2>(tiles_addr, rank, split, joined, m_out, n_out, out, accumulate);
        else if (joined.e >= 0)
            join_parts<kW, kMaxSplits>(tiles_addr, rank, split, joined, m_out, n_out, out,
                                       accumulate);
        __syncwarp();
        cluster_sync();  // nor while its part is read
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
    // the tile counter returns to zero for the next launch (the last pair out)
    if (!ctl->only && leader && threadIdx.x == 0) {
        __threadfence();
        const int before = atomicAdd(tile_counter + 1, 1);
        if (before == (int)(gridDim.x / 2) - 1) {
            atomicExch(tile_counter, 0);
            atomicExch(tile_counter + 1, 0);
        }
    }
}

template <int kMode, typename OutT, bool kFew, bool kLong>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    grouped_product_kernel(const __grid_constant__ CUtensorMap tmA,
                           const __grid_constant__ CUtensorMap tmB,
                           const __grid_constant__ CUtensorMap tmOut,
                           const int32_t* expert_offsets,
                           const int32_t* expert_counts, int E, int R, int K,
                           int m_out, int n_out, OutT* out, int accumulate,
                           int a_groups, int b_groups, int* err, int* tile_counter) {
    grouped_product<kMode, OutT, kFew, false, kLong>(tmA, tmB, tmOut, expert_offsets, expert_counts,
                                                     E, R, K, m_out, n_out, out, accumulate,
                                                     a_groups, b_groups, err, tile_counter, tmOut,
                                                     Gate{});
}
// Launched with clusters of 2 * splits CTAs.
template <int kMode, typename OutT, bool kFew, bool kLong>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_product_split_kernel(const __grid_constant__ CUtensorMap tmA,
                                 const __grid_constant__ CUtensorMap tmB,
                                 const __grid_constant__ CUtensorMap tmOut,
                                 const int32_t* expert_offsets,
                                 const int32_t* expert_counts, int E, int R, int K,
                                 int m_out, int n_out, OutT* out, int accumulate,
                                 int a_groups, int b_groups, int* err, int* tile_counter) {
    grouped_product<kMode, OutT, kFew, true, kLong>(tmA, tmB, tmOut, expert_offsets, expert_counts, E,
                                                    R, K, m_out, n_out, out, accumulate, a_groups,
                                                    b_groups, err, tile_counter, tmOut, Gate{});
}
// tmGu: gu as gate and up columns, [N*k][2][I]; tmOut: h, or the gradient of gu likewise.
template <int kMode, bool kFew>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gated_product_kernel(const __grid_constant__ CUtensorMap tmA,
                         const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmOut,
                         const __grid_constant__ CUtensorMap tmGu, const Gate gate,
                         const int32_t* expert_offsets, const int32_t* expert_counts, int E, int R,
                         int K, int I, int b_groups, int* err, int* tile_counter) {
    grouped_product<kMode, __nv_bfloat16, kFew, false, false>(
        tmA, tmB, tmOut, expert_offsets, expert_counts, E, R, K, 0, I,
        reinterpret_cast<__nv_bfloat16*>(gate.h), 0, 0, b_groups, err, tile_counter, tmGu, gate);
}

// dtopk_w of each pair: its row's sums of all 128-column parts, in their order.  A pair whose
// row no expert has keeps what is there; only where the experts have fewer rows than there are
// does a row look for its own.
__global__ void __launch_bounds__(256)
    gate_weight_grad_kernel(const float* parts, int n_parts, const int32_t* expert_offsets,
                            const int32_t* expert_counts, int E, const int32_t* pair_row,
                            long long R, float* dtopk_w) {
    __shared__ unsigned long long had[8];
    after_previous();
    long long rows = 0;
    for (int e = threadIdx.x; e < E; e += 256) rows += expert_counts[e];
#pragma unroll
    for (int o = 16; o; o >>= 1) rows += __shfl_xor_sync(0xffffffffu, rows, o);
    if ((threadIdx.x & 31) == 0) had[threadIdx.x >> 5] = (unsigned long long)rows;
    __syncthreads();
    rows = 0;
    for (int w = 0; w < 8; ++w) rows += (long long)had[w];
    const long long pair = (long long)blockIdx.x * 256 + threadIdx.x;
    if (pair >= R) return;
    const int row = pair_row[pair];
    if (row < 0 || row >= R) return;
    bool mine = rows >= R;
    for (int e = 0; !mine && e < E; ++e) {
        const int off = expert_offsets[e];
        mine = row >= off && row - off < expert_counts[e];
    }
    if (!mine) return;
    float sum = 0.0f;
#pragma unroll 8
    for (int p = 0; p < n_parts; ++p) sum += parts[p * R + row];
    dtopk_w[pair] = sum;
}

// Clusters of 2 * splits CTAs that the device holds at once; -1: the query failed.
template <typename Kernel>
int clusters_at_once(Kernel kernel, int splits, size_t smem) {
    cudaLaunchAttribute cluster[1];
    cluster[0].id = cudaLaunchAttributeClusterDimension;
    cluster[0].val.clusterDim.x = 2 * splits;
    cluster[0].val.clusterDim.y = cluster[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * splits);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = cluster;
    cfg.numAttrs = 1;
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n : -1;
}

template <int kMode, typename OutT, bool kFew, bool kLong>
moe_status launch_form(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o,
                  const GemmGroup& g, long long tiles, long long blocks,
                  int K, int m_out, int n_out, void* out, bool accumulate, int a_groups,
                  int b_groups, cudaStream_t st) {
    if (tiles >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
    // the attributes hold for the process and device: set once for each
    constexpr size_t smem = smem_bytes<kMode, kFew>();
    const auto split_kernel = grouped_product_split_kernel<kMode, OutT, kFew, kLong>;
    static OncePerDevice set;
    static std::atomic<int> held[kMaxDevices][2];  // clusters of 2 pairs and of 4, on each device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    if (dev >= kMaxDevices) return MOE_ERR_UNSUPPORTED;
    if (!set.done(dev)) {
        if (cudaFuncSetAttribute(grouped_product_kernel<kMode, OutT, kFew, kLong>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem) != cudaSuccess ||
            cudaFuncSetAttribute(split_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem) != cudaSuccess)
            return MOE_ERR_CUDA;
        const int two = clusters_at_once(split_kernel, 2, smem);
        const int four = clusters_at_once(split_kernel, kMaxSplits, smem);
        if (two < 0 || four < 0) return MOE_ERR_CUDA;
        held[dev][0].store(two, std::memory_order_relaxed);
        held[dev][1].store(four, std::memory_order_relaxed);
        set.finish(dev);
    }
    const int at_once[2] = {held[dev][0].load(std::memory_order_relaxed),
                            held[dev][1].load(std::memory_order_relaxed)};
    // Pairs that share a tile's contraction: as long as all clusters run side by side, and
    // what a pair no longer has to do, some 0.3 us a k-block, is more than what the
    // joining of the sums takes: 1 us for a few rows, 6 us for a tile's 256 (1 row, 4096 x
    // 3528: 25 us with one pair a tile, 16 us with four; K = 512: 8.1 and 7.8 us with two;
    // 256 x 256 sums of 1024 rows: 13.7 and 14.9 us with four, 4096 rows: 29 and 19 us).
    const long long m = kMode == kWeightsGrad ? m_out : kFew ? 0 : g.R;
    const long long join_blocks = 4 + 16 * (m < BT ? m : BT) / BT;
    int splits = 1;
    if (tiles <= at_once[1] && blocks * 3 > join_blocks * 4)
        splits = kMaxSplits;
    else if (tiles <= at_once[0] && blocks > join_blocks * 2)
        splits = 2;
    if (splits > 1)
        return cuda_status(launch_chained_clusters(
            split_kernel, 2 * splits, (int)(tiles * 2 * splits), kThreads, smem, st, a, b, o,
            g.offsets, g.counts, g.E, (int)g.R, K, m_out, n_out, reinterpret_cast<OutT*>(out),
            accumulate ? 1 : 0, a_groups, b_groups, g.err, (int*)nullptr));
    const long long pairs_max = sm_count() / 2;
    const long long pairs = tiles < pairs_max ? tiles : pairs_max;
    return cuda_status(launch_chained(
        grouped_product_kernel<kMode, OutT, kFew, kLong>, (int)(2 * (pairs > 0 ? pairs : 1)), kThreads,
        smem, st, a, b, o, g.offsets, g.counts, g.E, (int)g.R, K, m_out, n_out,
        reinterpret_cast<OutT*>(out), accumulate ? 1 : 0, a_groups, b_groups, g.err,
        g.prefix + g.E + 1));
}

// terms: the longest contraction that there may be.
template <int kMode, typename OutT, bool kFew = false>
moe_status launch(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o,
                  const GemmGroup& g, long long tiles, long long blocks, long long terms,
                  int K, int m_out, int n_out, void* out, bool accumulate, int a_groups,
                  int b_groups, cudaStream_t st) {
    const auto with = [&](auto form) {
        return form(a, b, o, g, tiles, blocks, K, m_out, n_out, out, accumulate, a_groups, b_groups,
                    st);
    };
    // bf16 outputs of what is surely one chain go without the code for more: 800 rows of 8
    // experts, 512 x 512, 7.9 us, 8.3 us with it
    if constexpr (sizeof(OutT) == 2 && !kFew) {
        if (terms > (long long)kChainBlocks<OutT> * BK)
            return with(launch_form<kMode, OutT, kFew, true>);
    }
    return with(launch_form<kMode, OutT, kFew, false>);
}

// A [outer, rows, cols] matrix (outer 0: [rows, cols]) in boxes of 64 columns.
bool map_rows(CUtensorMap* m, const void* ptr, long long outer, long long rows, long long cols,
              uint32_t box_rows) {
    const uint64_t sizes[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)outer};
    const uint64_t strides[2] = {(uint64_t)cols * 2, (uint64_t)(cols * rows) * 2};
    const uint32_t box[3] = {BK, box_rows, 1};
    return map_tiled(m, outer > 0 ? 3 : 2, ptr, sizes, strides, box);
}

// The same as an MN-major operand: boxes of 64 rows, box_cols columns (64 or 128) at a
// time where cols is a multiple of 64 (*groups), else 64.
bool map_mn(CUtensorMap* m, const void* ptr, long long outer, long long rows, long long cols,
            int box_cols, int* groups) {
    *groups = cols % 64 == 0;
    if (!*groups) return map_rows(m, ptr, outer, rows, cols, BK);
    const uint64_t sizes[4] = {64, (uint64_t)rows, (uint64_t)cols / 64, (uint64_t)outer};
    const uint64_t strides[3] = {(uint64_t)cols * 2, 128, (uint64_t)(cols * rows) * 2};
    const uint32_t box[4] = {64, BK, (uint32_t)box_cols / 64, 1};
    return map_tiled(m, outer > 0 ? 4 : 3, ptr, sizes, strides, box);
}

// The output ([outer,] rows, cols) in boxes of 32 lines of 128 bytes.
bool map_lines(CUtensorMap* m, const void* ptr, long long outer, long long rows, long long cols,
               bool f32) {
    const uint64_t es = f32 ? 4 : 2;
    const uint64_t sizes[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)outer};
    const uint64_t strides[2] = {(uint64_t)cols * es, (uint64_t)(cols * rows) * es};
    const uint32_t box[3] = {(uint32_t)(128 / es), 32, 1};
    return map_tiled(m, outer > 0 ? 3 : 2, ptr, sizes, strides, box, f32);
}

moe_status launch_rows(const uint16_t* rows, const GemmGroup& g, int c_in, int c_out,
                       const uint16_t* w, void* out, bool out_f32, bool input_grad,
                       cudaStream_t st) {
    const int K = input_grad ? c_out : c_in, n_out = input_grad ? c_in : c_out;
    CUtensorMap a, b, o;
    int groups = 0;
    const long long used = g.R < g.E ? g.R : g.E;  // experts with rows, at most
    const bool few = g.R <= kFewRows * used;
    const bool ok = map_rows(&a, rows, 0, g.R, K, few ? BF / 2 : BH) &&
                    (input_grad ? map_mn(&b, w, g.E, c_out, c_in,
                                         few ? BH : box_columns(n_out, true), &groups)
                                : map_rows(&b, w, g.E, c_out, c_in,
                                           few ? BH : box_columns(n_out, false))) &&
                    (few || map_lines(&o, out, 0, g.R, n_out, out_f32));
    if (!ok) return MOE_ERR_UNSUPPORTED;
    if (few) o = a;  // not used
    // at most as many row blocks as experts with rows and whole blocks besides
    const long long tiles = (used + (g.R - used) / (few ? BF : BT)) * blocks_of(n_out, BT);
    const long long blocks = blocks_of(K, BK);
    using bf16 = __nv_bfloat16;
    const auto with = [&](auto launch) {
        return launch(a, b, o, g, tiles, blocks, K, K, 0, n_out, out, false, 0, groups, st);
    };
    if (few)
        return input_grad ? (out_f32 ? with(launch<kRowsGrad, float, true>)
                                     : with(launch<kRowsGrad, bf16, true>))
                          : (out_f32 ? with(launch<kForward, float, true>)
                                     : with(launch<kForward, bf16, true>));
    return input_grad ? (out_f32 ? with(launch<kRowsGrad, float>) : with(launch<kRowsGrad, bf16>))
                      : (out_f32 ? with(launch<kForward, float>) : with(launch<kForward, bf16>));
}

moe_status launch_weights(const uint16_t* dout, const uint16_t* rows, const GemmGroup& g, int c_in,
                          int c_out, void* dw, bool out_f32, bool accumulate, cudaStream_t st) {
    CUtensorMap a, b, o;
    int a_groups = 0, b_groups = 0;
    if (!map_mn(&a, dout, 0, g.R, c_out, BH, &a_groups) ||
        !map_mn(&b, rows, 0, g.R, c_in, box_columns(c_in, true), &b_groups) ||
        !map_lines(&o, dw, g.E, c_out, c_in, out_f32))
        return MOE_ERR_UNSUPPORTED;
    const long long tiles =
        (long long)g.E * blocks_of(c_out, BT) * blocks_of(c_in, BT);
    const long long blocks = g.R / g.E / BK;  // of an expert, on average
    const auto with = [&](auto launch) {
        return launch(a, b, o, g, tiles, blocks, g.R, 0, c_out, c_in, dw, accumulate, a_groups,
                      b_groups, st);
    };
    return out_f32 ? with(launch<kWeightsGrad, float>) : with(launch<kWeightsGrad, __nv_bfloat16>);
}

// gu (or its gradient) [N*k, 2*I] as [N*k][2][I], in boxes of 32 rows of 64 or 32 columns of a
// half.
bool map_gu(CUtensorMap* m, const void* ptr, long long R, int I, int columns) {
    const uint64_t sizes[3] = {(uint64_t)I, 2, (uint64_t)R};
    const uint64_t strides[2] = {(uint64_t)I * 2, (uint64_t)I * 4};
    const uint32_t box[3] = {(uint32_t)columns, 1, 32};
    return map_typed(m, 3, ptr, sizes, strides, box, kMapBF16, columns * 2);
}

template <int kMode, bool kFew>
moe_status launch_gated(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& o,
                        const CUtensorMap& gu, const Gate& gate, const GemmGroup& g,
                        long long tiles, int K, int I, int b_groups, cudaStream_t st) {
    if (tiles >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
    constexpr size_t smem = smem_bytes<kMode, kFew>();
    static OncePerDevice set;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    if (!set.done(dev)) {
        if (cudaFuncSetAttribute(gated_product_kernel<kMode, kFew>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem) != cudaSuccess)
            return MOE_ERR_CUDA;
        set.finish(dev);
    }
    const long long pairs_max = sm_count() / 2;
    const long long pairs = tiles < pairs_max ? tiles : pairs_max;
    return cuda_status(launch_chained(gated_product_kernel<kMode, kFew>,
                                      (int)(2 * (pairs > 0 ? pairs : 1)), kThreads, smem, st, a, b,
                                      o, gu, gate, g.offsets, g.counts, g.E, (int)g.R, K, I,
                                      b_groups, g.err, g.prefix + g.E + 1));
}

moe_status launch_gated_forward(const uint16_t* rows, const GemmGroup& g, int c_in, int I,
                                const uint16_t* w, const Gate& gate, cudaStream_t st) {
    CUtensorMap a, b, o, gu;
    const long long used = g.R < g.E ? g.R : g.E;  // experts with rows, at most
    const bool few = g.R <= kFewRows * used;
    const uint64_t sizes[4] = {(uint64_t)c_in, (uint64_t)I, 2, (uint64_t)g.E};
    const uint64_t strides[3] = {(uint64_t)c_in * 2, (uint64_t)c_in * I * 2,
                                 (uint64_t)c_in * I * 4};
    const uint32_t box[4] = {BK, (uint32_t)(few ? 64 : BH), 1, 1};
    if (!map_rows(&a, rows, 0, g.R, c_in, few ? BF / 2 : BH) ||
        !map_tiled(&b, 4, w, sizes, strides, box) || !map_lines(&o, gate.h, 0, g.R, I, false))
        return MOE_ERR_UNSUPPORTED;
    gu = o;
    if (gate.gu && !map_gu(&gu, gate.gu, g.R, I, 64)) return MOE_ERR_UNSUPPORTED;
    const long long tiles = (used + (g.R - used) / (few ? BF : BT)) * blocks_of(I, BT / 2);
    return few ? launch_gated<kGated, true>(a, b, o, gu, gate, g, tiles, c_in, I, 0, st)
               : launch_gated<kGated, false>(a, b, o, gu, gate, g, tiles, c_in, I, 0, st);
}

moe_status launch_gated_grad(const uint16_t* dout, const GemmGroup& g, int c_out, int I,
                             const uint16_t* w, const Gate& gate, float* dtopk_w,
                             cudaStream_t st) {
    CUtensorMap a, b, o, gu;
    int groups = 0;
    if (!map_rows(&a, dout, 0, g.R, c_out, BH) ||
        !map_mn(&b, w, g.E, c_out, I, box_columns(I, true), &groups) ||
        !map_gu(&gu, gate.gu_in, g.R, I, kGateCols) || !map_gu(&o, gate.gu, g.R, I, kGateCols))
        return MOE_ERR_UNSUPPORTED;
    const long long used = g.R < g.E ? g.R : g.E;
    const long long tiles = (used + (g.R - used) / BT) * blocks_of(I, BT);
    MOE_TRY(launch_gated<kGatedGrad, false>(a, b, o, gu, gate, g, tiles, c_out, I, groups, st));
    if (!dtopk_w) return MOE_OK;
    return cuda_status(launch_chained(gate_weight_grad_kernel, (int)((g.R + 255) / 256), 256, 0, st,
                                      (const float*)gate.parts, blocks_of(I, kEpilogueCols),
                                      g.offsets, g.counts, g.E, gate.pair_row, g.R, dtopk_w));
}

// Contractions up to this are one chain of an accumulator (see "Precision").
constexpr int kMaxGateTerms = kChainBlocks<__nv_bfloat16> * BK;

// Columns of gu, and so its rows' pitch, are 32 bits.
constexpr int kMaxGateColumns = 1 << 28;

size_t gated_parts_offset(const moe_shape& s) { return workspace_layout(s).total; }

moe_status check_grouped(const moe_layout* layout, const moe_shape* shape, int32_t C_in,
                         int32_t C_out, int32_t out_type, void* ws, size_t ws_bytes) {
    MOE_TRY(check_shape(shape));
    MOE_TRY(check_layout(layout, shape));
    MOE_TRY(check_ws(shape, ws, ws_bytes));
    if (((uintptr_t)ws & 3u) != 0) return MOE_ERR_INVALID_ARG;  // its words are counted in
    if (C_in <= 0 || C_out <= 0) return MOE_ERR_INVALID_ARG;
    if (C_in % 8 != 0 || C_out % 8 != 0) return MOE_ERR_UNSUPPORTED;
    // a row block's coordinates, past the last row included, are 32 bits
    if ((long long)shape->N * shape->k > INT32_MAX - (1 << 20)) return MOE_ERR_UNSUPPORTED;
    if (out_type != MOE_TYPE_BF16 && out_type != MOE_TYPE_F32) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_grouped_gemm(const uint16_t* rows, const moe_layout* layout,
                            const moe_shape* shape, int32_t C_in, int32_t C_out,
                            const uint16_t* w, void* out, int32_t out_type, void* ws,
                            size_t ws_bytes, void* stream) {
    MOE_RANGE();
    MOE_TRY(check_grouped(layout, shape, C_in, C_out, out_type, ws, ws_bytes));
    if (shape->N == 0) return MOE_OK;
    if (!rows || !w || !out) return MOE_ERR_INVALID_ARG;
    if (!aligned16(rows, w, out)) return MOE_ERR_INVALID_ARG;
    return launch_rows(rows, routed_group(*layout, *shape, ws), C_in, C_out, w, out,
                       out_type == MOE_TYPE_F32, false, as_stream(stream));
}

moe_status moe_grouped_gemm_input_grad(const uint16_t* dout, const moe_layout* layout,
                                       const moe_shape* shape, int32_t C_in, int32_t C_out,
                                       const uint16_t* w, void* drows, int32_t out_type, void* ws,
                                       size_t ws_bytes, void* stream) {
    MOE_RANGE();
    MOE_TRY(check_grouped(layout, shape, C_in, C_out, out_type, ws, ws_bytes));
    if (shape->N == 0) return MOE_OK;
    if (!dout || !w || !drows) return MOE_ERR_INVALID_ARG;
    if (!aligned16(dout, w, drows)) return MOE_ERR_INVALID_ARG;
    return launch_rows(dout, routed_group(*layout, *shape, ws), C_in, C_out, w, drows,
                       out_type == MOE_TYPE_F32, true, as_stream(stream));
}

size_t moe_gated_workspace_bytes(const moe_shape* shape) {
    if (check_shape(shape) != MOE_OK) return 0;
    return gated_parts_offset(*shape) +
           align256((size_t)shape->N * shape->k * blocks_of(shape->I, kEpilogueCols) * 4);
}

moe_status moe_gated_gemm(const uint16_t* rows, const moe_layout* layout, const moe_shape* shape,
                          int32_t C_in, const uint16_t* w_gate_up, const float* topk_w,
                          uint16_t* gu, uint16_t* h, void* ws, size_t ws_bytes, void* stream) {
    MOE_RANGE();
    MOE_TRY(check_grouped(layout, shape, C_in, 8, MOE_TYPE_BF16, ws, ws_bytes));
    if (C_in > kMaxGateTerms || shape->I > kMaxGateColumns) return MOE_ERR_UNSUPPORTED;
    if (shape->N == 0) return MOE_OK;
    if (!rows || !w_gate_up || !h) return MOE_ERR_INVALID_ARG;
    if (!aligned16(rows, w_gate_up, gu, h)) return MOE_ERR_INVALID_ARG;
    const Gate gate = {topk_w, layout->row_token, layout->pair_row, shape->N, shape->k,
                       h,      gu,                nullptr,          nullptr};
    return launch_gated_forward(rows, routed_group(*layout, *shape, ws), C_in, shape->I, w_gate_up,
                                gate, as_stream(stream));
}

moe_status moe_gated_gemm_grad(const uint16_t* dout, const moe_layout* layout,
                               const moe_shape* shape, int32_t C_out, const uint16_t* w_down,
                               const float* topk_w, const uint16_t* gu, uint16_t* dgu,
                               float* dtopk_w, void* ws, size_t ws_bytes, void* stream) {
    MOE_RANGE();
    MOE_TRY(check_grouped(layout, shape, 8, C_out, MOE_TYPE_BF16, ws, ws_bytes));
    if (ws_bytes < moe_gated_workspace_bytes(shape)) return MOE_ERR_WORKSPACE;
    if (C_out > kMaxGateTerms || shape->I > kMaxGateColumns) return MOE_ERR_UNSUPPORTED;
    if (shape->N == 0) return MOE_OK;
    if (!dout || !w_down || !gu || !dgu) return MOE_ERR_INVALID_ARG;
    if (!aligned16(dout, w_down, gu, dgu)) return MOE_ERR_INVALID_ARG;
    float* parts = dtopk_w ? ws_ptr<float>(ws, gated_parts_offset(*shape)) : nullptr;
    const Gate gate = {topk_w,  layout->row_token, layout->pair_row, shape->N, shape->k,
                       nullptr, dgu,               gu,               parts};
    return launch_gated_grad(dout, routed_group(*layout, *shape, ws), C_out, shape->I, w_down, gate,
                             dtopk_w, as_stream(stream));
}

moe_status moe_grouped_gemm_weight_grad(const uint16_t* dout, const uint16_t* rows,
                                        const moe_layout* layout, const moe_shape* shape,
                                        int32_t C_in, int32_t C_out, void* dw, int32_t out_type,
                                        int32_t accumulate, void* ws, size_t ws_bytes,
                                        void* stream) {
    MOE_RANGE();
    MOE_TRY(check_grouped(layout, shape, C_in, C_out, out_type, ws, ws_bytes));
    if (accumulate && out_type != MOE_TYPE_F32) return MOE_ERR_UNSUPPORTED;
    if (!dw || !aligned16(dw)) return MOE_ERR_INVALID_ARG;
    const bool f32 = out_type == MOE_TYPE_F32;
    if (shape->N == 0) {
        if (accumulate) return MOE_OK;
        return cuda_status(cudaMemsetAsync(
            dw, 0, (size_t)shape->E * C_out * C_in * (f32 ? 4 : 2), as_stream(stream)));
    }
    if (!dout || !rows || !aligned16(dout, rows)) return MOE_ERR_INVALID_ARG;
    return launch_weights(dout, rows, routed_group(*layout, *shape, ws), C_in, C_out, dw, f32,
                          accumulate != 0, as_stream(stream));
}

}  // extern "C"
