// Products of few rows with matrices of 4-bit weights: the experts of a decoding step.
//
//   y[i, o] = sum over k of rows[i, k] * scale[e][o, k / group] * (q[e][o, k] - 8)
//
// with q in 0..15 and a scale for `group` weights of a matrix row; gated: the matrix holds I
// gate rows and I up rows, and h = w_i SiLU(g) u leaves instead of y.
//
// Memory bound: every weight is read once, 4 bits and its share of a scale.  So the packed
// layout (pack_kernel) is the order in which the kernel reads: tiles of 256 matrix rows, in
// chunks of 128 weights of each row, one chunk of a tile a contiguous piece of 17 to 18 KB that
// one bulk copy brings into a ring of shared memory, the scales beside the weights.  The rows'
// chunks come by TMA boxes of 8 rows.  A chunk's work: a warp has 32 rows of the matrix, whose
// weights become bf16 operands of mma.sync m16n8k16 in registers (q | 0x4300 is the number 128 +
// q, less 136: exact), the rows being its 8 columns; a group's products are summed in fp32 and
// then scaled once, in fp32.  tcgen05 would need the weights as bf16 in shared memory, four
// times the bytes that arrive, for MMAs of 8 columns.
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

constexpr int kSlabRows = 32;      // matrix rows of a warp
constexpr int kSlabs = 8;          // warps' slabs of a tile
constexpr int kChunk = 128;        // weights of a row in a chunk
constexpr int kNibbleBytes = kSlabRows * kChunk / 2;
constexpr int kConsumers = kSlabs * 32;
constexpr int kThreads = kConsumers + 32;
constexpr int kMaxBlocks = 304;

__host__ __device__ __forceinline__ int ceil_div(long long a, int b) {
    return (int)((a + b - 1) / b);
}
// A slab's chunk: nibbles, then its scales.
__host__ __device__ __forceinline__ int record_bytes(int group) {
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

// Byte offset of a tile's chunk within an expert's packed matrix; the slabs of a tile's chunk
// lie side by side.
__host__ __device__ __forceinline__ int tile_slabs(const Matrix& m, int tile) {
    return m.slabs - tile * kSlabs < kSlabs ? m.slabs - tile * kSlabs : kSlabs;
}
__host__ __device__ __forceinline__ long long chunk_at(const Matrix& m, int tile, int chunk) {
    return ((long long)tile * kSlabs * m.chunks + (long long)chunk * tile_slabs(m, tile)) * m.record;
}

// The matrix row of a slab's row r (0..31), or -1.  A lane of the MMA holds rows l / 4 and l / 4
// + 8 of two 16-row operands: those four are neighbours in the output, or two gate columns and
// their up columns (`up`: whether it is one of these).
__device__ __forceinline__ int matrix_row(const Matrix& m, int slab, int r, bool* up) {
    const int g = r & 7, which = r >> 3;  // which: 0, 1 first operand, 2, 3 second
    int o;
    if (m.gated) {
        o = slab * 16 + 2 * g + (which & 1);
        *up = which >= 2;
    } else {
        o = slab * 32 + 4 * g + which;
        *up = false;
    }
    return o < m.rows ? o : -1;
}

// Weight j (0..3) of MMA step s (0..3) that the lanes l with l % 4 == c hold, within a half
// chunk of 64: 16 neighbours a lane, or 8 of each group of 32.
__device__ __forceinline__ int weight_of(int group, int c, int s, int j) {
    return group == 32 ? (s >> 1) * 32 + c * 8 + (s & 1) * 4 + j : c * 16 + s * 4 + j;
}

// ---- the product ---------------------------------------------------------------------------

template <int kNT>
constexpr int kStagesOf = kNT == 1 ? 5 : kNT == 2 ? 4 : kNT == 4 ? 3 : 5;
template <int kNT>
constexpr int kBlocksPerSm = kNT <= 4 ? 2 : 1;
constexpr int kMaxRecord = kNibbleBytes + kSlabRows * 2 * 4;
constexpr int kWeightBytes = kSlabs * kMaxRecord;
// the rows' boxes of a stage: two halves of 64 columns, 8 * kNT rows of 128 bytes
template <int kNT>
constexpr int kRowBytes = 2 * kNT * 1024;
template <int kNT>
constexpr size_t smem_bytes(int E) {
    return 1024 + (size_t)kStagesOf<kNT> * (kWeightBytes + kRowBytes<kNT>) +
           (size_t)(E + 1) * sizeof(long long);
}

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
    int* counters;   // arrivals at a tile, one of each block's
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

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight nibbles to an operand: nibble r and nibble r + 4 are the halves of register r.
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&a)[4]) {
    const __nv_bfloat162 bias = __float2bfloat162_rn(136.0f);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const uint32_t v = ((w >> (4 * r)) & 0x000f000fu) | 0x43004300u;
        const __nv_bfloat162 x = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), bias);
        a[r] = *reinterpret_cast<const uint32_t*>(&x);
    }
}

// A run of chunks of one tile for up to 8 * kNT rows of an expert.
struct Piece {
    int e, tile, first_row, rows;  // rows from first_row of the expert's on
    int chunk0, chunk1;            // of the tile's chunks
    long long start;               // the tile's first unit
};

// Units are chunks: expert by expert, tile by tile, the passes over 8 * kNT rows each side by
// side (they read the same weights), chunk by chunk.
template <int kNT>
__device__ __forceinline__ Piece piece_at(const Args& a, const long long* prefix, long long u,
                                          long long end) {
    int lo = 0, hi = a.E;  // prefix[lo] <= u < prefix[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= u) lo = mid;
        else hi = mid;
    }
    Piece p;
    p.e = lo;
    const long long local = u - prefix[lo];
    const int cnt = a.counts[lo], passes = ceil_div(cnt, 8 * kNT);
    const long long run = local / a.m.chunks;  // tile * passes + pass
    p.chunk0 = (int)(local - run * a.m.chunks);
    p.tile = (int)(run / passes);
    const int pass = (int)(run - (long long)p.tile * passes);
    p.first_row = pass * 8 * kNT;
    p.rows = cnt - p.first_row < 8 * kNT ? cnt - p.first_row : 8 * kNT;
    p.start = u - p.chunk0;
    const long long left = end - u;
    p.chunk1 = left < a.m.chunks - p.chunk0 ? p.chunk0 + (int)left : a.m.chunks;
    return p;
}

// The unit at which block b's share starts.
__device__ __forceinline__ long long share(long long total, int b, int blocks) {
    return total * b / blocks;
}

template <int kNT>
struct Sums {
    float v[kNT][2][4];
};

// The sums of a tile's slab to their output.  w: the routing weights of rows `lane` and lane + 32.
template <int kNT, bool kGated>
__device__ __forceinline__ void write_out(const Args& a, const Piece& p, int slab,
                                          const Sums<kNT>& s, const float (&w)[2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const long long row0 = (long long)a.offsets[p.e] + p.first_row;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int n = nt * 8 + c * 2 + j;
            const float wn = __shfl_sync(0xffffffffu, w[nt / 4], n & 31);
            if (n >= p.rows) continue;
            // the lane's four matrix rows for this row
            const float v0 = s.v[nt][0][j], v1 = s.v[nt][0][2 + j];
            const float v2 = s.v[nt][1][j], v3 = s.v[nt][1][2 + j];
            const long long at = (row0 + n) * a.m.rows;
            if (kGated) {
                const int o = slab * 16 + 2 * g;
                if (o < a.m.rows)
                    *reinterpret_cast<uint32_t*>(a.gate.h + at + o) =
                        pack2(wn * (v0 * sigmoid(v0)) * v2, wn * (v1 * sigmoid(v1)) * v3);
            } else {
                const int o = slab * 32 + 4 * g;
                if (o >= a.m.rows) continue;
                if (a.out_f32)
                    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + o) =
                        make_float4(v0, v1, v2, v3);
                else
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at + o) =
                        make_uint2(pack2(v0, v1), pack2(v2, v3));
            }
        }
    }
}

__device__ __forceinline__ void consumers_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
}

// Each block takes an equal share of the units, whatever tiles they belong to.  A tile that
// several blocks share: each leaves its sums in a slot of the workspace, and the one that comes
// last adds them up in the order of the blocks and writes the tile out.  Nobody waits.
template <int kNT, int kGroup, bool kGated>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm<kNT>)
    w4_kernel(const __grid_constant__ CUtensorMap tmRows, const __grid_constant__ Args a) {
    constexpr int kStages = kStagesOf<kNT>;
    constexpr int kStageBytes = kWeightBytes + kRowBytes<kNT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ long long run_sums[kThreads / 32];
    __shared__ int abort_word, arrived;
    uint8_t* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    long long* prefix = reinterpret_cast<long long*>(ring + (size_t)kStages * kStageBytes);
    volatile int* abort_flag = &abort_word;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&empty[i]), kSlabs);
        }
        abort_word = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x == kConsumers) prefetch_map(&tmRows);
    after_previous();
    // prefix[e]: units before expert e; each thread sums a run of experts
    const int per = ceil_div(a.E, kThreads), e0 = threadIdx.x * per;
    const long long pass_units = (long long)a.m.tiles * a.m.chunks;
    long long mine = 0;
    const auto units = [&](int e) -> long long {
        const int off = a.offsets[e], cnt = a.counts[e];
        if (off < 0 || cnt < 0 || cnt > a.R || off > a.R - cnt) {
            set_error(a.err, MOE_ERR_INVALID_ARG);
            return 0;
        }
        return ceil_div(cnt, 8 * kNT) * pass_units;
    };
    for (int e = e0; e < e0 + per && e < a.E; ++e) mine += units(e);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) run_sums[warp] = incl;
    __syncthreads();
    long long before = incl - mine;
    for (int i = 0; i < warp; ++i) before += run_sums[i];
    for (int e = e0; e < e0 + per && e < a.E; ++e) {
        prefix[e] = before;
        before += units(e);
    }
    long long total = 0;
    for (int i = 0; i < kThreads / 32; ++i) total += run_sums[i];
    if (threadIdx.x == 0) prefix[a.E] = total;
    __syncthreads();
    // no block without a unit: those of a tile are all that arrive at its counter
    const int blocks = total < (long long)gridDim.x ? (int)total : (int)gridDim.x;
    const int block = (int)blockIdx.x;
    if (block >= blocks) return;
    const long long first = share(total, block, blocks), last = share(total, block + 1, blocks);

    if (warp == kSlabs) {
        // ---------------- producer ----------------
        if (lane != 0) return;
        int stage = 0;
        uint32_t phase = 0;
        for (long long u = first; u < last;) {
            const Piece p = piece_at<kNT>(a, prefix, u, last);
            const uint8_t* from = a.packed + (long long)p.e * a.expert_bytes;
            const int slabs = tile_slabs(a.m, p.tile), boxes = ceil_div(p.rows, 8);
            const int row = a.offsets[p.e] + p.first_row;
            const uint32_t weights = (uint32_t)(slabs * a.m.record);
            for (int c = p.chunk0; c < p.chunk1; ++c) {
                if (!wait_bar(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, a.err)) {
                    // let the copies in flight land before the block exits
                    const long long t0 = clock64();
                    while (clock64() - t0 < 4000000) {
                    }
                    return;
                }
                const uint32_t bar = smem_u32(&full[stage]);
                const uint32_t to = smem_u32(ring) + (uint32_t)(stage * kStageBytes);
                mbar_expect_tx(bar, weights + (uint32_t)(boxes * 2048));
                bulk_load(to + kRowBytes<kNT>, from + chunk_at(a.m, p.tile, c), weights, bar);
                for (int b = 0; b < boxes; ++b) {
                    tma_load_2d(to + b * 1024, &tmRows, bar, c * kChunk, row + b * 8);
                    tma_load_2d(to + (kNT + b) * 1024, &tmRows, bar, c * kChunk + 64, row + b * 8);
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            u += p.chunk1 - p.chunk0;
        }
        return;
    }
    // ---------------- consumers ----------------
    // One whose wait gives up goes on without its products: the others' barriers need it.
    bool alive = true;
    int stage = 0;
    uint32_t phase = 0;
    const int n = lane >> 2, c4 = lane & 3;
    for (long long u = first; u < last;) {
        const Piece p = piece_at<kNT>(a, prefix, u, last);
        const bool has = warp < tile_slabs(a.m, p.tile);
        const int slab = p.tile * kSlabs + warp, boxes = ceil_div(p.rows, 8);
        float w[2] = {0.0f, 0.0f};
        if (kGated) {
            const long long row = (long long)a.offsets[p.e] + p.first_row;
            if (lane < p.rows) w[0] = row_weight(a.gate, row + lane);
            if (kNT > 4 && lane + 32 < p.rows) w[1] = row_weight(a.gate, row + lane + 32);
        }
        Sums<kNT> sums = {};
        for (int c = p.chunk0; c < p.chunk1; ++c) {
            if (alive && !wait_bar(smem_u32(&full[stage]), phase, abort_flag, a.err)) alive = false;
            alive = __all_sync(0xffffffffu, alive);
            if (has && alive) {
                const uint8_t* rows = ring + (size_t)stage * kStageBytes;
                const uint8_t* rec = rows + kRowBytes<kNT> + warp * a.m.record;
                float part[kNT][2][4];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t q[2][4];
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        const uint4 v = *reinterpret_cast<const uint4*>(
                            rec + (hh * 2 + mt) * 512 + lane * 16);
                        q[mt][0] = v.x, q[mt][1] = v.y, q[mt][2] = v.z, q[mt][3] = v.w;
                    }
#pragma unroll
                    for (int sp = 0; sp < 2; ++sp) {
                        uint32_t x[2][2][4];  // steps 2 sp and 2 sp + 1, both operands
#pragma unroll
                        for (int s = 0; s < 2; ++s)
#pragma unroll
                            for (int mt = 0; mt < 2; ++mt) widen(q[mt][sp * 2 + s], x[s][mt]);
                        constexpr int kPairs = kChunk / kGroup;  // groups of a chunk
                        const bool starts = kPairs == 4 || (kPairs == 2 && sp == 0) ||
                                            (kPairs == 1 && sp == 0 && hh == 0);
                        const bool ends = kPairs == 4 || (kPairs == 2 && sp == 1) ||
                                          (kPairs == 1 && sp == 1 && hh == 1);
                        const int gi = kPairs == 4 ? hh * 2 + sp : kPairs == 2 ? hh : 0;
                        float4 scale;
                        if (ends) {
                            const uint2 v = *reinterpret_cast<const uint2*>(
                                rec + kNibbleBytes + gi * 64 + n * 8);
                            scale = make_float4(__uint_as_float(v.x << 16),
                                                __uint_as_float(v.x & 0xffff0000u),
                                                __uint_as_float(v.y << 16),
                                                __uint_as_float(v.y & 0xffff0000u));
                        }
                        const int piece = kGroup == 32 ? sp * 4 + c4 : c4 * 2 + sp;
                        const uint8_t* at = rows + hh * kNT * 1024 + n * 128 + ((piece ^ n) << 4);
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt) {
                            if (nt < boxes) {
                                const uint4 b = *reinterpret_cast<const uint4*>(at + nt * 1024);
                                if (starts) {
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        part[nt][0][i] = part[nt][1][i] = 0.0f;
                                }
                                mma_16816(part[nt][0], x[0][0], b.x, b.y);
                                mma_16816(part[nt][1], x[0][1], b.x, b.y);
                                mma_16816(part[nt][0], x[1][0], b.z, b.w);
                                mma_16816(part[nt][1], x[1][1], b.z, b.w);
                                if (ends) {
                                    float (&t)[2][4] = sums.v[nt];
#pragma unroll
                                    for (int i = 0; i < 2; ++i) {
                                        t[0][i] = fmaf(scale.x, part[nt][0][i], t[0][i]);
                                        t[0][2 + i] = fmaf(scale.y, part[nt][0][2 + i], t[0][2 + i]);
                                        t[1][i] = fmaf(scale.z, part[nt][1][i], t[1][i]);
                                        t[1][2 + i] = fmaf(scale.w, part[nt][1][2 + i], t[1][2 + i]);
                                    }
                                }
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&empty[stage]));
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        u += p.chunk1 - p.chunk0;
        if (p.chunk0 == 0 && p.chunk1 == a.m.chunks) {
            if (has) write_out<kNT, kGated>(a, p, slab, sums, w);
            continue;
        }
        // a tile of several blocks: those with units of [p.start, p.start + chunks)
        constexpr long long kSlot = (long long)kConsumers * kNT * 8;
        const long long tile_end = p.start + a.m.chunks;
        int owner = block, after = block;  // the first of them, the last
        while (share(total, owner, blocks) > p.start) --owner;
        while (share(total, after + 1, blocks) < tile_end) ++after;
        const auto slot = [&](int b) {
            const int s = b == owner && share(total, b, blocks) != p.start ? 1 : 0;
            return a.parts + ((long long)b * 2 + s) * kSlot + warp * (kNT * 8 * 32) + lane;
        };
        float* to = slot(block);
#pragma unroll
        for (int i = 0; i < kNT * 8; ++i)
            if (i / 8 < boxes) __stcg(to + i * 32, sums.v[i / 8][i / 4 % 2][i % 4]);
        __threadfence();
        consumers_sync();
        if (threadIdx.x == 0) {
            const int before_me = atomicAdd(a.counters + owner, 1);
            arrived = before_me;
            if (before_me == after - owner) a.counters[owner] = 0;  // the last: for the next call
            __threadfence();
        }
        consumers_sync();
        const bool finish = arrived == after - owner;
        consumers_sync();  // read before the next tile's
        if (finish && has) {
            __threadfence();
            Sums<kNT> all = {};
            for (int b = owner; b <= after; ++b) {
                const float* from = slot(b);
#pragma unroll
                for (int i = 0; i < kNT * 8; ++i)
                    if (i / 8 < boxes) all.v[i / 8][i / 4 % 2][i % 4] += __ldcg(from + i * 32);
            }
            write_out<kNT, kGated>(a, p, slab, all, w);
        }
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

// 16 bytes of the packed form a thread: 32 nibbles of a lane, or 8 scales.  Rows and columns
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
            const int hh = at >> 6, mt = at >> 5 & 1, lane = at & 31;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int r = matrix_row(m, slab, mt * 16 + half * 8 + (lane >> 2), &up);
                const uint8_t* from =
                    q + ((e * all_rows + (up ? m.rows : 0) + r) * (long long)m.C_in) / 2;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int k = chunk * kChunk + hh * 64 + weight_of(m.group, lane & 3, s, j);
                        uint32_t v = 8;
                        if (r >= 0 && k < m.C_in) v = (uint32_t)(from[k >> 1] >> (k % 2 * 4)) & 15u;
                        // register half + 2 (j / 2) of the operand, its low or high half
                        o[s] |= v << (4 * (half + 2 * (j >> 1) + 4 * (j & 1)));
                    }
                }
            }
        } else {
            const int first = (at - nibble_pieces) * 8;  // scale of [group][row / 4 of the lane][4]
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int s = first + j, gi = s >> 5, g = s >> 2 & 7, which = s & 3;
                const int r = matrix_row(m, slab, which * 8 + g, &up);
                const int grp = chunk * (kChunk / m.group) + gi;
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

// Boxes of 8 rows of a pass: enough for most experts' rows at once when they are spread as by
// chance around their average.
int boxes_of(long long R, int E) {
    const long long used = R < E ? R : E;
    const double mean = used > 0 ? (double)R / (double)used : 0.0;
    return mean <= 4.0 ? 1 : mean <= 10.0 ? 2 : mean <= 24.0 ? 4 : 8;
}

struct W4Work {
    size_t counters, parts, total;
};
W4Work w4_work(const moe_shape& s) {
    W4Work w;
    w.counters = workspace_layout(s).total;
    w.parts = w.counters + align256(kMaxBlocks * sizeof(int));
    w.total = w.parts + (size_t)kMaxBlocks * 2 * kConsumers * 8 * sizeof(float) *
                            boxes_of((long long)s.N * s.k, s.E);
    return w;
}

bool valid(const moe_w4_matrix* m) {
    return m && m->C_out > 0 && m->C_in > 0 &&
           (m->group == 32 || m->group == 64 || m->group == 128);
}
bool supported(const moe_w4_matrix* m) { return m->C_out % 8 == 0 && m->C_in % m->group == 0; }

long long packed_bytes(const moe_w4_matrix& m, int E) {
    const Matrix d = matrix_of(m);
    return (long long)E * d.slabs * d.chunks * d.record;
}

template <int kNT, int kGroup, bool kGated>
moe_status launch_as(const CUtensorMap& rows, const Args& a, long long units, cudaStream_t st) {
    const auto kernel = w4_kernel<kNT, kGroup, kGated>;
    static OncePerDevice set;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    if (!set.done(dev)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem_bytes<kNT>(kMaxE)) != cudaSuccess)
            return MOE_ERR_CUDA;
        set.finish(dev);
    }
    long long blocks = (long long)sm_count() * kBlocksPerSm<kNT>;
    if (blocks > kMaxBlocks) blocks = kMaxBlocks;
    if (blocks > units) blocks = units;
    return cuda_status(
        launch_chained(kernel, (int)blocks, kThreads, smem_bytes<kNT>(a.E), st, rows, a));
}

template <int kNT>
moe_status launch_w4(const CUtensorMap& rows, const Args& a, long long units, cudaStream_t st) {
    const bool gated = a.m.gated != 0;
    switch (a.m.group) {
        case 32:
            return gated ? launch_as<kNT, 32, true>(rows, a, units, st)
                         : launch_as<kNT, 32, false>(rows, a, units, st);
        case 64:
            return gated ? launch_as<kNT, 64, true>(rows, a, units, st)
                         : launch_as<kNT, 64, false>(rows, a, units, st);
        default:
            return gated ? launch_as<kNT, 128, true>(rows, a, units, st)
                         : launch_as<kNT, 128, false>(rows, a, units, st);
    }
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
    if (R > INT32_MAX - (1 << 20)) return MOE_ERR_UNSUPPORTED;
    if (R == 0) return MOE_OK;
    if (!rows || !packed || !out || !aligned16(rows, packed, out)) return MOE_ERR_INVALID_ARG;
    const GemmGroup g = routed_group(*layout, *shape, ws);
    Args a = {};
    a.packed = static_cast<const uint8_t*>(packed);
    a.m = matrix_of(*matrix);
    a.expert_bytes = (long long)a.m.slabs * a.m.chunks * a.m.record;
    a.gate = Gate{topk_w,  layout->row_token, layout->pair_row, shape->N, shape->k,
                  gated ? static_cast<uint16_t*>(out) : nullptr, nullptr, nullptr};
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
    const int nt = boxes_of(R, g.E);
    const long long used = R < g.E ? R : g.E;
    const long long units = (used + (R - used) / (8 * nt)) * a.m.tiles * a.m.chunks;
    const cudaStream_t st = as_stream(stream);
    return nt == 1   ? launch_w4<1>(map, a, units, st)
           : nt == 2 ? launch_w4<2>(map, a, units, st)
           : nt == 4 ? launch_w4<4>(map, a, units, st)
                     : launch_w4<8>(map, a, units, st);
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
    if (!q || !scales || !packed || !aligned16(q, scales, packed)) return MOE_ERR_INVALID_ARG;
    const long long pieces = packed_bytes(*matrix, E) / 16;
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
