// Tile queues of a CTA pair, shared by the kernels that take their tiles
// dynamically (grouped_gemm_2sm.cu, grouped_products.cu).
//
// A scheduler warp of the leader takes tile indices from a global counter and
// publishes them in a ring of kQ slots in both CTAs' shared memory; the peer's
// producer forwards each tile to the peer's other warps through a second,
// CTA-local ring, so that a tile costs one cluster-scope release each way.
// Ctl is the kernel's control block with the fields tile_q, tq_full, tq_empty,
// local_q, lq_full and lq_empty, kQ slots each.
#pragma once

#include "ptx.cuh"

namespace moe {
namespace ptx {

constexpr int kQ = 8;  // slots of the tile queues

// Leader's scheduler thread: wait until queue slot i % kQ is free in both CTAs, take
// the next tile from the counter (-1 once every tile is taken) and publish it
// to both CTAs.  Returns the tile, or -2 if the wait gave up.  first: the pair's
// first tile is its own index and the counter hands out the ones after the
// `first` pairs (0: every tile comes from the counter).
template <typename Ctl>
__device__ __forceinline__ int queue_publish(Ctl* ctl, int i, int* counter, int total,
                                             volatile int* abort, int* err, int first = 0) {
    const int slot = i % kQ;
    const uint32_t ph = (uint32_t)(i / kQ) & 1u;
    if (!wait_bar(smem_u32(&ctl->tq_empty[slot]), ph ^ 1u, abort, err)) return -2;
    int t = first > 0 && i == 0 ? (int)(blockIdx.x / 2) : first + atomicAdd(counter, 1);
    if (t >= total) t = -1;
    ctl->tile_q[slot] = t;
    st_shared_cluster(mapa_shared(smem_u32(&ctl->tile_q[slot]), 1), t);
    mbar_arrive(smem_u32(&ctl->tq_full[slot]));
    // release.cluster: the store into the peer's slot is visible before its arrival
    mbar_arrive_cluster(mapa_shared(smem_u32(&ctl->tq_full[slot]), 1));
    return t;
}

// Peer's producer: forward tile t to the peer's epilogue warps (local queue).
// Returns false if the wait gave up.
template <typename Ctl>
__device__ __forceinline__ bool local_publish(Ctl* ctl, int i, int t, volatile int* abort,
                                              int* err) {
    const int slot = i % kQ;
    const uint32_t ph = (uint32_t)(i / kQ) & 1u;
    if (!wait_bar(smem_u32(&ctl->lq_empty[slot]), ph ^ 1u, abort, err)) return false;
    ctl->local_q[slot] = t;
    mbar_arrive(smem_u32(&ctl->lq_full[slot]));
    return true;
}

// Peer's epilogue warp (lane 0): the tile in local queue slot i % kQ.
template <typename Ctl>
__device__ __forceinline__ int local_take(Ctl* ctl, int i, volatile int* abort, int* err) {
    const int slot = i % kQ;
    const uint32_t ph = (uint32_t)(i / kQ) & 1u;
    if (!wait_bar(smem_u32(&ctl->lq_full[slot]), ph, abort, err)) return -2;
    const int t = *reinterpret_cast<volatile int*>(&ctl->local_q[slot]);
    mbar_arrive(smem_u32(&ctl->lq_empty[slot]));
    return t;
}

// Reader of the leader's queue (the leader's producer, MMA thread and
// epilogue warps, the peer's producer): the tile in slot i % kQ (-1: none left), after which
// the slot is released to the leader.  Returns -2 if the wait gave up.
template <typename Ctl>
__device__ __forceinline__ int queue_take(Ctl* ctl, int i, bool leader, volatile int* abort,
                                          int* err) {
    const int slot = i % kQ;
    const uint32_t ph = (uint32_t)(i / kQ) & 1u;
    const uint32_t full = smem_u32(&ctl->tq_full[slot]);
    // the peer's copy was written by the leader: acquire at cluster scope
    if (!(leader ? wait_bar(full, ph, abort, err) : wait_bar_cluster(full, ph, abort, err)))
        return -2;
    const int t = *reinterpret_cast<volatile int*>(&ctl->tile_q[slot]);
    const uint32_t empty = smem_u32(&ctl->tq_empty[slot]);
    if (leader)
        mbar_arrive(empty);
    else
        mbar_arrive_cluster(mapa_shared(empty, 0));
    return t;
}

// Spin for about `cycles` SM clocks (lets copies in flight land on abort).
__device__ __forceinline__ void spin(long long cycles) {
    const long long t0 = clock64();
    while (clock64() - t0 < cycles) {
    }
}

}  // namespace ptx
}  // namespace moe
