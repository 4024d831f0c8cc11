// Argument checks and small helpers shared by the files that hold the C ABI's
// entry points (moe_api.cu and the training operators).
#pragma once

#include <nvtx3/nvToolsExt.h>

#include <atomic>

#include "moe_internal.cuh"

namespace moe {

inline moe_status check_shape(const moe_shape* s) {
    if (!s) return MOE_ERR_INVALID_ARG;
    if (s->N < 0 || s->H <= 0 || s->E <= 0 || s->k <= 0 || s->W <= 0 || s->I <= 0)
        return MOE_ERR_INVALID_ARG;
    if (s->k > s->E || s->E % s->W != 0) return MOE_ERR_INVALID_ARG;
    if (s->E > kMaxE || s->k > kMaxK) return MOE_ERR_UNSUPPORTED;
    if (s->H % 8 != 0 || s->I % 8 != 0) return MOE_ERR_UNSUPPORTED;
    if ((long long)s->N * s->k >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
    if (s->gemm != MOE_GEMM_AUTO && s->gemm != MOE_GEMM_SINGLE_CTA &&
        s->gemm != MOE_GEMM_CTA_PAIR && s->gemm != MOE_GEMM_FUSED)
        return MOE_ERR_INVALID_ARG;
    if (s->gemm == MOE_GEMM_FUSED && !fused_ffn_supported(s->H)) return MOE_ERR_UNSUPPORTED;
    if (s->weights != MOE_WEIGHTS_ROW_MAJOR && s->weights != MOE_WEIGHTS_PACKED)
        return MOE_ERR_INVALID_ARG;
    // the GEMMs address packed rows with 32-bit TMA coordinates
    if (s->weights == MOE_WEIGHTS_PACKED &&
        (packed_gate_up_rows(*s) >= (1LL << 31) || packed_down_rows(*s) >= (1LL << 31)))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// w_up is read only in the row-major layout (the packed gate/up weights hold both).
inline bool up_given(const moe_shape* s, const uint16_t* w_up) {
    return w_up != nullptr || s->weights == MOE_WEIGHTS_PACKED;
}

inline moe_status check_layout(const moe_layout* L, const moe_shape* s) {
    if (!L) return MOE_ERR_INVALID_ARG;
    if (!L->expert_counts || !L->expert_offsets || !L->rank_offsets || !L->row_token ||
        !L->pair_row)
        return MOE_ERR_INVALID_ARG;
    if (s->dedup && (!L->dedup_counts || !L->dedup_offsets || !L->dedup_row_token ||
                     !L->pair_dedup_row || !L->expand_src || !L->n_dedup_rows))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

inline moe_status check_ws(const moe_shape* s, void* ws, size_t ws_bytes) {
    if (!ws || ws_bytes < workspace_layout(*s).total) return MOE_ERR_WORKSPACE;
    return MOE_OK;
}

inline moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// The routed experts' GEMM problem: the plain expert-major rows of the layout.
inline GemmGroup routed_group(const moe_layout& L, const moe_shape& s, void* ws) {
    const Workspace wl = workspace_layout(s);
    return GemmGroup{L.expert_counts, L.expert_offsets, s.E, (long long)s.N * s.k,
                     ws_ptr<int32_t>(ws, wl.mblk_prefix), ws_ptr<int>(ws, wl.err),
                     s.weights == MOE_WEIGHTS_PACKED};
}

inline cudaStream_t as_stream(void* p) { return reinterpret_cast<cudaStream_t>(p); }

// The kernels move bf16 rows (and the fp32 accumulator) in 16-byte vectors,
// by TMA, cp.async or plain vector loads: a base address that is not 16-byte
// aligned is refused here instead of faulting on the device.  NULL passes
// (whether NULL is allowed is checked separately).
template <typename... T>
inline bool aligned16(const T*... p) {
    return ((((uintptr_t)p & 15u) == 0) && ...);
}

// An NVTX range named after the entry point around every call that enqueues
// work: profilers (Nsight Systems, ncu's NVTX filters) show the C ABI calls on
// the timeline.  With no tool attached a push/pop is a check of one function
// pointer.
struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

// Whether what a call sets up once for each device (function attributes, figures kept
// beside this) is set up.  Several host threads may make their first call together: each
// of them then does the set-up, to the same end, and a thread that sees another's finish()
// sees what that one has stored before.
constexpr int kMaxDevices = 64;
class OncePerDevice {
  public:
    bool done(int dev) const {
        return dev < kMaxDevices && done_[dev].load(std::memory_order_acquire);
    }
    void finish(int dev) {
        if (dev < kMaxDevices) done_[dev].store(true, std::memory_order_release);
    }

  private:
    std::atomic<bool> done_[kMaxDevices] = {};
};

// Launches a kernel whose blocks call after_previous(), in clusters of `cluster` blocks
// (0: as the kernel says).
template <typename... P, typename... A>
inline cudaError_t launch_chained_clusters(void (*kernel)(P...), int cluster, dim3 grid, int block,
                                           size_t smem, cudaStream_t st, const A&... args) {
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = cluster;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attrs;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
template <typename... P, typename... A>
inline cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, int block, size_t smem,
                                  cudaStream_t st, const A&... args) {
    return launch_chained_clusters(kernel, 0, grid, block, smem, st, args...);
}

#define MOE_RANGE() const NvtxRange _moe_nvtx_range(__func__)

#define MOE_TRY(...)                        \
    do {                                    \
        const moe_status _st = (__VA_ARGS__); \
        if (_st != MOE_OK) return _st;    \
    } while (0)

}  // namespace moe
