// lq_host.cuh -- host-side helpers shared by the library's sources: argument
// checks, launch attributes and grid sizes.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>
#include <utility>
#include <vector>

#include "lq_common.cuh"

namespace lq {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline lq_status check_config(const lq_config *c) {
    if (!c) return LQ_ERR_INVALID_ARG;
    if (c->num_slots <= 0 || c->num_heads <= 0 || c->dk <= 0 || c->dv <= 0 || c->window <= 0 ||
        c->num_comp < 0)
        return LQ_ERR_INVALID_ARG;
    if ((c->decay_kind | c->scale_dtype | c->smoothing | c->in_dtype | c->per_step) & ~1)
        return LQ_ERR_INVALID_ARG;
    if (c->per_step ? (c->bits != 8 && c->bits != 16)
                    : (c->bits != 4 && c->bits != 6 && c->bits != 8 && c->bits != 32))
        return LQ_ERR_INVALID_ARG;
    if ((int64_t)c->num_slots * c->num_heads > 0x7FFFFFFF) return LQ_ERR_UNSUPPORTED;
    if (c->dk != c->dv || (c->dk != 64 && c->dk != 128)) return LQ_ERR_UNSUPPORTED;
    if (c->window > kMaxWindow || c->num_comp > kMaxComp) return LQ_ERR_UNSUPPORTED;
    return LQ_OK;
}

inline Flags make_flags(const lq_config &c) {
    return Flags{c.decay_kind, c.scale_dtype, c.in_dtype, c.smoothing, c.window, c.num_comp};
}

// Allow a kernel more than 48 KB of dynamic shared memory (once per kernel
// and device).
struct SmemGrant {
    int dev;
    const void *fn;
    uint32_t bytes;
};

template <typename K>
cudaError_t allow_smem(K kernel, uint32_t bytes) {
    static std::mutex mu;
    static std::vector<SmemGrant> done;
    if (bytes <= 48u * 1024u) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const void *fn = reinterpret_cast<const void *>(kernel);
    std::lock_guard<std::mutex> lock(mu);
    for (const SmemGrant &g : done)
        if (g.dev == dev && g.fn == fn && g.bytes >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.push_back({dev, fn, bytes});
    return e;
}

// Launch with programmatic stream serialization: the kernel may start while
// the previous kernel on the stream drains; it waits for that kernel's
// completion (pdl_wait) before its first global-memory access.  `cluster`:
// CTAs of a thread-block cluster along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, int threads, int cluster, uint32_t smem, cudaStream_t s,
                       Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), int grid, int threads, uint32_t smem, cudaStream_t s, Args &&...args) {
    return launch_pdl(kernel, dim3((unsigned)grid), threads, 1, smem, s, std::forward<Args>(args)...);
}

inline lq_status launched(cudaError_t e) {
    if (e != cudaSuccess) return LQ_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? LQ_OK : LQ_ERR_CUDA;
}

// Persistent grid: as many CTAs as fit on the device at once, each walking
// a strided list of (slot, head) blobs.
template <typename K>
int persistent_grid(K kernel, int threads, uint32_t smem, int work) {
    static std::mutex mu;
    static std::vector<std::pair<std::pair<const void *, uint32_t>, int>> cache;
    const void *fn = reinterpret_cast<const void *>(kernel);
    int per_sm = 0, sms = 0, dev = 0;
    {
        std::lock_guard<std::mutex> lock(mu);
        for (auto &e : cache)
            if (e.first.first == fn && e.first.second == smem) per_sm = e.second;
    }
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return -1;
    if (per_sm == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess)
            return -1;
        if (per_sm < 1) per_sm = 1;
        std::lock_guard<std::mutex> lock(mu);
        cache.push_back({{fn, smem}, per_sm});
    }
    const long cap = (long)sms * per_sm;
    return (int)(work < cap ? work : cap);
}

}  // namespace lq
