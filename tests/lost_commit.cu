// The linear-attention entry points with one arrival left out: a chosen
// tcgen05.commit of one CTA is not made, so that what waits for it runs into its
// time limit.  Every wait is bounded and every CTA waits, bounded too, for what it
// has in flight before it leaves.
#include "lq_umma.cuh"

namespace lq {

__device__ char lost_name[48];
__device__ int lost_block, lost_segment, lost_nth, lost_seen;

__device__ __noinline__ bool commit_is_lost(const char *name) {
    if ((int)blockIdx.x != lost_block || (int)blockIdx.y != lost_segment) return false;
    for (int i = 0; i < (int)sizeof(lost_name); ++i) {
        if (name[i] != lost_name[i]) return false;
        if (name[i] == 0) return atomicAdd(&lost_seen, 1) == lost_nth;
    }
    return false;
}

}  // namespace lq

#define umma_commit(bar) \
    do {                 \
        if (!commit_is_lost(#bar)) (umma_commit)(bar); \
    } while (0)

#include "linear.cu"

// `name`: the barrier's expression in the kernel's source; the nth commit to it
// (from 0) by the CTA at (block, segment) is left out.  "": none.
extern "C" LQ_API int lose_commit(const char *name, int block, int segment, int nth) {
    char text[48] = {};
    for (int i = 0; name[i] && i < 47; ++i) text[i] = name[i];
    const int zero = 0;
    if (cudaMemcpyToSymbol(lq::lost_name, text, sizeof text) != cudaSuccess) return 1;
    if (cudaMemcpyToSymbol(lq::lost_block, &block, 4) != cudaSuccess) return 1;
    if (cudaMemcpyToSymbol(lq::lost_segment, &segment, 4) != cudaSuccess) return 1;
    if (cudaMemcpyToSymbol(lq::lost_nth, &nth, 4) != cudaSuccess) return 1;
    return cudaMemcpyToSymbol(lq::lost_seen, &zero, 4) == cudaSuccess ? 0 : 1;
}
