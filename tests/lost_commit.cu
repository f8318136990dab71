// The linear-attention entry points with one arrival left out: a chosen
// tcgen05.commit of one CTA is not made, a flag that nothing sets, so that what waits
// for it runs into its limit of a second and the status is seen.  Nothing else
// changes, so every access is one that the whole kernel makes: a role that gives up
// leaves before it reads or writes anything behind the wait, without an arrival, so
// no other role goes on to operands or chunk descriptions that are not there.  Every
// wait ends: those of the roles and those for loads and commits in flight, all
// through mbar_wait_bounded, then the block's barrier, which every warp reaches.  The
// products whose commit is left out were issued a second earlier, and the next commit
// of the same thread, where there is one, covers them before tensor memory is freed.
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
