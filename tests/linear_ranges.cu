// Host access to the index arithmetic of the linear-attention kernels.
#include "lq_linear.cuh"

extern "C" LQ_API int host_lin_stop(int run, int len, int t_begin, int t_end) {
    return lq::lin_stop(run != 0, len, t_begin, t_end);
}
