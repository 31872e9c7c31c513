// Attention over a cache of E4M3 values with a scale for each block of tokens and head.
#include "kv_attend.cuh"

cudaError_t moe::launch_attend_e4m3_blocks(const AttendArgs& a, const AttendPlan& p, cudaStream_t st) {
    return launch_attend_type<3>(a, p, st);
}
