// Attention over a cache of E4M3 values.
#include "kv_attend.cuh"

cudaError_t moe::launch_attend_e4m3(const AttendArgs& a, const AttendPlan& p, cudaStream_t st) {
    return launch_attend_type<2>(a, p, st);
}
