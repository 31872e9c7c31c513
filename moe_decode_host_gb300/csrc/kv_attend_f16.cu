// Attention over a cache of f16 values.
#include "kv_attend.cuh"

cudaError_t moe::launch_attend_f16(const AttendArgs& a, const AttendPlan& p, cudaStream_t st) {
    return launch_attend_type<1>(a, p, st);
}
