// Attention over a cache of bf16 values.
#include "kv_attend.cuh"

cudaError_t moe::launch_attend_bf16(const AttendArgs& a, const AttendPlan& p, cudaStream_t st) {
    return launch_attend_type<0>(a, p, st);
}
