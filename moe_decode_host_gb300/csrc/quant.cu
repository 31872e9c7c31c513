// Rows to E4M3 with one scale for each 128 elements.
//
//   s = max(max |x| / 448, 2^-126) over a group,  y = E4M3(x / s)
//
// Memory bound: each element once in and once out.  A half warp holds a group, 8 elements a
// lane, so that its maximum takes four exchanges and no shared memory; a half warp takes
// several groups so that their loads are in flight together.
//
// Measured on a GB300: 8192 x 4096 bf16 21.0 us (4.8 TB/s, 72% of a plain copy's rate), 512 x 4096 2.3, 777 x 5003
// fp32 at any alignment 5.5 (3.6 TB/s), 8 x 4096 1.3.
#include <algorithm>

#include "ptx.cuh"
#include "vec.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr float kE4M3Max = 448.f;

// The scale of a group with largest magnitude `top`, and the factor of its elements.  A NaN or
// an infinity among them: both NaN.
__device__ __forceinline__ float scale_of(float top, float& factor) {
    const float m = top < INFINITY ? top : __uint_as_float(0x7fc00000u);
    const float scale = m * (1.f / kE4M3Max);
    const bool floor = scale < 1.17549435e-38f;  // 2^-126; false for NaN
    factor = floor ? 8.50705917e+37f : kE4M3Max / m;
    return floor ? 1.17549435e-38f : scale;
}

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Group i of all: its row and its number there.
__device__ __forceinline__ int64_t row_of(int64_t i, int groups, int& g) {
    const int64_t row = i >> 32 ? i / groups : (int64_t)((uint32_t)i / (uint32_t)groups);
    g = (int)(i - row * groups);
    return row;
}

// Rows whose runs of 8 are aligned and whole.  U groups a half warp.
template <int XT, int U>
__global__ void __launch_bounds__(kThreads) quant_kernel(const QuantArgs a, int groups, int64_t total) {
    grid_launch_next();
    grid_dep_wait();
    const int half = threadIdx.x >> 4, lane = threadIdx.x & 15;
    const int64_t first = (int64_t)blockIdx.x * (kThreads / 16 * U) + half;
    Raw<8, XT == MOE_F32> r[U];
    int64_t row[U];
    int g[U];
    bool in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * (kThreads / 16);
        if (u == 0 || groups < kThreads / 16) {
            row[u] = row_of(i, groups, g[u]);
        } else {  // at most one row further
            const int next = g[u - 1] + kThreads / 16;
            row[u] = row[u - 1] + (next >= groups);
            g[u] = next >= groups ? next - groups : next;
        }
        in[u] = i < total && g[u] * kScaleGroup + lane * 8 < a.K;
        if (in[u]) r[u].load(a.x, row[u] * a.x_stride + g[u] * kScaleGroup + lane * 8, XT);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float v[8] = {}, top = 0.f, factor;
        if (in[u]) r[u].get(XT, v);
#pragma unroll
        for (int i = 0; i < 8; i += 2) top = max_nan(top, max_nan(fabsf(v[i]), fabsf(v[i + 1])));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float scale = scale_of(top, factor);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= factor;
        if (in[u]) {
            store_run<8>(a.y, row[u] * a.y_stride + g[u] * kScaleGroup + lane * 8, MOE_E4M3, v);
            if (lane == 0) a.scale[row[u] * a.scale_stride + g[u]] = scale;
        }
    }
}

// Any alignment and width: a warp a group, every 32nd element a lane.
__global__ void __launch_bounds__(kThreads) quant_any_kernel(const QuantArgs a, int groups, int64_t total) {
    grid_launch_next();
    grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (i >= total) return;  // the whole warp
    int g;
    const int64_t row = row_of(i, groups, g);
    constexpr int kEach = kScaleGroup / 32;
    const int k0 = g * kScaleGroup + lane;
    Raw<1> r[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (k0 + 32 * j < a.K) r[j].load(a.x, row * a.x_stride + k0 + 32 * j, a.x_type);
    float v[kEach], top = 0.f, factor;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        float one[1] = {0.f};
        if (k0 + 32 * j < a.K) r[j].get(a.x_type, one);
        v[j] = one[0];
        top = max_nan(top, fabsf(v[j]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float scale = scale_of(top, factor);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const float one[1] = {v[j] * factor};
        if (k0 + 32 * j < a.K) store_run<1>(a.y, row * a.y_stride + k0 + 32 * j, MOE_E4M3, one);
    }
    if (lane == 0) a.scale[row * a.scale_stride + g] = scale;
}

template <int XT>
cudaError_t launch(const QuantArgs& a, int groups, int64_t total, cudaStream_t st) {
    constexpr int each = kThreads / 16;
    if (total <= 32768) {  // few groups: all of the GPU rather than several a half warp (512 x 4096 2.3 us, 3.2 with four)
        return launch_pdl(quant_kernel<XT, 1>, dim3((unsigned)((total + each - 1) / each)), dim3(kThreads), 0, st, a, groups, total);
    }
    const int64_t grid = (total + 4 * each - 1) / (4 * each);
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_pdl(quant_kernel<XT, 4>, dim3((unsigned)grid), dim3(kThreads), 0, st, a, groups, total);
}

}  // namespace

cudaError_t launch_quant(const QuantArgs& a, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    const int groups = (a.K - 1) / kScaleGroup + 1;
    const int64_t total = (int64_t)a.T * groups;
    const bool vec = a.K % 8 == 0 && runs_aligned(a.x, a.x_type, 8, a.x_stride) && runs_aligned(a.y, MOE_E4M3, 8, a.y_stride);
    if (vec) {
        if (a.x_type == MOE_BF16) return launch<MOE_BF16>(a, groups, total, st);
        if (a.x_type == MOE_F16) return launch<MOE_F16>(a, groups, total, st);
        return launch<MOE_F32>(a, groups, total, st);
    }
    const int64_t grid = (total + kThreads / 32 - 1) / (kThreads / 32);
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_pdl(quant_any_kernel, dim3((unsigned)grid), dim3(kThreads), 0, st, a, groups, total);
}

}  // namespace moe
