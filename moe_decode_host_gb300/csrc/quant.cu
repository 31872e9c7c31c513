// Rows to E4M3 with one scale for each 128 elements.
//
//   s = max(max |x| / 448, 2^-126) over a group,  y = E4M3(x / s) with s as it is returned
//
// Memory bound: each element once in and once out.  A half warp holds a group, 8 elements a
// lane, so that its maximum takes four exchanges and no shared memory; a half warp takes
// several groups so that their loads are in flight together.
//
// Measured on a GB300: 8192 x 4096 bf16 22.0 us (4.6 TB/s, 69% of a plain copy's rate), 512 x 4096 2.5, 777 x 5003
// fp32 at any alignment 5.8 (3.4 TB/s), 8 x 4096 1.4.  A quotient takes two fused steps an
// element more than a product by one factor, with which the first took 20.9 us.
#include <algorithm>

#include "ptx.cuh"
#include "vec.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr float kE4M3Max = 448.f;

// The scale of a group with largest magnitude `top`.  A NaN or an infinity among them: NaN.
__device__ __forceinline__ float scale_of(float top) {
    const float m = top < INFINITY ? top : __uint_as_float(0x7fc00000u);
    const float scale = m * (1.f / kE4M3Max);
    return scale < 1.17549435e-38f ? 1.17549435e-38f : scale;  // 2^-126; NaN stays
}

// v /= scale, to nearest as fp32's division, so that a code is that of the quotient by the scale that the caller gets,
// at ties between codes too.  With r the scale's inverse to nearest, x r is within a step of the quotient, what it leaves
// of x is exact in a fused product, and adding that remainder's quotient rounds as the division does (P. Markstein, IBM
// J. Res. Dev. 34, 1990).  Scales near the smallest are taken 2^64 larger, with the values, so that the remainder is
// exact there too.  The remainder's sign is such that -0 stays.
template <int N>
__device__ __forceinline__ void divide(float (&v)[N], float scale) {
    if (scale < 8.67361738e-19f) {  // 2^-60
        scale *= 1.84467441e19f;    // 2^64
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= 1.84467441e19f;
    }
    const float r = 1.f / scale;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float q = v[i] * r;
        v[i] = fmaf(-fmaf(q, scale, -v[i]), r, q);
    }
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
        float v[8] = {}, top = 0.f;
        if (in[u]) r[u].get(XT, v);
#pragma unroll
        for (int i = 0; i < 8; i += 2) top = max_nan(top, max_nan(fabsf(v[i]), fabsf(v[i + 1])));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float scale = scale_of(top);
        divide(v, scale);
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
    float v[kEach], top = 0.f;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        float one[1] = {0.f};
        if (k0 + 32 * j < a.K) r[j].get(a.x_type, one);
        v[j] = one[0];
        top = max_nan(top, fabsf(v[j]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float scale = scale_of(top);
    divide(v, scale);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const float one[1] = {v[j]};
        if (k0 + 32 * j < a.K) store_run<1>(a.y, row * a.y_stride + k0 + 32 * j, MOE_E4M3, one);
    }
    if (lane == 0) a.scale[row * a.scale_stride + g] = scale;
}

template <int XT>
cudaError_t launch(const QuantArgs& a, int groups, int64_t total, cudaStream_t st) {
    constexpr int each = kThreads / 16;
    if (total <= 32768) {  // few groups: all of the GPU rather than several a half warp (512 x 4096 2.5 us, 3.5 with four)
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
