// Residual addition and root-mean-square norm, with an output in 16, 32 or 8 bits.
//
//   s = x + r,  y = s * rsqrt(mean(s^2) + eps) * w
//   8 bits: scale = max(max_j |y_j| / 448, 2^-126), y8 = E4M3(y / scale)
//
// Memory bound: x, r in, s, y out, each once.  The row stays in registers between the
// reduction and the outputs.  One reduction carries both statistics: the norm's factor
// is common to the row, so max |y| = rsqrt(...) * max |s * w| and the maximum can be
// taken before the factor is known.
#include "ptx.cuh"
#include "vec.cuh"

namespace moe {
namespace {

constexpr float kE4M3Max = 448.f;
constexpr int kNormThreads = 1024;

// A row is handled by blockDim.x threads (whole warps), NV runs of VEC elements each,
// blockDim.y rows a CTA.
template <int VEC, int NV>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const NormArgs a) {
    __shared__ float2 part[kNormThreads / 32];
    grid_launch_next();
    grid_dep_wait();
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < a.T;
    Raw<VEC> rx[NV], rr[NV], rw[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int e = (threadIdx.x + n * blockDim.x) * VEC;
        if (live && e < a.H) {
            rx[n].load(a.x, row * a.x_stride + e, a.x_type);
            if (a.res) rr[n].load(a.res, row * a.res_stride + e, a.res_type);
            if (a.w) rw[n].load(a.w, e, a.w_type);
        }
    }
    float s[NV][VEC];
    float ss = 0.f, top = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int e = (threadIdx.x + n * blockDim.x) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) s[n][i] = 0.f;
        if (live && e < a.H) {
            rx[n].get(a.x_type, s[n]);
            if (a.res) {
                float r[VEC];
                rr[n].get(a.res_type, r);
#pragma unroll
                for (int i = 0; i < VEC; ++i) s[n][i] += r[i];
            }
            if (a.sum) store_run<VEC>(a.sum, row * a.sum_stride + e, a.res_type, s[n]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) ss = fmaf(s[n][i], s[n][i], ss);
            if (a.w) {
                float w[VEC];
                rw[n].get(a.w_type, w);
#pragma unroll
                for (int i = 0; i < VEC; ++i) s[n][i] *= w[i];
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) top = fmaxf(top, fabsf(s[n][i]));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if (blockDim.x > 32) {
        const int warps = blockDim.x >> 5, w0 = threadIdx.y * warps;
        if ((threadIdx.x & 31) == 0) part[w0 + (threadIdx.x >> 5)] = make_float2(ss, top);
        __syncthreads();
        ss = 0.f;
        top = 0.f;
        for (int i = 0; i < warps; ++i) {  // the same order for every thread: one result a row
            const float2 p = part[w0 + i];
            ss += p.x;
            top = fmaxf(top, p.y);
        }
    }
    if (!live) return;
    float f = 1.f / sqrtf(ss / (float)a.H + a.eps);
    if (a.y_type == MOE_E4M3) {
        // a row with a NaN or an infinity gets a NaN scale (fmaxf alone would hide it)
        const float m = top * f;
        const float scale = m == m && f == f ? fmaxf(m / kE4M3Max, 1.17549435e-38f) : __uint_as_float(0x7fc00000u);
        if (threadIdx.x == 0) a.scale[row] = scale;
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[n][i] = s[n][i] * f / scale;
    } else {
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[n][i] *= f;
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int e = (threadIdx.x + n * blockDim.x) * VEC;
        if (e < a.H) store_run<VEC>(a.y, row * a.y_stride + e, a.y_type, s[n]);
    }
}

template <int VEC, int NV>
cudaError_t launch(const NormArgs& a, cudaStream_t st) {
    const int runs = (a.H + VEC - 1) / VEC;
    const int tx = ((runs + NV - 1) / NV + 31) / 32 * 32;
    const int ty = tx >= 128 ? 1 : 128 / tx;
    const int64_t grid = ((int64_t)a.T + ty - 1) / ty;
    return launch_pdl(norm_kernel<VEC, NV>, dim3((unsigned)grid), dim3(tx, ty), 0, st, a);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    const bool vec = a.H % 8 == 0 && runs_aligned(a.x, a.x_type, 8, a.x_stride) &&
                     (!a.res || runs_aligned(a.res, a.res_type, 8, a.res_stride)) &&
                     (!a.w || runs_aligned(a.w, a.w_type, 8)) &&
                     (!a.sum || runs_aligned(a.sum, a.res_type, 8, a.sum_stride)) &&
                     runs_aligned(a.y, a.y_type, 8, a.y_stride);
    if (vec) {
        if (a.H <= 8192) return launch<8, 1>(a, st);
        return launch<8, 4>(a, st);
    }
    if (a.H <= 1024) return launch<1, 1>(a, st);
    if (a.H <= 8192) return launch<1, 8>(a, st);
    return launch<1, 32>(a, st);
}

}  // namespace moe
