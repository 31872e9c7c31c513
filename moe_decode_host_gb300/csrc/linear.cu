// Matrix product with an epilogue: y = act(x W^T [* sx_t * sw_n] + bias) + residual.
//
// Plain form of the kernel: 16 x 16 tiles through shared memory, fp32 sums.
#include "ptx.cuh"
#include "vec.cuh"

namespace moe {
namespace {

constexpr int kTile = 16;

__device__ __forceinline__ float load_one(const void* p, int64_t at, int type) {
    if (type == MOE_E4M3) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(p)[at], __NV_E4M3);
        return __half2float(__half(h));
    }
    if (type == MOE_F32) return static_cast<const float*>(p)[at];
    return half_bits_to_f32(static_cast<const uint16_t*>(p)[at], type);
}

__device__ __forceinline__ float activate(float v, int act) {
    if (act == MOE_ACT_RELU) return v < 0.f ? 0.f : v;
    if (act == MOE_ACT_SILU) return v / (1.f + expf(-v));
    if (act == MOE_ACT_GELU) return 0.5f * v * (1.f + erff(v * 0.70710678f));
    return v;
}

__global__ void linear_kernel(const LinearArgs a) {
    __shared__ float sx[kTile][kTile + 1], sw[kTile][kTile + 1];
    grid_dep_wait();
    const int tx = threadIdx.x, ty = threadIdx.y;
    const int n = blockIdx.x * kTile + tx, t = blockIdx.y * kTile + ty, nr = blockIdx.x * kTile + ty;
    float acc = 0.f;
    for (int k = 0; k < a.K; k += kTile) {
        sx[ty][tx] = t < a.T && k + tx < a.K ? load_one(a.x, t * a.x_stride + k + tx, a.in_type) : 0.f;
        sw[ty][tx] = nr < a.N && k + tx < a.K ? load_one(a.w, nr * a.w_stride + k + tx, a.in_type) : 0.f;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kTile; ++i) acc = fmaf(sx[ty][i], sw[tx][i], acc);
        __syncthreads();
    }
    if (t >= a.T || n >= a.N) return;
    if (a.x_scale) acc *= a.x_scale[t] * a.w_scale[n];
    if (a.bias) acc += load_one(a.bias, n, a.bias_type);
    acc = activate(acc, a.act);
    if (a.res) acc += load_one(a.res, t * a.res_stride + n, a.y_type);
    const float r[1] = {acc};
    store_run<1>(a.y, t * a.y_stride + n, a.y_type, r);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    return launch_pdl(linear_kernel, dim3((a.N + kTile - 1) / kTile, (a.T + kTile - 1) / kTile), dim3(kTile, kTile), 0,
                      st, a);
}

}  // namespace moe
