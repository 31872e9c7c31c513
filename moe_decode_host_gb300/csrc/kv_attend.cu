// Attention of one new token per sequence over the paged cache.
//
//   o = sum_j softmax_j(scale * q . k_j) v_j,  j in [max(0, len - window), len)
//
// Plain form of the kernel: a CTA per query head and sequence, a warp per token, the
// running maximum and sum of the softmax per warp, joined at the end.
#include "ptx.cuh"
#include "vec.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxD = 256;

__device__ __forceinline__ float load_one(const void* p, int64_t at, int type) {
    if (type == MOE_F32) return static_cast<const float*>(p)[at];
    if (type == MOE_E4M3) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const uint8_t*>(p)[at], __NV_E4M3);
        return __half2float(__half(h));
    }
    return half_bits_to_f32(static_cast<const uint16_t*>(p)[at], type);
}

__global__ void __launch_bounds__(kWarps * 32) attend_kernel(const AttendArgs a) {
    __shared__ float so[kWarps][kMaxD], sm[kWarps], sl[kWarps];
    grid_dep_wait();
    const int h = blockIdx.x, b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kh = h / (a.kv.q_heads / a.kv.kv_heads), D = a.kv.head_dim;
    int n = a.lengths[b];
    const int64_t most = (int64_t)a.max_pages * a.kv.page_size;
    if (n < 0 || n > most) {
        if (threadIdx.x == 0) set_status(a.kv.status, MOE_ERR_BAD_INDEX);
        n = n < 0 ? 0 : (int)most;
    }
    const int first = a.window > 0 && n > a.window ? n - a.window : 0;
    float q[8], o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = lane + 32 * i;
        q[i] = d < D ? load_one(a.q, b * a.q_ts + h * a.q_hs + d, a.q_type) * a.scale : 0.f;
        o[i] = 0.f;
    }
    const float ks = a.kv.k_scale ? a.kv.k_scale[kh] : 1.f, vs = a.kv.v_scale ? a.kv.v_scale[kh] : 1.f;
    float m = -INFINITY, l = 0.f;
    for (int j = first + warp; j < n; j += kWarps) {
        const int page = a.page_table[b * a.table_stride + j / a.kv.page_size];
        if (page < 0 || page >= a.kv.n_pages) {
            if (lane == 0) set_status(a.kv.status, MOE_ERR_BAD_INDEX);
            continue;
        }
        const int64_t at = page * a.kv.page_stride + (j % a.kv.page_size) * a.kv.token_stride + kh * a.kv.head_stride;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int d = lane + 32 * i;
            if (d < D) s = fmaf(q[i], load_one(a.kv.k, at + d, a.kv.type), s);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= ks;
        const float mn = fmaxf(m, s);
        const float c = m == -INFINITY ? 0.f : expf(m - mn), p = mn == -INFINITY ? 0.f : expf(s - mn);
        l = l * c + p;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int d = lane + 32 * i;
            if (d < D) o[i] = o[i] * c + p * load_one(a.kv.v, at + d, a.kv.type);
        }
        m = mn;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) so[warp][lane + 32 * i] = o[i];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    __syncthreads();
    float mt = -INFINITY, lt = 0.f;
    for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, sm[w]);
    for (int w = 0; w < kWarps; ++w) lt += sm[w] == -INFINITY ? 0.f : sl[w] * expf(sm[w] - mt);
    const int d = threadIdx.x;
    if (d < D) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w)
            if (sm[w] != -INFINITY) v += so[w][d] * expf(sm[w] - mt);
        const float r[1] = {lt > 0.f ? v / lt * vs : 0.f};
        store_run<1>(a.out, b * a.out_ts + h * a.out_hs + d, a.q_type, r);
    }
    if (d == 0 && a.lse) a.lse[(int64_t)b * a.kv.q_heads + h] = lt > 0.f ? mt + logf(lt) : -INFINITY;
}

}  // namespace

size_t attend_workspace(const KvView&, int, int) { return 256; }

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t st) {
    if (a.B == 0) return cudaSuccess;
    return launch_pdl(attend_kernel, dim3(a.kv.q_heads, a.B), dim3(kWarps * 32), 0, st, a);
}

}  // namespace moe
