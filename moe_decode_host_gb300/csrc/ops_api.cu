// Host side of the decoder-layer operators of moehost.h: argument checks, the cache
// handle, launches.
#include <cmath>
#include <new>

#include "host.cuh"
#include "vec.cuh"

using namespace moe;

struct moe_kv {
    KvView view;
    int max_batch;
    int sm_count;
    void* workspace = nullptr;  // one allocation: moe_kv_attend's workspace, then the status word
    int* d_status = nullptr;
};

namespace {

// SMs of the current device; asked once a device (ordinals below 64), as the answer
// does not change.
int sm_count_now(int* out) {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return MOE_ERR_CUDA;
        }
        if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    }
    *out = n;
    return MOE_OK;
}

// Most tokens and outputs of a moe_linear call: tile counts and grid dimensions stay in range.
constexpr int kMaxExtent = 1 << 22;

bool whole16(const void* p, int type, int64_t s0, int64_t s1) {
    return aligned(p, 16) && s0 * type_bytes(type) % 16 == 0 && s1 * type_bytes(type) % 16 == 0;
}

// moe_kv_create and moe_kv_create_blocks (scale_tokens > 0).
int create_cache(const moe_kv_params* pp, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                 int scale_tokens, moe_kv** out) {
    if (!pp || !out) return MOE_ERR_INVALID_ARG;
    const moe_kv_params p = *pp;
    if (!is_float16(p.type) && p.type != MOE_E4M3) return MOE_ERR_INVALID_ARG;
    if (p.n_pages < 1 || p.page_size < 1 || p.page_size > 65536 || p.kv_heads < 1 || p.q_heads < p.kv_heads ||
        p.q_heads > 65535 || p.q_heads % p.kv_heads || p.head_dim < 16 || p.head_dim > 256 || p.head_dim % 16 ||
        p.max_batch < 1 || p.max_batch > 65535)
        return MOE_ERR_INVALID_ARG;
    if (p.page_stride < 0 || p.token_stride < 0 || p.head_stride < 0) return MOE_ERR_INVALID_ARG;
    if (!k_cache || !v_cache || !whole16(k_cache, p.type, p.page_stride, p.token_stride) ||
        !whole16(v_cache, p.type, p.head_stride, 0) || !is_device_ptr(k_cache) || !is_device_ptr(v_cache))
        return MOE_ERR_INVALID_ARG;
    const bool scaled = p.type == MOE_E4M3;
    if (scaled != (k_scale != nullptr) || scaled != (v_scale != nullptr)) return MOE_ERR_INVALID_ARG;
    if (scaled && (!is_device_ptr(k_scale) || !is_device_ptr(v_scale) || !aligned(k_scale, 4) || !aligned(v_scale, 4)))
        return MOE_ERR_INVALID_ARG;
    moe_kv* kv = new (std::nothrow) moe_kv;
    if (!kv) return MOE_ERR_NOMEM;
    kv->view = KvView{k_cache, v_cache, k_scale, v_scale, p.type, p.n_pages, p.page_size, p.kv_heads, p.q_heads,
                      p.head_dim, p.page_stride, p.token_stride, p.head_stride, nullptr, scale_tokens,
                      scale_tokens ? p.page_size / scale_tokens : 0,
                      scale_tokens > 1 ? (uint32_t)(((1ull << 32) + scale_tokens - 1) / scale_tokens) : 0u};
    kv->max_batch = p.max_batch;
    if (!attend_fits(kv->view)) {
        delete kv;
        return MOE_ERR_INVALID_ARG;
    }
    if (sm_count_now(&kv->sm_count) != MOE_OK) {
        delete kv;
        return MOE_ERR_CUDA;
    }
    const size_t ws = (attend_workspace(kv->view, kv->sm_count) + 15) / 16 * 16;
    cudaError_t err = cudaMalloc(&kv->workspace, ws + sizeof(int));
    err = err ? err : cudaMemset(kv->workspace, 0, ws + sizeof(int));
    err = err ? err : cudaStreamSynchronize(nullptr);  // done before a call on any stream
    if (err != cudaSuccess) {
        cudaGetLastError();
        moe_kv_destroy(kv);
        return err == cudaErrorMemoryAllocation ? MOE_ERR_NOMEM : MOE_ERR_CUDA;
    }
    kv->d_status = reinterpret_cast<int*>(static_cast<uint8_t*>(kv->workspace) + ws);
    kv->view.status = kv->d_status;
    *out = kv;
    return MOE_OK;
}

// moe_kv_append and moe_kv_append_axes (axis_of_pair given).
int append(moe_kv* kv, int type, const void* q, int64_t q_ts, int64_t q_hs, const void* k, int64_t k_ts, int64_t k_hs,
           const void* v, int64_t v_ts, int64_t v_hs, const int32_t* positions, int64_t positions_stride, int n_axes,
           const uint8_t* axis_of_pair, const int64_t* slots, const float* cos_sin, int n_positions, int rot_dim,
           int interleaved, int T, void* q_out, int64_t qo_ts, int64_t qo_hs, void* stream) {
    if (!kv || T < 0 || !is_float_type(type)) return MOE_ERR_INVALID_ARG;
    if (rot_dim < 0 || rot_dim > kv->view.head_dim || rot_dim % 2 || n_positions < 0) return MOE_ERR_INVALID_ARG;
    if (interleaved != 0 && interleaved != 1) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!q || !k || !v || !slots || !q_out) return MOE_ERR_INVALID_ARG;
    if (rot_dim > 0 && (!positions || !cos_sin)) return MOE_ERR_INVALID_ARG;
    if (T == 1) q_ts = k_ts = v_ts = qo_ts = 0;  // of no meaning for one token, or one head
    if (kv->view.q_heads == 1) q_hs = qo_hs = 0;
    if (kv->view.kv_heads == 1) k_hs = v_hs = 0;
    uint32_t axis[8] = {};
    if (axis_of_pair) {
        for (int i = 0; i < rot_dim / 2; ++i) {
            if (axis_of_pair[i] >= n_axes) return MOE_ERR_INVALID_ARG;
            axis[i >> 4] |= (uint32_t)axis_of_pair[i] << (2 * (i & 15));
        }
    }
    AppendArgs a{kv->view, q, k, v, type, q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, positions, slots, cos_sin, n_positions,
                 rot_dim, interleaved, T, q_out, qo_ts, qo_hs, kv->sm_count, n_axes, positions_stride, {}};
    for (int i = 0; i < 8; ++i) a.axis[i] = axis[i];
    return cuda_status(kv->view.scale_tokens ? launch_append_blocks(a, S(stream)) : launch_append(a, S(stream)));
}

// What moe_linear and moe_linear_blocks check alike; `nothing`: a call without tokens, done.
int linear_args(const void* x, int64_t x_stride, const void* w, int64_t w_stride, int in_type, int T, int N, int K,
                const float* x_scale, const float* w_scale, const void* bias, int bias_type, int act,
                const void* residual, int64_t res_stride, void* y, int y_type, int64_t y_stride, int* status_dev,
                LinearArgs& a, bool& nothing) {
    if (T < 0 || N < 1 || K < 1 || N > kMaxExtent || T > kMaxExtent) return MOE_ERR_INVALID_ARG;
    if ((!is_float16(in_type) && in_type != MOE_E4M3) || !is_float_type(y_type)) return MOE_ERR_INVALID_ARG;
    if (act < MOE_ACT_NONE || act > MOE_ACT_GELU) return MOE_ERR_INVALID_ARG;
    if (bias && !is_float_type(bias_type)) return MOE_ERR_INVALID_ARG;
    nothing = T == 0;
    if (nothing) return MOE_OK;
    if (!x || !w || !y) return MOE_ERR_INVALID_ARG;
    const bool scaled = in_type == MOE_E4M3;
    if (scaled != (x_scale != nullptr) || scaled != (w_scale != nullptr)) return MOE_ERR_INVALID_ARG;
    if (T == 1) x_stride = K;  // of no meaning for one row
    if (N == 1) w_stride = K;
    if (x_stride < K || w_stride < K || (int64_t)K * type_bytes(in_type) % 16) return MOE_ERR_INVALID_ARG;
    if (!whole16(x, in_type, x_stride, 0) || !whole16(w, in_type, w_stride, 0)) return MOE_ERR_INVALID_ARG;
    a = LinearArgs{x, w, in_type, x_stride, w_stride, T, N, K, x_scale, w_scale, bias, bias_type, act, residual,
                   res_stride, y, y_type, y_stride, status_dev, 0};
    return sm_count_now(&a.sm_count);
}

}  // namespace

extern "C" {

int moe_add_rms_norm(const void* x, int x_type, int64_t x_stride, const void* residual, int res_type,
                     int64_t res_stride, const void* weight, int weight_type, float eps, int T, int H, void* sum_out,
                     int64_t sum_stride, void* y, int y_type, int64_t y_stride, float* y_scale, void* stream) {
    if (T < 0 || H < 1 || H > 32768 || !(eps >= 0.f) || std::isinf(eps)) return MOE_ERR_INVALID_ARG;
    if (!is_float_type(x_type) || (!is_float_type(y_type) && y_type != MOE_E4M3)) return MOE_ERR_INVALID_ARG;
    if ((residual || sum_out) && !is_float_type(res_type)) return MOE_ERR_INVALID_ARG;
    if (weight && !is_float_type(weight_type)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!x || !y || (y_type == MOE_E4M3) != (y_scale != nullptr)) return MOE_ERR_INVALID_ARG;
    if (T == 1) x_stride = res_stride = sum_stride = y_stride = 0;  // of no meaning for one row
    NormArgs a{x, residual, weight, x_type, res_type, weight_type, x_stride, res_stride, eps, T, H, sum_out,
               sum_stride, y, y_type, y_stride, y_scale, 1.f / (float)H, 0};
    const int rc = sm_count_now(&a.sm_count);
    if (rc != MOE_OK) return rc;
    return cuda_status(launch_norm(a, S(stream)));
}

int moe_kv_create(const moe_kv_params* pp, void* k_cache, void* v_cache, const float* k_scale, const float* v_scale,
                  moe_kv** out) {
    // written by the appends of block-scaled caches alone
    return create_cache(pp, k_cache, v_cache, const_cast<float*>(k_scale), const_cast<float*>(v_scale), 0, out);
}

int moe_kv_create_blocks(const moe_kv_params* pp, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                         int scale_tokens, moe_kv** out) {
    if (!pp || pp->type != MOE_E4M3 || scale_tokens < 1 || scale_tokens > kMaxScaleTokens || pp->page_size < 1 ||
        pp->page_size % scale_tokens)
        return MOE_ERR_INVALID_ARG;
    return create_cache(pp, k_cache, v_cache, k_scale, v_scale, scale_tokens, out);
}

int moe_kv_destroy(moe_kv* kv) {
    if (!kv) return MOE_ERR_INVALID_ARG;
    cudaFree(kv->workspace);
    delete kv;
    return MOE_OK;
}

int moe_kv_append(moe_kv* kv, int type, const void* q, int64_t q_ts, int64_t q_hs, const void* k, int64_t k_ts,
                  int64_t k_hs, const void* v, int64_t v_ts, int64_t v_hs, const int32_t* positions,
                  const int64_t* slots, const float* cos_sin, int n_positions, int rot_dim, int interleaved, int T,
                  void* q_out, int64_t qo_ts, int64_t qo_hs, void* stream) {
    return append(kv, type, q, q_ts, q_hs, k, k_ts, k_hs, v, v_ts, v_hs, positions, 0, 1, nullptr, slots, cos_sin,
                  n_positions, rot_dim, interleaved, T, q_out, qo_ts, qo_hs, stream);
}

int moe_kv_append_axes(moe_kv* kv, int type, const void* q, int64_t q_ts, int64_t q_hs, const void* k, int64_t k_ts,
                       int64_t k_hs, const void* v, int64_t v_ts, int64_t v_hs, const int32_t* positions,
                       int64_t positions_stride, int n_axes, const uint8_t* axis_of_pair, const int64_t* slots,
                       const float* cos_sin, int n_positions, int rot_dim, int interleaved, int T, void* q_out,
                       int64_t qo_ts, int64_t qo_hs, void* stream) {
    if (!axis_of_pair || n_axes < 1 || n_axes > kMaxAxes || rot_dim < 2) return MOE_ERR_INVALID_ARG;
    return append(kv, type, q, q_ts, q_hs, k, k_ts, k_hs, v, v_ts, v_hs, positions, positions_stride, n_axes, axis_of_pair,
                  slots, cos_sin, n_positions, rot_dim, interleaved, T, q_out, qo_ts, qo_hs, stream);
}

int moe_kv_attend(moe_kv* kv, const void* q, int q_type, int64_t q_ts, int64_t q_hs, const int32_t* page_table,
                  int64_t table_stride, int max_pages, const int32_t* lengths, int B, float scale, int window,
                  void* out, int64_t out_ts, int64_t out_hs, float* lse, void* stream) {
    if (!kv || B < 0 || B > kv->max_batch || max_pages < 0 || window < 0 || table_stride < 0) return MOE_ERR_INVALID_ARG;
    if (!is_float16(q_type) || (kv->view.type != MOE_E4M3 && kv->view.type != q_type)) return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
    if (B == 0) return MOE_OK;
    if (!q || !lengths || !out || (max_pages > 0 && !page_table)) return MOE_ERR_INVALID_ARG;
    if (q == out) return MOE_ERR_INVALID_ARG;  // several CTAs read a query whose output one of them writes
    if (B == 1) q_ts = out_ts = table_stride = 0;  // of no meaning for one sequence, or one head
    if (kv->view.q_heads == 1) q_hs = out_hs = 0;
    if (!whole16(q, q_type, q_ts, q_hs) || !whole16(out, q_type, out_ts, out_hs)) return MOE_ERR_INVALID_ARG;
    AttendArgs a{kv->view, q, q_type, q_ts, q_hs, page_table, table_stride, max_pages, lengths, B, scale, window, out,
                 out_ts, out_hs, lse, kv->sm_count, kv->workspace};
    return cuda_status(launch_attend(a, S(stream)));
}

int moe_quant_e4m3(const void* x, int x_type, int64_t x_stride, int T, int K, void* y, int64_t y_stride, float* scale,
                   int64_t scale_stride, void* stream) {
    if (T < 0 || K < 1 || !is_float_type(x_type)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!x || !y || !scale) return MOE_ERR_INVALID_ARG;
    if (y == x || scale == x || scale == y) return MOE_ERR_INVALID_ARG;  // a group's codes would lie on another's elements
    if (T == 1) x_stride = y_stride = scale_stride = 0;  // of no meaning for one row
    QuantArgs a{x, x_type, x_stride, T, K, y, y_stride, scale, scale_stride};
    return cuda_status(launch_quant(a, S(stream)));
}

int moe_kv_get_status(moe_kv* kv, int* status) {
    if (!kv || !status) return MOE_ERR_INVALID_ARG;
    return cuda_status(cudaMemcpy(status, kv->d_status, sizeof(int), cudaMemcpyDeviceToHost));
}

int moe_kv_clear_status(moe_kv* kv) {
    if (!kv) return MOE_ERR_INVALID_ARG;
    cudaError_t err = cudaMemset(kv->d_status, 0, sizeof(int));
    return cuda_status(err ? err : cudaStreamSynchronize(nullptr));
}

int moe_linear(const void* x, int64_t x_stride, const void* w, int64_t w_stride, int in_type, int T, int N, int K,
               const float* x_scale, const float* w_scale, const void* bias, int bias_type, int act,
               const void* residual, int64_t res_stride, void* y, int y_type, int64_t y_stride, int* status_dev,
               void* stream) {
    LinearArgs a;
    bool nothing;
    const int rc = linear_args(x, x_stride, w, w_stride, in_type, T, N, K, x_scale, w_scale, bias, bias_type, act, residual,
                               res_stride, y, y_type, y_stride, status_dev, a, nothing);
    if (rc != MOE_OK || nothing) return rc;
    return cuda_status(launch_linear(a, S(stream)));
}

int moe_linear_blocks(const void* x, int64_t x_stride, const void* w, int64_t w_stride, int T, int N, int K,
                      const float* x_scale, int64_t x_scale_stride, const float* w_scale, int64_t w_scale_stride,
                      const void* bias, int bias_type, int act, const void* residual, int64_t res_stride, void* y,
                      int y_type, int64_t y_stride, int* status_dev, void* stream) {
    LinearArgs a;
    bool nothing;
    const int rc = linear_args(x, x_stride, w, w_stride, MOE_E4M3, T, N, K, x_scale, w_scale, bias, bias_type, act, residual,
                               res_stride, y, y_type, y_stride, status_dev, a, nothing);
    if (rc != MOE_OK || nothing) return rc;
    if (T == 1) x_scale_stride = 0;
    if (N <= kScaleGroup) w_scale_stride = 0;
    return cuda_status(launch_linear_blocks(a, x_scale_stride, w_scale_stride, S(stream)));
}

}  // extern "C"
