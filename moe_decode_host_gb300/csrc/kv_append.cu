// Position rotation of queries and keys, and the append of keys and values to a paged
// cache.
//
//   (a, b) -> (a cos - b sin, a sin + b cos)
//
// over the pairs (i, i + rot/2) or (2i, 2i + 1) of the first rot elements of a head,
// with the cosines and sines of the token's position from a table in fp32; then
// q -> q_out, k and v -> the token's slot of the cache, in 16 bits or as E4M3 of the
// value over the head's scale.
//
// Memory bound: q, k, v in, q_out and the slots out, each once.  An item is 2 * VEC
// elements of one head that hold VEC whole pairs (two runs rot/2 apart, or one double
// run), so in both pairings item j uses table entries [j VEC, j VEC + VEC).  Thread x of
// a CTA keeps item x % items of its token and walks the heads: its table entries are
// read once.
#include "ptx.cuh"
#include "vec.cuh"

namespace moe {
namespace {

constexpr int kAppendThreads = 256;

template <int VEC>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
    grid_launch_next();
    grid_dep_wait();
    const int t = blockIdx.x;
    const int items = a.kv.head_dim / (2 * VEC);  // of one head
    const int j = threadIdx.x % items;
    const int step = kAppendThreads / items;
    if (threadIdx.x >= step * items) return;
    const int half = a.rot / 2;
    const bool turn = j * VEC < half;  // whether the item is rotated, else copied
    // element offsets of the item's two runs
    int e0, e1;
    if (!turn || a.interleaved) {
        e0 = 2 * j * VEC;
        e1 = e0 + VEC;
    } else {
        e0 = j * VEC;
        e1 = e0 + half;
    }
    const int pos = a.rot > 0 ? a.positions[t] : 0;
    if (a.rot > 0 && (pos < 0 || pos >= a.n_positions)) {  // no table row: nothing of this token is written
        if (threadIdx.x == 0) set_status(a.kv.status, MOE_ERR_BAD_INDEX);
        return;
    }
    const int64_t slot = a.slots[t];
    bool put = slot >= 0;  // a negative slot: the token is not appended
    int64_t dst = 0;
    if (put) {
        const int64_t page = slot / a.kv.page_size;
        if (page >= a.kv.n_pages) {
            put = false;
            if (threadIdx.x == 0) set_status(a.kv.status, MOE_ERR_BAD_INDEX);
        } else {
            dst = page * a.kv.page_stride + (slot - page * a.kv.page_size) * a.kv.token_stride;
        }
    }
    float cs[VEC], sn[VEC];
    if (turn) {
        const float* row = a.cos_sin + (int64_t)pos * a.rot + j * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            cs[i] = row[i];
            sn[i] = row[half + i];
        }
    }
    const int hq = a.kv.q_heads, hkv = a.kv.kv_heads;
    for (int h = threadIdx.x / items; h < hq + 2 * hkv; h += step) {
        const int kind = h < hq ? 0 : (h < hq + hkv ? 1 : 2);
        if (kind != 0 && !put) continue;
        const int hh = kind == 0 ? h : (kind == 1 ? h - hq : h - hq - hkv);
        const void* src = kind == 0 ? a.q : (kind == 1 ? a.k : a.v);
        const int64_t at = kind == 0   ? t * a.q_ts + hh * a.q_hs
                           : kind == 1 ? t * a.k_ts + hh * a.k_hs
                                       : t * a.v_ts + hh * a.v_hs;
        Raw<VEC> r0, r1;
        r0.load(src, at + e0, a.type);
        r1.load(src, at + e1, a.type);
        float x0[VEC], x1[VEC];
        r0.get(a.type, x0);
        r1.get(a.type, x1);
        if (turn && kind != 2) {
            if (a.interleaved) {
                // pair i is elements 2i, 2i + 1 of the double run
                if constexpr (VEC == 1) {
                    const float p = x0[0], q = x1[0];
                    x0[0] = p * cs[0] - q * sn[0];
                    x1[0] = p * sn[0] + q * cs[0];
                } else {
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i) {
                        const float p = x0[2 * i], q = x0[2 * i + 1], u = x1[2 * i], v = x1[2 * i + 1];
                        x0[2 * i] = p * cs[i] - q * sn[i];
                        x0[2 * i + 1] = p * sn[i] + q * cs[i];
                        x1[2 * i] = u * cs[VEC / 2 + i] - v * sn[VEC / 2 + i];
                        x1[2 * i + 1] = u * sn[VEC / 2 + i] + v * cs[VEC / 2 + i];
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float p = x0[i], q = x1[i];
                    x0[i] = p * cs[i] - q * sn[i];
                    x1[i] = p * sn[i] + q * cs[i];
                }
            }
        }
        if (kind == 0) {
            store_run<VEC>(a.q_out, t * a.qo_ts + hh * a.qo_hs + e0, a.type, x0);
            store_run<VEC>(a.q_out, t * a.qo_ts + hh * a.qo_hs + e1, a.type, x1);
        } else {
            const float* scale = kind == 1 ? a.kv.k_scale : a.kv.v_scale;
            if (scale) {
                const float s = scale[hh];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    x0[i] = x0[i] / s;
                    x1[i] = x1[i] / s;
                }
            }
            void* cache = kind == 1 ? a.kv.k : a.kv.v;
            store_run<VEC>(cache, dst + hh * a.kv.head_stride + e0, a.kv.type, x0);
            store_run<VEC>(cache, dst + hh * a.kv.head_stride + e1, a.kv.type, x1);
        }
    }
}

// Whether every run of `vec` elements of the call is aligned.
bool fits(const AppendArgs& a, int vec) {
    return a.rot / 2 % vec == 0 && a.kv.head_dim % (2 * vec) == 0 && runs_aligned(a.q, a.type, vec, a.q_ts, a.q_hs) &&
           runs_aligned(a.k, a.type, vec, a.k_ts, a.k_hs) && runs_aligned(a.v, a.type, vec, a.v_ts, a.v_hs) &&
           runs_aligned(a.q_out, a.type, vec, a.qo_ts, a.qo_hs);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    if (fits(a, 8)) return launch_pdl(append_kernel<8>, dim3(a.T), dim3(kAppendThreads), 0, st, a);
    if (fits(a, 4)) return launch_pdl(append_kernel<4>, dim3(a.T), dim3(kAppendThreads), 0, st, a);
    return launch_pdl(append_kernel<1>, dim3(a.T), dim3(kAppendThreads), 0, st, a);
}

}  // namespace moe
