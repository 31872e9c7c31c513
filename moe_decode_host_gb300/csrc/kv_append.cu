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
// a token's CTA keeps item x % items and takes heads x / items + i * step, kHeads of them
// at once: their loads are issued before the token's position is known, and its table
// entries are read once.
#include "ptx.cuh"
#include "vec.cuh"

namespace moe {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kHeads = 4;

// WIDE: q, k and v may be fp32.
template <int VEC, bool WIDE>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
    grid_launch_next();
    grid_dep_wait();
    const int t = blockIdx.x;
    const int items = a.kv.head_dim / (2 * VEC);  // of one head
    const int j = threadIdx.x % items;
    const int step = blockDim.x / items;
    const int g = threadIdx.x / items;
    if (g >= step) return;
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
    const int hq = a.kv.q_heads, hkv = a.kv.kv_heads, heads = hq + 2 * hkv;
    Raw<VEC, WIDE> r0[kHeads], r1[kHeads];
    auto fetch = [&](int h0) {
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            const int h = h0 + i * step;
            if (h >= heads) break;
            const void* src = h < hq ? a.q : (h < hq + hkv ? a.k : a.v);
            const int64_t at = h < hq         ? t * a.q_ts + h * a.q_hs
                               : h < hq + hkv ? t * a.k_ts + (h - hq) * a.k_hs
                                              : t * a.v_ts + (h - hq - hkv) * a.v_hs;
            r0[i].load(src, at + e0, a.type);
            r1[i].load(src, at + e1, a.type);
        }
    };
    fetch(g);
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
    for (int h0 = g; h0 < heads; h0 += kHeads * step) {
        if (h0 != g) fetch(h0);
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            const int h = h0 + i * step;
            if (h >= heads) break;
            const int kind = h < hq ? 0 : (h < hq + hkv ? 1 : 2);
            if (kind != 0 && !put) continue;
            const int hh = kind == 0 ? h : (kind == 1 ? h - hq : h - hq - hkv);
            float x0[VEC], x1[VEC];
            r0[i].get(a.type, x0);
            r1[i].get(a.type, x1);
            if (turn && kind != 2) {
                if (a.interleaved) {
                    // pair i is elements 2i, 2i + 1 of the double run
                    if constexpr (VEC == 1) {
                        const float p = x0[0], q = x1[0];
                        x0[0] = p * cs[0] - q * sn[0];
                        x1[0] = p * sn[0] + q * cs[0];
                    } else {
#pragma unroll
                        for (int j = 0; j < VEC / 2; ++j) {
                            const float p = x0[2 * j], q = x0[2 * j + 1], u = x1[2 * j], v = x1[2 * j + 1];
                            x0[2 * j] = p * cs[j] - q * sn[j];
                            x0[2 * j + 1] = p * sn[j] + q * cs[j];
                            x1[2 * j] = u * cs[VEC / 2 + j] - v * sn[VEC / 2 + j];
                            x1[2 * j + 1] = u * sn[VEC / 2 + j] + v * cs[VEC / 2 + j];
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float p = x0[j], q = x1[j];
                        x0[j] = p * cs[j] - q * sn[j];
                        x1[j] = p * sn[j] + q * cs[j];
                    }
                }
            }
            if (kind == 0) {
                store_run<VEC>(a.q_out, t * a.qo_ts + hh * a.qo_hs + e0, a.type, x0);
                store_run<VEC>(a.q_out, t * a.qo_ts + hh * a.qo_hs + e1, a.type, x1);
            } else {
                const float* scale = kind == 1 ? a.kv.k_scale : a.kv.v_scale;
                if (scale) {
                    const float inv = 1.f / scale[hh];
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        x0[j] *= inv;
                        x1[j] *= inv;
                    }
                }
                void* cache = kind == 1 ? a.kv.k : a.kv.v;
                store_run<VEC>(cache, dst + hh * a.kv.head_stride + e0, a.kv.type, x0);
                store_run<VEC>(cache, dst + hh * a.kv.head_stride + e1, a.kv.type, x1);
            }
        }
    }
}

// Whether every run of `vec` elements of the call is aligned.
bool fits(const AppendArgs& a, int vec) {
    return a.rot / 2 % vec == 0 && a.kv.head_dim % (2 * vec) == 0 && runs_aligned(a.q, a.type, vec, a.q_ts, a.q_hs) &&
           runs_aligned(a.k, a.type, vec, a.k_ts, a.k_hs) && runs_aligned(a.v, a.type, vec, a.v_ts, a.v_hs) &&
           runs_aligned(a.q_out, a.type, vec, a.qo_ts, a.qo_hs);
}

template <int VEC>
cudaError_t launch(const AppendArgs& a, cudaStream_t st) {
    const int items = a.kv.head_dim / (2 * VEC), heads = a.kv.q_heads + 2 * a.kv.kv_heads;
    int threads = (items * ((heads + kHeads - 1) / kHeads) + 31) / 32 * 32;
    if (threads > kAppendThreads) threads = kAppendThreads;
    if (a.type == MOE_F32) return launch_pdl(append_kernel<VEC, true>, dim3(a.T), dim3(threads), 0, st, a);
    return launch_pdl(append_kernel<VEC, false>, dim3(a.T), dim3(threads), 0, st, a);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    return fits(a, 8) ? launch<8>(a, st) : fits(a, 4) ? launch<4>(a, st) : launch<1>(a, st);
}

}  // namespace moe
