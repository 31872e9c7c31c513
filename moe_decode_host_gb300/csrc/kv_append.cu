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
// run), so in both pairings item j uses table entries [j VEC, j VEC + VEC).  A thread
// keeps one item and takes kHeads heads of a token at once, so that it reads its table
// entries once.
//
// Measured on a GB300: 8192 tokens of 32 + 8 + 8 heads of 128, bf16 into an E4M3 cache, 32.6
// us (5.8 TB/s, 85% of a plain copy's rate); 8 tokens 2.8 us.
#include <algorithm>

#include "ptx.cuh"
#include "vec.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;
constexpr int kStages = 2;  // three leave an SM fewer CTAs: 38.8 us instead of 32.3 for 8192 tokens into E4M3

// Element offsets of item j's two runs in a head, and whether it is rotated (else copied).
template <int VEC>
struct Item {
    int j, e0, e1;
    bool turn;
    __device__ __forceinline__ Item(const AppendArgs& a, int item) : j(item) {
        const int half = a.rot / 2;
        turn = j * VEC < half;
        e0 = !turn || a.interleaved ? 2 * j * VEC : j * VEC;
        e1 = !turn || a.interleaved ? e0 + VEC : e0 + half;
    }
};

// Head h of a token: 0 query, 1 key, 2 value, and its number there.
__device__ __forceinline__ int kind_of(const AppendArgs& a, int h, int& n) {
    const int hq = a.kv.q_heads, hkv = a.kv.kv_heads;
    const int kind = h < hq ? 0 : (h < hq + hkv ? 1 : 2);
    n = kind == 0 ? h : (kind == 1 ? h - hq : h - hq - hkv);
    return kind;
}
__device__ __forceinline__ const void* source(const AppendArgs& a, int64_t t, int h, int64_t& at) {
    int n;
    const int kind = kind_of(a, h, n);
    at = kind == 0 ? t * a.q_ts + n * a.q_hs : kind == 1 ? t * a.k_ts + n * a.k_hs : t * a.v_ts + n * a.v_hs;
    return kind == 0 ? a.q : (kind == 1 ? a.k : a.v);
}

// Where a token goes: its offset in the cache, or put = false.
struct Slot {
    int64_t at;
    bool put;
};
__device__ __forceinline__ Slot slot_of(const AppendArgs& a, int64_t slot, bool tell) {
    Slot s{0, slot >= 0};  // a negative slot: the token is not appended
    if (s.put) {
        const int64_t page = slot >> 32 ? slot / a.kv.page_size : (uint32_t)slot / (uint32_t)a.kv.page_size;
        if (page >= a.kv.n_pages) {
            s.put = false;
            if (tell) set_status(a.kv.status, MOE_ERR_BAD_INDEX);
        } else {
            s.at = page * a.kv.page_stride + (slot - page * a.kv.page_size) * a.kv.token_stride;
        }
    }
    return s;
}

// The scale of head h's values in an E4M3 cache, and what they are multiplied by on their way there.
__device__ __forceinline__ float scale_of(const AppendArgs& a, int h) {
    int n;
    const int kind = kind_of(a, h, n);
    return kind == 0 || a.kv.type != MOE_E4M3 ? 1.f : (kind == 1 ? a.kv.k_scale : a.kv.v_scale)[n];
}
__device__ __forceinline__ float inverse_scale(const AppendArgs& a, int h) { return 1.f / scale_of(a, h); }

// Rotates an item of head h (raw runs in r0, r1) and writes it where it belongs.
template <int VEC, class R>
__device__ __forceinline__ void finish(const AppendArgs& a, int64_t t, int h, const Item<VEC>& it, const Slot& slot,
                                       const R& r0, const R& r1, const float (&cs)[VEC], const float (&sn)[VEC],
                                       float inv, int xt, int ct) {
    int n;
    const int kind = kind_of(a, h, n);
    if (kind != 0 && !slot.put) return;
    float x0[VEC], x1[VEC];
    r0.get(xt, x0);
    r1.get(xt, x1);
    if (it.turn && kind != 2) {
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
        store_run<VEC>(a.q_out, t * a.qo_ts + n * a.qo_hs + it.e0, xt, x0);
        store_run<VEC>(a.q_out, t * a.qo_ts + n * a.qo_hs + it.e1, xt, x1);
    } else {
        if (ct == MOE_E4M3) {
            if (fabsf(inv) == INFINITY) {  // a scale below 2^-128: its inverse is past fp32, the quotients need not be
                const float scale = scale_of(a, h);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    x0[i] /= scale;
                    x1[i] /= scale;
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    x0[i] *= inv;
                    x1[i] *= inv;
                }
            }
        }
        void* cache = kind == 1 ? a.kv.k : a.kv.v;
        store_run<VEC>(cache, slot.at + n * a.kv.head_stride + it.e0, ct, x0);
        store_run<VEC>(cache, slot.at + n * a.kv.head_stride + it.e1, ct, x1);
    }
}

// Any types and alignment: a CTA a token.
template <int VEC>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a) {
    grid_launch_next();
    grid_dep_wait();
    const int64_t t = blockIdx.x;
    const int items = a.kv.head_dim / (2 * VEC), heads = a.kv.q_heads + 2 * a.kv.kv_heads;
    const int step = blockDim.x / items, g = threadIdx.x / items;
    if (g >= step) return;
    const Item<VEC> it(a, threadIdx.x % items);
    const int pos = a.rot > 0 ? a.positions[t] : 0;
    if (a.rot > 0 && (pos < 0 || pos >= a.n_positions)) {  // no table row: nothing of this token is written
        if (threadIdx.x == 0) set_status(a.kv.status, MOE_ERR_BAD_INDEX);
        return;
    }
    const Slot slot = slot_of(a, a.slots[t], threadIdx.x == 0);
    float cs[VEC], sn[VEC];
    if (it.turn) {
        const float* row = a.cos_sin + (int64_t)pos * a.rot + it.j * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            cs[i] = row[i];
            sn[i] = row[a.rot / 2 + i];
        }
    }
    for (int h = g; h < heads; h += step) {
        int64_t at;
        const void* src = source(a, t, h, at);
        Raw<VEC> r0, r1;
        r0.load(src, at + it.e0, a.type);
        r1.load(src, at + it.e1, a.type);
        finish<VEC>(a, t, h, it, slot, r0, r1, cs, sn, inverse_scale(a, h), a.type, a.kv.type);
    }
}

__device__ __forceinline__ void cp_async16_l1(uint4* dst, const void* src) {  // read by the whole CTA: through L1
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// 16-bit q, k and v in runs of 8, the cache of their type (CT = XT) or E4M3.  CTAs walk the
// (token, block of heads) pairs; a thread's runs and table entries of the next pair come
// through a ring in shared memory that it alone reads, and the position that a copy of the
// table needs is fetched one step before.
template <int XT, int CT>
__global__ void __launch_bounds__(kThreads) append_ring_kernel(const AppendArgs a) {
    constexpr int VEC = 8, kPieces = 2 * kHeads + 4;
    extern __shared__ uint4 ring[];  // [stage][piece][thread]
    grid_launch_next();
    grid_dep_wait();
    const int items = a.kv.head_dim / (2 * VEC), heads = a.kv.q_heads + 2 * a.kv.kv_heads;
    const int step = blockDim.x / items, g = threadIdx.x / items;
    if (g >= step) return;
    const Item<VEC> it(a, threadIdx.x % items);
    const int blocks = (heads + step * kHeads - 1) / (step * kHeads);  // of heads, a token
    const int64_t total = (int64_t)a.T * blocks;
    auto token = [&](int64_t n) { return blocks == 1 ? n : n / blocks; };
    auto piece = [&](int stage, int i) { return ring + (stage * kPieces + i) * blockDim.x + threadIdx.x; };
    auto position = [&](int64_t n) { return a.rot > 0 && n < total ? a.positions[token(n)] : 0; };
    auto valid = [&](int pos) { return a.rot == 0 || (pos >= 0 && pos < a.n_positions); };
    auto copy = [&](int64_t n, int pos, int stage) {
        if (n < total) {
            const int64_t t = token(n);
            const int h0 = (int)(n - t * blocks) * step * kHeads + g;
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                const int h = h0 + i * step;
                if (h >= heads) break;
                int64_t at;
                const uint16_t* src = static_cast<const uint16_t*>(source(a, t, h, at));
                cp_async16(piece(stage, 2 * i), src + at + it.e0);
                cp_async16(piece(stage, 2 * i + 1), src + at + it.e1);
            }
            if (it.turn && valid(pos)) {
                const float* row = a.cos_sin + (int64_t)pos * a.rot + it.j * VEC;
#pragma unroll
                for (int i = 0; i < 4; ++i) cp_async16_l1(piece(stage, 2 * kHeads + i), row + (i & 1) * 4 + (i >> 1) * (a.rot / 2));
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int64_t n = blockIdx.x;
    // positions and slots of this step and the next ones
    int pos[kStages];
    int64_t slots[kStages];
    auto look = [&](int64_t m, int i) {
        pos[i] = position(m);
        slots[i] = m < total ? a.slots[token(m)] : -1;
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) look(n + (int64_t)i * gridDim.x, i);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) copy(n + (int64_t)i * gridDim.x, pos[i], i);
    float inv[kHeads];
    int inv_h0 = -1;
    for (int stage = 0; n < total; n += gridDim.x, stage = stage + 1 == kStages ? 0 : stage + 1) {
        copy(n + (int64_t)(kStages - 1) * gridDim.x, pos[kStages - 1], stage == 0 ? kStages - 1 : stage - 1);
        const int64_t t = token(n);
        const int h0 = (int)(n - t * blocks) * step * kHeads + g;
        const int p0 = pos[0];
        const Slot slot = slot_of(a, slots[0], threadIdx.x == 0);
#pragma unroll
        for (int i = 0; i + 1 < kStages; ++i) {
            pos[i] = pos[i + 1];
            slots[i] = slots[i + 1];
        }
        look(n + (int64_t)kStages * gridDim.x, kStages - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        if (!valid(p0)) {  // no table row: nothing of this token is written
            if (threadIdx.x == 0) set_status(a.kv.status, MOE_ERR_BAD_INDEX);
            continue;
        }
        if (CT == MOE_E4M3 && h0 != inv_h0) {
#pragma unroll
            for (int i = 0; i < kHeads; ++i) inv[i] = h0 + i * step < heads ? inverse_scale(a, h0 + i * step) : 1.f;
            inv_h0 = h0;
        }
        float cs[VEC], sn[VEC];
        if (it.turn) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 c = *piece(stage, 2 * kHeads + i), s = *piece(stage, 2 * kHeads + 2 + i);
                cs[4 * i] = __uint_as_float(c.x), cs[4 * i + 1] = __uint_as_float(c.y);
                cs[4 * i + 2] = __uint_as_float(c.z), cs[4 * i + 3] = __uint_as_float(c.w);
                sn[4 * i] = __uint_as_float(s.x), sn[4 * i + 1] = __uint_as_float(s.y);
                sn[4 * i + 2] = __uint_as_float(s.z), sn[4 * i + 3] = __uint_as_float(s.w);
            }
        }
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            const int h = h0 + i * step;
            if (h >= heads) break;
            Raw<VEC, false> r0, r1;
            r0.set(piece(stage, 2 * i), 0);
            r1.set(piece(stage, 2 * i + 1), 0);
            finish<VEC>(a, t, h, it, slot, r0, r1, cs, sn, inv[i], XT, CT);
        }
    }
}

// Whether every run of `vec` elements of the call is aligned, and the table's too.
bool fits(const AppendArgs& a, int vec) {
    return a.rot / 2 % vec == 0 && a.kv.head_dim % (2 * vec) == 0 && runs_aligned(a.q, a.type, vec, a.q_ts, a.q_hs) &&
           runs_aligned(a.k, a.type, vec, a.k_ts, a.k_hs) && runs_aligned(a.v, a.type, vec, a.v_ts, a.v_hs) &&
           runs_aligned(a.q_out, a.type, vec, a.qo_ts, a.qo_hs);
}

int threads_of(const AppendArgs& a, int vec, int each) {  // one item of `each` heads a thread
    const int items = a.kv.head_dim / (2 * vec), heads = a.kv.q_heads + 2 * a.kv.kv_heads;
    return std::min(kThreads, (items * ((heads + each - 1) / each) + 31) / 32 * 32);
}

template <int VEC>
cudaError_t launch(const AppendArgs& a, cudaStream_t st) {
    return launch_pdl(append_kernel<VEC>, dim3(a.T), dim3(threads_of(a, VEC, 2)), 0, st, a);
}

template <int XT, int CT>
cudaError_t launch_ring(const AppendArgs& a, cudaStream_t st) {
    const auto kernel = append_ring_kernel<XT, CT>;
    const int threads = threads_of(a, 8, kHeads), warps = threads / 32;
    const int smem = kStages * (2 * kHeads + 4) * threads * 16;
    static std::atomic<uint64_t> configured;
    cudaError_t err = ensure_smem_limit((const void*)kernel, kStages * (2 * kHeads + 4) * kThreads * 16, configured, true);
    if (err != cudaSuccess) return err;
    // one round of CTAs, each walking its share of the tokens
    static std::atomic<int> resident[kThreads / 32 + 1];  // CTAs an SM holds, by warps
    int per_sm = resident[warps].load(std::memory_order_relaxed);
    if (per_sm == 0) {
        err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
        if (err != cudaSuccess) return err;
        if (per_sm < 1) per_sm = 1;
        resident[warps].store(per_sm, std::memory_order_relaxed);
    }
    const int items = a.kv.head_dim / 16, heads = a.kv.q_heads + 2 * a.kv.kv_heads, step = threads / items;
    const int64_t total = (int64_t)a.T * ((heads + step * kHeads - 1) / (step * kHeads));
    const int64_t grid = std::min<int64_t>(total, (int64_t)per_sm * a.sm_count);
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(threads), smem, st, a);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    const bool table16 = a.rot == 0 || (reinterpret_cast<uintptr_t>(a.cos_sin) % 16 == 0 && a.rot % 8 == 0);
    if (fits(a, 8) && table16 && is_float16(a.type) && (a.kv.type == a.type || a.kv.type == MOE_E4M3)) {
        if (a.type == MOE_BF16)
            return a.kv.type == MOE_BF16 ? launch_ring<MOE_BF16, MOE_BF16>(a, st) : launch_ring<MOE_BF16, MOE_E4M3>(a, st);
        return a.kv.type == MOE_F16 ? launch_ring<MOE_F16, MOE_F16>(a, st) : launch_ring<MOE_F16, MOE_E4M3>(a, st);
    }
    return fits(a, 8) ? launch<8>(a, st) : fits(a, 4) ? launch<4>(a, st) : launch<1>(a, st);
}

}  // namespace moe
