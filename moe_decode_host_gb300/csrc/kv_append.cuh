// What the appends share: a token's heads, its position's axes and its rows of the rotation table.
#pragma once

#include "ptx.cuh"
#include "vec.cuh"

namespace moe {
namespace {

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

__device__ __forceinline__ void cp_async16_l1(uint4* dst, const void* src) {  // read by the whole CTA: through L1
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// A token's position along its axes; valid: the table has a row for each.
struct Place {
    int pos[kMaxAxes];
    bool valid;
    __device__ __forceinline__ int at(int axis) const {  // no indexing of registers
        return axis == 0 ? pos[0] : (axis == 1 ? pos[1] : (axis == 2 ? pos[2] : pos[3]));
    }
};
__device__ __forceinline__ Place place_of(const AppendArgs& a, int64_t t) {
    Place p{{0, 0, 0, 0}, true};
    if (a.rot == 0) return p;
    if (a.axes == 1) {
        p.pos[0] = a.positions[t];
        p.valid = p.pos[0] >= 0 && p.pos[0] < a.n_positions;
        return p;
    }
#pragma unroll
    for (int i = 0; i < kMaxAxes; ++i)
        if (i < a.axes) {
            p.pos[i] = a.positions[i * a.pos_stride + t];
            p.valid = p.valid && p.pos[i] >= 0 && p.pos[i] < a.n_positions;
        }
    return p;
}

// Cosines and sines of N pairs from `pair` on.  FOURS: aligned fours of pairs have one axis, and the
// table's rows are aligned for reads of four (fours_of).
template <int N, bool FOURS = false>
__device__ __forceinline__ void turn_of(const AppendArgs& a, const Place& p, int pair, float (&cs)[N], float (&sn)[N]) {
    if constexpr (FOURS) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const int axis = a.axes == 1 ? 0 : axis_of(a, pair + i);
            const float* at = a.cos_sin + (int64_t)p.at(axis) * a.rot + pair + i;
            const float4 c = *reinterpret_cast<const float4*>(at), s = *reinterpret_cast<const float4*>(at + a.rot / 2);
            cs[i] = c.x, cs[i + 1] = c.y, cs[i + 2] = c.z, cs[i + 3] = c.w;
            sn[i] = s.x, sn[i + 1] = s.y, sn[i + 2] = s.z, sn[i + 3] = s.w;
        }
    } else if (a.axes == 1) {
        const float* row = a.cos_sin + (int64_t)p.pos[0] * a.rot + pair;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            cs[i] = row[i];
            sn[i] = row[a.rot / 2 + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float* at = a.cos_sin + (int64_t)p.at(axis_of(a, pair + i)) * a.rot + pair + i;
            cs[i] = at[0];
            sn[i] = at[a.rot / 2];
        }
    }
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

// Turns the pairs of two runs: element i of both where not interleaved, else 2i and 2i + 1 of the
// double run that they form.
template <int VEC>
__device__ __forceinline__ void rotate(bool interleaved, float (&x0)[VEC], float (&x1)[VEC], const float (&cs)[VEC],
                                       const float (&sn)[VEC]) {
    if (interleaved) {
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

// Whether every run of `vec` elements of the call is aligned.
inline bool append_fits(const AppendArgs& a, int vec) {
    return a.rot / 2 % vec == 0 && a.kv.head_dim % (2 * vec) == 0 && runs_aligned(a.q, a.type, vec, a.q_ts, a.q_hs) &&
           runs_aligned(a.k, a.type, vec, a.k_ts, a.k_hs) && runs_aligned(a.v, a.type, vec, a.v_ts, a.v_hs) &&
           runs_aligned(a.q_out, a.type, vec, a.qo_ts, a.qo_hs);
}
// Whether aligned fours of pairs turn by one axis each.
inline bool one_axis_fours(const AppendArgs& a) {
    if (a.axes > 1)
        for (int i = 0; i < a.rot / 2; ++i)
            if (axis_of(a, i) != axis_of(a, i & ~3)) return false;
    return true;
}
inline bool fours_of(const AppendArgs& a) {
    return reinterpret_cast<uintptr_t>(a.cos_sin) % 16 == 0 && a.rot % 8 == 0 && one_axis_fours(a);
}

}  // namespace
}  // namespace moe
