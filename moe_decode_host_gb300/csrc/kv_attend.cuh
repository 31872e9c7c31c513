// Attention of one new token per sequence over the paged cache.
//
//   o = sum_j softmax_j(scale * q . k_j) v_j,  j in [max(0, len - window), len)
//
// Bound by the cache's bytes, each read once for a block of up to 32 query heads of a key
// head (16 from head_dim 144 on).  Measured on a GB300, with the share of a plain copy's
// rate: 32 ragged sequences (1.1 GB of bf16) 174 us (94%); 64 long ones in E4M3, 16 query
// heads a key head (1.6 GB) 295 us (81%: issue latency); one sequence of 4097 tokens 13.5 us, 15.1
// with its rows in memory and not in L2, a chain of latencies.
//
// Split.  The attended tokens of a (sequence, key head, block of query heads) form a
// segment of units of 16 tokens (32 where a row is at most 128 bytes), and a few places more
// for the cost of starting it; the segments of a call are laid end to end and every CTA gets
// the same number of places of that line, whatever the lengths.  A CTA walks its stretch as
// pieces of segments.  A segment inside one CTA is finished there; the parts of one that
// spans CTAs go to a workspace, and the CTA that arrives last joins them, always in the
// order of the line, so the result does not depend on timing.
//
// A piece.  Each warp takes every fourth unit through a ring of its own (cp.async, no
// barrier between warps) with its own running maximum and sum; the warps are joined in
// shared memory at the piece's end.  The transposed products keep the padding small:
//   S^T [16 tokens x 8 heads] = K Q^T,   O^T [16 dims x 8 heads] += V^T P^T
// put the query heads in the 8-wide side of m16n8k16, and a head's statistics in the
// same lanes for S and O, so rescaling needs no exchange.  E4M3 keys and values become
// f16 in registers (exactly): the order of dimensions within a 16-wide step of the
// contraction is free, so a lane's four consecutive bytes serve as its four elements, in the
// tokens of V^T P^T as in the dimensions of K Q^T.  The weights P are two 16-bit terms each.
// mma.sync suffices: the products take 14% (bf16) and 46% (E4M3, 16 heads) of the tensor pipe,
// and their operands come from registers.
#pragma once

#include <algorithm>

#include "attend_plan.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace moe {
namespace {

constexpr int kWarps = kAttendWarps, kThreads = kWarps * 32;

// 16-bit types: rows are read 8 in a row.  E4M3: values 8 in a row, keys in the order of
// token_of (rows 0, 1, 4, 5, 8, 9, 12, 13 and the others); the three bits tell both apart.
template <bool F8>
__device__ __forceinline__ int swap_of(int row) {
    return F8 ? (row & 1) | (row >> 1 & 2) | (((row >> 1) ^ (row >> 3)) & 1) << 2 : row & 7;
}
// The token of a 16-token tile in row r of S^T.  E4M3: rows 2c, 2c + 1, 2c + 8, 2c + 9 hold
// tokens 4c .. 4c + 3, the order in which the byte-wise ldmatrix.trans delivers values.
template <bool F8>
__device__ __forceinline__ int token_of(int r) {
    return F8 ? (r >> 1 & 3) * 4 + (r & 1) + (r >> 3) * 2 : r;
}

// 16 bytes of a row of the cache, or zeros where `bytes` is 0.  Rows are read whole: 128 bytes at a time from L2.
__device__ __forceinline__ void cp_row16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cp_row16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// Two 16 x 16 byte matrices transposed: lane (g, c) gets rows (dims) g, g + 8 of the first,
// then of the second, columns (tokens) 4c .. 4c + 3.
__device__ __forceinline__ void ldsm_bytes_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What a part with maximum m counts under the joint maximum (a part may have seen nothing).
__device__ __forceinline__ float part_weight(float m, float top) { return m == -INFINITY ? 0.f : fast_exp2(m - top); }

// Two E4M3 codes (the low or high half of w) as f16x2.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// Attended tokens of sequence b: [first, first + count).
struct Span {
    int first, count;
};
__host__ __device__ __forceinline__ int64_t room_of(const AttendArgs& a) {  // tokens that a row of the table can hold
    const int64_t room = (int64_t)a.max_pages * a.kv.page_size;
    return room < kMaxTokens ? room : kMaxTokens;
}
__device__ __forceinline__ Span span_of(const AttendArgs& a, int b) {
    const int64_t room = room_of(a);
    int64_t n = a.lengths[b];
    n = n < 0 ? 0 : (n > room ? room : n);
    const int first = a.window > 0 && n > a.window ? (int)n - a.window : 0;
    return {first, (int)n - first};
}
// Places of one of its segments on the line: kStart for what a piece costs, then its units.
__device__ __forceinline__ int places_of(const Span& s, int unit) {
    return s.count > 0 ? (s.count + unit - 1) / unit + kStart : 0;
}

// T: 0 bf16, 1 f16, 2 E4M3 (computed in f16).  DP: head_dim (EXACT) or a bound of it; with
// the dimension known no step of the products is conditional, and they overlap.  NT: blocks
// of 8 query heads.
template <int T, int DP, int NT, bool EXACT>
__global__ void __launch_bounds__(kThreads, ctas_an_sm(DP, T == 2 ? 1 : 2, NT))
    attend_kernel(const AttendArgs a, const AttendPlan p) {
    constexpr bool BF = T == 0, F8 = T == 2;
    constexpr float lift = BF ? 0.f : kLift;
    constexpr int HC = 8 * NT;
    constexpr int ES = F8 ? 1 : 2;
    constexpr int U = unit_tokens(DP * ES), MT = U / 16;  // tokens of a unit, in tiles of 16
    constexpr uint32_t kAll = U == 32 ? 0xffffffffu : 0xffffu;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_m[kWarps][HC], s_l[kWarps][HC], s_scale[HC], s_inv[HC];
    __shared__ uint32_t s_mask[kWarps][kMaxStages];
    __shared__ long long s_sum[kWarps], s_rest[kWarps], s_before;
    __shared__ int s_b, s_last, s_longest[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    constexpr int CPR = DP * ES / 16;
    const int D = EXACT ? DP : a.kv.head_dim, steps = D / 16;
    const int qpitch = D * 2 + 16;
    const int pitch = EXACT ? row_pitch(CPR) : p.pitch, swizzle = EXACT ? row_swizzle(CPR) : p.swizzle;
    const int cpr = EXACT ? CPR : p.cpr;
    const int unit_bytes = 2 * U * pitch;
    uint8_t* s_q = smem;
    uint8_t* ring = smem + HC * (DP * 2 + 16) + warp * p.stages * unit_bytes;
    const uint32_t ring_u = smem_u32(ring), q_u = smem_u32(s_q);
    const int heads = a.kv.q_heads, group = heads / a.kv.kv_heads;
    const int per_b = a.kv.kv_heads * p.chunks;  // segments of a sequence
    grid_launch_next();
    grid_dep_wait();

    // ---- this CTA's stretch of the line: a scan over the lengths, kThreads at a time ----
    const int own = blockIdx.x < a.B ? a.lengths[blockIdx.x] : 1;  // its own share of the empty sequences, below
    // sums of places, with the number of sequences that have any above kOne
    constexpr long long kOne = 1ll << 44;
    const int u0 = tid < a.B ? places_of(span_of(a, tid), U) : 0;
    long long rest = 0;  // behind the first kThreads sequences
    for (int b = kThreads + tid; b < a.B; b += kThreads) {
        const int u = places_of(span_of(a, b), U);
        rest += u > 0 ? u + kOne : 0;
    }
    auto scan = [&](long long x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        return x;
    };
    const long long x0 = scan(u0 > 0 ? u0 + kOne : 0);
    if (a.B > kThreads) rest = scan(rest);
    const int longest = __reduce_max_sync(0xffffffffu, u0);
    if (lane == 31) {
        s_sum[warp] = x0;
        s_rest[warp] = rest;
        s_longest[warp] = longest;
    }
    __syncthreads();
    long long ahead = 0, chunk = 0, total = 0;  // places ahead of this warp, of the first kThreads sequences, of all
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) ahead += s_sum[w];
        chunk += s_sum[w];
        total += s_rest[w];
    }
    total += chunk;
    // short segments, no more than CTAs: a CTA each, which costs less than joining parts.  They all
    // get the places of the longest such segment
    bool level = a.B <= kThreads && (total >> 44) * per_b <= gridDim.x;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) level = level && s_longest[w] <= kWhole + kStart;
    const long long units = ((total & (kOne - 1)) - (total >> 44) * kStart) * per_b;
    long long ctas = (units + kMinUnits - 1) / kMinUnits;
    if (ctas > gridDim.x) ctas = gridDim.x;
    if (level) ctas = (total >> 44) * per_b;
    total = level ? ctas * (kWhole + kStart) : (total & (kOne - 1)) * per_b;
    chunk &= kOne - 1;
    long long u_begin = 0, u_end = 0;
    if ((long long)blockIdx.x < ctas) {
        if (total < 1 << 21) {  // in 32 bits: a grid is below 2^11
            u_begin = (uint32_t)total * blockIdx.x / (uint32_t)ctas;
            u_end = (uint32_t)total * (blockIdx.x + 1) / (uint32_t)ctas;
        } else {
            u_begin = total * blockIdx.x / ctas;
            u_end = total * (blockIdx.x + 1) / ctas;
        }
        // the sequence that holds place u_begin
        const int here = level ? kWhole + kStart : u0;
        const long long lo = (level ? (((ahead + x0) >> 44) - 1) * here : ((ahead + x0) & (kOne - 1)) - here) * per_b;
        if (u0 > 0 && u_begin >= lo && u_begin < lo + (long long)here * per_b) {
            s_b = tid;
            s_before = lo;
        }
        for (int b0 = kThreads; !level && chunk * per_b <= u_begin; b0 += kThreads) {
            const int b = b0 + tid, u = b < a.B ? places_of(span_of(a, b), U) : 0;
            const long long x = scan(u);
            __syncthreads();
            if (lane == 31) s_sum[warp] = x;
            __syncthreads();
            long long at = chunk + x - u;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) at += s_sum[w];
                chunk += s_sum[w];
            }
            if (u > 0 && u_begin >= at * per_b && u_begin < (at + u) * per_b) {
                s_b = b;
                s_before = at * per_b;
            }
        }
    }
    // ---- sequences without a token, and lengths out of range ----
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const int n = b == (int)blockIdx.x ? own : a.lengths[b];
        if ((n < 0 || n > room_of(a)) && tid == 0) set_status(a.kv.status, MOE_ERR_BAD_INDEX);
        if (n > 0 && room_of(a) > 0) continue;
        for (int i = tid; i < heads * (D / 2); i += kThreads) {
            const int h = i / (D / 2), d = i % (D / 2) * 2;
            uint16_t* o = static_cast<uint16_t*>(a.out) + b * a.out_ts + h * a.out_hs + d;
            *reinterpret_cast<uint32_t*>(o) = 0u;
        }
        if (a.lse)
            for (int h = tid; h < heads; h += kThreads) a.lse[(int64_t)b * heads + h] = -INFINITY;
    }

    if ((long long)blockIdx.x >= ctas) return;
    __syncthreads();
    int b = s_b;
    long long before = s_before;  // places ahead of sequence b
    Span span = span_of(a, b);
    int ub = 0, nu = 0;  // its places and its units
    auto measure = [&]() {
        ub = places_of(span, U);
        nu = ub - kStart;
        if (level && ub > 0) ub = kWhole + kStart;
    };
    measure();

    for (long long u = u_begin; u < u_end;) {
        while (u >= before + (long long)ub * per_b) {  // next sequence with a token
            before += (long long)ub * per_b;
            ++b;
            span = span_of(a, b);
            measure();
        }
        const int seg = (int)((u - before) / ub);
        const long long seg_begin = before + (long long)seg * ub;
        const int last_place = (int)((u_end < seg_begin + ub ? u_end : seg_begin + ub) - seg_begin);
        const int first_u = max(0, (int)(u - seg_begin) - kStart), last_u = min(nu, max(0, last_place - kStart));
        u = seg_begin + last_place;
        if (last_u == first_u) continue;  // nothing but the start of a segment
        const int kh = seg / p.chunks, h0 = kh * group + seg % p.chunks * p.chunk;
        const int nh = min(p.chunk, kh * group + group - h0);  // query heads of this segment

        // ---- loads: unit x of this warp is first_u + warp + kWarps * x ----
        const int n_mine = (last_u - first_u - warp + kWarps - 1) / kWarps;
        const uint8_t* kb = static_cast<const uint8_t*>(a.kv.k) + kh * a.kv.head_stride * ES;
        const uint8_t* vb = static_cast<const uint8_t*>(a.kv.v) + kh * a.kv.head_stride * ES;
        const int32_t* table = a.page_table + b * a.table_stride;
        int next_page = -1, next_entry = 0;  // the page and entry of row `lane` of the next unit
        auto look_up = [&](int x) {
            const int j = (first_u + warp + kWarps * x) * U + lane;
            if (lane < U && x < n_mine && j < span.count) {
                const uint32_t t = span.first + j, pg = (uint32_t)((uint64_t)t * p.page_mul >> p.page_shift);
                next_entry = t - pg * a.kv.page_size;
                next_page = table[pg];
            }
        };
        auto issue = [&](int x, int slot) {  // the unit that look_up last saw
            if (x < n_mine) {
                const bool in = lane < U && (first_u + warp + kWarps * x) * U + lane < span.count;
                const bool ok = in && next_page >= 0 && next_page < a.kv.n_pages;
                if (in && !ok) set_status(a.kv.status, MOE_ERR_BAD_INDEX);
                const uint32_t off =
                    ok ? (uint32_t)(((next_page * a.kv.page_stride + next_entry * a.kv.token_stride) * ES) >> p.shift) : 0u;
                const uint32_t mask = __ballot_sync(0xffffffffu, ok);
                if (lane == 0) s_mask[warp][slot] = mask;
                const uint32_t dst = ring_u + slot * unit_bytes;
                if (EXACT && mask == kAll) {
                    static_assert(!EXACT || U * CPR % 32 == 0, "whole rounds of the warp");
                    const uint64_t unit = 1ull << p.shift;
#pragma unroll
                    for (int i0 = 0; i0 < U * CPR; i0 += 32) {
                        const int r = (i0 + lane) / CPR, col = (i0 + lane) % CPR * 16;
                        const uint64_t o = __shfl_sync(0xffffffffu, off, r) * unit + col;
                        const uint32_t at = dst + r * pitch + (col ^ (swap_of<F8>(r) & swizzle) << 4);
                        cp_row16(at, kb + o);
                        cp_row16(at + U * pitch, vb + o);
                    }
                } else {
                    for (int i0 = 0; i0 < U * cpr; i0 += 32) {
                        const int i = i0 + lane;
                        const int row = EXACT ? i / CPR : (int)((uint32_t)i * p.inv >> 20), col = (i - row * cpr) * 16;
                        const uint64_t o = ((uint64_t)__shfl_sync(0xffffffffu, off, row & (U - 1)) << p.shift) + col;
                        if (row < U) {
                            const uint32_t bytes = (mask >> row & 1u) ? 16u : 0u;  // rows left out are zeros
                            const uint32_t at = dst + row * pitch + (col ^ (swap_of<F8>(row) & swizzle) << 4);
                            cp_row16(at, kb + o, bytes);
                            cp_row16(at + U * pitch, vb + o, bytes);
                        }
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // queries first, so that they are on their way together with the first units
        constexpr int HW = HC / kWarps;  // heads a warp brings: warp, warp + kWarps, ...
        uint16_t raw[HW][DP / 32];
        const float k_scale = F8 ? a.kv.k_scale[kh] : 1.f, v_scale = F8 ? a.kv.v_scale[kh] : 1.f;
#pragma unroll
        for (int x = 0; x < HW; ++x) {
            const int h = warp + kWarps * x;
            const uint16_t* src = static_cast<const uint16_t*>(a.q) + b * a.q_ts + (h0 + h) * a.q_hs;
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) raw[x][i] = h < nh && lane + 32 * i < D ? src[lane + 32 * i] : (uint16_t)0;
        }
        look_up(0);
        for (int x = 0; x < p.stages - 1; ++x) {
            issue(x, x);
            look_up(x + 1);
        }
#pragma unroll
        for (int x = 0; x < HW; ++x) {
            const int h = warp + kWarps * x;
            float v[DP / 32], top = 0.f;
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) {
                v[i] = half_bits_to_f32(raw[x][i], a.q_type);
                top = fmaxf(top, fabsf(v[i]));
            }
            int e = 0;
            if constexpr (F8) {
                // q becomes f16 scaled by a power of two to a largest magnitude in [2^14, 2^15): a bf16
                // keeps all its bits down to 2^-28 of the largest
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                e = prescale_exp(top);
            }
            // the sign of the scores' factor is folded into q, so that the largest raw score is the
            // largest score
            const float factor = a.scale * kLog2e * k_scale;
            const float down = copysignf(F8 ? pow2i(-e) : 1.f, factor);
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) {
                const int d = lane + 32 * i;
                if (d < D)
                    reinterpret_cast<uint16_t*>(s_q + h * qpitch)[d] =
                        (uint16_t)(BF ? pack_bf16(v[i] * down, 0.f) : pack_f16(v[i] * down, 0.f));
            }
            // never zero: a score left out (-inf) must stay -inf under it.  NaN stays NaN
            const float up = fabsf(factor) * (F8 ? pow2i(e) : 1.f);
            if (lane == 0) s_scale[h] = up < 1e-37f ? 1e-37f : up;
        }
        __syncthreads();

        float o[DP / 16][NT][4], m[NT][2], l[NT][2], sc[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int i = 0; i < DP / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][t][j] = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[t][j] = -INFINITY;
                l[t][j] = 0.f;
                sc[t][j] = s_scale[8 * t + 2 * c + j];
            }
        }

        // where ldmatrix lanes read.  Keys: row lane % 16 of S^T, the 16-byte piece lane / 16 further on;
        // pieces come in pairs, so piece 2j + x is in place 2j ^ (x ^ swap)
        const int k_row = token_of<F8>(lane & 15), k_x = (lane >> 4) ^ (swap_of<F8>(k_row) & swizzle);
        // values: E4M3 as keys but in order; else tokens of half lane / 16, pieces of lane / 8 % 2
        const int v_row = F8 ? lane & 15 : (lane & 7) + ((lane >> 4) << 3);
        const int v_x = (F8 ? lane >> 4 : lane >> 3 & 1) ^ (swap_of<F8>(v_row) & swizzle);
        for (int x = 0, slot = 0; x < n_mine; ++x, slot = slot + 1 == p.stages ? 0 : slot + 1) {
            issue(x + p.stages - 1, slot == 0 ? p.stages - 1 : slot - 1);
            look_up(x + p.stages);
            cp_wait(p.stages - 1);
            __syncwarp();
            const uint32_t ku = ring_u + slot * unit_bytes, vu = ku + U * pitch;
            const uint32_t mask = s_mask[warp][slot];
            float s[MT][NT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int t = 0; t < NT; ++t) s[i][t][0] = s[i][t][1] = s[i][t][2] = s[i][t][3] = 0.f;
            // matrices of a load: halves of the tile's rows for a 16-byte piece, then for the next one
            const uint32_t k_at = ku + k_row * pitch, v_at = vu + v_row * pitch;
            if constexpr (F8) {
#pragma unroll
                for (int kk = 0; kk < DP / 16; kk += 2) {
                    if (kk < steps) {
                        uint32_t r[MT][4];
#pragma unroll
                        for (int i = 0; i < MT; ++i) ldsm4(r[i], k_at + i * 16 * pitch + ((kk ^ k_x) << 4));
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (kk + h < steps) {
                                uint2 q[NT];
#pragma unroll
                                for (int t = 0; t < NT; ++t)
                                    q[t] = *reinterpret_cast<const uint2*>(s_q + (8 * t + g) * qpitch + (kk + h) * 32 + c * 8);
#pragma unroll
                                for (int i = 0; i < MT; ++i) {
                                    const uint32_t f[4] = {e4m3_lo(r[i][2 * h]), e4m3_lo(r[i][2 * h + 1]),
                                                           e4m3_hi(r[i][2 * h]), e4m3_hi(r[i][2 * h + 1])};
#pragma unroll
                                    for (int t = 0; t < NT; ++t) mma16816<BF>(s[i][t], f, q[t].x, q[t].y);
                                }
                            }
                        }
                    }
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk) {
                    if (kk < steps) {
                        uint32_t r[MT][4];
#pragma unroll
                        for (int i = 0; i < MT; ++i) ldsm4(r[i], k_at + i * 16 * pitch + (((2 * kk) ^ k_x) << 4));
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const uint8_t* q = s_q + (8 * t + g) * qpitch + kk * 32 + c * 4;
                            const uint32_t q0 = *reinterpret_cast<const uint32_t*>(q);
                            const uint32_t q1 = *reinterpret_cast<const uint32_t*>(q + 16);
#pragma unroll
                            for (int i = 0; i < MT; ++i) mma16816<BF>(s[i][t], r[i], q0, q1);
                        }
                    }
                }
            }
            // softmax: lane (g, c) holds rows g, g + 8 of each tile, heads 2c, 2c + 1 of each block
            if (mask != kAll) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (!(mask >> (16 * i + token_of<F8>(g + 8 * (j >> 1))) & 1u)) {
#pragma unroll
                            for (int t = 0; t < NT; ++t) s[i][t][j] = -INFINITY;
                        }
            }
            float keep[NT][2];
            bool grown = false;
            uint32_t pb[MT][NT][2][2];  // two terms
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float top = fmaxf(s[0][t][j], s[0][t][2 + j]);
#pragma unroll
                    for (int i = 1; i < MT; ++i) top = fmaxf(top, fmaxf(s[i][t][j], s[i][t][2 + j]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    // the reference moves only when weights would pass 2^(kSlack + lift): any reference near the
                    // maximum does, and moving it costs a pass over the sums
                    const bool move = (top - m[t][j]) * sc[t][j] > kSlack;  // false where nothing was seen yet
                    const float mn = move ? top : m[t][j];
                    const float ref = mn == -INFINITY ? 0.f : fmaf(mn, sc[t][j], -lift);  // then every weight is 0
                    keep[t][j] = move ? fast_exp2(fmaf(m[t][j], sc[t][j], -ref) - lift) : 1.f;
                    grown |= move;
                    m[t][j] = mn;
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        s[i][t][j] = fast_exp2(fmaf(s[i][t][j], sc[t][j], -ref));
                        s[i][t][2 + j] = fast_exp2(fmaf(s[i][t][2 + j], sc[t][j], -ref));
                        sum += s[i][t][j] + s[i][t][2 + j];
                    }
                    l[t][j] = fmaf(l[t][j], keep[t][j], sum);
                }
                // a weight goes to the tensor cores as two terms of the values' 16-bit type, the nearest and
                // its remainder (2^-16 of the weight are lost with bf16, 2^-22 with f16): one term alone added
                // as much error as the output's rounding and, where one key outweighs the rest, took its own
                // rounding into every output (32 ragged 172.6 us with one term, 173.5 with two)
                auto pack = [](float x, float y) { return BF ? pack_bf16(x, y) : pack_f16(x, y); };
                auto low = [](uint32_t p) { return half_bits_to_f32(p & 0xffffu, BF ? MOE_BF16 : MOE_F16); };
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float x = s[i][t][2 * j], y = s[i][t][2 * j + 1];
                        const uint32_t p = pack(x, y);
                        pb[i][t][0][j] = transpose8x8(p);
                        pb[i][t][1][j] = transpose8x8(pack(x - low(p), y - low(p >> 16)));
                    }
            }
            if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
                for (int i = 0; i < DP / 16; ++i)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[i][t][j] *= keep[t][j & 1];
            }
#pragma unroll
            for (int k = 0; k < MT; ++k) {
                if constexpr (F8) {
#pragma unroll
                    for (int i = 0; i < DP / 16; i += 2) {
                        if (i < steps) {
                            uint32_t r[4];
                            ldsm_bytes_t(r, v_at + 16 * k * pitch + ((i ^ v_x) << 4));
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (i + h < steps) {
                                    const uint32_t f[4] = {e4m3_lo(r[2 * h]), e4m3_lo(r[2 * h + 1]), e4m3_hi(r[2 * h]),
                                                           e4m3_hi(r[2 * h + 1])};
#pragma unroll
                                    for (int t = 0; t < NT; ++t)
#pragma unroll
                                        for (int j = 0; j < 2; ++j) mma16816<BF>(o[i + h][t], f, pb[k][t][j][0], pb[k][t][j][1]);
                                }
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < DP / 16; ++i) {
                        if (i < steps) {
                            uint32_t r[4];
                            ldsm4_t(r, v_at + 16 * k * pitch + (((2 * i) ^ v_x) << 4));
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int j = 0; j < 2; ++j) mma16816<BF>(o[i][t], r, pb[k][t][j][0], pb[k][t][j][1]);
                        }
                    }
                }
            }
            __syncwarp();
        }
        // maxima of scores from here on, in powers of two, less the lift
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (m[t][j] != -INFINITY) m[t][j] = fmaf(m[t][j], sc[t][j], -lift);

        // ---- join the warps ----
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float y = l[t][j];
                y += __shfl_xor_sync(0xffffffffu, y, 4);
                y += __shfl_xor_sync(0xffffffffu, y, 8);
                y += __shfl_xor_sync(0xffffffffu, y, 16);
                if (g == 0) {
                    s_m[warp][8 * t + 2 * c + j] = m[t][j];
                    s_l[warp][8 * t + 2 * c + j] = y;
                }
            }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        float* mine_o = reinterpret_cast<float*>(ring);  // [HC][D + 4]; the ring is empty now
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int h = 8 * t + 2 * c + j;
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][h]);
                const float f = m[t][j] == -INFINITY ? 0.f : fast_exp2(m[t][j] - top);
#pragma unroll
                for (int i = 0; i < DP / 16; ++i) {
                    if (i < steps) {
                        mine_o[h * (D + 4) + 16 * i + g] = o[i][t][j] * f;
                        mine_o[h * (D + 4) + 16 * i + g + 8] = o[i][t][2 + j] * f;
                    }
                }
            }
        __syncthreads();
        const bool whole = first_u == 0 && last_u == nu;
        float* slot_base = nullptr;
        int i0 = 0, i1 = 0;
        if (!whole) {
            // CTAs that hold the segment's first and last unit
            i0 = (int)(((seg_begin + kStart + 1) * ctas - 1) / total);
            i1 = (int)(((seg_begin + ub) * ctas - 1) / total);
            const int slot = 2 * blockIdx.x + ((int)blockIdx.x == i0 ? 1 : 0);
            slot_base = static_cast<float*>(a.workspace) + p.slots + (int64_t)slot * HC * (D + 2);
        }
        if (tid < HC) {
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][tid]);
            // a warp with no maximum has seen nothing (sum 0) or NaN alone (sum NaN, which has to stay)
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += s_l[w][tid] * part_weight(s_m[w][tid], top);
            if (whole) {
                s_inv[tid] = v_scale / sum;
                if (!(sum != 0.f)) s_inv[tid] = 0.f;
                if (a.lse && tid < nh) a.lse[(int64_t)b * heads + h0 + tid] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
            } else {
                slot_base[tid] = top;
                slot_base[HC + tid] = sum;
            }
        }
        __syncthreads();
        {
            const float* all = reinterpret_cast<const float*>(smem + HC * (DP * 2 + 16));
            const int step = p.stages * unit_bytes / 4;
            for (int i = tid; i < nh * (D / 2); i += kThreads) {
                const int h = i / (D / 2), d = i % (D / 2) * 2;
                float2 v = make_float2(0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 y = *reinterpret_cast<const float2*>(all + w * step + h * (D + 4) + d);
                    v.x += y.x;
                    v.y += y.y;
                }
                if (whole) {
                    const float f = s_inv[h];
                    uint16_t* dst = static_cast<uint16_t*>(a.out) + b * a.out_ts + (h0 + h) * a.out_hs + d;
                    *reinterpret_cast<uint32_t*>(dst) =
                        a.q_type == MOE_BF16 ? pack_bf16(v.x * f, v.y * f) : pack_f16(v.x * f, v.y * f);
                } else {
                    *reinterpret_cast<float2*>(slot_base + 2 * HC + h * D + d) = v;
                }
            }
        }
        if (!whole) {
            // ---- join the CTAs: the last to arrive, in the order of the line ----
            __threadfence();
            __syncthreads();
            int* counters = static_cast<int*>(a.workspace);
            if (tid == 0) {
                const int parts = i1 - i0 + 1;
                s_last = atomicAdd(counters + i0, 1) == parts - 1;
                if (s_last) counters[i0] = 0;  // as the next call expects it
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                const float* base = static_cast<const float*>(a.workspace) + p.slots;
                auto part = [&](int i) { return base + (int64_t)(2 * i + (i == i0 ? 1 : 0)) * HC * (D + 2); };
                // the parts' sums come through the idle ring, as many as it holds at once; a thread adds up
                // what it copied itself.  Meanwhile a warp a head and a lane a part find the joint
                // maximum and sum, then every part's weight
                constexpr int IT = (HC * DP / 4 + kThreads - 1) / kThreads;  // 4-wide pieces of a thread
                const int parts = i1 - i0 + 1, pieces = nh * (D / 4);
                float* weights = reinterpret_cast<float*>(smem + HC * (DP * 2 + 16));  // [nh][parts]
                float4* room = reinterpret_cast<float4*>(weights + (nh * parts + 3) / 4 * 4);
                const int fit = (kWarps * p.stages * unit_bytes / 4 - (nh * parts + 3) / 4 * 4) / (nh * D);
                const int stride = 2 * HC * (D + 2);  // floats from a CTA's slots to the next one's
                auto bring = [&](int k0) {
                    // the first part is in its CTA's second slot, the others in the first ones
                    const float* from = part(i0 + k0) + 2 * HC + 4 * tid;
                    uint32_t to = smem_u32(room + tid);
#pragma unroll 4
                    for (int k = k0; k < min(parts, k0 + fit); ++k) {
#pragma unroll
                        for (int x = 0; x < IT; ++x)
                            if (tid + x * kThreads < pieces) cp_row16(to + x * kThreads * 16, from + 4 * x * kThreads);
                        from += k == 0 ? stride / 2 : stride;
                        to += pieces * 16;
                    }
                };
                bring(0);
                for (int h = warp; h < nh; h += kWarps) {
                    float top = -INFINITY, sum = 0.f;
#pragma unroll 4
                    for (int i = lane; i < parts; i += 32) {
                        const float mi = part(i0 + i)[h], li = part(i0 + i)[HC + h];
                        const float mn = fmaxf(top, mi);
                        sum = sum * part_weight(top, mn) + li * part_weight(mi, mn);
                        top = mn;
                        weights[h * parts + i] = mi;
                    }
                    float all = top;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
                    sum *= part_weight(top, all);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    for (int i = lane; i < parts; i += 32) weights[h * parts + i] = part_weight(weights[h * parts + i], all);
                    if (lane == 0) {
                        s_inv[h] = sum != 0.f ? v_scale / sum : 0.f;
                        if (a.lse) a.lse[(int64_t)b * heads + h0 + h] = sum == 0.f ? -INFINITY : (all + log2f(sum)) * kLn2;
                    }
                }
                __syncthreads();
                float4 v[IT];
                const float* w[IT];
#pragma unroll
                for (int x = 0; x < IT; ++x) {
                    v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                    w[x] = weights + min(tid + x * kThreads, pieces - 1) / (D / 4) * parts;
                }
                for (int k0 = 0; k0 < parts; k0 += fit) {
                    if (k0 > 0) bring(k0);
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    const float4* y0 = room + tid;
#pragma unroll 4
                    for (int k = k0; k < min(parts, k0 + fit); ++k, y0 += pieces) {
#pragma unroll
                        for (int x = 0; x < IT; ++x) {
                            if (tid + x * kThreads < pieces) {
                                const float f = w[x][k];
                                const float4 y = y0[x * kThreads];
                                v[x].x = fmaf(y.x, f, v[x].x);
                                v[x].y = fmaf(y.y, f, v[x].y);
                                v[x].z = fmaf(y.z, f, v[x].z);
                                v[x].w = fmaf(y.w, f, v[x].w);
                            }
                        }
                    }
                }
#pragma unroll
                for (int x = 0; x < IT; ++x) {
                    const int i = tid + x * kThreads;
                    if (i < pieces) {
                        const int h = i / (D / 4), d = i % (D / 4) * 4;
                        const float f = s_inv[h];
                        float r[4] = {v[x].x * f, v[x].y * f, v[x].z * f, v[x].w * f};
                        store_run<4>(a.out, b * a.out_ts + (h0 + h) * a.out_hs + d, a.q_type, r);
                    }
                }
            }
        }
        __syncthreads();  // shared memory is free for the next piece
    }
}

template <int T, int DP, int NT, bool EXACT>
cudaError_t launch(const AttendArgs& a, const AttendPlan& p, cudaStream_t st) {
    constexpr int ES = T == 2 ? 1 : 2;
    const auto kernel = attend_kernel<T, DP, NT, EXACT>;
    static std::atomic<uint64_t> configured;
    // one limit serves every launch of the kernel; the CTAs share the SM's whole memory
    cudaError_t err =
        ensure_smem_limit((const void*)kernel, budget_of(ctas_an_sm(DP, ES, NT)) + 2048, configured, true);
    if (err != cudaSuccess) return err;
    const int64_t per_b = (int64_t)a.kv.kv_heads * p.chunks;
    const int64_t room = room_of(a);
    const int64_t most = a.window > 0 && room > a.window ? a.window : room;
    const int unit = unit_tokens(DP * ES);
    const int64_t units = (most + unit - 1) / unit * per_b * a.B;
    const int64_t grid = std::min<int64_t>(p.slots, std::max((units + kMinUnits - 1) / kMinUnits, per_b * a.B));
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kThreads), p.smem, st, a, p);
}

template <int T, int DP, bool EXACT>
cudaError_t heads(const AttendArgs& a, const AttendPlan& p, cudaStream_t st) {
    if (p.blocks == 1) return launch<T, DP, 1, EXACT>(a, p, st);
    if constexpr (DP <= 128) {
        if (p.blocks == 4) return launch<T, DP, 4, EXACT>(a, p, st);
    }
    return launch<T, DP, 2, EXACT>(a, p, st);
}

template <int T>
cudaError_t launch_attend_type(const AttendArgs& a, const AttendPlan& p, cudaStream_t st) {
    switch (a.kv.head_dim) {  // p.dp is the same, or 128 or 256
        case 64: return heads<T, 64, true>(a, p, st);
        case 96: return heads<T, 96, true>(a, p, st);
        case 128: return heads<T, 128, true>(a, p, st);
        case 192: return heads<T, 192, true>(a, p, st);
        case 256: return heads<T, 256, true>(a, p, st);
        default: return a.kv.head_dim < 128 ? heads<T, 128, false>(a, p, st) : heads<T, 256, false>(a, p, st);
    }
}

}  // namespace
}  // namespace moe
