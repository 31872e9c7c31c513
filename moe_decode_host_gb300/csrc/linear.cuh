// What the matrix products share: clusters, stages of operands by TMA, the tensor cores'
// instructions and the parts of the epilogue.
#pragma once

#include <algorithm>

#include "ptx.cuh"
#include "vec.cuh"

namespace moe {
namespace {

constexpr int kRowBytes = 128;         // bytes of K in a stage
constexpr int kABytes = 128 * kRowBytes;
constexpr int kEpiWarps = 8;           // warps 2-9 read the accumulators and finish the outputs
constexpr int kThreads = 64 + 32 * kEpiWarps;  // warp 0 loads, warp 1 issues
constexpr int kMaxStages = 12;
// Bytes of the split kernel's ring, CTAS of which share an SM: two while a token block's
// sums ([128][128] fp32 at most) fit the smaller ring, so that more clusters run at once.
__host__ __device__ constexpr int split_ring(int ctas) { return ctas == 2 ? 104 * 1024 : 192 * 1024; }
constexpr int kSplitMax = 8;           // CTAs of a cluster
constexpr int kTileRing = 192 * 1024;  // bytes of the tiled kernel's ring
constexpr int kEpiBytes = 32 * 32 * 4;  // staging of an epilogue warp of the tiled kernel: 32 tokens x 32 outputs

// Barriers of the stages and of ACC accumulators, and the rest of what the warps share.
template <int ACC>
struct Head {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[ACC], acc_empty[ACC];
    uint32_t tmem;
    int abort;
};
constexpr int kMaxAcc = 8;
constexpr int split_smem(int ctas) { return 1024 + split_ring(ctas) + (int)sizeof(Head<kMaxAcc>); }
constexpr int kTileSmem = 1024 + kTileRing + kEpiWarps * kEpiBytes + (int)sizeof(Head<kMaxAcc>);
static_assert(kTileSmem <= 227 * 1024, "shared memory of a CTA");

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// From a CTA of the cluster where `on`, else zeros: no branch for the parts that there are not.
__device__ __forceinline__ float4 ld_cluster(uint32_t addr, bool on) {
    float4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.f32 %0, 0f00000000;\n\tmov.f32 %1, 0f00000000;\n\t"
        "mov.f32 %2, 0f00000000;\n\tmov.f32 %3, 0f00000000;\n\t@p ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "=&f"(v.x), "=&f"(v.y), "=&f"(v.z), "=&f"(v.w)
        : "r"(addr), "r"((uint32_t)on)
        : "memory");
    return v;
}

__device__ __forceinline__ float ld_cluster1(uint32_t addr, bool on) {
    float v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.f32 %0, 0f00000000;\n\t@p ld.shared::cluster.f32 %0, [%1];\n\t}"
        : "=&f"(v)
        : "r"(addr), "r"((uint32_t)on)
        : "memory");
    return v;
}

// A stage's four k-steps and the commit that frees it, by an elected lane of a converged warp;
// with CG == 2 the commit arrives on the barrier at this place in both CTAs.  One election a
// stage takes the issuing warp 250 cycles beside its wait, one for each instruction 285.
#define MOE_MMA_STAGE(CG, KIND, COMMIT)                                                        \
    asm volatile(                                                                              \
        "{\n\t.reg .pred e, p, t;\n\t.reg .b64 x, y;\n\t.reg .b16 m;\n\t"                      \
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.eq.u32 t, %3, %3;\n\t"   \
        "mov.u16 m, 3;\n\t"                                                                    \
        "@e tcgen05.mma.cta_group::" CG ".kind::" KIND " [%0], %1, %2, %3, p;\n\t"             \
        "add.u64 x, %1, 2;\n\tadd.u64 y, %2, 2;\n\t"                                           \
        "@e tcgen05.mma.cta_group::" CG ".kind::" KIND " [%0], x, y, %3, t;\n\t"               \
        "add.u64 x, %1, 4;\n\tadd.u64 y, %2, 4;\n\t"                                           \
        "@e tcgen05.mma.cta_group::" CG ".kind::" KIND " [%0], x, y, %3, t;\n\t"               \
        "add.u64 x, %1, 6;\n\tadd.u64 y, %2, 6;\n\t"                                           \
        "@e tcgen05.mma.cta_group::" CG ".kind::" KIND " [%0], x, y, %3, t;\n\t"               \
        COMMIT "\n\t}" ::"r"(d),                                                               \
        "l"(ad), "l"(bd), "r"(idesc), "r"(acc), "r"(smem_u32(bar))                             \
        : "memory")
#define MOE_COMMIT_ONE "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];"
#define MOE_COMMIT_PAIR "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%5], m;"
template <bool F8, int CG, bool COMMIT = true>
__device__ __forceinline__ void mma_stage(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc, uint64_t* bar) {
    if constexpr (F8 && CG == 1) MOE_MMA_STAGE("1", "f8f6f4", MOE_COMMIT_ONE);
    else if constexpr (CG == 1) MOE_MMA_STAGE("1", "f16", MOE_COMMIT_ONE);
    else if constexpr (F8 && COMMIT) MOE_MMA_STAGE("2", "f8f6f4", MOE_COMMIT_PAIR);
    else if constexpr (F8) MOE_MMA_STAGE("2", "f8f6f4", "");
    else if constexpr (COMMIT) MOE_MMA_STAGE("2", "f16", MOE_COMMIT_PAIR);
    else MOE_MMA_STAGE("2", "f16", "");
}
#undef MOE_COMMIT_ONE
#undef MOE_COMMIT_PAIR
#undef MOE_MMA_STAGE

// Instruction descriptor: fp32 sums, operand formats (f16 and E4M3 are 0, bf16 is 1),
// M rows and N columns.
__device__ __forceinline__ uint32_t mma_idesc(int in_type, int m, int n) {
    const uint32_t f = in_type == MOE_BF16 ? 1u : 0u;
    return (1u << 4) | (f << 7) | (f << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Two fp32 operations an instruction.
struct Pair {
    uint64_t v;
};
__device__ __forceinline__ Pair pair(float a, float b) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(Pair p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v)); }
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// GELU of two values, v Phi(v) = max(v, 0) - |v| Phi(-|v|), so that small results keep their
// precision.  With x = |v| and t = 1 / (1 + 0.3 x),
//   Phi(-x) = exp(-x^2 / 2) t P(t),
// P the polynomial of degree 7 nearest to the quotient in relative terms for x up to 14.5
// (Remez exchange; 1.6e-7).  The exponent -x^2 log2(e) / 2 reaches 126, where fp32 alone would
// lose 2^-17 of the result: what its two products round off is brought back as a factor.  In
// all 2^-18 of the value at most, wherever it is a normal fp32 number (2048 x 4096 x 512 23.8 us;
// 22.2 with Abramowitz and Stegun 7.1.28, which is good to 5e-7 absolutely alone).  At 64 the tail has long
// vanished; the argument is held there, so that no infinity is multiplied by 0.
__device__ __forceinline__ void gelu2(float& v0, float& v1) {
    const float x0 = fabsf(v0), x1 = fabsf(v1);
    const Pair x = pair(fminf(x0, 64.f), fminf(x1, 64.f));
    auto both = [](float c) { return pair(c, c); };
    float d0, d1;
    unpair(fma2(x, both(0.3f), both(1.f)), d0, d1);
    const Pair t = pair(fast_rcp(d0), fast_rcp(d1));
    Pair p = fma2(t, both(0.0354237072f), both(-0.156158343f));
    p = fma2(p, t, both(0.204556614f));
    p = fma2(p, t, both(-0.0520338714f));
    p = fma2(p, t, both(0.127691701f));
    p = fma2(p, t, both(0.100175969f));
    p = fma2(p, t, both(0.120712131f));
    p = fma2(p, t, both(0.119632006f));
    constexpr float kC = 0.72134752f;  // log2(e) / 2
    const Pair xc = mul2(x, both(-kC)), z = mul2(xc, x), minus_z = mul2(z, both(-1.f));
    const Pair rest = fma2(fma2(x, both(-kC), mul2(xc, both(-1.f))), x, fma2(xc, x, minus_z));
    float z0, z1;
    unpair(z, z0, z1);
    Pair tail = mul2(pair(fast_exp2(z0), fast_exp2(z1)), mul2(p, t));
    tail = fma2(tail, mul2(rest, both(0.693147181f)), tail);
    const Pair pos = fma2(pair(v0, v1), both(0.5f), mul2(pair(x0, x1), both(0.5f)));
    unpair(fma2(mul2(x, both(-1.f)), tail, pos), v0, v1);
}

// SiLU of two values, v / (1 + exp(-v)), by the exponential that cannot overflow: v / (1 + e) above 0
// and v e / (1 + e) below, e = exp(-|v|) = 2^z with what z loses to rounding brought back as a
// factor.  2^-20 of the value at most.  At 256 e has long vanished, and no infinity meets another.
__device__ __forceinline__ void silu2(float& v0, float& v1) {
    constexpr float kL = 1.4426950216293335f, kRest = 1.925963033500011e-08f;  // log2(e) and the rest of it
    auto both = [](float c) { return pair(c, c); };
    const float x0 = fminf(fabsf(v0), 256.f), x1 = fminf(fabsf(v1), 256.f);
    const Pair down = pair(-x0, -x1), z = mul2(down, both(kL)), minus_z = mul2(pair(x0, x1), both(kL));
    const Pair rest = fma2(down, both(kRest), fma2(down, both(kL), minus_z));
    float z0, z1, d0, d1, e0, e1;
    unpair(z, z0, z1);
    Pair e = pair(fast_exp2(z0), fast_exp2(z1));
    e = fma2(e, mul2(rest, both(0.693147181f)), e);
    unpair(fma2(e, both(1.f), both(1.f)), d0, d1);
    unpair(e, e0, e1);
    const Pair up = mul2(pair(v0, v1), pair(v0 > 0.f ? 1.f : e0, v1 > 0.f ? 1.f : e1));
    unpair(mul2(up, pair(fast_rcp(d0), fast_rcp(d1))), v0, v1);
}

template <int VEC>
__device__ __forceinline__ void activate(float (&v)[VEC], int act) {
    if (act == MOE_ACT_NONE) return;
    if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) gelu2(v[i], v[i + 1]);
    } else if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) silu2(v[i], v[i + 1]);
    } else if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];
    }
}

// Scales and biases of VEC outputs from n on, `inc` apart (1 and 0 where there are none).
template <int VEC>
struct Columns {
    float scale[VEC], bias[VEC];
    __device__ __forceinline__ void load(const LinearArgs& a, int n, int inc) {  // past N: the last one's
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            scale[i] = 1.f;
            bias[i] = 0.f;
        }
        if (a.w_scale) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) scale[i] = a.w_scale[min(n + i * inc, a.N - 1)];
        }
        if (a.bias) {
            if (a.bias_type == MOE_F32) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) bias[i] = static_cast<const float*>(a.bias)[min(n + i * inc, a.N - 1)];
            } else {
                uint16_t h[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) h[i] = static_cast<const uint16_t*>(a.bias)[min(n + i * inc, a.N - 1)];
#pragma unroll
                for (int i = 0; i < VEC; ++i) bias[i] = half_bits_to_f32(h[i], a.bias_type);
            }
        }
    }
};

__device__ __forceinline__ void finish_one(const LinearArgs& a, int64_t t, int n, float v) {
    if (a.res) {
        Raw<1> r;
        float f[1];
        r.load(a.res, t * a.res_stride + n, a.y_type);
        r.get(a.y_type, f);
        v += f[0];
    }
    const float one[1] = {v};
    store_run<1>(a.y, t * a.y_stride + n, a.y_type, one);
}

// A wait taken by a whole converged warp; false when it ran out.
template <int ACC>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, unsigned parity, Head<ACC>& hd, int* status, int where, int slot) {
    return __all_sync(0xffffffffu,
                      mbar_wait_fast(bar, parity, &hd.abort, status, nullptr, where, slot, 0, 0));
}

// The loading warp's end, at ring position (s, ph) after `loads` stages: waits until the
// products have read every stage (the last arrivals on these barriers), or after an abort
// until the copies have landed, so that nothing reaches the CTA's memory after it ended.
template <int ACC>
__device__ __forceinline__ void drain(Head<ACC>& hd, int s, unsigned ph, int stages, int64_t loads) {
    const bool gone = *reinterpret_cast<volatile int*>(&hd.abort) != 0;
    if ((threadIdx.x & 31) == 0)
        for (int k = 0; k < stages && k < loads; ++k) mbar_drain(gone ? &hd.full[k] : &hd.empty[k], k < s ? ph : ph ^ 1u);
    __syncwarp();
}

// The end of a block of 128 outputs whose sums the CTAs of a cluster share: rank r finishes the tokens
// [c0, c1) of the block; each epilogue warp finishes every eighth, four outputs a lane (a run where rows
// are aligned, else 32 apart), and has their scales, biases and first residuals in hand before the sums
// are.  AHEAD: tokens at a time, two where there are registers for the parts of both on their way together.
template <int AHEAD>
struct SplitOut {
    int S, t0, c0, c1, inc, mine;
    bool vec, whole;
    Columns<4> col;
    Raw<4> res[AHEAD];
    float sx[2];
    uint32_t peer[kSplitMax];  // this lane's first output of the block's first token, in each rank's sums

    // sums: [token][128 outputs] of this CTA
    __device__ __forceinline__ void prepare(const LinearArgs& a, const uint8_t* sums, int warp, int lane, int rank, int ranks,
                                            int n0, int first_token, int cols, bool aligned) {
        S = ranks, t0 = first_token, vec = aligned;
        c0 = cols * rank / S, c1 = cols * (rank + 1) / S;
        inc = vec ? 1 : 32, mine = n0 + (vec ? lane * 4 : lane);
        whole = vec && mine + 4 <= a.N;
        sx[0] = sx[1] = 1.f;
        if (warp < 2) return;
#pragma unroll
        for (int j = 0; j < kSplitMax; ++j) peer[j] = map_rank(smem_u32(sums) + lane * (vec ? 16 : 4), min(j, S - 1));
        col.load(a, mine, inc);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int c = c0 + warp - 2 + kEpiWarps * k;
            if (c < c1) {
                if (a.res && whole) res[k].load(a.res, (int64_t)(t0 + c) * a.res_stride + mine, a.y_type);
                if (a.x_scale) sx[k] = a.x_scale[t0 + c];
            }
        }
    }

    // The parts in rank order, then the epilogue; branches are taken once for all the tokens in hand
    // (256 x 1024 x 4096 bf16 10.4 us; with one for each part, flag and run 11.7).
    __device__ __forceinline__ void finish(const LinearArgs& a, int warp) {
        for (int c = c0 + warp - 2, k = 0; c < c1 && mine < a.N; c += AHEAD * kEpiWarps, ++k) {
            float4 p[AHEAD][kSplitMax];
            const bool there[2] = {true, c + kEpiWarps < c1};
            if (vec) {
#pragma unroll
                for (int j = 0; j < kSplitMax; ++j)
#pragma unroll
                    for (int h = 0; h < AHEAD; ++h) p[h][j] = ld_cluster(peer[j] + (c + kEpiWarps * h) * 512, j < S && there[h]);
            } else {
#pragma unroll
                for (int j = 0; j < kSplitMax; ++j)
#pragma unroll
                    for (int h = 0; h < AHEAD; ++h) {
                        const uint32_t at = peer[j] + (c + kEpiWarps * h) * 512;
                        const bool on = j < S && there[h];
                        p[h][j] = make_float4(ld_cluster1(at, on), ld_cluster1(at + 128, on), ld_cluster1(at + 256, on),
                                              ld_cluster1(at + 384, on));
                    }
            }
            if (k > 0) {
                if (a.x_scale) {
#pragma unroll
                    for (int h = 0; h < AHEAD; ++h)
                        if (there[h]) sx[h] = a.x_scale[t0 + c + kEpiWarps * h];
                }
                if (a.res && whole) {
#pragma unroll
                    for (int h = 0; h < AHEAD; ++h)
                        if (there[h])
                            res[h].load(a.res, (int64_t)(t0 + c + kEpiWarps * h) * a.res_stride + mine, a.y_type);
                }
            }
            float v[4 * AHEAD];
#pragma unroll
            for (int h = 0; h < AHEAD; ++h) {
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < kSplitMax; ++j) {
                    sum[0] += p[h][j].x;
                    sum[1] += p[h][j].y;
                    sum[2] += p[h][j].z;
                    sum[3] += p[h][j].w;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) v[4 * h + i] = fmaf(sum[i], sx[h] * col.scale[i], col.bias[i]);
            }
            activate<4 * AHEAD>(v, a.act);
            if (!whole) {  // element by element; with inc = 32 a warp still writes and reads whole lines
                auto out = [&](int type) {
                    if (a.res) {
                        Raw<1> r[4 * AHEAD];
#pragma unroll
                        for (int i = 0; i < 4 * AHEAD; ++i)
                            if (there[i / 4] && mine + i % 4 * inc < a.N)
                                r[i].load(a.res, (int64_t)(t0 + c + kEpiWarps * (i / 4)) * a.res_stride + mine + i % 4 * inc, type);
#pragma unroll
                        for (int i = 0; i < 4 * AHEAD; ++i) {
                            float f[1];
                            r[i].get(type, f);
                            v[i] += f[0];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4 * AHEAD; ++i) {
                        const float one[1] = {v[i]};
                        if (there[i / 4] && mine + i % 4 * inc < a.N)
                            store_run<1>(a.y, (int64_t)(t0 + c + kEpiWarps * (i / 4)) * a.y_stride + mine + i % 4 * inc, type, one);
                    }
                };
                if (a.y_type == MOE_BF16) out(MOE_BF16);
                else if (a.y_type == MOE_F16) out(MOE_F16);
                else out(MOE_F32);
            } else {
                auto out = [&](int type) {
                    if (a.res) {
#pragma unroll
                        for (int h = 0; h < AHEAD; ++h) {
                            float f[4];
                            res[h].get(type, f);
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[4 * h + i] += f[i];
                        }
                    }
#pragma unroll
                    for (int h = 0; h < AHEAD; ++h) {
                        const float w[4] = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
                        if (there[h]) store_run<4>(a.y, (int64_t)(t0 + c + kEpiWarps * h) * a.y_stride + mine, type, w);
                    }
                };
                if (a.y_type == MOE_BF16) out(MOE_BF16);
                else if (a.y_type == MOE_F16) out(MOE_F16);
                else out(MOE_F32);
            }
        }
    }
};

// 32 x 32 sums into an epilogue warp's staging: a lane holds a token.  16-byte piece j of its row goes to piece
// j ^ (row % 8): no side of the exchange meets a bank twice within 8 lanes.
__device__ __forceinline__ void stage_row(uint8_t* stage, int lane, const float (&v0)[16], const float (&v1)[16]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        *reinterpret_cast<float4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) =
            make_float4(v0[4 * j], v0[4 * j + 1], v0[4 * j + 2], v0[4 * j + 3]);
        *reinterpret_cast<float4*>(stage + lane * 128 + (((j + 4) ^ (lane & 7)) << 4)) =
            make_float4(v1[4 * j], v1[4 * j + 1], v1[4 * j + 2], v1[4 * j + 3]);
    }
    __syncwarp();
}

// An epilogue warp's outputs: 32 tokens from t0, up to 32 outputs from n0 + c of the tile's `cols`.
// exchange() brings their sums into `stage` (stage_row).
template <class Exchange>
__device__ __forceinline__ void finish_chunk(const LinearArgs& a, uint8_t* stage, int lane, int t0, int n0, int c, int cols,
                                             bool vec, const Exchange& exchange) {
    if (vec) {
        // out: a lane takes 8 outputs of every eighth token; their scales, biases and residuals
        // are fetched while the sums go through shared memory
        const int nn = n0 + c + (lane & 3) * 8;
        const bool in = nn < n0 + cols, whole = nn + 8 <= a.N;
        Columns<8> col;
        Raw<8> res[4];
        float sx[4];
        if (in) {
            col.load(a, nn, 1);
            const int r0 = t0 + (lane >> 2);
#pragma unroll
            for (int k = 0; k < 4; ++k) sx[k] = 1.f;
            if (a.x_scale) {
#pragma unroll
                for (int k = 0; k < 4; ++k) sx[k] = a.x_scale[min(r0 + 8 * k, a.T - 1)];
            }
            if (a.res && whole) {
                auto fetch = [&](int type) {  // past T: the last token's
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        res[k].load(a.res, (int64_t)min(r0 + 8 * k, a.T - 1) * a.res_stride + nn, type);
                };
                if (a.y_type == MOE_F32) fetch(MOE_F32);
                else fetch(MOE_BF16);  // 16 bits either way
            }
        }
        exchange();
        if (in) {
            float v[32];  // all four runs at once: a branch on flags and types for 32 values
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = (lane >> 2) + 8 * k;
                const uint8_t* row = stage + r * 128;
                const float4 lo = *reinterpret_cast<const float4*>(row + (((2 * (lane & 3)) ^ (r & 7)) << 4));
                const float4 hi = *reinterpret_cast<const float4*>(row + (((2 * (lane & 3) + 1) ^ (r & 7)) << 4));
                const float w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) v[8 * k + i] = fmaf(w[i], sx[k] * col.scale[i], col.bias[i]);
            }
            activate<32>(v, a.act);
            if (!whole) {  // the run that N ends in: through this lane's own places, one by one
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = (lane >> 2) + 8 * k;
                    uint8_t* row = stage + r * 128;
                    *reinterpret_cast<float4*>(row + (((2 * (lane & 3)) ^ (r & 7)) << 4)) =
                        make_float4(v[8 * k], v[8 * k + 1], v[8 * k + 2], v[8 * k + 3]);
                    *reinterpret_cast<float4*>(row + (((2 * (lane & 3) + 1) ^ (r & 7)) << 4)) =
                        make_float4(v[8 * k + 4], v[8 * k + 5], v[8 * k + 6], v[8 * k + 7]);
                }
#pragma unroll 1
                for (int j = 0; j < 32; ++j) {
                    const int r = (lane >> 2) + 8 * (j >> 3), i = j & 7;
                    if (t0 + r < a.T && nn + i < a.N)
                        finish_one(a, t0 + r, nn + i,
                                   *reinterpret_cast<const float*>(
                                       stage + r * 128 + (((2 * (lane & 3) + (i >> 2)) ^ (r & 7)) << 4) + (i & 3) * 4));
                }
            } else {
                auto out = [&](int type) {
                    if (a.res) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float f[8];
                            res[k].get(type, f);
#pragma unroll
                            for (int i = 0; i < 8; ++i) v[8 * k + i] += f[i];
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int t = t0 + (lane >> 2) + 8 * k;
                        const float(&w)[8] = *reinterpret_cast<const float(*)[8]>(v + 8 * k);
                        if (t < a.T) store_run<8>(a.y, (int64_t)t * a.y_stride + nn, type, w);
                    }
                };
                if (a.y_type == MOE_BF16) out(MOE_BF16);
                else if (a.y_type == MOE_F16) out(MOE_F16);
                else out(MOE_F32);
            }
        }
    } else {
        // rows of any alignment: a lane takes one output of every token, so that a warp's
        // stores and residuals are consecutive (8087 outputs of 6116 x 1424, fp32 with
        // residual: 180 us; with a branch on types and flags for each output 278, with 8
        // outputs a lane, element by element, 541)
        const int nn = n0 + c + lane;
        const bool in = nn < n0 + cols;
        Columns<1> col;
        Raw<1> res[32];
        if (in) {
            col.load(a, nn, 1);
            if (a.res) {
                auto fetch = [&](int type) {  // past T: the last token's
#pragma unroll
                    for (int r = 0; r < 32; ++r)
                        res[r].load(a.res, (int64_t)min(t0 + r, a.T - 1) * a.res_stride + nn, type);
                };
                if (a.y_type == MOE_F32) fetch(MOE_F32);
                else fetch(MOE_BF16);  // 16 bits either way
            }
        }
        exchange();
        if (in) {
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += 8) {
                float v[8], sx[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) sx[i] = 1.f;
                if (a.x_scale) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) sx[i] = a.x_scale[min(t0 + r0 + i, a.T - 1)];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float sum = *reinterpret_cast<const float*>(stage + (r0 + i) * 128 +
                                                                      (((lane >> 2) ^ i) << 4) + (lane & 3) * 4);
                    v[i] = fmaf(sum, sx[i] * col.scale[0], col.bias[0]);
                }
                activate<8>(v, a.act);
                auto out = [&](int type) {
                    if (a.res) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float one[1];
                            res[r0 + i].get(type, one);
                            v[i] += one[0];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float one[1] = {v[i]};
                        if (t0 + r0 + i < a.T)
                            store_run<1>(a.y, (int64_t)(t0 + r0 + i) * a.y_stride + nn, type, one);
                    }
                };
                if (a.y_type == MOE_BF16) out(MOE_BF16);
                else if (a.y_type == MOE_F16) out(MOE_F16);
                else out(MOE_F32);
            }
        }
    }
    __syncwarp();
}

// A stage's two copies by an elected lane of a converged warp.
__device__ __forceinline__ void load_stage(uint64_t* bar, uint32_t bytes, uint32_t dw, const CUtensorMap* wmap, uint32_t dx,
                                           const CUtensorMap* xmap, int k, int n, int t, uint64_t wpolicy, uint64_t xpolicy) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%2], [%3, {%6, %7}], [%0], %9;\n\t"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%4], [%5, {%6, %8}], [%0], %10;\n\t}" ::"r"(smem_u32(bar)),
        "r"(bytes), "r"(dw), "l"(wmap), "r"(dx), "l"(xmap), "r"(k), "r"(n), "r"(t), "l"(wpolicy), "l"(xpolicy)
        : "memory");
}

// The two copies of a block of K by an elected lane of a converged warp; they arrive on `bar`,
// which may be the peer's.  With `announce` (the leader, at a stage's first block) the bytes of
// both CTAs are first announced on its own barrier.
__device__ __forceinline__ void load_pair_block(uint64_t* own, bool announce, uint32_t bytes, uint32_t bar, uint32_t dx,
                                                const CUtensorMap* xmap, uint32_t dw, const CUtensorMap* wmap, int k, int t,
                                                int n, uint64_t policy) {
    asm volatile(
        "{\n\t.reg .pred e, f;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.and.u32 f, %1, 0, e;\n\t"
        "@f mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %2;\n\t"
        "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%4], [%5, {%8, %9}], [%3], %11;\n\t"
        "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%6], [%7, {%8, %10}], [%3], %11;\n\t}" ::"r"(smem_u32(own)),
        "r"((uint32_t)announce), "r"(bytes), "r"(bar), "r"(dx), "l"(xmap), "r"(dw), "l"(wmap), "r"(k), "r"(t), "r"(n), "l"(policy)
        : "memory");
}
// Arrives on the barrier at this place in both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair_elect(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\telect.sync _|e, 0xffffffff;\n\tmov.u16 m, 3;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
            smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

bool encode_rows(CUtensorMap* map, const LinearArgs& a, const void* p, int rows, int64_t stride, int box) {
    const int es = type_bytes(a.in_type);
    const CUtensorMapDataType dt = a.in_type == MOE_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : a.in_type == MOE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    return encode_tmap_2d(map, dt, p, (uint64_t)a.K, (uint64_t)rows, (uint64_t)(stride * es), kRowBytes / es, box,
                          CU_TENSOR_MAP_SWIZZLE_128B);
}

// A cluster's CTAs: the most (up to kSplitMax and the blocks of K) with which all blocks of
// outputs still run at once, for a second round costs more than a longer pass over K
// (32 x 6144 x 4096 E4M3, 48 blocks: 8.1 us with 2, 6.7 with 3 to 5, 11.4 with 6, of which
// 46 fit).  How many clusters of a size run at once is asked of the runtime, once a device,
// for a kernel of the same footprint without tensor memory: for one that allocates tensor
// memory the runtime answers as if each CTA took all 512 columns.
template <int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) footprint_kernel() {}

int split_stages(int ctas, int bn) { return std::min(kMaxStages, split_ring(ctas) / (kABytes + bn * kRowBytes)); }

template <int CTAS>
cudaError_t cluster_size(int64_t blocks, int nkb, int* out) {
    static std::atomic<int> known[64][kSplitMax + 1];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    static std::atomic<uint64_t> configured;
    err = ensure_smem_limit((const void*)footprint_kernel<CTAS>, split_smem(CTAS), configured, true);
    if (err != cudaSuccess) return err;
    *out = 1;
    for (int s = min(kSplitMax, nkb); s > 1; --s) {
        std::atomic<int>* slot = dev < 64 ? &known[dev][s] : nullptr;
        int n = slot ? slot->load(std::memory_order_relaxed) : 0;
        if (n == 0) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(s);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = split_smem(CTAS);
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = s;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            err = cudaOccupancyMaxActiveClusters(&n, footprint_kernel<CTAS>, &cfg);
            if (err != cudaSuccess) return err;
            if (n < 1) n = 1;
            if (slot) slot->store(n, std::memory_order_relaxed);
        }
        if (n >= blocks) {
            *out = s;
            break;
        }
    }
    return cudaSuccess;
}

}  // namespace
}  // namespace moe
