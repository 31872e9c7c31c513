// Matrix product of E4M3 operands with a scale for each block of 128:
//
//   y = act(sum_g sx[t][g] sw[n / 128][g] (sum_{k in g} x w) + bias) + residual
//
// The two kernels are the plain product's (linear.cu): TMA, tcgen05 kind::f8f6f4, a split kernel for
// few tiles and a kernel of CTA pairs for many.  What differs is that the tensor cores' sums last for
// one block of K only, the 128 bytes of a stage: each block's products go to an accumulator of their
// own in a ring in tensor memory, from where warps add them, times their two scales, to fp32 sums in
// registers.  The scales are any fp32 numbers, which the block-scaled MMA forms (powers of two for 32
// elements) could not take, and the registers' sums are rounded to nearest, so that a long K loses less
// than in the tensor cores' own sums.
//
// Measured on a GB300 (launches of a graph): 8192 x 6144 x 4096 with bias 173 us (2385 TFLOP/s; the plain
// E4M3 product 115), with ReLU 209, with GELU 243, 4096 x 4096 x 4096 64, 1024 x 4096 x 4096 20, 777 x 5003 x 1424 f16 with
// GELU 27.5,
// 32 x 6144 x 4096 7.6, 1 x 4096 x 4096 5.1 (6.3 with its weights in memory and not in L2).
// What bounds the tiles is a circle of two accumulators: products (some 600 cycles for 256 x 256 outputs
// and a block of K), their commit, the additions up to the last read of the accumulator (some 450) and the
// arrival that lets the next products have it, 1500 cycles for two blocks of K.  The additions alone
// are 256 cycles of fp32 work a block.
#include <algorithm>

#include "linear.cuh"

namespace moe {
namespace {

struct BlockScales {
    const float *x, *w;  // [T][groups], [ceil(N / 128)][groups]
    int64_t x_stride, w_stride;
    bool fours;  // rows of both are aligned for reads of four
};

// ---- split kernel ------------------------------------------------------------

// Grid: x the cluster's K parts, y blocks of 128 outputs, z blocks of bn tokens.  An epilogue warp holds the
// sums of 32 outputs (a lane each) and, of the bn tokens, CH chunks of 16: every other one.
template <int CTAS, int CH>
__global__ void __launch_bounds__(kThreads, CTAS)
    blocks_split_kernel(const LinearArgs a, const BlockScales sc, const __grid_constant__ CUtensorMap wmap,
                        const __grid_constant__ CUtensorMap xmap, int bn, int stages, bool vec) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ float4 s_f[kEpiWarps][CH][4];  // a warp's factors of this block of K
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Head<kMaxAcc>& hd = *reinterpret_cast<Head<kMaxAcc>*>(base + split_ring(CTAS));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = gridDim.x, rank = blockIdx.x;
    const int n0 = blockIdx.y * 128, t0 = blockIdx.z * bn;
    const int nkb = (a.K + kRowBytes - 1) / kRowBytes;
    const int kb0 = (int)((int64_t)nkb * rank / S), kb1 = (int)((int64_t)nkb * (rank + 1) / S);
    const int stage_bytes = kABytes + bn * kRowBytes;
    constexpr int kPitch = 32 * CH;  // columns of an accumulator
    constexpr int kAccs = CTAS * kPitch >= 256 ? 2 : 4;
    constexpr int kCols = kAccs * kPitch;
    static_assert(CTAS * kCols <= 512 && kAccs <= kMaxAcc, "tensor memory of an SM");
    if (threadIdx.x == 0) {
        prefetch_tmap(&wmap);
        prefetch_tmap(&xmap);
        hd.abort = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(&hd.full[s], 1);
            mbar_init(&hd.empty[s], 1);
        }
        for (int s = 0; s < kAccs; ++s) {
            mbar_init(&hd.acc_full[s], 1);
            mbar_init(&hd.acc_empty[s], kEpiWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&hd.tmem)),
                     "r"(kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = hd.tmem;
    grid_launch_next();
    grid_dep_wait();
    const int cols = min(bn, a.T - t0);
    SplitOut<CTAS == 1 ? 2 : 1> out;
    out.prepare(a, base, warp, lane, rank, S, n0, t0, cols, vec);
    if (warp == 0) {
        const uint64_t first = l2_policy_evict_first(), last = l2_policy_evict_last();
        int s = 0;
        unsigned ph = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!wait_warp(&hd.empty[s], ph ^ 1u, hd, a.status, 2, s)) break;
            const uint32_t st = smem_u32(base) + (uint32_t)(s * stage_bytes);
            load_stage(&hd.full[s], stage_bytes, st, &wmap, st + kABytes, &xmap, kb * kRowBytes, n0, t0, first, last);
            advance(s, ph, stages);
        }
        drain(hd, s, ph, stages, kb1 - kb0);
    } else if (warp == 1) {
        const uint32_t idesc = mma_idesc(a.in_type, 128, bn);
        int s = 0, buf = 0;
        unsigned ph = 0, aph = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!wait_warp(&hd.acc_empty[buf], aph ^ 1u, hd, a.status, 4, buf)) break;
            if (!wait_warp(&hd.full[s], ph, hd, a.status, 1, s)) break;
            tc_fence_after();
            const uint64_t ad = sw128_desc(smem_u32(base + (size_t)s * stage_bytes));
            const uint64_t bd = sw128_desc(smem_u32(base + (size_t)s * stage_bytes + kABytes));
            mma_stage<true, 1>(tmem + buf * kPitch, ad, bd, idesc, 0, &hd.empty[s]);
            tc_commit_elect(&hd.acc_full[buf]);
            advance(s, ph, stages);
            advance(buf, aph, kAccs);
        }
    }
    // ---- sums of the blocks of K ----
    float sum[CH][16];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[c][i] = 0.f;
    const int q = warp & 3, half = warp >= 6 ? 1 : 0;  // warps 2-5 take the even chunks, 6-9 the odd ones
    bool ok = true;
    if (warp >= 2) {
        // lane l brings the factors of token l % 16 of chunks l / 16, l / 16 + 2, ..., two blocks of K ahead
        constexpr int kMine = (CH + 1) / 2;
        const float* xs[kMine];
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
            const int c = 16 * (2 * (lane / 16 + 2 * j) + half) + lane % 16;
            xs[j] = sc.x + (int64_t)(t0 + min(c, cols - 1)) * sc.x_stride;
        }
        const float* ws = sc.w + (int64_t)blockIdx.y * sc.w_stride;
        float ahead[2][kMine];
        auto fetch = [&](int kb, float (&f)[kMine]) {
            const int k = min(kb, nkb - 1);
            const float w = ws[k];
#pragma unroll
            for (int j = 0; j < kMine; ++j) f[j] = xs[j][k] * w;
        };
        fetch(kb0, ahead[0]);
        fetch(kb0 + 1, ahead[1]);
        float* mine = reinterpret_cast<float*>(s_f[warp - 2]);
        int buf = 0;
        unsigned aph = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
#pragma unroll
            for (int j = 0; j < kMine; ++j) {
                if (lane / 16 + 2 * j < CH) mine[(lane / 16 + 2 * j) * 16 + lane % 16] = ahead[0][j];
                ahead[0][j] = ahead[1][j];
            }
            fetch(kb + 2, ahead[1]);
            __syncwarp();
            if (!wait_warp(&hd.acc_full[buf], aph, hd, a.status, 3, buf)) {
                ok = false;
                break;
            }
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                if (16 * (2 * c + half) < bn) {  // the same in the whole warp
                    float v[16];
                    tc_ld16(tmem + ((uint32_t)(q * 32) << 16) + buf * kPitch + 16 * (2 * c + half), v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 f = s_f[warp - 2][c][i];
                        sum[c][4 * i] = fmaf(v[4 * i], f.x, sum[c][4 * i]);
                        sum[c][4 * i + 1] = fmaf(v[4 * i + 1], f.y, sum[c][4 * i + 1]);
                        sum[c][4 * i + 2] = fmaf(v[4 * i + 2], f.z, sum[c][4 * i + 2]);
                        sum[c][4 * i + 3] = fmaf(v[4 * i + 3], f.w, sum[c][4 * i + 3]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&hd.acc_empty[buf]);
            advance(buf, aph, kAccs);
        }
    }
    // ---- to shared memory, [token][128 outputs], once all products have read the ring ----
    __syncthreads();
    float* dump = reinterpret_cast<float*>(base);
    if (warp >= 2 && ok) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int at = 16 * (2 * c + half);
            if (at < cols) {
#pragma unroll
                for (int i = 0; i < 16; ++i) dump[(at + i) * 128 + q * 32 + lane] = sum[c][i];
            }
        }
    }
    __syncwarp();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
    }
    if (warp >= 2) out.finish(a, warp);
    __syncwarp();
    cluster_sync();  // the others may still read this CTA's sums
}

// ---- tiled kernel --------------------------------------------------------------

struct Tiles {
    int tm, tn;  // tiles along tokens (of 256) and outputs
    int stages;
};

// Tile i: bands of 8 token tiles, the outputs' tiles walked within a band, so that the
// tiles in flight share operands in L2.
__device__ __forceinline__ void tile_of(const Tiles& g, int i, int& m, int& n) {
    const int band = 8 * g.tn, b = i / band, r = i - b * band;
    const int rows = min(8, g.tm - 8 * b);
    n = r / rows;
    m = 8 * b + r - n * rows;
}

// Warp 0 loads, warp 1 issues, warp 2 brings the scales, warps 4-11 add up and finish.
constexpr int kBlockThreads = 32 * (4 + kEpiWarps);
// Registers of a thread (setmaxnreg) of the first four warps and of the others, out of the launch's 168.  The
// adding warps hold up to 128 sums and must not spill: the L1 that is left beside the ring does not hold it (with
// 50 bytes spilled 8192 x 6144 x 4096 took 270 us).
__host__ __device__ constexpr int few_regs(int bn) { return bn == 256 ? 56 : 88; }
__host__ __device__ constexpr int many_regs(int bn) { return bn == 256 ? 224 : 208; }
static_assert(4 * few_regs(256) + kEpiWarps * many_regs(256) <= (4 + kEpiWarps) * 168 &&
                  4 * few_regs(128) + kEpiWarps * many_regs(128) <= (4 + kEpiWarps) * 168,
              "registers of the CTA at its launch");
constexpr int kBlockRing = 144 * 1024;  // bytes of the ring of operands
constexpr int kBatch = 8;               // blocks of K whose scales come together
constexpr int kPiece = 32 * 64;         // bytes of 32 rows of 64 bytes of outputs
constexpr int kPieces = 4;              // of an adding warp: all its 16-bit outputs

// What the warps of a tile share beside the operands and the staging.
struct Shared {
    float x[2][kBatch][128];  // scales of the CTA's tokens, of two batches
    float w[2][kBatch][2];    // and of the tile's one or two blocks of outputs
    float beyond[2];          // read behind the last batch, and not used
    alignas(16) float bias[3][256];  // of three tiles, for a tile's is read when the next one's scales are all in use
    uint64_t scales_full[2], scales_empty[2], res_full[kEpiWarps];
    Head<kMaxAcc> head;
};
constexpr int kBlockSmem = 1024 + kBlockRing + kEpiWarps * kPieces * kPiece + (int)sizeof(Shared);
static_assert(kBlockSmem <= 227 * 1024, "shared memory of a CTA");

// s += f * 32 columns of this thread's lane: two loads, their wait and the arithmetic in one piece, so that the
// loaded values need not be moved to registers of the compiler's choice (which took as many instructions again).
__device__ __forceinline__ void add_columns(uint32_t at, float f, float (&s0)[16], float (&s1)[16]) {
    asm volatile(
        "{\n\t.reg .b32 a<16>, b<16>;\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {a0,a1,a2,a3,a4,a5,a6,a7,a8,a9,a10,a11,a12,a13,a14,a15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {b0,b1,b2,b3,b4,b5,b6,b7,b8,b9,b10,b11,b12,b13,b14,b15}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n\t"
        "fma.rn.f32 %0, a0, %34, %0;\n\tfma.rn.f32 %1, a1, %34, %1;\n\tfma.rn.f32 %2, a2, %34, %2;\n\tfma.rn.f32 %3, a3, %34, %3;\n\t"
        "fma.rn.f32 %4, a4, %34, %4;\n\tfma.rn.f32 %5, a5, %34, %5;\n\tfma.rn.f32 %6, a6, %34, %6;\n\tfma.rn.f32 %7, a7, %34, %7;\n\t"
        "fma.rn.f32 %8, a8, %34, %8;\n\tfma.rn.f32 %9, a9, %34, %9;\n\tfma.rn.f32 %10, a10, %34, %10;\n\tfma.rn.f32 %11, a11, %34, %11;\n\t"
        "fma.rn.f32 %12, a12, %34, %12;\n\tfma.rn.f32 %13, a13, %34, %13;\n\tfma.rn.f32 %14, a14, %34, %14;\n\tfma.rn.f32 %15, a15, %34, %15;\n\t"
        "fma.rn.f32 %16, b0, %34, %16;\n\tfma.rn.f32 %17, b1, %34, %17;\n\tfma.rn.f32 %18, b2, %34, %18;\n\tfma.rn.f32 %19, b3, %34, %19;\n\t"
        "fma.rn.f32 %20, b4, %34, %20;\n\tfma.rn.f32 %21, b5, %34, %21;\n\tfma.rn.f32 %22, b6, %34, %22;\n\tfma.rn.f32 %23, b7, %34, %23;\n\t"
        "fma.rn.f32 %24, b8, %34, %24;\n\tfma.rn.f32 %25, b9, %34, %25;\n\tfma.rn.f32 %26, b10, %34, %26;\n\tfma.rn.f32 %27, b11, %34, %27;\n\t"
        "fma.rn.f32 %28, b12, %34, %28;\n\tfma.rn.f32 %29, b13, %34, %29;\n\tfma.rn.f32 %30, b14, %34, %30;\n\tfma.rn.f32 %31, b15, %34, %31;\n\t"
        "}"
        : "+f"(s0[0]), "+f"(s0[1]), "+f"(s0[2]), "+f"(s0[3]), "+f"(s0[4]), "+f"(s0[5]), "+f"(s0[6]), "+f"(s0[7]),
          "+f"(s0[8]), "+f"(s0[9]), "+f"(s0[10]), "+f"(s0[11]), "+f"(s0[12]), "+f"(s0[13]), "+f"(s0[14]), "+f"(s0[15]),
          "+f"(s1[0]), "+f"(s1[1]), "+f"(s1[2]), "+f"(s1[3]), "+f"(s1[4]), "+f"(s1[5]), "+f"(s1[6]), "+f"(s1[7]),
          "+f"(s1[8]), "+f"(s1[9]), "+f"(s1[10]), "+f"(s1[11]), "+f"(s1[12]), "+f"(s1[13]), "+f"(s1[14]), "+f"(s1[15])
        : "r"(at), "r"(at + 16), "f"(f)
        : "memory");
}

// The waits of linear.cuh without a call: a kernel that shifts registers between its warps may not hold any.  What is
// usual takes one poll and one vote.
__device__ __forceinline__ bool wait_inline(uint64_t* bar, unsigned parity, Head<kMaxAcc>& hd, int* status) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t since = globaltimer();
#pragma unroll 1
    for (unsigned it = 1; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++it) {
        if ((it & 63u) == 0) {
            bool gone = *reinterpret_cast<volatile int*>(&hd.abort) != 0;
            if (!gone && globaltimer() - since > kTimeoutNs) {
                *reinterpret_cast<volatile int*>(&hd.abort) = 1;
                set_status(status, MOE_ERR_TIMEOUT);
                gone = true;
            }
            if (__any_sync(0xffffffffu, gone)) return false;
        }
    }
    return true;
}
// Both waits of the issuing warp: two polls on their way at once, and the waits themselves where they fail.
__device__ __forceinline__ bool wait_both(uint64_t* one, unsigned one_parity, uint64_t* other, unsigned other_parity, Head<kMaxAcc>& hd,
                                          int* status) {
    unsigned got;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 a, [%1], %2;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 b, [%3], %4;\n\t"
        "and.pred a, a, b;\n\tselp.u32 %0, 1, 0, a;\n\t}"
        : "=r"(got)
        : "r"(smem_u32(one)), "r"(one_parity), "r"(smem_u32(other)), "r"(other_parity)
        : "memory");
    if (__all_sync(0xffffffffu, got != 0)) return true;
    return wait_inline(one, one_parity, hd, status) && wait_inline(other, other_parity, hd, status);
}
__device__ __forceinline__ void drain_inline(Head<kMaxAcc>& hd, int s, unsigned ph, int stages, int64_t loads) {
    if ((threadIdx.x & 31) == 0)
#pragma unroll 1
        for (int k = 0; k < stages && k < loads; ++k) {
            const uint64_t since = globaltimer();
            while (!mbar_try_wait(&hd.empty[k], k < s ? ph : ph ^ 1u) && globaltimer() - since < kTimeoutNs) {
            }
        }
    __syncwarp();
}

// 16 values to 16 columns of this thread's lane.
__device__ __forceinline__ void keep_columns(uint32_t at, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
}

// A piece holds 32 rows (a lane each) of 64 bytes; 16-byte part j of row r is in place j ^ (r / 2 % 4), as TMA's
// 64-byte swizzle has it, so that 8 lanes meet every bank once.
__device__ __forceinline__ uint4* part_of(uint8_t* piece, int row, int j) {
    return reinterpret_cast<uint4*>(piece + row * 64 + ((j ^ (row >> 1 & 3)) << 4));
}

// One lane's copy of a piece's box (column x, row y) of an output or residual.
__device__ __forceinline__ void store_piece(const CUtensorMap* map, const uint8_t* piece, int x, int y) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n\t"
        "@e cp.async.bulk.commit_group;\n\t}" ::"l"(map),
        "r"(smem_u32(piece)), "r"(x), "r"(y)
        : "memory");
}
// Residuals of `count` pieces side by side; they arrive on `bar` together.
__device__ __forceinline__ void load_pieces(uint8_t* pieces, const CUtensorMap* map, int x, int y, int count, uint64_t* bar) {
    mbar_arrive_expect_tx_elect(bar, count * kPiece);
    for (int i = 0; i < count; ++i)
        asm volatile(
            "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
            "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(
                smem_u32(pieces + i * kPiece)),
            "l"(map), "r"(x + 64 * i), "r"(y), "r"(smem_u32(bar))
            : "memory");
}
// Until this warp's stores have read their pieces (the electing instruction picks the same lane each time; the others
// have nothing to wait for).
__device__ __forceinline__ void stores_read() {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
}

// 16 outputs of a lane's token into its row of a piece, from part `first` on, `res`: onto the residuals there.
template <int YT>
__device__ __forceinline__ void put_row(uint8_t* piece, int lane, int first, float (&v)[16], bool res) {
    constexpr int kRun = YT == MOE_F32 ? 4 : 8;  // values of a part
#pragma unroll
    for (int j = 0; j < 16 / kRun; ++j) {
        uint4* at = part_of(piece, lane, first + j);
        if (res) {
            float f[kRun];
            if constexpr (YT == MOE_F32) {
                const float4 r = *reinterpret_cast<const float4*>(at);
                f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w;
            } else {
                Raw<8, false> r;
                r.set(at, 0);
                r.get(YT, f);
            }
#pragma unroll
            for (int i = 0; i < kRun; ++i) v[kRun * j + i] += f[i];
        }
        store_run<kRun>(at, 0, YT, *reinterpret_cast<const float(*)[kRun]>(v + kRun * j));
    }
}

// Outputs [n0, n1) (at most 32) of 32 tokens from t0, rows of any alignment, from sums that `stage` holds (stage_row): a
// lane takes an output of every token, so that a warp's stores and residuals are consecutive.
template <int YT>
__device__ __forceinline__ void put_columns(const LinearArgs& a, const uint8_t* stage, int lane, int t0, int n0, int n1) {
    constexpr int kSize = YT == MOE_F32 ? 4 : 2;
    const int rows = min(32, a.T - t0);
    if (n0 + lane < n1) {
        uint8_t* to = static_cast<uint8_t*>(a.y) + ((int64_t)t0 * a.y_stride + n0 + lane) * kSize;
        const uint8_t* from = static_cast<const uint8_t*>(a.res) + ((int64_t)t0 * a.res_stride + n0 + lane) * kSize;
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += 16) {
            Raw<1> raw[16];
            if (a.res) {
#pragma unroll
                for (int i = 0; i < 16; ++i, from += a.res_stride * kSize)
                    if (r0 + i < rows) raw[i].load(from, 0, YT);
            }
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] = *reinterpret_cast<const float*>(stage + (r0 + i) * 128 + (((lane >> 2) ^ (i & 7)) << 4) + (lane & 3) * 4);
            if (a.res) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float f[1] = {0.f};
                    if (r0 + i < rows) raw[i].get(YT, f);
                    v[i] += f[0];
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i, to += a.y_stride * kSize) {
                const float one[1] = {v[i]};
                if (r0 + i < rows) store_run<1>(to, 0, YT, one);
            }
        }
    }
    __syncwarp();
}

// The end of an adding warp's tile: 32 tokens from t0 and 16 W outputs from n0, from sums in tensor memory at `sums`.
// Aligned rows: as many pieces as there are room for, two chunks of 16 at a time so that one's way hides the other's,
// then their stores; the residuals of the first ones are on their way since the tile began.
template <int YT, int W, bool LEAN>
__device__ __forceinline__ void finish_tile(const LinearArgs& a, const CUtensorMap* ymap, const CUtensorMap* rmap, uint8_t* pieces,
                                            uint64_t* res_full, unsigned& res_phase, const float* bias, int lane, int t0, int n0,
                                            uint32_t sums, bool vec, Head<kMaxAcc>& hd) {
    constexpr int kSize = YT == MOE_F32 ? 4 : 2, kPer = YT == MOE_F32 ? 1 : 2;  // chunks of 16 in a piece
    constexpr int kRound = W < kPieces * kPer ? W : kPieces * kPer;             // chunks between stores
    const auto value = [&](int c, float (&v)[16], int act) {
        tc_ld16(sums + 16 * c, v);
        if (a.bias) {
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                const float4 p = *reinterpret_cast<const float4*>(bias + 16 * c + j);
                v[j] += p.x, v[j + 1] += p.y, v[j + 2] += p.z, v[j + 3] += p.w;
            }
        }
        activate<16>(v, act);
    };
    if (t0 >= a.T || n0 >= a.N) return;
    if (LEAN || vec) {
#pragma unroll 1
        for (int c0 = 0; c0 < W && n0 + 16 * c0 < a.N; c0 += kRound) {
            const int x = (n0 + 16 * c0) * kSize, count = min(kRound / kPer, (a.N * kSize - x + 63) / 64);
            if (a.res) {
                if (c0 > 0) {
                    stores_read();
                    load_pieces(pieces, rmap, x, t0, count, res_full);
                }
                if (!wait_inline(res_full, res_phase, hd, a.status)) return;
                res_phase ^= 1u;
            } else {
                stores_read();
            }
#pragma unroll 2
            for (int c = 0; c < kRound; ++c) {
                float v[16];
                value(c0 + c, v, LEAN ? MOE_ACT_NONE : a.act);
                put_row<YT>(pieces + c / kPer * kPiece, lane, c % kPer * 2, v, a.res != nullptr);
            }
            fence_proxy_async_shared();
            __syncwarp();
            for (int i = 0; i < count; ++i) store_piece(ymap, pieces + i * kPiece, x + 64 * i, t0);
        }
    } else {
#pragma unroll 1
        for (int c = 0; c < W && n0 + 16 * c < a.N; c += 2) {
            float v0[16], v1[16];
            value(c, v0, a.act);
            value(c + 1, v1, a.act);
            stage_row(pieces, lane, v0, v1);
            put_columns<YT>(a, pieces, lane, t0, n0 + 16 * c, min(n0 + 16 * c + 32, a.N));
        }
    }
}

// The sums are in registers when this arrives (tcgen05.wait::ld): nothing in memory has to be released, and a
// release at the cluster's scope would wait for the scales' loads that are on their way.
__device__ __forceinline__ void arrive_cluster_relaxed(uint32_t bar, bool on) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar),
                 "r"((uint32_t)on)
                 : "memory");
}

// A block of K into a new accumulator, and the commits that announce it and free its stage in both CTAs, under one
// election.
__device__ __forceinline__ void mma_block(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint64_t* free, uint64_t* done) {
    asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b64 x, y;\n\t.reg .b16 m;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 p, %3, %3;\n\tsetp.eq.u32 t, %3, %3;\n\tmov.u16 m, 3;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
        "add.u64 x, %1, 2;\n\tadd.u64 y, %2, 2;\n\t@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], x, y, %3, t;\n\t"
        "add.u64 x, %1, 4;\n\tadd.u64 y, %2, 4;\n\t@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], x, y, %3, t;\n\t"
        "add.u64 x, %1, 6;\n\tadd.u64 y, %2, 6;\n\t@e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], x, y, %3, t;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%5], m;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%4], m;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"(smem_u32(free)), "r"(smem_u32(done))
        : "memory");
}

// A CTA pair works on 256 tokens x BN outputs; each CTA has 128 tokens, an adding warp 32 of them (a lane each) and
// half of the outputs.  LEAN: rows that TMA takes and no activation, whose code costs the sums' loop registers (8192 x
// 6144 x 4096 196 us with it there).
template <int BN, bool LEAN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kBlockThreads, 1)
    blocks_tile_kernel(const LinearArgs a, const BlockScales sc, const __grid_constant__ CUtensorMap wmap,
                       const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap ymap,
                       const __grid_constant__ CUtensorMap rmap, const Tiles g, bool vec) {
    constexpr int kAccs = 512 / BN, W = BN / 32;  // accumulators; chunks of 16 outputs of an adding warp
    static_assert(kAccs <= kMaxAcc, "barriers of the accumulators");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* epi = base + kBlockRing;
    constexpr int kStageBytes = kABytes + BN / 2 * kRowBytes;
    Shared& sh = *reinterpret_cast<Shared*>(epi + kEpiWarps * kPieces * kPiece);
    Head<kMaxAcc>& hd = sh.head;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int nkb = (a.K + kRowBytes - 1) / kRowBytes;
    const int tiles = g.tm * g.tn, pairs = gridDim.x / 2, pair_id = blockIdx.x / 2;
    if (threadIdx.x == 0) {
        prefetch_tmap(&wmap);
        prefetch_tmap(&xmap);
        hd.abort = 0;
        for (int s = 0; s < g.stages; ++s) {
            mbar_init(&hd.full[s], 1);
            mbar_init(&hd.empty[s], 1);
        }
        for (int s = 0; s < kAccs; ++s) {
            mbar_init(&hd.acc_full[s], 1);
            mbar_init(&hd.acc_empty[s], 2 * kEpiWarps);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.scales_full[s], 32);
            mbar_init(&sh.scales_empty[s], kEpiWarps);
        }
        for (int w = 0; w < kEpiWarps; ++w) mbar_init(&sh.res_full[w], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&hd.tmem)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = hd.tmem;
    grid_launch_next();
    grid_dep_wait();
    bool ok = true;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(few_regs(BN)));
        if (warp == 0) {
            // each CTA stages its half: 128 tokens and BN / 2 outputs; the leader's barrier counts both
            const uint64_t keep = l2_policy_evict_last();
            int s = 0;
            unsigned ph = 0;
            for (int i = pair_id; i < tiles && ok; i += pairs) {
                int m, n;
                tile_of(g, i, m, n);
                const int t0 = m * 256 + (int)rank * 128, n0 = n * BN + (int)rank * (BN / 2);
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!wait_inline(&hd.empty[s], ph ^ 1u, hd, a.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t st = smem_u32(base) + (uint32_t)(s * kStageBytes);
                    load_pair_block(&hd.full[s], rank == 0, 2u * kStageBytes, map_rank(smem_u32(&hd.full[s]), 0), st, &xmap,
                                    st + kABytes, &wmap, kb * kRowBytes, t0, n0, keep);
                    advance(s, ph, g.stages);
                }
            }
            if (ok) drain_inline(hd, s, ph, g.stages, (int64_t)nkb * ((tiles - pair_id + pairs - 1) / pairs));
        } else if (warp == 1 && rank == 0) {
            const uint32_t idesc = mma_idesc(a.in_type, 256, BN);
            const uint64_t a0 = sw128_desc(smem_u32(base)), b0 = sw128_desc(smem_u32(base) + kABytes);
            int s = 0, buf = 0;
            unsigned ph = 0, aph = 0;
            for (int i = pair_id; i < tiles && ok; i += pairs) {
#pragma unroll 1
                for (int kb = 0; kb < nkb; ++kb) {
                    ok = wait_both(&hd.full[s], ph, &hd.acc_empty[buf], aph ^ 1u, hd, a.status);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t at = s * (kStageBytes >> 4);
                    mma_block(tmem + buf * BN, a0 + at, b0 + at, idesc, &hd.empty[s], &hd.acc_full[buf]);
                    advance(s, ph, g.stages);
                    advance(buf, aph, kAccs);
                }
            }
        } else if (warp == 2) {
            // the scales of kBatch blocks of K at a time: four tokens a lane, one after the other; with a
            // tile's first ones its bias
            int s = 0, slot = 0;
            unsigned ph = 0;
            for (int i = pair_id; i < tiles && ok; i += pairs) {
                int m, n;
                tile_of(g, i, m, n);
                const int t0 = m * 256 + (int)rank * 128 + lane;
                for (int kb = 0; kb < nkb; kb += kBatch) {
                    if (!wait_inline(&sh.scales_empty[s], ph ^ 1u, hd, a.status)) {
                        ok = false;
                        break;
                    }
                    const int left = nkb - kb;
                    if (kb == 0 && a.bias) {
#pragma unroll 1
                        for (int j = lane; j < BN; j += 32) {
                            const int at = min(n * BN + j, a.N - 1);
                            sh.bias[slot][j] = a.bias_type == MOE_F32
                                                   ? static_cast<const float*>(a.bias)[at]
                                                   : half_bits_to_f32(static_cast<const uint16_t*>(a.bias)[at], a.bias_type);
                        }
                    }
                    if (lane < 2 * kBatch && lane / 2 < left)
                        sh.w[s][lane / 2][lane & 1] =
                            sc.w[(int64_t)min(n * BN / 128 + (lane & 1), (a.N - 1) / 128) * sc.w_stride + kb + lane / 2];
#pragma unroll 1
                    for (int j = 0; j < 4; ++j) {
                        const float* x = sc.x + (int64_t)min(t0 + 32 * j, a.T - 1) * sc.x_stride + kb;
                        float v[kBatch];
                        if (sc.fours && left >= kBatch) {
#pragma unroll
                            for (int k = 0; k < kBatch; k += 4) {
                                const float4 p = *reinterpret_cast<const float4*>(x + k);
                                v[k] = p.x, v[k + 1] = p.y, v[k + 2] = p.z, v[k + 3] = p.w;
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < kBatch; ++k) v[k] = k < left ? x[k] : 0.f;
                        }
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) sh.x[s][k][lane + 32 * j] = v[k];
                    }
                    mbar_arrive(&sh.scales_full[s]);
                    advance(s, ph, 2);
                }
                slot = slot == 2 ? 0 : slot + 1;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(many_regs(BN)));
        const int q = warp & 3, half = (warp - 4) >> 2, n_mine = half * (BN / 2);
        uint8_t* pieces = epi + (warp - 4) * kPieces * kPiece;
        uint64_t* res_full = &sh.res_full[warp - 4];
        const uint32_t acc_empty = map_rank(smem_u32(hd.acc_empty), 0);
        const uint32_t mine = tmem + ((uint32_t)(q * 32) << 16) + n_mine;
        int buf = 0, batch = 0, slot = 0;
        unsigned aph = 0, sph = 0, rph = 0;
        for (int i = pair_id; i < tiles && ok; i += pairs) {
            int m, n;
            tile_of(g, i, m, n);
            const int t0 = m * 256 + (int)rank * 128 + q * 32, n0 = n * BN + n_mine;
            if ((LEAN || vec) && a.res && t0 < a.T && n0 < a.N) {  // the first pieces' residuals
                const int size = a.y_type == MOE_F32 ? 4 : 2;
                stores_read();
                load_pieces(pieces, &rmap, n0 * size, t0, min(min(kPieces, W * size / 4), ((a.N - n0) * size + 63) / 64), res_full);
            }
            float sum[W][16];
#pragma unroll
            for (int c = 0; c < W; ++c)
#pragma unroll
                for (int j = 0; j < 16; ++j) sum[c][j] = 0.f;
            for (int kb = 0; kb < nkb && ok; kb += kBatch) {
                ok = wait_inline(&sh.scales_full[batch], sph, hd, a.status);
                const float* x = &sh.x[batch][0][q * 32 + lane];
                const float* w = &sh.w[batch][0][BN == 256 ? half : 0];
                const int end = min(kBatch, nkb - kb);
                float f = x[0] * w[0];
#pragma unroll 1
                for (int j = 0; j < end && ok; ++j) {
                    x += 128, w += 2;  // of the next block of K; behind the batch's last one nothing uses them
                    const float x1 = x[0], w1 = w[0];
                    ok = wait_inline(&hd.acc_full[buf], aph, hd, a.status);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < W; c += 2) add_columns(mine + buf * BN + 16 * c, f, sum[c], sum[c + 1]);
                    // the warp's loads are done (tcgen05.wait::ld): the next products may have the accumulator
                    tc_fence_before();
                    if (kb + j + 1 < nkb) {
                        arrive_cluster_relaxed(acc_empty + 8 * buf, lane == 0);
                        f = x1 * w1;
                        advance(buf, aph, kAccs);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.scales_empty[batch]);
                advance(batch, sph, 2);
            }
            if (!ok) break;
            // The sums go to the last accumulator, which is held until the tile is finished: in registers they would
            // leave none to the epilogue.  The next tile's first products go to another one meanwhile.
            const uint32_t held = mine + buf * BN;
#pragma unroll
            for (int c = 0; c < W; ++c) keep_columns(held + 16 * c, sum[c]);
            tc_wait_st();
            const float* bias = sh.bias[slot] + n_mine;
            slot = slot == 2 ? 0 : slot + 1;
            if (a.y_type == MOE_BF16) finish_tile<MOE_BF16, W, LEAN>(a, &ymap, &rmap, pieces, res_full, rph, bias, lane, t0, n0, held, vec, hd);
            else if (a.y_type == MOE_F16) finish_tile<MOE_F16, W, LEAN>(a, &ymap, &rmap, pieces, res_full, rph, bias, lane, t0, n0, held, vec, hd);
            else finish_tile<MOE_F32, W, LEAN>(a, &ymap, &rmap, pieces, res_full, rph, bias, lane, t0, n0, held, vec, hd);
            tc_fence_before();
            __syncwarp();
            arrive_cluster_relaxed(acc_empty + 8 * buf, lane == 0);
            advance(buf, aph, kAccs);
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // the stores are done before the CTA's memory goes
    }
    __syncwarp();
    __syncthreads();
    if (*reinterpret_cast<volatile int*>(&hd.abort)) {
        // a wait ran out: give the copies still in flight time to land before the CTA ends
        const uint64_t t = globaltimer();
        while (globaltimer() - t < 1000000ull) {
        }
    }
    tc_fence_before();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <int CTAS, int CH>
cudaError_t launch_split(const LinearArgs& a, const BlockScales& sc, int bn, int ksplit, bool vec, cudaStream_t st) {
    CUtensorMap wmap, xmap;
    if (!encode_rows(&wmap, a, a.w, a.N, a.w_stride, 128) || !encode_rows(&xmap, a, a.x, a.T, a.x_stride, bn))
        return cudaErrorInvalidValue;
    const auto kernel = blocks_split_kernel<CTAS, CH>;
    static std::atomic<uint64_t> configured;
    cudaError_t err = ensure_smem_limit((const void*)kernel, split_smem(CTAS), configured, true);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ksplit, (a.N + 127) / 128, (a.T + bn - 1) / bn);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = split_smem(CTAS);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ksplit;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a, sc, wmap, xmap, bn, split_stages(CTAS, bn), vec);
}

template <int CTAS>
cudaError_t launch_split_chunks(const LinearArgs& a, const BlockScales& sc, int bn, int ksplit, bool vec, cudaStream_t st) {
    if (bn <= 32) return launch_split<CTAS, 1>(a, sc, bn, ksplit, vec, st);
    if (bn <= 64) return launch_split<CTAS, 2>(a, sc, bn, ksplit, vec, st);
    return launch_split<CTAS, 4>(a, sc, bn, ksplit, vec, st);  // bn <= 128
}

template <int BN>
cudaError_t launch_tiles(const LinearArgs& a, const BlockScales& sc, bool vec, cudaStream_t st) {
    CUtensorMap wmap, xmap, ymap = {}, rmap = {};
    if (!encode_rows(&wmap, a, a.w, a.N, a.w_stride, BN / 2) || !encode_rows(&xmap, a, a.x, a.T, a.x_stride, 128))
        return cudaErrorInvalidValue;
    // pieces of 64 bytes x 32 tokens; rows that TMA does not take are stored one by one, and so are those that end
    // inside 16 bytes, for it writes the rest of these
    const int size = type_bytes(a.y_type);
    const auto pieces = [&](CUtensorMap* map, const void* p, int64_t stride) {
        return stride >= a.N && encode_tmap_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, (uint64_t)a.N * size, (uint64_t)a.T,
                                               (uint64_t)(stride * size), 64, 32, CU_TENSOR_MAP_SWIZZLE_64B);
    };
    vec = vec && (int64_t)a.N * size % 16 == 0 && pieces(&ymap, a.y, a.y_stride) && (!a.res || pieces(&rmap, a.res, a.res_stride));
    const Tiles g{(a.T + 255) / 256, (a.N + BN - 1) / BN, std::min(kMaxStages, kBlockRing / (kABytes + BN / 2 * kRowBytes))};
    const int pairs = std::min(a.sm_count / 2, g.tm * g.tn);
    const auto go = [&](auto kernel, std::atomic<uint64_t>& configured) {
        cudaError_t err = ensure_smem_limit((const void*)kernel, kBlockSmem, configured);
        if (err != cudaSuccess) return err;
        return launch_pdl(kernel, dim3(2 * pairs), dim3(kBlockThreads), kBlockSmem, st, a, sc, wmap, xmap, ymap, rmap, g, vec);
    };
    static std::atomic<uint64_t> configured[2];
    return vec && a.act == MOE_ACT_NONE ? go(blocks_tile_kernel<BN, true>, configured[1]) : go(blocks_tile_kernel<BN, false>, configured[0]);
}

}  // namespace

// Which kernel, by what each is expected to take in ns (fitted to products of 96 to 4096 tokens, 512 to 8192 outputs
// and depths of 512 to 8192):
//  tiles  2600 + rounds * (blocks of K * step + epilogue), step 470, 290 and 245 and epilogue 4000, 2400 and 1500 for
//         tiles of 256, 128 and 64 outputs.  1024 x 1024 x 1024 10.4, 7.2 and 6.9 us; 4096 x 2048 x 8192 67, 78 and 117.
//  split  3000 + rounds * (45 bn for the join + blocks of K of a CTA * (200 + 1.2 bn)).  128 x 4096 x 4096 11.2 us
//         against 12.0 in tiles, 128 x 1024 x 1024 8.8 against 6.0.
// Fitted before the kernel without activation was an instance of its own, which takes less (8192 x 6144 x 4096 173 us, 212
// by the formula), and blind to activations and unaligned rows, which take more (777 x 5003 x 1424 27 us, 20).
cudaError_t launch_linear_blocks(const LinearArgs& args, int64_t xs_stride, int64_t ws_stride, cudaStream_t st) {
    if (args.T == 0) return cudaSuccess;
    const BlockScales sc{args.x_scale, args.w_scale, xs_stride, ws_stride,
                         runs_aligned(args.x_scale, MOE_F32, 4, xs_stride) && runs_aligned(args.w_scale, MOE_F32, 4, ws_stride)};
    LinearArgs a = args;
    a.x_scale = a.w_scale = nullptr;  // none are left for the epilogue
    const bool vec = runs_aligned(a.y, a.y_type, 8, a.y_stride) && (!a.res || runs_aligned(a.res, a.y_type, 8, a.res_stride));
    const bool vec4 = runs_aligned(a.y, a.y_type, 4, a.y_stride) && (!a.res || runs_aligned(a.res, a.y_type, 4, a.res_stride));
    const int nkb = (a.K + kRowBytes - 1) / kRowBytes, pairs = a.sm_count / 2;
    const int tm = (a.T + 255) / 256;
    int64_t tiles_ns = INT64_MAX;
    int width = 256;
    for (int bn = 256; bn >= 64; bn /= 2) {
        const int64_t rounds = ((int64_t)tm * ((a.N + bn - 1) / bn) + pairs - 1) / pairs;
        const int64_t step = bn == 256 ? 470 : (bn == 128 ? 290 : 245), end = bn == 256 ? 4000 : (bn == 128 ? 2400 : 1500);
        const int64_t ns = 2600 + rounds * (nkb * step + end);
        if (ns < tiles_ns) {
            tiles_ns = ns;
            width = bn;
        }
    }
    // split: token blocks as even as they come, and K over what is left of the GPU.  Two CTAs an SM while the
    // smaller ring is as deep as a short pass over K needs
    const int tz = (a.T + 127) / 128, bn = ((a.T + tz - 1) / tz + 15) / 16 * 16;
    const int64_t blocks = (int64_t)((a.N + 127) / 128) * tz;
    int ksplit = 1;
    cudaError_t err = cluster_size<2>(blocks, nkb, &ksplit);
    const bool two = bn <= 32 || (nkb + ksplit - 1) / ksplit <= split_stages(2, bn);
    if (err == cudaSuccess && !two) err = cluster_size<1>(blocks, nkb, &ksplit);
    if (err != cudaSuccess) return err;
    const int64_t at_once = (int64_t)a.sm_count * (two ? 2 : 1), rounds = (blocks * ksplit + at_once - 1) / at_once;
    const int64_t split_ns = 3000 + rounds * (45 * bn + ((nkb + ksplit - 1) / ksplit) * (200 + bn * 12 / 10));
    if (a.T > 64 && tiles_ns < split_ns) {
        if (width == 256) return launch_tiles<256>(a, sc, vec, st);
        return width == 128 ? launch_tiles<128>(a, sc, vec, st) : launch_tiles<64>(a, sc, vec, st);
    }
    return two ? launch_split_chunks<2>(a, sc, bn, ksplit, vec4, st) : launch_split_chunks<1>(a, sc, bn, ksplit, vec4, st);
}

}  // namespace moe
