// Matrix product of E4M3 operands with a scale for each block of 128:
//
//   y = act(sum_g sx[t][g] sw[n / 128][g] (sum_{k in g} x w) + bias) + residual
//
// The two kernels are the plain product's (linear.cu): TMA, tcgen05 kind::f8f6f4, a split kernel for
// few tiles and a kernel of CTA pairs for many.  What differs is that the tensor cores' sums last for
// one block of K only, the 128 bytes of a stage: each block's products go to an accumulator of their
// own in a ring in tensor memory, from where the epilogue warps add them, times their two scales, to
// fp32 sums in registers.  The scales are any fp32 numbers, which the block-scaled MMA forms (powers of
// two for 32 elements) could not take, and the registers' sums are rounded to nearest, so that a long K
// loses less than in the tensor cores' own sums.
//
// An addition for every output and block of K keeps the fp32 units busy for half of the products' time
// at 256 x 256 outputs a pair (128 x 256 a CTA: 256 cycles of 512), and so does reading the accumulators
// from tensor memory; both run beside the products as long as there are two accumulators.
#include <algorithm>

#include "linear.cuh"

namespace moe {
namespace {

struct BlockScales {
    const float *x, *w;  // [T][groups], [ceil(N / 128)][groups]
    int64_t x_stride, w_stride;
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
    constexpr int kPitch = CH == 1 ? 32 : 32 * CH;  // columns of an accumulator
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

// A CTA pair works on 256 tokens x 64 NC outputs; each CTA has 128 tokens, an epilogue warp 32 of them (a lane
// each) and half of the outputs, NC chunks of 32.
template <int NC>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    blocks_tile_kernel(const LinearArgs a, const BlockScales sc, const __grid_constant__ CUtensorMap wmap,
                       const __grid_constant__ CUtensorMap xmap, const Tiles g, bool vec) {
    constexpr int kBn = 64 * NC, kPitch = NC == 3 ? 256 : kBn, kAccs = 512 / kPitch;
    static_assert(kAccs <= kMaxAcc, "barriers of the accumulators");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* epi = base + kTileRing;
    constexpr int kStageBytes = kABytes + kBn / 2 * kRowBytes;
    Head<kMaxAcc>& hd = *reinterpret_cast<Head<kMaxAcc>*>(epi + kEpiWarps * kEpiBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int nkb = (a.K + kRowBytes - 1) / kRowBytes;
    const int tiles = g.tm * g.tn, pairs = gridDim.x / 2, pair = blockIdx.x / 2;
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
    if (warp == 0) {
        // each CTA stages its half: 128 tokens and kBn / 2 outputs; the leader's barrier counts both
        const uint64_t keep = l2_policy_evict_last();
        int s = 0;
        unsigned ph = 0;
        for (int i = pair; i < tiles && ok; i += pairs) {
            int m, n;
            tile_of(g, i, m, n);
            const int t0 = m * 256 + (int)rank * 128, n0 = n * kBn + (int)rank * (kBn / 2);
            for (int kb = 0; kb < nkb; ++kb) {
                if (!wait_warp(&hd.empty[s], ph ^ 1u, hd, a.status, 2, s)) {
                    ok = false;
                    break;
                }
                const uint32_t st = smem_u32(base) + (uint32_t)(s * kStageBytes);
                load_pair_block(&hd.full[s], rank == 0, 2u * kStageBytes, map_rank(smem_u32(&hd.full[s]), 0), st, &xmap,
                                st + kABytes, &wmap, kb * kRowBytes, t0, n0, keep);
                advance(s, ph, g.stages);
            }
        }
        if (ok) drain(hd, s, ph, g.stages, (int64_t)nkb * ((tiles - pair + pairs - 1) / pairs));
    } else if (warp == 1 && rank == 0) {
        const uint32_t idesc = mma_idesc(a.in_type, 256, kBn);
        int s = 0, buf = 0;
        unsigned ph = 0, aph = 0;
        for (int i = pair; i < tiles && ok; i += pairs) {
            for (int kb = 0; kb < nkb; ++kb) {
                if (!wait_warp(&hd.acc_empty[buf], aph ^ 1u, hd, a.status, 4, buf) ||
                    !wait_warp(&hd.full[s], ph, hd, a.status, 1, s)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t ad = sw128_desc(smem_u32(base) + s * kStageBytes);
                const uint64_t bd = sw128_desc(smem_u32(base) + s * kStageBytes + kABytes);
                mma_stage<true, 2>(tmem + buf * kPitch, ad, bd, idesc, 0, &hd.empty[s]);
                commit_pair_elect(&hd.acc_full[buf]);
                advance(s, ph, g.stages);
                advance(buf, aph, kAccs);
            }
        }
    } else if (warp >= 2) {
        const int q = warp & 3, half = warp >= 6 ? 1 : 0;
        uint8_t* stage = epi + (warp - 2) * kEpiBytes;
        int buf = 0;
        unsigned aph = 0;
        for (int i = pair; i < tiles && ok; i += pairs) {
            int m, n;
            tile_of(g, i, m, n);
            const int t0 = m * 256 + (int)rank * 128 + q * 32, n0 = n * kBn, c0 = half * (kBn / 2);
            // this lane's token's scales, and those of the one or two blocks that its outputs lie in
            const float* xs = sc.x + (int64_t)min(t0 + lane, a.T - 1) * sc.x_stride;
            const int nb = (n0 + c0) / 128, last = (a.N - 1) / 128;
            const float* ws0 = sc.w + min(nb, last) * sc.w_stride;
            const float* ws1 = sc.w + min(nb + 1, last) * sc.w_stride;
            float fx[2], fw[2][2];  // two blocks of K ahead
            auto fetch = [&](int kb, int at) {
                const int k = min(kb, nkb - 1);
                fx[at] = xs[k];
                fw[at][0] = ws0[k];
                if (NC == 3) fw[at][1] = ws1[k];
            };
            fetch(0, 0);
            fetch(1, 1);
            float sum[NC][32];
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int j = 0; j < 32; ++j) sum[c][j] = 0.f;
            for (int kb = 0; kb < nkb; ++kb) {
                const float f0 = fx[0] * fw[0][0], f1 = NC == 3 ? fx[0] * fw[0][1] : f0;
                fx[0] = fx[1], fw[0][0] = fw[1][0];
                if (NC == 3) fw[0][1] = fw[1][1];
                fetch(kb + 2, 1);
                if (!wait_warp(&hd.acc_full[buf], aph, hd, a.status, 3, buf)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    float v0[16], v1[16];
                    const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + buf * kPitch + c0 + 32 * c;
                    tc_ld16x2(at, at + 16, v0, v1);
                    const float f = (n0 + c0 + 32 * c) / 128 == nb ? f0 : f1;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        sum[c][j] = fmaf(v0[j], f, sum[c][j]);
                        sum[c][16 + j] = fmaf(v1[j], f, sum[c][16 + j]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(map_rank(smem_u32(&hd.acc_empty[buf]), 0));
                advance(buf, aph, kAccs);
            }
            if (!ok) break;
            const int cols = min(kBn, a.N - n0);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (c0 + 32 * c < cols)
                    finish_chunk(a, stage, lane, t0, n0, c0 + 32 * c, cols, vec, [&]() {
                        float v0[16], v1[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            v0[j] = sum[c][j];
                            v1[j] = sum[c][16 + j];
                        }
                        stage_row(stage, lane, v0, v1);
                    });
            }
        }
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
    if (CTAS == 2 || bn <= 128) return launch_split<CTAS, 4>(a, sc, bn, ksplit, vec, st);
    if constexpr (CTAS == 1) return launch_split<1, 8>(a, sc, bn, ksplit, vec, st);
    return cudaErrorInvalidValue;
}

template <int NC>
cudaError_t launch_tiles(const LinearArgs& a, const BlockScales& sc, bool vec, cudaStream_t st) {
    CUtensorMap wmap, xmap;
    if (!encode_rows(&wmap, a, a.w, a.N, a.w_stride, 32 * NC) || !encode_rows(&xmap, a, a.x, a.T, a.x_stride, 128))
        return cudaErrorInvalidValue;
    const auto kernel = blocks_tile_kernel<NC>;
    static std::atomic<uint64_t> configured;
    cudaError_t err = ensure_smem_limit((const void*)kernel, kTileSmem, configured);
    if (err != cudaSuccess) return err;
    const Tiles g{(a.T + 255) / 256, (a.N + 64 * NC - 1) / (64 * NC), std::min(kMaxStages, kTileRing / (kABytes + 32 * NC * kRowBytes))};
    const int pairs = std::min(a.sm_count / 2, g.tm * g.tn);
    return launch_pdl(kernel, dim3(2 * pairs), dim3(kThreads), kTileSmem, st, a, sc, wmap, xmap, g, vec);
}

}  // namespace

cudaError_t launch_linear_blocks(const LinearArgs& args, int64_t xs_stride, int64_t ws_stride, cudaStream_t st) {
    if (args.T == 0) return cudaSuccess;
    const BlockScales sc{args.x_scale, args.w_scale, xs_stride, ws_stride};
    LinearArgs a = args;
    a.x_scale = a.w_scale = nullptr;  // none are left for the epilogue
    const bool vec = runs_aligned(a.y, a.y_type, 8, a.y_stride) && (!a.res || runs_aligned(a.res, a.y_type, 8, a.res_stride));
    const bool vec4 = runs_aligned(a.y, a.y_type, 4, a.y_stride) && (!a.res || runs_aligned(a.res, a.y_type, 4, a.res_stride));
    const int nkb = (a.K + kRowBytes - 1) / kRowBytes, pairs = a.sm_count / 2;
    const int tm = (a.T + 255) / 256;
    int64_t tiles_ns = INT64_MAX;
    int nc = 4;
    for (int c = 4; c >= 1; --c) {
        const int bn = 64 * c;
        const int64_t tn = (a.N + bn - 1) / bn, rounds = (tm * tn + pairs - 1) / pairs;
        const int64_t pass = nkb * (int64_t)std::max(170, bn * 12 / 10), epi = 1000 + 14 * bn;
        const int64_t ns = 1600 + rounds * (pass + epi);
        if (ns < tiles_ns) {
            tiles_ns = ns;
            nc = c;
        }
    }
    const int tz = (a.T + 255) / 256, bn = ((a.T + tz - 1) / tz + 15) / 16 * 16;
    const int64_t blocks = (int64_t)((a.N + 127) / 128) * tz;
    int ksplit = 1;
    cudaError_t err = bn <= 128 ? cluster_size<2>(blocks, nkb, &ksplit) : cudaSuccess;
    const bool two = bn <= 32 || (bn <= 128 && (nkb + ksplit - 1) / ksplit <= split_stages(2, bn));
    if (err == cudaSuccess && !two) err = cluster_size<1>(blocks, nkb, &ksplit);
    if (err != cudaSuccess) return err;
    const int64_t at_once = (int64_t)a.sm_count * (two ? 2 : 1), rounds = (blocks * ksplit + at_once - 1) / at_once;
    const int64_t split_ns = 2500 + rounds * (20 * bn + ((nkb + ksplit - 1) / ksplit) * (200 + bn * 12 / 10));
    if (a.T > 64 && tiles_ns < split_ns) {
        switch (nc) {
            case 1: return launch_tiles<1>(a, sc, vec, st);
            case 2: return launch_tiles<2>(a, sc, vec, st);
            case 3: return launch_tiles<3>(a, sc, vec, st);
            default: return launch_tiles<4>(a, sc, vec, st);
        }
    }
    return two ? launch_split_chunks<2>(a, sc, bn, ksplit, vec4, st) : launch_split_chunks<1>(a, sc, bn, ksplit, vec4, st);
}

}  // namespace moe
