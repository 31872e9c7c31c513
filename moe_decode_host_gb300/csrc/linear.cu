// Matrix product with an epilogue: y = act(x W^T [* sx_t * sw_n] + bias) + residual.
//
// Both kernels run on tcgen05 with operands staged by TMA (128-byte rows of K, 128-byte
// swizzle) and fp32 accumulators in tensor memory; bf16 and f16 use kind::f16, E4M3
// kind::f8f6f4, whose stages and descriptors are the same bytes (a step is 32 bytes of
// K either way).  Rows past T and N and bytes past K arrive as zeros.
//
//  split kernel   few output tiles: the weights' bytes (or the latency of one pass over
//                 K) bound the call.  The weight rows take the 128-wide side of the MMA
//                 and the tokens its free side (a multiple of 16), so a token tile costs
//                 what it holds; K is split over the CTAs of a cluster, which join their
//                 sums through distributed shared memory in rank order.
//  tiled kernel   many tiles: the tensor cores bound the call.  A CTA pair works on 256
//                 tokens x up to 256 outputs (cta_group::2: each CTA stages half of both
//                 operands), persistent, with two accumulators so that the epilogue of a
//                 tile runs under the next tile's products.
//
// Measured on a GB300 (launches of a graph): 1 x 4096 x 4096 bf16 with residual 7.2 us over three
// sets of weights, of which L2 holds much, 8.2 us over 24 (4.1 TB/s, launch and fill included); 32 x
// 6144 x 4096 E4M3 6.5 and 8.6 us; 8192 x 6144 x 4096 bf16 with bias, GELU and residual 235 us
// (1750 TFLOP/s; 262 us back to back under the power cap), E4M3 with bias 115 us (3580 TFLOP/s;
// 130 back to back).  Between them 128 x 4096 x 4096 10.8 us (cuBLAS 7.6), 512 17.4 (11.6), 1024 24.3
// (19.8).
//
// The tensor cores' fp32 sums round towards zero, a step of 32 bytes of K at a time: fp32 outputs of
// bf16 products are off by 1.0e-6 at K = 1024 and 9.1e-6 at 8192 in tiles, as the library's are, and by
// less where K is split.
#include <algorithm>

#include "linear.cuh"

namespace moe {
namespace {

// Outputs of a tile up to which a stage holds two blocks of K: the loading and the issuing warp
// take about 170 ns a stage, more than the products of narrow tiles (one and two blocks: 256 x
// 1024 x 4096 14.5 and 11.5 us with 64 outputs a tile; 1024 x 4096 x 4096 23.9 and 24.7 with 256).
constexpr int kTwoBlocks = 128;

// ---- split kernel ------------------------------------------------------------

// Grid: x the cluster's K parts, y blocks of 128 outputs, z blocks of bn tokens.
template <bool F8, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS)
    linear_split_kernel(const LinearArgs a, const __grid_constant__ CUtensorMap wmap,
                        const __grid_constant__ CUtensorMap xmap, int bn, int stages, bool vec) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    Head<2>& hd = *reinterpret_cast<Head<2>*>(base + split_ring(CTAS));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = gridDim.x, rank = blockIdx.x;
    const int n0 = blockIdx.y * 128, t0 = blockIdx.z * bn;
    const int nkb = (int)(((int64_t)a.K * (F8 ? 1 : 2) + kRowBytes - 1) / kRowBytes);
    const int kb0 = (int)((int64_t)nkb * rank / S), kb1 = (int)((int64_t)nkb * (rank + 1) / S);
    const int stage_bytes = kABytes + bn * kRowBytes;
    const int tcols = bn <= 32 ? 32 : (bn <= 64 ? 64 : (bn <= 128 ? 128 : 256));
    if (threadIdx.x == 0) {
        prefetch_tmap(&wmap);
        prefetch_tmap(&xmap);
        hd.abort = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(&hd.full[s], 1);
            mbar_init(&hd.empty[s], 1);
        }
        mbar_init(&hd.acc_full[0], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&hd.tmem)),
                     "r"(tcols)
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
            load_stage(&hd.full[s], stage_bytes, st, &wmap, st + kABytes, &xmap, kb * (F8 ? 128 : 64), n0, t0, first, last);
            advance(s, ph, stages);
        }
        drain(hd, s, ph, stages, kb1 - kb0);
    } else if (warp == 1) {
        const uint32_t idesc = mma_idesc(a.in_type, 128, bn);
        int s = 0;
        unsigned ph = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!wait_warp(&hd.full[s], ph, hd, a.status, 1, s)) break;
            tc_fence_after();
            const uint64_t ad = sw128_desc(smem_u32(base + (size_t)s * stage_bytes));
            const uint64_t bd = sw128_desc(smem_u32(base + (size_t)s * stage_bytes + kABytes));
            mma_stage<F8, 1>(tmem, ad, bd, idesc, kb > kb0, &hd.empty[s]);
            advance(s, ph, stages);
        }
        tc_commit_elect(&hd.acc_full[0]);
    }
    // ---- sums to shared memory, [token][128 outputs]; the ring is idle by then ----
    float* dump = reinterpret_cast<float*>(base);
    if (warp >= 2) {
        const int q = warp & 3;
        wait_warp(&hd.acc_full[0], 0, hd, a.status, 3, 0);
        tc_fence_after();
        for (int c = (warp - 2) / 4 * 16; c < cols; c += 64) {  // two warps share a quarter of the lanes
            const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + c;
            float v[16], w[16];
            float* to = dump + c * 128 + q * 32 + lane;
            if (c + 32 < cols) {
                tc_ld16x2(at, at + 32, v, w);
#pragma unroll
                for (int i = 0; i < 16; ++i) to[(32 + i) * 128] = w[i];
            } else {
                tc_ld16(at, v);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) to[i * 128] = v[i];
        }
        tc_fence_before();
    }
    __syncwarp();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(tcols) : "memory");
    }
    if (warp >= 2) out.finish(a, warp);
    __syncwarp();
    cluster_sync();  // the others may still read this CTA's sums
}

// ---- tiled kernel --------------------------------------------------------------

struct TileGrid {
    int tm, tn, bn;  // tiles along tokens (of 256) and outputs (of bn)
    int stages;
};

// Tile i: bands of 8 token tiles, the outputs' tiles walked within a band, so that the
// tiles in flight share operands in L2.
__device__ __forceinline__ void tile_at(const TileGrid& g, int i, int& m, int& n) {
    const int band = 8 * g.tn, b = i / band, r = i - b * band;
    const int rows = min(8, g.tm - 8 * b);
    n = r / rows;
    m = 8 * b + r - n * rows;
}

template <bool F8, int SUB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    linear_tile_kernel(const LinearArgs a, const __grid_constant__ CUtensorMap wmap,
                       const __grid_constant__ CUtensorMap xmap, const TileGrid g, bool vec) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* epi = base + kTileRing;
    const int w_bytes = g.bn / 2 * kRowBytes, stage_bytes = SUB * (kABytes + w_bytes);
    Head<2>& hd = *reinterpret_cast<Head<2>*>(epi + kEpiWarps * kEpiBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int nkb = (int)(((int64_t)a.K * (F8 ? 1 : 2) + kRowBytes - 1) / kRowBytes);
    const int tiles = g.tm * g.tn, pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    if (threadIdx.x == 0) {
        prefetch_tmap(&wmap);
        prefetch_tmap(&xmap);
        hd.abort = 0;
        for (int s = 0; s < g.stages; ++s) {
            mbar_init(&hd.full[s], 1);
            mbar_init(&hd.empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
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
        // each CTA stages its half: 128 tokens and bn / 2 outputs; the leader's barrier counts both
        const uint64_t keep = l2_policy_evict_last();
        const int half = g.bn / 2;
        const unsigned bytes = 2u * (unsigned)stage_bytes;
        int s = 0;
        unsigned ph = 0;
        for (int i = pair; i < tiles && ok; i += pairs) {
            int m, n;
            tile_at(g, i, m, n);
            const int t0 = m * 256 + (int)rank * 128, n0 = n * g.bn + (int)rank * half;
            for (int kb = 0; kb < nkb; kb += SUB) {
                if (!wait_warp(&hd.empty[s], ph ^ 1u, hd, a.status, 2, s)) {
                    ok = false;
                    break;
                }
                const uint32_t st = smem_u32(base) + (uint32_t)(s * stage_bytes);
#pragma unroll
                for (int u = 0; u < SUB; ++u)  // a block past the last is zeros
                    load_pair_block(&hd.full[s], rank == 0 && u == 0, bytes, map_rank(smem_u32(&hd.full[s]), 0),
                                    st + u * kABytes, &xmap, st + SUB * kABytes + u * w_bytes, &wmap,
                                    (kb + u) * (F8 ? 128 : 64), t0, n0, keep);
                advance(s, ph, g.stages);
            }
        }
        if (ok) drain(hd, s, ph, g.stages, (int64_t)((nkb + SUB - 1) / SUB) * ((tiles - pair + pairs - 1) / pairs));
    } else if (warp == 1 && rank == 0) {
        const uint32_t idesc = mma_idesc(a.in_type, 256, g.bn);
        int s = 0, buf = 0;
        unsigned ph = 0, accph = 0;
        for (int i = pair; i < tiles && ok; i += pairs) {
            if (!wait_warp(&hd.acc_empty[buf], ((accph >> buf) & 1u) ^ 1u, hd, a.status, 4, buf)) break;
            accph ^= 1u << buf;
            tc_fence_after();
            for (int kb = 0; kb < nkb; kb += SUB) {
                if (!wait_warp(&hd.full[s], ph, hd, a.status, 1, s)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t ad = sw128_desc(smem_u32(base) + s * stage_bytes);
                const uint64_t bd = sw128_desc(smem_u32(base) + s * stage_bytes + SUB * kABytes);
                if constexpr (SUB == 2)
                    mma_stage<F8, 2, false>(tmem + buf * 256, ad, bd, idesc, kb > 0, &hd.empty[s]);
                mma_stage<F8, 2>(tmem + buf * 256, ad + (SUB - 1) * (kABytes >> 4), bd + (SUB - 1) * (w_bytes >> 4), idesc,
                                 SUB == 2 || kb > 0, &hd.empty[s]);
                advance(s, ph, g.stages);
            }
            if (!ok) break;
            commit_pair_elect(&hd.acc_full[buf]);
            buf ^= 1;
        }
    } else if (warp >= 2) {
        const int q = warp & 3;
        uint8_t* stage = epi + (warp - 2) * kEpiBytes;
        int buf = 0;
        unsigned accph = 0;
        for (int i = pair; i < tiles; i += pairs) {
            int m, n;
            tile_at(g, i, m, n);
            const int t0 = m * 256 + (int)rank * 128 + q * 32, n0 = n * g.bn;
            if (!wait_warp(&hd.acc_full[buf], (accph >> buf) & 1u, hd, a.status, 3, buf)) break;
            accph ^= 1u << buf;
            tc_fence_after();
            const int cols = min(g.bn, a.N - n0);
            // two warps share a quarter of the lanes and take every other 32 outputs
            for (int c = (warp - 2) / 4 * 32; c < cols; c += 64) {
                finish_chunk(a, stage, lane, t0, n0, c, cols, vec, [&]() {
                    float v0[16], v1[16];
                    const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + buf * 256 + c;
                    tc_ld16x2(at, at + 16, v0, v1);
                    stage_row(stage, lane, v0, v1);
                });
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(map_rank(smem_u32(&hd.acc_empty[buf]), 0));
            buf ^= 1;
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

template <bool F8, int CTAS>
cudaError_t launch_split(const LinearArgs& a, int bn, int ksplit, bool vec, cudaStream_t st) {
    CUtensorMap wmap, xmap;
    if (!encode_rows(&wmap, a, a.w, a.N, a.w_stride, 128) || !encode_rows(&xmap, a, a.x, a.T, a.x_stride, bn))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> configured;
    cudaError_t err = ensure_smem_limit((const void*)linear_split_kernel<F8, CTAS>, split_smem(CTAS), configured, true);
    if (err != cudaSuccess) return err;
    const int tz = (a.T + bn - 1) / bn, stages = split_stages(CTAS, bn);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ksplit, (a.N + 127) / 128, tz);
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
    return cudaLaunchKernelEx(&cfg, linear_split_kernel<F8, CTAS>, a, wmap, xmap, bn, stages, vec);
}

template <bool F8, int SUB>
cudaError_t launch_tiles(const LinearArgs& a, TileGrid g, bool vec, cudaStream_t st) {
    CUtensorMap wmap, xmap;
    if (!encode_rows(&wmap, a, a.w, a.N, a.w_stride, g.bn / 2) || !encode_rows(&xmap, a, a.x, a.T, a.x_stride, 128))
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> configured;
    cudaError_t err = ensure_smem_limit((const void*)linear_tile_kernel<F8, SUB>, kTileSmem, configured);
    if (err != cudaSuccess) return err;
    const int pairs = min(a.sm_count / 2, g.tm * g.tn);
    g.stages = std::min(kMaxStages, kTileRing / (SUB * (kABytes + g.bn / 2 * kRowBytes)));
    return launch_pdl(linear_tile_kernel<F8, SUB>, dim3(2 * pairs), dim3(kThreads), kTileSmem, st, a, wmap, xmap, g, vec);
}

}  // namespace

// Which kernel, by what each is expected to take in ns (measured on bf16 products of 64 to
// 8192 tokens, 256 to 8192 outputs and depths of 256 to 8192; a block of K is the 128 bytes of a stage):
//  tiles  1600 + blocks of K * step + (rounds - 1) * max(blocks of K * step, epilogue) + epilogue,
//         for an epilogue is hidden under the next tile's products but for the last.  Epilogue:
//         1000 + 14 bn.  Step, the most of: 50 + 1.15 bn to 128 outputs and 0.62 for each beyond
//         them (the issuing warps, then the tensor cores); the stage of all CTAs at the 17 TB/s
//         that L2 gives.  512 x 4096 x 4096: 16.7 us against 20.3 split.
//  split  2500 + rounds * (20 bn for the join + blocks of K of a CTA * (200 + 0.8 bn)).
//         128 x 4096 x 4096: 10.7 us against 13.8 in tiles.
cudaError_t launch_linear(const LinearArgs& a, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    const bool f8 = a.in_type == MOE_E4M3;
    const bool vec = runs_aligned(a.y, a.y_type, 8, a.y_stride) && (!a.res || runs_aligned(a.res, a.y_type, 8, a.res_stride));
    const bool vec4 = runs_aligned(a.y, a.y_type, 4, a.y_stride) && (!a.res || runs_aligned(a.res, a.y_type, 4, a.res_stride));
    const int nkb = (int)(((int64_t)a.K * type_bytes(a.in_type) + kRowBytes - 1) / kRowBytes);
    const int pairs = a.sm_count / 2;
    TileGrid g{(a.T + 255) / 256, 0, 0, 0};
    int64_t tiles_ns = INT64_MAX;
    for (int bn = 256; bn >= 64; bn -= 32) {  // the width that leaves the least work to the last round
        const int64_t tn = (a.N + bn - 1) / bn, rounds = (g.tm * tn + pairs - 1) / pairs;
        const int64_t ctas = 2 * std::min<int64_t>(pairs, g.tm * tn);
        const int64_t l2 = ctas * (kABytes + bn / 2 * kRowBytes) / 17000, epi = 1000 + 14 * bn;
        const int64_t pass = nkb * std::max<int64_t>(l2, bn <= 128 ? 50 + bn * 115 / 100 : 197 + (bn - 128) * 62 / 100);
        const int64_t ns = 1600 + pass + (rounds - 1) * std::max(pass, epi) + epi;
        if (ns < tiles_ns) {
            tiles_ns = ns;
            g.tn = (int)tn;
            g.bn = bn;
        }
    }
    // split: token blocks as even as they come, and K over what is left of the GPU.  Two CTAs an SM
    // while the smaller ring is as deep as the narrow blocks (or a short pass over K) need
    const int tz = (a.T + 255) / 256, bn = ((a.T + tz - 1) / tz + 15) / 16 * 16;
    const int64_t blocks = (int64_t)((a.N + 127) / 128) * tz;
    int ksplit = 1;
    cudaError_t err = bn <= 128 ? cluster_size<2>(blocks, nkb, &ksplit) : cudaSuccess;
    const bool two = bn <= 32 || (bn <= 128 && (nkb + ksplit - 1) / ksplit <= split_stages(2, bn));
    if (err == cudaSuccess && !two) err = cluster_size<1>(blocks, nkb, &ksplit);
    if (err != cudaSuccess) return err;
    const int64_t at_once = (int64_t)a.sm_count * (two ? 2 : 1), rounds = (blocks * ksplit + at_once - 1) / at_once;
    const int64_t split_ns = 2500 + rounds * (20 * bn + ((nkb + ksplit - 1) / ksplit) * (200 + bn * 8 / 10));
    if (a.T > 64 && tiles_ns < split_ns) {
        if (g.bn <= kTwoBlocks) return f8 ? launch_tiles<true, 2>(a, g, vec, st) : launch_tiles<false, 2>(a, g, vec, st);
        return f8 ? launch_tiles<true, 1>(a, g, vec, st) : launch_tiles<false, 1>(a, g, vec, st);
    }
    if (two) return f8 ? launch_split<true, 2>(a, bn, ksplit, vec4, st) : launch_split<false, 2>(a, bn, ksplit, vec4, st);
    return f8 ? launch_split<true, 1>(a, bn, ksplit, vec4, st) : launch_split<false, 1>(a, bn, ksplit, vec4, st);
}

}  // namespace moe
