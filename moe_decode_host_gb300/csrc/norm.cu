// Residual addition and root-mean-square norm, with an output in 16, 32 or 8 bits.
//
//   s = x + r,  y = s * rsqrt(mean(s^2) + eps) * w
//   8 bits: scale = max(max_j |y_j| / 448, 2^-126), y8 = E4M3(y / scale)
//
// Memory bound: x, r in, s, y out, each once.  The row stays in registers between the
// reduction and the outputs.  One reduction carries both statistics: the norm's factor
// is common to the row, so max |y| = rsqrt(...) * max |s * w| and the maximum can be
// taken before the factor is known.
//
// Measured on a GB300: 8192 x 4096 bf16 with residual to E4M3 38.2 us (6.2 TB/s, 91% of a
// plain copy's rate), 777 x 5003 f16 with an fp32 residual (rows at odd addresses) 13.8 us
// (3.4 TB/s), one row 1.7 us.
#include <algorithm>

#include "ptx.cuh"
#include "vec.cuh"

namespace moe {
namespace {

constexpr float kE4M3Max = 448.f;
constexpr int kRingBytes = 48 * 1024;  // of a CTA, where two stages fit
constexpr int kAny = -1;  // a type known only at run time

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A row is handled by blockDim.x threads (whole warps) with NV runs of VEC elements each,
// blockDim.y rows a CTA at a time.  A CTA walks rows gridDim.x * blockDim.y apart; the next
// row's loads are issued before the current row is reduced, so that reads stay in flight
// through the reduction and the stores.  The usual types are template arguments: with the
// types at run time the conversions made the kernel issue bound (52 instructions an
// element and 77 us for 8192 x 4096 to E4M3).
// FULL: residual, sum and weights are all there and the runs of a CTA's threads are the row,
// so that nothing in the loop is conditional.
template <int VEC, int NV, int THREADS, int XT, int RT, int WT, int YT, bool FULL>
__global__ void __launch_bounds__(THREADS) norm_kernel(const NormArgs a, int stages) {
    constexpr bool kRing = VEC == 8 && THREADS <= 256;
    constexpr bool kAhead = !kRing && THREADS * NV * VEC <= 8192;  // registers for the next row
    constexpr bool XW = XT == kAny || XT == MOE_F32, RW = RT == kAny || RT == MOE_F32;
    constexpr int kPlanes = (XW ? 2 : 1) + (RW ? 2 : 1);  // 16-byte pieces of a run of x and r
    extern __shared__ uint4 ring[];  // [stage][run][piece][thread]
    __shared__ float2 part[2][THREADS / 32];
    const int xt = XT == kAny ? a.x_type : XT, rt = RT == kAny ? a.res_type : RT;
    const int wt = WT == kAny ? a.w_type : WT, yt = YT == kAny ? a.y_type : YT;
    grid_launch_next();
    grid_dep_wait();
    const int warps = blockDim.x >> 5, w0 = threadIdx.y * warps;
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int e0 = threadIdx.x * VEC, de = blockDim.x * VEC;
    const bool has_res = FULL || a.res, has_sum = FULL || a.sum, has_w = FULL || a.w;
    auto in = [&](int n) { return FULL || e0 + n * de < a.H; };  // run n is in the row
    const int all = blockDim.x * blockDim.y, me = threadIdx.y * blockDim.x + threadIdx.x;
    Raw<VEC, XW> rx[NV];
    Raw<VEC, RW> rr[NV];
    // a thread reads back only what it copied itself: no barrier but its own wait
    const uint8_t* gx = static_cast<const uint8_t*>(a.x) + (row * a.x_stride + e0) * type_bytes(xt);
    const uint8_t* gr = static_cast<const uint8_t*>(a.res) + (row * a.res_stride + e0) * type_bytes(rt);
    const int64_t gx_step = step * a.x_stride * type_bytes(xt), gr_step = step * a.res_stride * type_bytes(rt);
    auto copy = [&](int64_t r, int stage) {  // the next row, r, that gx and gr stand at
        if (r < a.T) {
#pragma unroll
            for (int n = 0; n < NV; ++n)
                if (in(n)) {
                    uint4* d = ring + (stage * NV + n) * kPlanes * all + me;
                    const uint8_t* px = gx + n * de * type_bytes(xt);
                    cp_async16(d, px);
                    if (XW && xt == MOE_F32) cp_async16(d + all, px + 16);
                    if (has_res) {
                        const uint8_t* pr = gr + n * de * type_bytes(rt);
                        cp_async16(d + (XW ? 2 : 1) * all, pr);
                        if (RW && rt == MOE_F32) cp_async16(d + (XW ? 3 : 2) * all, pr + 16);
                    }
                }
        }
        gx += gx_step;
        gr += gr_step;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto take = [&](int stage) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const uint4* d = ring + (stage * NV + n) * kPlanes * all + me;
            if constexpr (VEC == 8) {
                rx[n].set(d, all);
                if (has_res) rr[n].set(d + (XW ? 2 : 1) * all, all);
            }
        }
    };
    auto fetch = [&](int64_t r) {
        if (r >= a.T) return;
#pragma unroll
        for (int n = 0; n < NV; ++n)
            if (in(n)) {
                rx[n].load(a.x, r * a.x_stride + e0 + n * de, xt);
                if (has_res) rr[n].load(a.res, r * a.res_stride + e0 + n * de, rt);
            }
    };
    if (kAhead) fetch(row);
    if (kRing)
        for (int i = 0; i < stages - 1; ++i) copy(row + i * step, i);
    int slot = 0;
    uint8_t* ps = static_cast<uint8_t*>(a.sum) + (row * a.sum_stride + e0) * type_bytes(rt);
    uint8_t* py = static_cast<uint8_t*>(a.y) + (row * a.y_stride + e0) * type_bytes(yt);
    const int64_t ps_step = step * a.sum_stride * type_bytes(rt), py_step = step * a.y_stride * type_bytes(yt);
    // every thread of the CTA makes the same number of rounds (their barriers)
    int flip = 0;
    for (int64_t first = (int64_t)blockIdx.x * blockDim.y; first < a.T;
         first += step, row += step, ps += ps_step, py += py_step, flip ^= 1) {
        const bool live = FULL || row < a.T;
        Raw<VEC, WT == kAny || WT == MOE_F32> rw[NV];
        if (kRing) {
            const int next = slot == 0 ? stages - 1 : slot - 1;  // the slot of the row before
            copy(row + (stages - 1) * step, next);
            cp_wait(stages - 1);
            take(slot);
            slot = slot + 1 == stages ? 0 : slot + 1;
        } else if (!kAhead) {
            fetch(row);
        }
#pragma unroll
        for (int n = 0; n < NV; ++n)
            if (has_w && in(n)) rw[n].load(a.w, e0 + n * de, wt);
        float s[NV][VEC];
        float ss = 0.f, top = 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[n][i] = 0.f;
            if (live && in(n)) {
                rx[n].get(xt, s[n]);
                if (has_res) {
                    float r[VEC];
                    rr[n].get(rt, r);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) s[n][i] += r[i];
                }
            }
        }
        if (kAhead) fetch(row + step);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            if (in(n)) {
                if (has_sum && live) store_run<VEC>(ps, n * de, rt, s[n]);
#pragma unroll
                for (int i = 0; i < VEC; ++i) ss = fmaf(s[n][i], s[n][i], ss);
                if (has_w) {
                    float w[VEC];
                    rw[n].get(wt, w);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) s[n][i] *= w[i];
                }
                if (yt == MOE_E4M3) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) top = max_nan(top, fabsf(s[n][i]));
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (yt == MOE_E4M3) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        }
        if (warps > 1) {
            // two sets of partials: the next round's writes meet no reader of this round's
            if ((threadIdx.x & 31) == 0) part[flip][w0 + (threadIdx.x >> 5)] = make_float2(ss, top);
            __syncthreads();
            // lane i takes partial i, the rest add nothing: the same tree in every warp, one result a row
            constexpr int kMost = THREADS / 32 > 16 ? 32 : (THREADS / 32 > 8 ? 16 : 8);
            const int lane = threadIdx.x & (kMost - 1);
            const float2 v = lane < warps ? part[flip][w0 + lane] : make_float2(0.f, 0.f);
            ss = v.x;
            top = v.y;
#pragma unroll
            for (int o = kMost / 2; o > 0; o >>= 1) {
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (yt == MOE_E4M3) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
            }
        }
        if (!live) continue;
        const float square = fmaf(ss, a.inv_h, a.eps);
        float f = rsqrtf(square), after = 1.f;
        if (yt == MOE_E4M3) {
            // a NaN anywhere, or a square past fp32 (f would be 0): a NaN scale and NaN codes
            const float m = square < INFINITY ? top * f : __uint_as_float(0x7fc00000u);
            const float scale = m == m ? fmaxf(m * (1.f / kE4M3Max), 1.17549435e-38f) : m;
            if (threadIdx.x == 0) a.scale[row] = scale;
            if (m != m) {
                f = m;
            } else if (top > 1e-30f && scale > 1.17549435e-38f) {
                f = kE4M3Max / top;  // = f / scale: one factor
            } else {
                after = 1.f / scale;  // finite, as scale >= 2^-126
            }
        }
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[n][i] *= f;
        if (yt == MOE_E4M3 && after != 1.f) {  // f / scale may be past fp32: y first, then over the scale
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int i = 0; i < VEC; ++i) s[n][i] *= after;
        }
#pragma unroll
        for (int n = 0; n < NV; ++n)
            if (in(n)) store_run<VEC>(py, n * de, yt, s[n]);
    }
}

template <int VEC, int NV, int THREADS, int XT, int RT, int WT, int YT, bool FULL = false>
cudaError_t launch(const NormArgs& a, cudaStream_t st) {
    const int runs = (a.H + VEC - 1) / VEC;
    const int tx = ((runs + NV - 1) / NV + 31) / 32 * 32;
    const int ty = tx >= 128 ? 1 : 128 / tx;
    if constexpr (!FULL && VEC == 8 && THREADS <= 256 && XT != kAny) {
        if (a.res && a.sum && a.w && ty == 1 && tx * NV * VEC == a.H)
            return launch<VEC, NV, THREADS, XT, RT, WT, YT, true>(a, st);
    }
    const auto kernel = norm_kernel<VEC, NV, THREADS, XT, RT, WT, YT, FULL>;
    // one round of CTAs: a CTA that had to wait for another to end would walk its rows alone
    static std::atomic<int> resident[THREADS / 32 + 1];  // CTAs an SM holds, by warps
    const int warps = tx * ty / 32;
    constexpr bool kRing = VEC == 8 && THREADS <= 256;
    constexpr int kPlanes = (XT == kAny || XT == MOE_F32 ? 2 : 1) + (RT == kAny || RT == MOE_F32 ? 2 : 1);
    const int stage_bytes = NV * kPlanes * 32 * warps * 16;
    const int stages = kRing ? std::max(2, std::min(4, kRingBytes / stage_bytes)) : 0;
    const int smem = stages * stage_bytes;
    if (kRing) {
        static std::atomic<uint64_t> configured;
        cudaError_t err = ensure_smem_limit((const void*)kernel, std::max(kRingBytes, 2 * NV * kPlanes * THREADS * 16), configured, true);
        if (err != cudaSuccess) return err;
    }
    int per_sm = resident[warps].load(std::memory_order_relaxed);
    if (per_sm == 0) {
        cudaError_t err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, 32 * warps, smem);
        if (err != cudaSuccess) return err;
        if (per_sm < 1) per_sm = 1;
        resident[warps].store(per_sm, std::memory_order_relaxed);
    }
    int64_t grid = ((int64_t)a.T + ty - 1) / ty;
    if (grid > (int64_t)per_sm * a.sm_count) grid = (int64_t)per_sm * a.sm_count;
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(tx, ty), smem, st, a, stages);
}

// The weights of x's type and y of x's type or E4M3: types as template arguments.
template <int VEC, int NV, int THREADS, int XT>
cudaError_t typed(const NormArgs& a, cudaStream_t st) {
    const bool wide = (a.res || a.sum) && a.res_type == MOE_F32;
    if (a.y_type == MOE_E4M3)
        return wide ? launch<VEC, NV, THREADS, XT, MOE_F32, XT, MOE_E4M3>(a, st)
                    : launch<VEC, NV, THREADS, XT, XT, XT, MOE_E4M3>(a, st);
    return wide ? launch<VEC, NV, THREADS, XT, MOE_F32, XT, XT>(a, st) : launch<VEC, NV, THREADS, XT, XT, XT, XT>(a, st);
}

template <int VEC, int NV, int THREADS>
cudaError_t pick(const NormArgs& a, cudaStream_t st) {
    const bool usual = (!a.w || a.w_type == a.x_type) && (a.y_type == a.x_type || a.y_type == MOE_E4M3) &&
                       (!(a.res || a.sum) || a.res_type == a.x_type || a.res_type == MOE_F32);
    if (usual && a.x_type == MOE_BF16) return typed<VEC, NV, THREADS, MOE_BF16>(a, st);
    if (usual && a.x_type == MOE_F16) return typed<VEC, NV, THREADS, MOE_F16>(a, st);
    if (usual && a.x_type == MOE_F32) return typed<VEC, NV, THREADS, MOE_F32>(a, st);
    return launch<VEC, NV, THREADS, kAny, kAny, kAny, kAny>(a, st);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    const bool vec = a.H % 8 == 0 && runs_aligned(a.x, a.x_type, 8, a.x_stride) &&
                     (!a.res || runs_aligned(a.res, a.res_type, 8, a.res_stride)) &&
                     (!a.w || runs_aligned(a.w, a.w_type, 8)) &&
                     (!a.sum || runs_aligned(a.sum, a.res_type, 8, a.sum_stride)) &&
                     runs_aligned(a.y, a.y_type, 8, a.y_stride);
    if (vec) {
        if (a.H <= 2048) return pick<8, 1, 256>(a, st);
        if (a.H <= 4096) return pick<8, 2, 256>(a, st);
        if (a.H <= 8192) return pick<8, 4, 256>(a, st);
        return launch<8, 4, 1024, kAny, kAny, kAny, kAny>(a, st);
    }
    // Single elements: a thread holds five while 1024 threads then cover the row, and eight above.
    // Five against eight, f16 with an fp32 residual: 4000 x 4099 49.9 and 60.0 us, 4000 x 5119 56.3 and
    // 62.2, 777 x 4501 13.5 and 14.8; bf16 to E4M3 4000 x 4099 60.8 and 66.8, 4000 x 5119 70.3 and 69.2.
    // (Six to 6144 gain 10% just above 5120 and lose as much below it.)
    if (a.H <= 5120) return pick<1, 5, 1024>(a, st);
    if (a.H <= 8192) return pick<1, 8, 1024>(a, st);
    return launch<1, 32, 1024, kAny, kAny, kAny, kAny>(a, st);
}

}  // namespace moe
