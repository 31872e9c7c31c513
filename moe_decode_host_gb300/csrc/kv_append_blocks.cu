// Position rotation and append to an E4M3 cache with a scale for each block of tokens and head.
//
//   scale = 2^e, e the smallest with max |values| <= 448 * 2^e;  code = E4M3(value / scale)
//
// over the values that the call puts into the block; a block that had tokens keeps its scale if
// that is as large in magnitude, and else its other codes are rewritten under the new one.  Powers of two
// lose nothing in the rewriting but low bits of codes that become subnormal, and E4M3 has as many
// bits under them as under any other scale.  (Codes under a scale of the caller's own that is no power
// of two are rounded again.)
//
// Memory bound: q, k, v in, q_out and the codes out, each once.  The tokens of a block follow one
// another in the call, so a team of threads (a warp where that is little, else four) takes what
// the call puts into one block of one head of k or v: it turns the values, keeps them in shared memory
// while their maximum is found, and writes codes and scale.  Teams look for the blocks that begin
// in their window of tokens, so nothing has to be counted or sorted beforehand.  The queries of small
// calls are turned by further CTAs of the same launch, those of large ones by the plain append's kernel.
//
// Measured on a GB300, bf16 of 32 + 8 + 8 heads of 128 into blocks whose scales stay: 8192 tokens into blocks of 64 63 us
// (in the profiler 24 for the queries' launch and 36 for the keys' and values'; the rest passes between the two), of 128 75,
// of 16 80, of 4 72, of 1 183; into blocks of 32 8 tokens 3.6, 64 sequences 4.2, 512 sequences 11.6; 256 tokens of one into
// blocks of 64 10.9.  Over 30 caches in turn, whose blocks all have to be rewritten under larger scales, and the same calls
// afterwards: 8 tokens 6.8 and 3.6, 512 sequences 34 and 13.9, 8192 tokens of 32 sequences 67.5 and 65.
#include <algorithm>

#include "kv_append.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kAny = -1;   // a type known only at run time
constexpr int kChecks = 256;  // most CTAs that look at runs

// The smallest power of two s with top <= 448 s, from 2^-126 to 2^119.  448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_for(float top) {
    const uint32_t b = __float_as_uint(top);
    int e = (int)(b >> 23) + ((b & 0x7fffffu) > 0x600000u ? 1 : 0) - 8;  // biased
    e = e < 1 ? 1 : (e > 127 + 119 ? 127 + 119 : e);
    return __uint_as_float((uint32_t)e << 23);
}

// The block that a slot lies in, as the slot of its first entry; negative: the token is not appended.
struct Home {
    int64_t first;
    int page, block;
};
__device__ __forceinline__ Home home_of(const AppendArgs& a, int64_t slot) {
    Home h{-1, 0, 0};
    if (slot < 0) return h;
    const int64_t page = slot >> 32 ? slot / a.kv.page_size : (int64_t)((uint32_t)slot / (uint32_t)a.kv.page_size);
    if (page >= a.kv.n_pages) {
        set_status(a.kv.status, MOE_ERR_BAD_INDEX);
        return h;
    }
    const int entry = (int)(slot - page * a.kv.page_size);
    h.page = (int)page;
    h.block = block_of(a.kv, entry);
    h.first = slot - entry + h.block * a.kv.scale_tokens;
    return h;
}

// Four codes as fp32.
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float (&v)[4]) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

// Calls whose tokens may go to different teams each: up to some warps for each that the GPU holds at once.
bool few(const AppendArgs& a) { return (int64_t)a.T * 2 * a.kv.kv_heads <= 16384; }

// TEAM threads, 32 or all of the CTA.
template <int TEAM>
__device__ __forceinline__ void team_sync() {
    if constexpr (TEAM == 32) __syncwarp();
    else __syncthreads();
}

// What a thread has brought of KEEP tokens at a time, in shared memory that it alone reads: two runs of a head and,
// for keys, the cosines and sines of their pairs, and the tokens' entries in the block.
template <int KEEP>
struct Kept {
    uint4 piece[KEEP][6][kThreads];  // two runs; four of the table, or the turned values
    int at[KEEP][kThreads];  // -1: not appended
};

// The runs of tokens of one block that begin among `window` tokens from w0 on (at most 32), the same in every warp.
struct Window {
    int64_t mine;     // lane i: the slot of token w0 + i
    Home home;        // and its home
    uint32_t begins;  // bit i: a run begins with token w0 + i
};
__device__ __forceinline__ bool within(const AppendArgs& a, int64_t slot, int64_t first) {
    return (uint64_t)(slot - first) < (uint64_t)a.kv.scale_tokens;
}
__device__ __forceinline__ Window window_of(const AppendArgs& a, int64_t w0, int window) {
    const int lane = threadIdx.x & 31;
    Window w;
    // a block is scale_tokens slots in a row, so that only this takes a division: a run begins where the token before
    // is in another one
    w.mine = lane < window && w0 + lane < a.T ? a.slots[w0 + lane] : -1;
    int64_t before = __shfl_up_sync(0xffffffffu, w.mine, 1);
    if (lane == 0) before = w0 > 0 ? a.slots[w0 - 1] : -1;
    w.home = home_of(a, w.mine);
    w.begins = __ballot_sync(0xffffffffu, w.home.first >= 0 && (before < 0 || !within(a, before, w.home.first)));
    return w;
}

// Whether the runs that begin with tokens [w0, w0 + 32) are their blocks' only ones in the call, told in the status:
// teams of their own would take two at a time.  One that begins with its block's first entry needs no look, for any
// other of that block begins behind it; so a prompt has one to look for, a decode step as many as it has sequences.
// CTAs of their own do it beside the others: 8 tokens 3.55 us (3.4 without), 512 sequences 11.5 (11.5), 8192 sequences
// 441 (432), or 47 (37) with one key head; looking in every team before it writes took 512 sequences 15.2 us.
__device__ __forceinline__ void check_runs(const AppendArgs& a, int64_t w0) {
    const int lane = threadIdx.x & 31;
    const auto slot_at = [&](int64_t t) { return t < a.T ? a.slots[t] : -1; };
    int64_t next = slot_at(threadIdx.x);
    const Window win = window_of(a, w0, 32);
    const uint32_t starts = __ballot_sync(0xffffffffu, (win.begins >> lane & 1u) && win.mine != win.home.first);
    if (!starts) return;
    const uint32_t low = (uint32_t)win.home.first;
    const bool many = __popc(starts) > 4;  // then all without branches
    for (int64_t t = threadIdx.x; t - lane < a.T; t += kThreads) {
        const int64_t slot = next;
        next = slot_at(t + kThreads);
        uint32_t near = 0;  // starts whose block this token's slot lies in, by the low halves of both
        const auto look = [&](int j) {
            if ((uint32_t)slot - __shfl_sync(0xffffffffu, low, j) < (uint32_t)a.kv.scale_tokens) near |= 1u << j;
        };
        if (many) {
#pragma unroll
            for (int j = 0; j < 32; ++j) look(j);
        } else {
            for (uint32_t left = starts; left; left &= left - 1) look(__ffs(left) - 1);
        }
        near &= starts;
        if (t >= w0 && t < w0 + 32) near &= ~(1u << (t - w0));  // itself
        for (uint32_t left = __reduce_or_sync(0xffffffffu, near); left; left &= left - 1) {
            const int j = __ffs(left) - 1;
            const int64_t first = __shfl_sync(0xffffffffu, win.home.first, j);
            // another token of the block: one that does not go on with a run begins another
            if ((near >> j & 1u) && within(a, slot, first) && (t == 0 || !within(a, a.slots[t - 1], first)))
                set_status(a.kv.status, MOE_ERR_BAD_INDEX);
        }
    }
}

// A team's share of k and v: the runs `begins` of the window, of head `head` of k (side 0) or v (side 1).
// KEEP > 0: 16-bit values and table rows that can be copied 16 bytes at a time, KEEP tokens of a thread at
// once, so that a block that they hold is read once; 0: read twice.
template <int XT, int VEC, int TEAM, int KEEP, bool FOURS>
__device__ __forceinline__ void append_block_runs(const AppendArgs& a, const Window& win, uint32_t begins, int64_t w0,
                                                  int window, int side, int head, uint32_t* mask,
                                                  float (*part)[kThreads / 32], Kept<KEEP ? KEEP : 1>& kept) {
    const int me = threadIdx.x % TEAM, lane = threadIdx.x & 31;
    const int items = a.kv.head_dim / (2 * VEC), step = TEAM / items, g = me / items;
    const bool works = g < step;
    const Item<VEC> it(a, me % items);
    const int xt = XT == kAny ? a.type : XT;
    const void* src = side ? a.v : a.k;
    const int64_t ts = side ? a.v_ts : a.k_ts, hs = side ? a.v_hs : a.k_hs;
    uint8_t* cache = static_cast<uint8_t*>(side ? a.kv.v : a.kv.k) + head * a.kv.head_stride;
    float* scales = side ? a.kv.v_scale : a.kv.k_scale;
    const bool turn = it.turn && side == 0;
    const int64_t mine = win.mine;
    while (begins) {  // the same in every warp of the team
        const int i0 = __ffs(begins) - 1;
        begins &= begins - 1;
        const int64_t t0 = w0 + i0, first = __shfl_sync(0xffffffffu, win.home.first, i0);
        const int page = __shfl_sync(0xffffffffu, win.home.page, i0), block = __shfl_sync(0xffffffffu, win.home.block, i0);
        // the run's end: the next token of another home, maybe behind the window
        const uint32_t others = __ballot_sync(0xffffffffu, lane > i0 && (mine < 0 || !within(a, mine, first)));
        int64_t t1 = others ? w0 + __ffs(others) - 1 : w0 + 32;
        if (!others || t1 >= w0 + window) {
            t1 = w0 + window;
            for (bool on = true; on && t1 < a.T;) {
                const int64_t t = t1 + lane;
                const uint32_t same = __ballot_sync(0xffffffffu, t < a.T && within(a, a.slots[t], first));
                on = same == 0xffffffffu;
                t1 += on ? 32 : __ffs(~same) - 1;
            }
            if (t1 > a.T) t1 = a.T;
        }
        const int64_t base = (int64_t)page * a.kv.page_stride + (int64_t)(block * a.kv.scale_tokens) * a.kv.token_stride;
        float* scale_at = scales + ((int64_t)page * a.kv.blocks + block) * a.kv.kv_heads + head;
        const float old = *scale_at;

        // the entry of a token in the block, or -1 where it has no position in the table
        auto entry_of = [&](int64_t t, Place& place) {
            place = place_of(a, t);
            if (place.valid) return (int)(a.slots[t] - first);
            set_status(a.kv.status, MOE_ERR_BAD_INDEX);
            return -1;
        };
        // KEEP tokens of this thread from t on
        auto bring = [&](int64_t t) {
            if constexpr (KEEP > 0) {
#pragma unroll
                for (int k = 0; k < KEEP; ++k, t += step) {
                    int at = -1;
                    if (works && t < t1) {
                        Place place;
                        at = entry_of(t, place);
                        const uint16_t* x = static_cast<const uint16_t*>(src) + t * ts + head * hs;
                        cp_async16(&kept.piece[k][0][threadIdx.x], x + it.e0);
                        cp_async16(&kept.piece[k][1][threadIdx.x], x + it.e1);
                        if (turn && at >= 0) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int pair = it.j * VEC + (i & 1) * 4;
                                const int axis = a.axes == 1 ? 0 : axis_of(a, pair);
                                cp_async16_l1(&kept.piece[k][2 + i][threadIdx.x],
                                              a.cos_sin + (int64_t)place.at(axis) * a.rot + pair + (i >> 1) * (a.rot / 2));
                            }
                        }
                    }
                    kept.at[k][threadIdx.x] = at;
                }
                asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
            }
        };
        // values of token t, or of the k-th of those kept, turned; its entry, or -1.  Turned ones take the table's place
        // in what is kept; `again`: they are there
        auto values = [&](int64_t t, int k, bool again, float (&x0)[VEC], float (&x1)[VEC]) {
            if constexpr (KEEP > 0) {
                const int at = kept.at[k][threadIdx.x];
                if (at < 0) return at;
                uint4* piece = &kept.piece[k][0][threadIdx.x];
                if (turn && again) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float* x = i < 2 ? x0 + 4 * i : x1 + 4 * (i - 2);
                        const float4 v = *reinterpret_cast<const float4*>(piece + (2 + i) * kThreads);
                        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
                    }
                    return at;
                }
                Raw<VEC, false> r0, r1;
                r0.set(&kept.piece[k][0][threadIdx.x], 0);
                r1.set(&kept.piece[k][1][threadIdx.x], 0);
                r0.get(XT, x0);
                r1.get(XT, x1);
                if (turn) {
                    float cs[VEC], sn[VEC];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 c = kept.piece[k][2 + i][threadIdx.x], s = kept.piece[k][4 + i][threadIdx.x];
                        cs[4 * i] = __uint_as_float(c.x), cs[4 * i + 1] = __uint_as_float(c.y);
                        cs[4 * i + 2] = __uint_as_float(c.z), cs[4 * i + 3] = __uint_as_float(c.w);
                        sn[4 * i] = __uint_as_float(s.x), sn[4 * i + 1] = __uint_as_float(s.y);
                        sn[4 * i + 2] = __uint_as_float(s.z), sn[4 * i + 3] = __uint_as_float(s.w);
                    }
                    rotate<VEC>(a.interleaved, x0, x1, cs, sn);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float* x = i < 2 ? x0 + 4 * i : x1 + 4 * (i - 2);
                        *reinterpret_cast<float4*>(piece + (2 + i) * kThreads) = make_float4(x[0], x[1], x[2], x[3]);
                    }
                }
                return at;
            } else {
                Place place;
                const int at = entry_of(t, place);
                if (at < 0) return at;
                Raw<VEC, XT == kAny || XT == MOE_F32> r0, r1;
                r0.load(src, t * ts + head * hs + it.e0, xt);
                r1.load(src, t * ts + head * hs + it.e1, xt);
                r0.get(xt, x0);
                r1.get(xt, x1);
                if (turn) {
                    float cs[VEC], sn[VEC];
                    turn_of<VEC, FOURS>(a, place, it.j * VEC, cs, sn);
                    rotate<VEC>(a.interleaved, x0, x1, cs, sn);
                }
                return at;
            }
        };
        float top = 0.f;
        bool anew = false;
        constexpr int kEach = KEEP > 0 ? KEEP : 1;  // tokens of a thread at a time
        const bool once = t1 - t0 <= (int64_t)kEach * step;
        auto all = [&](bool again, auto&& use) {  // every token of this thread
#pragma unroll 1
            for (int64_t c = t0; c < t1; c += (int64_t)kEach * step) {
                if (!again || !once) bring(c + g);
#pragma unroll 1
                for (int k = 0; k < kEach; ++k) {
                    const int64_t t = c + g + (int64_t)k * step;
                    if (!works || t >= t1) break;
                    float x0[VEC], x1[VEC];
                    if constexpr (KEEP > 0) {
                        // the largest magnitude of 16-bit values that are not turned, from their bits: two an instruction
                        if (!again && !turn) {
                            const int at = kept.at[k][threadIdx.x];
                            if (at < 0) continue;
                            constexpr uint32_t kInf = XT == MOE_BF16 ? 0x7f80u : 0x7c00u;
                            const uint4 p = kept.piece[k][0][threadIdx.x], q = kept.piece[k][1][threadIdx.x];
                            const uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
                            uint32_t most = 0;
#pragma unroll
                            for (int i = 0; i < 8; ++i) most = __vmaxu2(most, w[i] & 0x7fff7fffu);
                            most = max(most & 0xffffu, most >> 16);
                            if (most <= kInf) {  // else there is a NaN, which does not count: one by one
                                top = fmaxf(top, half_bits_to_f32(most, XT));
                                anew = anew || at == 0;
                                continue;
                            }
                        }
                    }
                    const int at = values(t, k, again && once, x0, x1);
                    if (at >= 0) use(x0, x1, at);
                }
            }
        };
        all(false, [&](const float (&x0)[VEC], const float (&x1)[VEC], int entry) {
            anew = anew || entry == 0;
#pragma unroll
            for (int i = 0; i < VEC; ++i) top = fmaxf(top, fmaxf(fabsf(x0[i]), fabsf(x1[i])));  // NaN does not count
        });
        top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));  // not negative: ordered as its bits
        anew = __any_sync(0xffffffffu, anew);
        if constexpr (TEAM > 32) {
            if (lane == 0) {
                part[0][threadIdx.x >> 5] = top;
                part[1][threadIdx.x >> 5] = anew ? 1.f : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int w = 0; w < TEAM / 32; ++w) {
                top = fmaxf(top, part[0][w]);
                anew = anew || part[1][w] != 0.f;
            }
        }
        const float need = scale_for(top);
        // one of the caller's own may be negative, or large enough though less than the power of two
        const float had = fabsf(old);
        const bool enough = had >= need || (had >= 1.17549435e-38f && top <= 448.f * had);  // 2^-126
        const float scale = anew || !enough ? need : old;
        const float inv = 1.f / scale;
        all(true, [&](float (&x0)[VEC], float (&x1)[VEC], int entry) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                x0[i] *= inv;
                x1[i] *= inv;
            }
            const int64_t to = base + (int64_t)entry * a.kv.token_stride;
            store_run<VEC>(cache, to + it.e0, MOE_E4M3, x0);
            store_run<VEC>(cache, to + it.e1, MOE_E4M3, x1);
        });
        if (!anew && scale != old) {  // the block's other entries keep their values
            const int n = a.kv.scale_tokens;
            for (int i = me; i < (n + 31) / 32; i += TEAM) mask[i] = 0;
            team_sync<TEAM>();
            for (int64_t t = t0 + me; t < t1; t += TEAM)
                if (place_of(a, t).valid) {
                    const int entry = (int)(a.slots[t] - first);
                    atomicOr(mask + (entry >> 5), 1u << (entry & 31));
                }
            team_sync<TEAM>();
            const float factor = old * inv;
            const int pieces = a.kv.head_dim / 16;
            for (int i = me; i < n * pieces; i += TEAM) {
                const int entry = i / pieces;
                if (mask[entry >> 5] >> (entry & 31) & 1u) continue;
                uint4* p = reinterpret_cast<uint4*>(cache + base + (int64_t)entry * a.kv.token_stride) + i % pieces;
                uint4 w = *p;
                auto again = [&](uint32_t& c) {
                    float v[4];
                    e4m3x4_to_f32(c, v);
                    c = pack_e4m3(v[0] * factor, v[1] * factor) | pack_e4m3(v[2] * factor, v[3] * factor) << 16;
                };
                again(w.x), again(w.y), again(w.z), again(w.w);
                *p = w;
            }
        }
        team_sync<TEAM>();  // the parts and the mask are free, and every thread has read the old scale
        if (me == 0) *scale_at = scale;
    }
}

// The first CTAs look whether runs are their blocks' only ones, the next take k and v, a team per (window of tokens,
// head of either); the others, where there are any, a token's queries each.  FEW: a CTA per window of as many tokens as it has warps, which take a run each; the last run
// is the only one that can reach behind the window, and if it does all of them take it (a prompt of 256 tokens
// 10.9 us, 28 by a warp a block; 512 sequences of a token each 11.6 us, 11.0).
template <int XT, int VEC, int TEAM, int KEEP, bool FOURS, bool FEW>
__global__ void __launch_bounds__(kThreads) append_blocks_kernel(const AppendArgs a, int window, int checks, int kv_ctas) {
    static_assert(!FEW || TEAM == 32, "a run a warp");
    __shared__ uint32_t mask[kThreads / TEAM][kMaxScaleTokens / 32];
    __shared__ float part[2][kThreads / 32];
    extern __shared__ __align__(16) uint8_t room[];
    grid_launch_next();
    grid_dep_wait();
    const int xt = XT == kAny ? a.type : XT;
    if ((int)blockIdx.x < checks) {
        for (int64_t w0 = 32 * (int64_t)blockIdx.x; w0 < a.T; w0 += 32 * (int64_t)checks) check_runs(a, w0);
        return;
    }
    const uint32_t cta = blockIdx.x - checks;
    if ((int)cta < kv_ctas) {
        const int heads = 2 * a.kv.kv_heads, team = threadIdx.x / TEAM;
        const uint32_t unit = FEW ? cta : cta * (kThreads / TEAM) + team, w32 = unit / (uint32_t)heads;
        const int64_t w0 = (int64_t)w32 * window;
        const int h = (int)(unit - w32 * heads), side = h >= a.kv.kv_heads, head = side ? h - a.kv.kv_heads : h;
        Kept<KEEP ? KEEP : 1>& kept = *reinterpret_cast<Kept<KEEP ? KEEP : 1>*>(room);
        if (w0 >= a.T) return;  // a team of one warp leaves alone; a CTA's has the same window
        const Window win = window_of(a, w0, window);
        if constexpr (FEW) {
            if (!win.begins) return;  // the whole CTA
            const int last = 31 - __clz(win.begins);
            const int64_t first = __shfl_sync(0xffffffffu, win.home.first, last);
            const bool beyond = w0 + window < a.T && within(a, a.slots[w0 + window], first) &&
                                !__any_sync(0xffffffffu, threadIdx.x % 32 > last && threadIdx.x % 32 < window && !within(a, win.mine, first));
            uint32_t own = beyond ? win.begins & ~(1u << last) : win.begins;
            for (int i = 0; i < team; ++i) own &= own - 1;
            if (own) append_block_runs<XT, VEC, 32, KEEP, FOURS>(a, win, own & -own, w0, window, side, head, mask[team], part, kept);
            if (beyond) append_block_runs<XT, VEC, kThreads, KEEP, FOURS>(a, win, 1u << last, w0, window, side, head, mask[0], part, kept);
        } else {
            append_block_runs<XT, VEC, TEAM, KEEP, FOURS>(a, win, win.begins, w0, window, side, head, mask[team], part, kept);
        }
        return;
    }
    const int64_t t = cta - kv_ctas;
    const int items = a.kv.head_dim / (2 * VEC), step = kThreads / items, g = threadIdx.x / items;
    if (g >= step) return;
    const Item<VEC> it(a, threadIdx.x % items);
    const Place place = place_of(a, t);
    if (!place.valid) {  // no table row: nothing of this token is written
        if (threadIdx.x == 0) set_status(a.kv.status, MOE_ERR_BAD_INDEX);
        return;
    }
    float cs[VEC], sn[VEC];
    if (it.turn) turn_of<VEC, FOURS>(a, place, it.j * VEC, cs, sn);
#pragma unroll 2
    for (int h = g; h < a.kv.q_heads; h += step) {
        Raw<VEC, XT == kAny || XT == MOE_F32> r0, r1;
        r0.load(a.q, t * a.q_ts + h * a.q_hs + it.e0, xt);
        r1.load(a.q, t * a.q_ts + h * a.q_hs + it.e1, xt);
        float x0[VEC], x1[VEC];
        r0.get(xt, x0);
        r1.get(xt, x1);
        if (it.turn) rotate<VEC>(a.interleaved, x0, x1, cs, sn);
        store_run<VEC>(a.q_out, t * a.qo_ts + h * a.qo_hs + it.e0, xt, x0);
        store_run<VEC>(a.q_out, t * a.qo_ts + h * a.qo_hs + it.e1, xt, x1);
    }
}

template <int XT, int VEC, int TEAM, int KEEP, bool FOURS, bool FEW = false>
cudaError_t launch(const AppendArgs& a, cudaStream_t st) {
    // short windows while there are warps for all tokens, so that sequences' tokens go to teams of their own; else as
    // long as a block, where most windows begin one
    const int window = FEW ? kThreads / 32 : few(a) ? 1 : std::min(32, a.kv.scale_tokens);
    const int64_t teams = ((int64_t)a.T + window - 1) / window * 2 * a.kv.kv_heads, per = FEW ? 1 : kThreads / TEAM;
    const int64_t kv_ctas = (teams + per - 1) / per;
    // many queries go faster through the ring of the plain append's kernel, as tokens that are not appended
    const bool alone = !few(a);
    if (alone) {
        AppendArgs q = a;
        q.kv.kv_heads = 0;
        q.kv.type = a.type;
        cudaError_t err = launch_append(q, st);
        if (err != cudaSuccess) return err;
    }
    const int checks = a.kv.scale_tokens > 1 ? std::min(kChecks, (a.T - 1) / 32 + 1) : 0;
    const int64_t grid = checks + kv_ctas + (alone ? 0 : a.T);
    if (grid > 0x3fffffff) return cudaErrorInvalidValue;  // teams are numbered in 32 bits
    const auto kernel = append_blocks_kernel<XT, VEC, TEAM, KEEP, FOURS, FEW>;
    constexpr int smem = KEEP ? (int)sizeof(Kept<KEEP ? KEEP : 1>) : 0;
    static std::atomic<uint64_t> configured;
    cudaError_t err = ensure_smem_limit((const void*)kernel, smem, configured, true);
    if (err != cudaSuccess) return err;
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kThreads), smem, st, a, window, checks, (int)kv_ctas);
}

template <int XT, bool FOURS>
cudaError_t launch_team(const AppendArgs& a, cudaStream_t st) {
    constexpr bool ring = FOURS && XT != MOE_F32;
    // a warp turns 512 / head_dim tokens at a time: few for a long block, which four warps share, and enough
    // for a short one
    if (few(a)) return launch<XT, 8, 32, ring ? 2 : 0, FOURS, true>(a, st);
    return a.kv.scale_tokens <= 8 ? launch<XT, 8, 32, ring ? 2 : 0, FOURS>(a, st)
                                  : launch<XT, 8, kThreads, ring ? 4 : 0, FOURS>(a, st);
}

template <int XT>
cudaError_t launch_fours(const AppendArgs& a, cudaStream_t st) {
    return fours_of(a) ? launch_team<XT, true>(a, st) : launch_team<XT, false>(a, st);
}

}  // namespace

cudaError_t launch_append_blocks(const AppendArgs& a, cudaStream_t st) {
    if (a.T == 0) return cudaSuccess;
    if (append_fits(a, 8)) {
        if (a.type == MOE_BF16) return launch_fours<MOE_BF16>(a, st);
        if (a.type == MOE_F16) return launch_fours<MOE_F16>(a, st);
        return launch_fours<MOE_F32>(a, st);
    }
    return append_fits(a, 4) ? launch<kAny, 4, kThreads, 0, false>(a, st) : launch<kAny, 1, kThreads, 0, false>(a, st);
}

}  // namespace moe
