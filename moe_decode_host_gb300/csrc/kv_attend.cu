// Attention over the paged cache: what is derived from a cache's geometry before a launch.
#include <algorithm>

#include "attend_plan.cuh"
#include "vec.cuh"

namespace moe {
namespace {

// The unit of the rows' offsets: what page and token stride are both multiples of.
int row_shift(const KvView& kv) {
    const uint64_t bytes = (uint64_t)(kv.page_stride | kv.token_stride) * type_bytes(kv.type);
    int s = 4;
    while (s < 30 && !(bytes >> s & 1)) ++s;
    return s;
}

AttendPlan plan_of(const KvView& kv, int sm_count) {
    AttendPlan p;
    const int D = kv.head_dim, es = type_bytes(kv.type), group = kv.q_heads / kv.kv_heads;
    p.dp = D % 64 == 0 || D == 96 ? D : (D < 128 ? 128 : 256);
    p.blocks = group <= 8 ? 1 : (group <= 16 || p.dp > 128 ? 2 : 4);
    const int hc = 8 * p.blocks;
    p.chunks = (group + hc - 1) / hc;
    p.chunk = (group + p.chunks - 1) / p.chunks;
    p.cpr = D * es / 16;
    p.inv = ((1u << 20) + p.cpr - 1) / p.cpr;
    p.swizzle = row_swizzle(p.cpr);
    p.pitch = row_pitch(p.cpr);
    int lg = 0;
    while ((1u << lg) < (uint32_t)kv.page_size) ++lg;
    p.page_shift = 30 + lg;
    p.page_mul = (uint32_t)(((1ull << p.page_shift) + kv.page_size - 1) / kv.page_size);
    p.shift = row_shift(kv);
    const int ctas = ctas_an_sm(p.dp, es, p.blocks);
    p.slots = (ctas * sm_count + 3) / 4 * 4;  // the sums behind the counters are read in fours
    // as many units in flight as fit beside the other CTAs of the SM; the ring also holds the
    // warp's [hc][head_dim + 4] sums when a piece ends, and when a segment is joined the parts'
    // weights (hc * slots floats at most) with the sums of one part or more (hc * head_dim floats)
    const int tokens = unit_tokens(p.dp * es);
    const int unit = 2 * tokens * p.pitch + (kv.scale_tokens ? scale_bytes(tokens) : 0), fixed = hc * (p.dp * 2 + 16) + 16;
    const int least = std::max((hc * (D + 4) * 4 + unit - 1) / unit,
                               (hc * (p.slots + D) * 4 + kAttendWarps * unit - 1) / (kAttendWarps * unit));
    p.stages = kMaxStages;
    while (p.stages > 2 && p.stages > least && fixed + kAttendWarps * p.stages * unit > budget_of(ctas)) --p.stages;
    p.smem = fixed + kAttendWarps * p.stages * unit;
    return p;
}

}  // namespace

bool attend_fits(const KvView& kv) {
    const uint64_t last = ((uint64_t)(kv.n_pages - 1) * kv.page_stride + (uint64_t)(kv.page_size - 1) * kv.token_stride) *
                          type_bytes(kv.type);
    return last >> row_shift(kv) <= 0xffffffffull;
}

// A counter a CTA, then two slots of partial sums a CTA: maxima and sums of the block's
// heads, and their [heads][head_dim] outputs.
size_t attend_workspace(const KvView& kv, int sm_count) {
    const AttendPlan p = plan_of(kv, sm_count);
    return sizeof(float) * ((size_t)p.slots + (size_t)2 * p.slots * 8 * p.blocks * (kv.head_dim + 2));
}

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t st) {
    if (a.B == 0) return cudaSuccess;
    const AttendPlan p = plan_of(a.kv, a.sm_count);
    if (a.kv.type == MOE_BF16) return launch_attend_bf16(a, p, st);
    if (a.kv.type == MOE_F16) return launch_attend_f16(a, p, st);
    return a.kv.scale_tokens ? launch_attend_e4m3_blocks(a, p, st) : launch_attend_e4m3(a, p, st);
}

}  // namespace moe
