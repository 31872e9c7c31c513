// Sizes that the attention kernels and their host side share.
#pragma once

#include "internal.cuh"

namespace moe {

constexpr int kAttendWarps = 4;  // of a CTA
// CTAs that share an SM, by the registers that their sums take (nt blocks of 8 heads of dp)
// and the shared memory of a useful ring (es: bytes of an element).
__host__ __device__ constexpr int ctas_an_sm(int dp, int es, int nt) {
    return dp <= 128 ? (nt > 2 ? 2 : 3) : (es == 1 ? 2 : 1);
}
constexpr int budget_of(int ctas) { return ctas == 3 ? 73 * 1024 : (ctas == 2 ? 111 * 1024 : 222 * 1024); }

// Tokens of a unit, for rows of `bytes` (head_dim rounded up): the wider unit halves the
// work a token that does not depend on its row (page look-up, the maxima's exchange).
__host__ __device__ constexpr int unit_tokens(int bytes) { return bytes <= 128 ? 32 : 16; }
constexpr int kMaxStages = 8;    // units of a warp's ring
constexpr int kMinUnits = 4;     // units worth a CTA of its own: one a warp
// Units that a CTA could stream in the time that starting and ending a piece takes (about 5
// us): each segment is that much longer on the line that the CTAs share out, or those with
// several pieces would end last (0, 6, 10, 16: 172.8, 168.8, 167.8, 168.4 us for 32 ragged
// sequences, 24.5, 21.1, 20.7, 20.1 us for the windowed batch of 19).
constexpr int kStart = 12;
// Units of a segment that a CTA takes whole, where there is a CTA for each segment: 16 units are
// done in less time than parts are joined, 24 are not (whole against split, D 128: one sequence of
// 1 token 4.2 and 10.5 us, of 256 6.4 and 7.6, of 384 7.9 and 7.7; 8 of 100 to 300 7.7 and 8.8, of
// 10 to 380 9.3 and 8.8).
constexpr int kWhole = 20;
constexpr int64_t kMaxTokens = 1 << 30;  // of a sequence: token indexes stay in 32 bits
constexpr float kSlack = 8.f;    // of the maximum over its reference, in powers of two
// f16 weights are kept 2^kLift larger than the softmax has them, up to 2^14: what f16 can no longer
// hold is then below 2^-31 of the largest.  (Unlifted, 2^18 weights of 2^-25 beside one of 1 vanish.)
constexpr float kLift = 6.f;
constexpr float kLog2e = 1.44269504f;
constexpr float kLn2 = 0.69314718f;

// What the host derives from the cache and the call.
struct AttendPlan {
    int dp, blocks;  // the kernel's DP and NT
    int smem;
    int chunk;      // query heads of a segment, at most 8 NT
    int chunks;     // segments of a key head
    int pitch, swizzle;  // bytes of a row in the ring, and whether its pieces change places (row_pitch)
    int stages;
    int cpr;        // 16-byte pieces of a row
    uint32_t inv;   // 2^20 / cpr rounded up: row of piece i = i * inv >> 20 (i <= 512)
    uint32_t page_mul;  // t / page_size = t * page_mul >> page_shift for t < 2^30
    int page_shift;
    int shift;      // offsets of rows in the cache are kept in units of 2^shift bytes
    int slots;      // CTAs the workspace has room for
};

// ldmatrix reads one 16-byte piece of 8 rows at a time.  Rows of whole 128 bytes keep piece i
// in place i ^ swap_of(row) (swizzle 7), others are an odd number of pieces apart (swizzle 0).
__host__ __device__ constexpr int row_swizzle(int pieces) { return pieces % 8 ? 0 : 7; }
__host__ __device__ constexpr int row_pitch(int pieces) {
    return pieces % 8 ? ((pieces | 1) < 3 ? 3 : (pieces | 1)) * 16 : pieces * 16;
}
// One launcher per cache type, each in a translation unit of its own.
cudaError_t launch_attend_bf16(const AttendArgs& a, const AttendPlan& p, cudaStream_t st);
cudaError_t launch_attend_f16(const AttendArgs& a, const AttendPlan& p, cudaStream_t st);
cudaError_t launch_attend_e4m3(const AttendArgs& a, const AttendPlan& p, cudaStream_t st);

}  // namespace moe
