/*
 * moehost.h -- C ABI of the GB300 (sm_103a) library for the mixture-of-experts
 * layer of a decode step whose experts do not all fit in HBM.
 *
 * Method (from "DeepSeek-V4.1-Flash on One GB300 Without the Second GPU: What the
 * Sidecar Is Worth", section 1, The idea): the router picks the top-k experts per
 * token; cold experts live in pinned host memory; one kernel per layer copies only
 * the routed cold experts into a shared HBM slot scratch and remaps their ids; one
 * grouped SwiGLU expert call then runs over all experts as if they were resident;
 * outputs are combined with the router weights; between steps a residency manager
 * promotes often-picked cold experts and demotes quiet hot ones.
 *
 * Conventions
 *  - Every call returns an int status: MOE_OK (0) or a negative MOE_ERR_* code.
 *    A call that returns MOE_ERR_INVALID_ARG has launched nothing; after
 *    MOE_ERR_CUDA part of its work may already be enqueued.  Where a call lists no
 *    errors, a null handle or pointer gives MOE_ERR_INVALID_ARG and a failed CUDA
 *    call MOE_ERR_CUDA.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *    All device work is enqueued on it; nothing synchronises the stream except
 *    residency_update on an acting step in the synchronous residency mode (it
 *    reads the pick counters on the host), moe_get_status, moe_layer_get_loc and
 *    moe_layer_get_counts.  In the default deferred mode residency_update waits
 *    (host side) only for the previous acting call's counter copy.
 *  - Errors found by a kernel after launch (non-finite logits, an expert id out of
 *    range) are written to the layer's device status word (first error wins);
 *    moe_get_status reads it.
 *  - Ownership: the caller owns every buffer it passes (device memory, and host
 *    blobs that are pinned and mapped, e.g. cudaHostAlloc or torch pin_memory).
 *    The library borrows raw pointers for the life of the layer and owns only its
 *    handles and small internal tables (placement map, phys-id pointer table, pick
 *    counters, status word), freed by the destroy calls.
 *  - Shapes: H and I multiples of 128; 1 <= k <= 32; k <= E <= 1024.
 *  - Host threads: a layer (and the scratch it shares) keeps host-side state
 *    (placement map, pending-copy flag, step count), so calls on one layer, or on
 *    layers sharing a scratch, must not run concurrently from several host
 *    threads; distinct layers with distinct scratches may.  moe_combine,
 *    moe_quant_mxfp4 and moe_residency_plan hold no state.
 *
 * Expert blob format (one contiguous blob per expert, every plane 16-byte aligned):
 *   w13 nibbles [2I][H/2] | w13 scales [2I][H/32] | w2 nibbles [H][I/2] | w2 scales [H][I/32]
 *   MXFP4: E2M1 elements, E8M0 scale per 32-element block along the reduction
 *   dimension ("A 475 GB Model Across Two Workstations, With the Table on Disk",
 *   Abstract: routed experts ship in MXFP4).  w13 rows 0..I-1 are the gate
 *   projection, rows I..2I-1 the up projection (the fused w13/w2 planes of "Milo
 *   and James Try Inference Engineering", offload flag table).  Rows are K-major:
 *   element k of a row is in byte k/2, low nibble when k is even.  Scale byte b
 *   of a row is the exponent of elements 32b..32b+31.
 *
 * Placement: loc[e] in [0, n_hot) is an HBM slot; loc[e] = n_hot + c is cold slot
 * c, whose bytes live in host blob c and are copied to scratch slot c when routed.
 * The physical id of a pick is loc of its expert.
 */
#ifndef MOEHOST_H
#define MOEHOST_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_OK 0
#define MOE_ERR_INVALID_ARG (-1)
#define MOE_ERR_CUDA (-2)
#define MOE_ERR_NONFINITE (-3)
#define MOE_ERR_BAD_EXPERT (-4)
#define MOE_ERR_TIMEOUT (-5)
#define MOE_ERR_NOMEM (-6)
#define MOE_ERR_INJECTED (-7)
#define MOE_ERR_SCRATCH_TOO_SMALL (-8)
#define MOE_ERR_BAD_INDEX (-9)

/* Element types of the decoder-layer operators (moe_add_rms_norm, moe_quant_e4m3, moe_kv_*,
 * moe_linear, moe_linear_blocks).  MOE_E4M3 is the 8-bit float with 4 exponent and 3 mantissa bits,
 * largest value 448; conversions to it round to nearest, ties to even, and saturate. */
#define MOE_BF16 0
#define MOE_F16 1
#define MOE_F32 2
#define MOE_E4M3 3

/* Activations of moe_linear.  GELU is the exact form, v * Phi(v).  It is computed to 2^-18 of its
 * value and SiLU to 2^-20 (where that is a normal fp32 number) before the output is rounded. */
#define MOE_ACT_NONE 0
#define MOE_ACT_RELU 1
#define MOE_ACT_SILU 2
#define MOE_ACT_GELU 3

/* Layer parameters.
 *  E, k        experts and picks per token ("Milo and James Try Inference
 *              Engineering", the mixture-of-experts paragraph: 384 experts, 6 per
 *              token).
 *  H, I        hidden and expert intermediate sizes.
 *  n_hot       experts resident in HBM; n_cold = E - n_hot in pinned host memory
 *              ("DeepSeek-V4.1-Flash on One GB300 ...", section 1: 255 / 129).
 *  renorm      0: pick weight = softmax probability; 1: divided by the sum over
 *              the k picks.
 *  swap_every  residency_update acts on every swap_every-th call (0 = never).
 *  max_swaps   at most this many swaps per acting update (<= 64).
 *  hysteresis  a cold expert is promoted over a hot one only when its window
 *              count exceeds hysteresis times the hot one's (same page, section 3:
 *              3.0 is the published default).
 *  host_mirror 0: cold_blobs_host holds the n_cold cold slots' blobs and a swap
 *              exchanges bytes between an HBM slot and a host blob.  1:
 *              cold_blobs_host holds a pinned copy of every expert, indexed by
 *              expert id (E blobs); a demotion moves no bytes and a promotion
 *              copies the expert into its HBM slot from its scratch slot when that
 *              slot still holds this layer's copy of it, else from its host copy.
 *              The host copies must equal the HBM-resident experts' bytes.
 *  zero_copy   0: cold_gather copies the picked cold experts into their scratch
 *              slots and moe_grouped_ffn reads them there.  1 (calls of at most 64
 *              tokens): cold_gather only remaps, and moe_grouped_ffn reads the
 *              picked cold experts' weights in place from their pinned host blobs,
 *              on the layer's copy stream alongside the experts in HBM ("Milo and
 *              James Try Inference Engineering": reading expert rows from pinned
 *              host memory over the link; "Running High-Quality DeepSeek V4 Flash
 *              on One 96 GB GPU": mapped host planes read in place).  Larger calls
 *              copy as with 0. */
typedef struct moe_params {
    int E, k, H, I, n_hot, n_cold;
    int renorm;
    int swap_every;
    int max_swaps;
    float hysteresis;
    int host_mirror;
    int zero_copy;
} moe_params;

typedef struct moe_scratch moe_scratch;
typedef struct moe_layer moe_layer;

/* Bytes of one expert blob for (H, I): 3*H*I/2 nibble bytes + 3*H*I/32 scale
 * bytes.  Returns 0 if H or I is not a positive multiple of 128. */
size_t moe_expert_bytes(int H, int I);

/* Shared cold-slot scratch ("DeepSeek-V4.1-Flash on One GB300 ...", section 1:
 * one scratch area with a slot per cold expert, shared by all layers because they
 * run one after another).  slot_dev: caller-owned device memory of
 * n_slots * expert_bytes bytes, 256-byte aligned; slot c starts at
 * slot_dev + c * expert_bytes.  All layers that share it must run their
 * cold_gather and moe_grouped_ffn calls in stream order.  The library keeps a
 * small device table of which layer last copied into each slot.
 * Errors: MOE_ERR_INVALID_ARG (null, n_slots < 0, misaligned, not device memory),
 * MOE_ERR_CUDA, MOE_ERR_NOMEM. */
int moe_scratch_create(int n_slots, size_t expert_bytes, void* slot_dev, moe_scratch** out);
int moe_scratch_destroy(moe_scratch* s);

/* One MoE layer.  hot_blobs_dev[h] (h < n_hot): device pointer of HBM slot h's
 * blob.  cold_blobs_host[c] (c < n_cold): host pointer of cold slot c's blob,
 * pinned and mapped; with host_mirror = 1 instead cold_blobs_host[e] (e < E) is
 * the host copy of expert e.  init_loc: host array [E], a bijection onto [0, E).
 * The scratch must have at least n_cold slots of moe_expert_bytes(H, I) bytes.
 * Validates shapes, 16-byte alignment, memory kinds (cudaPointerGetAttributes)
 * and the map.  Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA, MOE_ERR_NOMEM. */
int moe_layer_create(const moe_params* p, moe_scratch* scratch, void* const* hot_blobs_dev,
                     void* const* cold_blobs_host, const int32_t* init_loc, moe_layer** out);
int moe_layer_destroy(moe_layer* L);

/* Router: top-k, softmax weights and token-to-expert bucketing for T tokens
 * ("Milo and James Try Inference Engineering", the mixture-of-experts paragraph;
 * "DeepSeek-V4.1-Flash on One GB300 ...", section 1: the copy kernel looks at
 * which experts the router picked).
 *  logits   device fp32 [T][E] row-major.
 *  topk_ids device int32 [T][k]: expert e is picked iff fewer than k experts have
 *           a larger logit or an equal logit and a lower index; listed by that
 *           rank (descending logit, ties to the lower index).
 *  topk_w   device fp32 [T][k]: softmax probability of each pick over all E
 *           (renorm: divided by the sum over the picks).
 *  counts   device int32 [E]; offsets device int32 [E+1] (exclusive prefix);
 *  entries  device int32 [T*k]: pick ids t*k+j grouped by expert, ascending.
 * Also adds the picks to the layer's window counters used by residency_update.
 * A token with a non-finite logit gets ids 0..k-1 and weights 0, and the status
 * word becomes MOE_ERR_NONFINITE.  T = 0 is valid (offsets become all zero).
 * Errors: MOE_ERR_INVALID_ARG (null pointer with T > 0, T < 0), MOE_ERR_CUDA. */
int moe_route(moe_layer* L, const float* logits, int T, int32_t* topk_ids, float* topk_w, int32_t* counts,
              int32_t* offsets, int32_t* entries, void* stream);

/* Cold dedupe, id remap and gather ("DeepSeek-V4.1-Flash on One GB300 ...",
 * section 1: one small kernel copies just the routed cold experts into their
 * slots; section 3: that copy was 2.60 ms of a 10.49 ms step).
 *  topk_ids      device int32 [T][k].
 *  phys_ids      device int32 [T][k] out: loc of each pick's expert (-1 for an id
 *                outside [0, E), which also sets MOE_ERR_BAD_EXPERT in the status).
 *  cold_list     device int32 [min(n_cold, T*k)] out: distinct cold slots picked,
 *                ascending.
 *  n_cold_picked device int32 [1] out.
 * Every listed slot of the scratch is overwritten with the bytes of its host blob,
 * read zero-copy with 16-byte loads; unlisted slots are left as they were.  With
 * moe_params.zero_copy set and T <= 64 nothing is copied (moe_grouped_ffn reads the
 * cold experts in place) and only the outputs above are produced.
 * phys_ids, cold_list and n_cold_picked are ready in `stream` order.  The byte
 * copy itself runs on the layer's own copy stream, forked from `stream` at this
 * call, so that moe_grouped_ffn can work on the experts in HBM while the link
 * streams the cold ones; it moves every picked blob's gate/up planes (w13 nibbles
 * and scales) first and its down planes second, so that moe_grouped_ffn can run
 * the cold experts' gate/up phase while the down planes stream.
 * moe_grouped_ffn and residency_update on this layer join it, and so does
 * moe_gather_join.  A layer sharing the scratch must not call
 * cold_gather before this layer's copy has been joined into `stream`.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA. */
int cold_gather(moe_layer* L, const int32_t* topk_ids, int T, int32_t* phys_ids, int32_t* cold_list,
                int32_t* n_cold_picked, void* stream);

/* Makes `stream` wait for the layer's work in flight on its copy stream: the cold
 * copy, and a deferred residency move with its map upload (no-op when none).
 * Needed only to read the scratch slots, the expert bytes or the placement
 * without calling cold_gather or moe_grouped_ffn. */
int moe_gather_join(moe_layer* L, void* stream);

/* Device workspace bytes moe_grouped_ffn needs for T tokens. */
int moe_ffn_workspace_bytes(const moe_layer* L, int T, size_t* bytes);

/* Grouped SwiGLU expert FFN over all picks ("DeepSeek-V4.1-Flash on One GB300
 * ...", section 1: the layer runs all experts in a single call).  For pick
 * i = t*k + j with expert blob B = blob of physical id phys_ids[i]:
 *   g = W_gate x_t, u = W_up x_t, h = SiLU(g) * u, y_i = W2 h.
 *  x        device bf16 [T][H].
 *  phys_ids device int32 [T][k] (from cold_gather); counts/offsets/entries from
 *           moe_route.
 *  y        device fp32 [T*k][H] out, row i = pick i.
 *  workspace device memory of at least moe_ffn_workspace_bytes(L, T) bytes,
 *           256-byte aligned; its contents are overwritten.
 * Each distinct expert's weights are streamed once per call (with
 * moe_params.zero_copy set and T <= 64, the picked cold experts' straight from their
 * pinned host blobs, on the layer's copy stream, joined into `stream` before the
 * call returns).  Errors:
 * MOE_ERR_INVALID_ARG (null, T < 0, workspace too small), MOE_ERR_CUDA. */
int moe_grouped_ffn(moe_layer* L, const void* x, int T, const int32_t* phys_ids, const int32_t* counts,
                    const int32_t* offsets, const int32_t* entries, float* y, void* workspace,
                    size_t workspace_bytes, void* stream);

/* Arithmetic of calls with more than 64 tokens (prefill-sized buckets).
 *  kind 0 (default): weights expanded exactly from MXFP4 to f16 and multiplied with
 *         f16 activations on tcgen05 kind::f16 tensor cores (buckets above 64
 *         tokens; smaller ones on the decode kernel), fp32 accumulation: the result
 *         of the unquantised layer within rounding.
 *  kind 1 (all-FP4): x and h are converted to MXFP4 as well (each 32-element block
 *         of a row gets the exponent floor(log2(max |v|)) - 2 clamped to
 *         [-127, 127], each element the nearest E2M1 value, ties to the even code,
 *         saturating at 6), and every bucket of the call runs on block-scaled
 *         tcgen05 kind::mxf4 tensor cores with fp32 accumulation ("A 475 GB Model
 *         Across Two Workstations, With the Table on Disk", Abstract: the experts
 *         ship in MXFP4).  The result is the layer with both activations
 *         quantised, which differs from the unquantised layer by the quantisation
 *         of x and h.
 * Calls of at most 64 tokens follow moe_layer_set_decode_kind.
 * moe_ffn_workspace_bytes follows the kinds; set them before sizing the workspace.
 * Errors: MOE_ERR_INVALID_ARG (null, kind not 0 or 1). */
int moe_layer_set_prefill_kind(moe_layer* L, int kind);

/* Arithmetic of calls with at most 64 tokens (decode-sized).
 *  kind 1: the dequant-GEMV kernel (E2M1 weights expanded to f16 in registers, f16
 *         activations, mma.sync).
 *  kind 2: every bucket on block-scaled tcgen05 kind::mxf4 tensor cores, which
 *         decode the MXFP4 weights themselves; each activation (x, then h) is
 *         written as a sum of four MXFP4 terms, the first the activation rounded to
 *         MXFP4 and each further one the remainder of those before, with block
 *         exponents chosen so that no element saturates (each remainder is exact in
 *         fp32), so the result is the unquantised layer's to about 2e-4 relative.
 *  kind 0 (default): kind 2 (on a GB300 the block-scaled kernels are the faster at
 *         every decode size of H = 4096, I = 3072, k = 6, from one token up).
 * Layers that read cold experts in place (moe_params.zero_copy) run kind 1 for
 * calls with cold experts.  Errors: MOE_ERR_INVALID_ARG (null, kind not 0, 1 or 2). */
int moe_layer_set_decode_kind(moe_layer* L, int kind);

/* moe_grouped_ffn for callers that cannot allocate device memory (an engine that
 * has given all free HBM to its own pools and forbids later allocations, code
 * running during a global-mode stream capture, embedders with their own
 * allocator).  No counterpart in the published method: same arguments and results as
 * moe_grouped_ffn minus the workspace, which here is a fixed array of
 * MOE_NOALLOC_SCRATCH_BYTES inside the library's device image (every GPU that
 * loads the library holds one copy until the process exits).  The call
 * allocates nothing: no cudaMalloc, no cudaFree, no allocating library routine.
 * The first call on a device looks up the array's device address (with that
 * device current); make that first call before any stream capture.  All calls on
 * a device share the array and it keeps the previous call's contents (the FFN
 * clears what must start at zero itself), so calls that overlap on the GPU race:
 * order them on one stream or otherwise serialise them.
 * Errors: MOE_ERR_SCRATCH_TOO_SMALL when T needs more than the array holds
 * (moe_ffn_workspace_bytes(L, T) > MOE_NOALLOC_SCRATCH_BYTES; each of the T*k picks
 * takes 2*max(H, I) + 4*I + 4 bytes, each section rounded up to 256 bytes, so
 * T <= 68 at H=4096, I=3072, k=6), MOE_ERR_INVALID_ARG, MOE_ERR_CUDA. */
#define MOE_NOALLOC_SCRATCH_BYTES (8u << 20)
int moe_grouped_ffn_noalloc(moe_layer* L, const void* x, int T, const int32_t* phys_ids, const int32_t* counts,
                            const int32_t* offsets, const int32_t* entries, float* y, void* stream);

/* Combine ("DeepSeek-V4.1-Flash on One GB300 ...", section 4: contributions are
 * summed; the order only moves the last decimal places).  out[t] = sum over
 * j = 0..k-1, in that order, of topk_w[t][j] * y[t*k+j], in fp32.
 *  y device fp32 [T*k][H]; topk_w device fp32 [T][k];
 *  out device [T][H]: bf16 (round to nearest even) when out_fp32 = 0, else fp32.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA. */
int moe_combine(const float* y, const float* topk_w, int T, int k, int H, void* out, int out_fp32, void* stream);

/* Adaptive residency ("DeepSeek-V4.1-Flash on One GB300 ...", section 1: between
 * steps a manager swaps often-picked experts into the hot set and quiet ones out;
 * section 3: hysteresis 3.0 as the published default).  Call once per step, after
 * the layer's moe_grouped_ffn (and moe_combine) on the same stream.  Every
 * swap_every-th call closes a window of pick counts; the plan pairs cold experts
 * picked at least once (count desc, id asc) with hot experts (count asc, id asc)
 * and swaps pair i while count(cold) > hysteresis * count(hot) (at most
 * max_swaps, stopping at the first pair that fails); applying a pair moves the
 * bytes (host_mirror 0: exchanges the two experts' bytes in place between the
 * HBM slot and the host blob; host_mirror 1: copies the promoted expert into the
 * HBM slot, see moe_params) and rewrites the placement map.  Each expert is in at
 * most one pair, so any prefix of a plan is a valid placement.
 *  Deferred mode (default, moe_layer_set_residency_defer 1): the closing call
 *  enqueues a copy of the window's counters to the host and starts the next
 *  window in a second counter buffer, without synchronising; the layer's next
 *  call (one step later) makes the plan from those counts and the current
 *  placement.  The plan's n pairs land in plan order, paced over the calls
 *  before the next window closes: pair i at the plan's call floor(i * span / n)
 *  (call 0 being the one that made it, span = max(1, swap_every - 1)); pairs
 *  still unapplied when the next plan is made land first.  Each landing moves
 *  its bytes on the layer's copy stream, after the work already on `stream`,
 *  while later layers run; the layer's next cold_gather or moe_grouped_ffn waits
 *  for the move.  The promoted expert is read from its host blob (host copy),
 *  never from the shared scratch.  The counts and plans are those of the
 *  synchronous mode; only the times at which the pairs land differ.
 *  Synchronous mode (0): the closing call synchronises `stream`, reads the
 *  counters, and moves the bytes on `stream` at once; with host copies it
 *  promotes from the scratch slot while that slot still holds this layer's copy.
 *  Layers sharing a scratch must make this call before a later layer's
 *  cold_gather on the same stream order (it may read a slot).
 *  n_swaps_out host int32 [1] out: the swaps applied by this call (deferred: by
 *  the plan of the previous closing call).
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA, MOE_ERR_INJECTED (test hook: on a
 * closing call, before anything is enqueued or applied). */
int residency_update(moe_layer* L, int32_t* n_swaps_out, void* stream);

/* Selects the residency mode of residency_update: 1 deferred (default), 0
 * synchronous.  A plan already pending is applied at the next call either way.
 * Errors: MOE_ERR_INVALID_ARG (null, defer not 0 or 1). */
int moe_layer_set_residency_defer(moe_layer* L, int defer);

/* The plan one acting residency_update applies, computed on the host with no
 * device work (callable without a GPU): the same ranking, pairing and stopping
 * rule, from a window's pick counts and a placement.
 *  counts    host int32 [E], each >= 0.
 *  loc       host int32 [E]: a placement (a permutation of 0..E-1; values below
 *            n_hot are HBM slots).
 *  loc_out   host int32 [E] out: the placement after the swaps (may equal loc).
 *  promoted, demoted  host int32 [max_swaps] out (may be NULL when max_swaps is
 *            0): pair i moved promoted[i] into demoted[i]'s HBM slot and
 *            demoted[i] into promoted[i]'s cold slot.
 *  1 <= E <= 1024, 0 <= n_hot <= E, 0 <= max_swaps <= 64, hysteresis finite >= 0.
 * Returns the number of swaps (>= 0), or MOE_ERR_INVALID_ARG (bad sizes, a
 * negative count, or loc not a permutation). */
int moe_residency_plan(const int32_t* counts, const int32_t* loc, int E, int n_hot, int max_swaps, float hysteresis,
                       int32_t* loc_out, int32_t* promoted, int32_t* demoted);

/* MXFP4 quantisation of bf16 activation rows, the first step of the all-FP4
 * prefill mode (a block-scaled FP4 x FP4 tensor-core product takes both operands
 * in MXFP4).  Each 32-element block of a row gets the shared exponent
 * floor(log2(max |v|)) - 2 clamped to [-127, 127] (an all-zero block: -127),
 * stored as scale byte exponent + 127; each element gets |v| / 2^exponent rounded
 * to the nearest E2M1 magnitude {0, 0.5, 1, 1.5, 2, 3, 4, 6}, ties to the even
 * code, above 6 saturating to 6, with v's sign bit (the OCP Microscaling
 * conversion for E2M1).  Output in the weights' row layout.
 *  x_bf16  device bf16 [rows][K], finite values; K a positive multiple of 32.
 *  nib     device uint8 [rows][K/2] out: element k of a row in byte k/2, low
 *          nibble when k is even.
 *  scales  device uint8 [rows][K/32] out.
 * rows = 0 is valid.  Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA. */
int moe_quant_mxfp4(const void* x_bf16, int rows, int K, uint8_t* nib, uint8_t* scales, void* stream);

/* ---- The rest of a decoder layer -------------------------------------------------
 * The MoE layer takes router logits and activations and returns the experts' sum.
 * These entry points are what a decoder layer runs around it: residual addition and
 * norm, position rotation with the append to a paged key-value cache, attention of
 * one new token per sequence over that cache, and the dense products between them.
 * All strides are in elements, the innermost dimension is contiguous, and no call
 * allocates device memory or synchronises, so all can be captured in a graph.  Every call
 * runs on the calling thread's current device, which has to be the one that its buffers,
 * its stream and its cache handle belong to (the Python binding refuses others).  Sums,
 * statistics and accumulators are fp32; each output is rounded once. */

/* Residual addition and root-mean-square norm:
 *   s = x + residual;  sum_out = s;  y = s * rsqrt(mean(s^2) + eps) * weight
 * with s kept in fp32 (the norm is of the unrounded sum).  Each row is independent.
 *  x         device [T][H] of x_type (MOE_BF16, MOE_F16 or MOE_F32), rows x_stride apart.
 *  residual  device [T][H] of res_type (same three types), rows res_stride apart, or
 *            NULL (s = x).
 *  weight    device [H] of weight_type (same three types), or NULL (ones).
 *  sum_out   device [T][H] of res_type, rows sum_stride apart, or NULL; may be
 *            residual or x themselves (same rows, type and stride).
 *  y         device [T][H] of y_type, rows y_stride apart; may be x itself likewise.
 *            MOE_E4M3: y holds y / y_scale[t] with y_scale[t] = max(max_j |y_tj| / 448,
 *            2^-126); a row with a NaN in s * weight, or with a sum of squares past fp32's
 *            range, gets a NaN scale and NaN codes.  In the other types such a sum (elements
 *            from about 2^64 / sqrt(H) up) leaves zeros, and NaN where s is infinite.
 *  y_scale   device fp32 [T], MOE_E4M3 only (else NULL).
 * 1 <= H <= 32768, eps finite and >= 0; T = 0 is valid.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA. */
int moe_add_rms_norm(const void* x, int x_type, int64_t x_stride, const void* residual, int res_type,
                     int64_t res_stride, const void* weight, int weight_type, float eps, int T, int H, void* sum_out,
                     int64_t sum_stride, void* y, int y_type, int64_t y_stride, float* y_scale, void* stream);

/* Rows to E4M3 with one fp32 scale for each 128 elements, the operands of moe_linear_blocks:
 *   scale[t][g] = max(max_k |x_tk| / 448, 2^-126),  y_tk = x_tk / scale[t][g],  k in [128 g, 128 g + 128)
 * scale as it is returned (a product with 1 / 448: within 2^-23), the quotient an fp32 division's.  A group with a NaN
 * or an infinity gets a NaN scale and NaN codes.  Each group is independent.
 *  x     device [T][K] of x_type (MOE_BF16, MOE_F16 or MOE_F32), rows x_stride apart.
 *  y     device E4M3 [T][K], rows y_stride apart.
 *  scale device fp32 [T][ceil(K / 128)], rows scale_stride apart.
 * The outputs must not share memory with x nor with one another (an output at another's or at x's address is
 * refused).  K >= 1; T = 0 is valid.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA. */
int moe_quant_e4m3(const void* x, int x_type, int64_t x_stride, int T, int K, void* y, int64_t y_stride, float* scale,
                   int64_t scale_stride, void* stream);

/* A paged key-value cache of one layer.  Token slot s is entry s % page_size of page
 * s / page_size; element d of key head h there is at
 *   k_cache[(s / page_size) * page_stride + (s % page_size) * token_stride + h * head_stride + d]
 * and of v_cache likewise, so both orders of tokens and heads within a page fit.
 *  type       MOE_BF16, MOE_F16, or MOE_E4M3 with one fp32 scale per key head (value =
 *             scale * code; the scale may have either sign).
 *  q_heads    a multiple of kv_heads; query head h reads key head
 *             h / (q_heads / kv_heads).
 *  head_dim   a multiple of 16, at most 256.
 *  page_size  any from 1 to 65536.
 *  max_batch  most sequences of one moe_kv_attend call, 1 to 65535.
 * The last token's offset must be below 2^32 times the largest power of two (in bytes)
 * that divides both page and token stride: 64 GB for the narrowest rows of 16 bytes, more
 * than the GPU holds for any row of 128 bytes. */
typedef struct moe_kv_params {
    int n_pages, page_size, kv_heads, q_heads, head_dim, type, max_batch;
    int64_t page_stride, token_stride, head_stride;
} moe_kv_params;

typedef struct moe_kv moe_kv;

/* Creates the handle: k_cache, v_cache (device, 16-byte aligned, strides whole
 * 16-byte units) and the scales (device fp32 [kv_heads], both or none: MOE_E4M3 needs
 * them, the other types take NULL) are borrowed for its life.  The handle owns a
 * status word and the workspace in which moe_kv_attend joins parts of a sequence, so
 * calls of moe_kv_attend on one handle must be ordered on one stream or by events.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA, MOE_ERR_NOMEM. */
int moe_kv_create(const moe_kv_params* p, void* k_cache, void* v_cache, const float* k_scale, const float* v_scale,
                  moe_kv** out);
int moe_kv_destroy(moe_kv* kv);

/* A cache of MOE_E4M3 with one fp32 scale for each block of scale_tokens tokens of a page and key
 * head, so that no scale has to be known before the tokens are:
 *   value = scale[page][entry / scale_tokens][h] * code,
 * k_scale and v_scale device fp32 [n_pages][page_size / scale_tokens][kv_heads], contiguous, which
 * moe_kv_append writes and moe_kv_attend reads (a scale of the caller's own making may have either
 * sign).  scale_tokens: 1 to 1024, a divisor of page_size.  The rest as moe_kv_create, and the handle
 * is used in the same calls:
 *  moe_kv_append  gives a block the smallest power of two with which the largest magnitude among the
 *    tokens that it takes in, at most 448 * scale, held to 2^-126 and 2^119 (larger values, infinities among
 *    them, saturate; NaN stays NaN and does not count).  A block whose first entry is among them starts anew:
 *    what else it held means nothing any more, though its bytes stay.  Any other block keeps its scale
 *    where its magnitude is large enough; where it is not, the codes of its other entries are rewritten under the
 *    new one, so the block's scale has to be initialised (zero will do) before a block is begun in its middle.
 *    Rewriting codes under a power of two, as the append's own scales are, is exact but where codes of less than
 *    2^-6 lose their low bits; under any other scale it rounds each once more.
 *    The tokens of a call that go to one block have to follow one another in the call, with none between them
 *    that goes elsewhere or nowhere.  Where they do not, MOE_ERR_BAD_INDEX is set in the handle's status, and what
 *    that block holds is not defined.  Calls that append to one block have to be ordered.
 *  moe_kv_attend  takes scales up to 2^96 in magnitude, keys and values of 2^104; a NaN among those of
 *    attended tokens shows in that head's outputs.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA, MOE_ERR_NOMEM. */
int moe_kv_create_blocks(const moe_kv_params* p, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                         int scale_tokens, moe_kv** out);

/* Position rotation and append.  For each token t: the first rot_dim elements of
 * every head of q and k are turned by the token's position,
 *   (a, b) -> (a cos - b sin, a sin + b cos),
 * over the pairs (i, i + rot_dim/2), or (2i, 2i + 1) when interleaved is 1; q goes to
 * q_out, k and v to cache slot slots[t] (E4M3 caches: divided by the head's scale).
 *  q [T][q_heads][head_dim], k and v [T][kv_heads][head_dim], q_out as q: device, of
 *  `type` (MOE_BF16, MOE_F16 or MOE_F32), token strides *_ts and head strides *_hs;
 *  q_out may be q itself.
 *  positions device int32 [T]; cos_sin device fp32 [n_positions][rot_dim], the row's
 *  rot_dim/2 cosines, then its sines (both NULL when rot_dim is 0).
 *  slots device int64 [T]: a negative slot appends nothing (q_out is still written);
 *  two tokens of a call must not share a slot.
 * A position outside the table, or a slot past the last page, sets MOE_ERR_BAD_INDEX in
 * the handle's status: of the first token nothing is written, of the second q_out
 * alone.  0 <= rot_dim <= head_dim, even; T = 0 is valid.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA. */
int moe_kv_append(moe_kv* kv, int type, const void* q, int64_t q_ts, int64_t q_hs, const void* k, int64_t k_ts,
                  int64_t k_hs, const void* v, int64_t v_ts, int64_t v_hs, const int32_t* positions,
                  const int64_t* slots, const float* cos_sin, int n_positions, int rot_dim, int interleaved, int T,
                  void* q_out, int64_t qo_ts, int64_t qo_hs, void* stream);

/* moe_kv_append where a token's position has several axes (time, height and width of an image's or a
 * video's tokens): pair i of a head is turned by the table's row of position positions[axis_of_pair[i]][t].
 *  positions     device int32 [n_axes][T], rows positions_stride apart.  A token with any position
 *                outside the table is left out.
 *  axis_of_pair  host uint8 [rot_dim / 2], each below n_axes; read during the call.
 *  1 <= n_axes <= 4, and rot_dim > 0.  The rest as moe_kv_append.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA. */
int moe_kv_append_axes(moe_kv* kv, int type, const void* q, int64_t q_ts, int64_t q_hs, const void* k, int64_t k_ts,
                       int64_t k_hs, const void* v, int64_t v_ts, int64_t v_hs, const int32_t* positions,
                       int64_t positions_stride, int n_axes, const uint8_t* axis_of_pair, const int64_t* slots,
                       const float* cos_sin, int n_positions, int rot_dim, int interleaved, int T, void* q_out,
                       int64_t qo_ts, int64_t qo_hs, void* stream);

/* Attention of one query token per sequence over the cache:
 *   out[b][h] = sum_j softmax_j(scale * q[b][h] . k_j) v_j,  j in [max(0, n - window), n)
 * with n = lengths[b] tokens (window = 0: all of them), k_j and v_j of key head
 * h / (q_heads / kv_heads) at slot page_table[b][j / page_size] * page_size + j % page_size.
 *  q, out  device [B][q_heads][head_dim] of type q_type: MOE_BF16 or MOE_F16, the
 *          cache's own type unless the cache is MOE_E4M3; strides *_ts per sequence and
 *          *_hs per head; 16-byte aligned, strides whole 16-byte units.  out must not share
 *          elements with q (out = q is refused): parts of a sequence read its query at any time.
 *  page_table device int32 [B][max_pages], rows table_stride apart (0: one row for all);
 *          entries past a sequence's last page (or wholly before its window) are not read.
 *  lengths device int32 [B].  A sequence of length 0 gets zeros and a log-sum of -inf.
 *  lse     device fp32 [B][q_heads] out, contiguous: log sum_j exp(scale * q . k_j), or NULL.
 * Several query tokens of one sequence are several rows with their own lengths and the
 * same page-table row.  A page id outside [0, n_pages) or a length outside
 * [0, max_pages * page_size] (or above 2^30) sets MOE_ERR_BAD_INDEX in the handle's status; the page's
 * tokens are left out, the length is clamped.  The result does not depend on the
 * timing of the GPU: the same call gives the same bits.
 * 0 <= B <= max_batch; scale finite.  The softmax is fp32; its weights meet the values as two
 * 16-bit terms each, which lose at most 2^-16 of a weight (bf16 caches), or 2^-22 of it and
 * 2^-31 of the largest one (f16, E4M3; with scales of blocks 2^-31 of the largest weight times the
 * largest scale of a value met before it).
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA. */
int moe_kv_attend(moe_kv* kv, const void* q, int q_type, int64_t q_ts, int64_t q_hs, const int32_t* page_table,
                  int64_t table_stride, int max_pages, const int32_t* lengths, int B, float scale, int window,
                  void* out, int64_t out_ts, int64_t out_hs, float* lse, void* stream);

/* Reads (0 = no error so far) and clears the handle's status word.  Both return when done;
 * neither waits for work of streams that do not synchronise with the legacy default
 * stream: synchronise those first. */
int moe_kv_get_status(moe_kv* kv, int* status);
int moe_kv_clear_status(moe_kv* kv);

/* Matrix product with its epilogue: y = act(x W^T + bias) + residual, and for E4M3
 * operands y = act(x_scale[t] * w_scale[n] * (x W^T) + bias) + residual.
 *  x device [T][K], w device [N][K] (one row per output), both of in_type: MOE_BF16,
 *    MOE_F16 or MOE_E4M3; 16-byte aligned, row strides and K * element size multiples
 *    of 16 bytes (pad K with zeros otherwise).
 *  x_scale [T], w_scale [N] device fp32: MOE_E4M3 only, both (else NULL).
 *  bias device [N] of bias_type (MOE_BF16, MOE_F16, MOE_F32), or NULL.
 *  act MOE_ACT_*.
 *  residual device [T][N] of y_type, rows res_stride apart, or NULL; may be y itself.
 *  y device [T][N] of y_type (MOE_BF16, MOE_F16, MOE_F32), rows y_stride apart.
 *  status_dev device int, or NULL: set to MOE_ERR_TIMEOUT when a bounded device wait ran
 *    out (zero it first; y is then undefined).
 * The sums are the tensor cores' fp32 accumulators, which round towards zero at every step of 32
 * bytes of K (bf16 and f16: about 1e-9 K of the output's size).
 * T, N (at most 2^22) and the strides of y and residual are free; x and w rows are at least K
 * apart; T = 0 is valid; N, K >= 1.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA. */
int moe_linear(const void* x, int64_t x_stride, const void* w, int64_t w_stride, int in_type, int T, int N, int K,
               const float* x_scale, const float* w_scale, const void* bias, int bias_type, int act,
               const void* residual, int64_t res_stride, void* y, int y_type, int64_t y_stride, int* status_dev,
               void* stream);

/* moe_linear on E4M3 operands with a scale for each block of 128: with G = ceil(K / 128),
 *   y = act(sum_g x_scale[t][g] * w_scale[n / 128][g] * (sum_{k in g} x_tk w_nk) + bias) + residual
 *  x device E4M3 [T][K], w device E4M3 [N][K], as in moe_linear.
 *  x_scale device fp32 [T][G], rows x_scale_stride apart; w_scale device fp32 [ceil(N / 128)][G], rows
 *    w_scale_stride apart: any numbers.  The product of the two is an fp32 number (below 2^-126 it loses bits, from
 *    2^128 it is infinite).
 * The rest as moe_linear.  The products of a block of K are summed by the tensor cores (fp32, towards zero
 * at every 32 of K), the blocks, times their two scales' product, in fp32 to nearest.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA. */
int moe_linear_blocks(const void* x, int64_t x_stride, const void* w, int64_t w_stride, int T, int N, int K,
                      const float* x_scale, int64_t x_scale_stride, const float* w_scale, int64_t w_scale_stride,
                      const void* bias, int bias_type, int act, const void* residual, int64_t res_stride, void* y,
                      int y_type, int64_t y_stride, int* status_dev, void* stream);

/* Copies the placement map to host int32 [E] (synchronous). */
int moe_layer_get_loc(moe_layer* L, int32_t* loc_host);

/* Copies the window pick counters to host int32 [E] (synchronous). */
int moe_layer_get_counts(moe_layer* L, int32_t* counts_host);

/* Reads the layer's device status word (synchronous); 0 = no error so far. */
int moe_get_status(moe_layer* L, int* status);

/* Clears the device status word and the diagnostic record (synchronous). */
int moe_clear_status(moe_layer* L);

/* Copies the diagnostic record of the first device-side wait that ran out of
 * time (set together with MOE_ERR_TIMEOUT) to host int32 [16]: [0] 1 when set,
 * [1] block, [2] warp, [3] wait kind (1 stage full, 2 stage empty), [4] ring slot,
 * [5] parity waited for, [6] stage index, [7] task << 8 | token columns,
 * [8] 1 if the other parity had completed.  All zero when nothing timed out. */
int moe_get_diag(moe_layer* L, int32_t* diag_host);

/* Text for a status code. */
const char* moe_strerror(int code);

/* Number of CTAs the cold copy kernel runs on (0 = the default, 3/16 of the SMs:
 * enough to keep the host link busy on GB300).  A zero-copy layer's cold FFN chain
 * runs on the same number of CTAs, or a quarter of the SMs if that is more.
 * The copy shares the GPU with the FFN over HBM-resident experts. */
int moe_layer_set_copy_ctas(moe_layer* L, int ctas);

/* Timing: after moe_layer_profile(L, n) (which first waits for the device to go
 * idle) the next n cold_gather calls record CUDA events around their byte copy on
 * the layer's copy stream, and the next n moe_grouped_ffn calls record events
 * around their kernels on the caller's stream; n = 0 stops and frees them.
 * moe_layer_profile_read waits for the copy records and writes up to `max`
 * durations in ms to host float copy_ms[] and their number to *n_out.
 * moe_layer_profile_read_ffn does the same for the FFN calls: each duration is the
 * call's kernel time without the waits for the cold copy (the work before the join
 * of the cold gate/up planes, between that join and the join of the rest, and
 * after it).  0 <= n <= 2^20, else MOE_ERR_INVALID_ARG. */
int moe_layer_profile(moe_layer* L, int max_records);
int moe_layer_profile_read(moe_layer* L, float* copy_ms, int max, int* n_out);
int moe_layer_profile_read_ffn(moe_layer* L, float* ffn_ms, int max, int* n_out);

/* Test hook for host-side fault injection: what = 1 makes the next acting
 * residency_update fail with MOE_ERR_INJECTED before any copy or map change (as a
 * failed host copy would); what = 0 clears it.  Never set in normal use. */
int moe_layer_inject_fault(moe_layer* L, int what);

/* Host-link probe: copies `bytes` (a multiple of 16) from mapped pinned host
 * memory `src_host` to device memory `dst_dev` with the same zero-copy 16-byte
 * load loop as cold_gather, on `ctas` CTAs (0 = one per SM).  Used to measure
 * the link peak the cold gather is reported against. */
int moe_link_probe(const void* src_host, void* dst_dev, size_t bytes, int ctas, void* stream);

/* Dense block-scaled FP4 tensor-core rate probe (the denominator the all-FP4
 * prefill path is reported against): `ctas` CTAs (0 = one per SM) each issue
 * `iters` back-to-back tcgen05 kind::mxf4 MMAs of M = 128, N = 256, K = 64
 * (2 * 128 * 256 * 64 flops each) on operands resident in shared memory; the
 * caller times the launch on `stream`.  status_dev: device int, set to
 * MOE_ERR_TIMEOUT if the kernel's bounded wait for its MMAs ran out (zero it
 * first).  1 <= iters <= 2^20.  Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA. */
int moe_mxf4_peak_probe(int iters, int ctas, int* status_dev, void* stream);

/* Test hook for the bounded device waits of the pipelined kernels: launches one
 * thread that waits on an mbarrier phase that nothing completes.  The wait gives
 * up at its deadline (2 s), writes its record to diag_dev (device int32 [16], the
 * layout moe_get_diag describes; zero it first) and MOE_ERR_TIMEOUT to
 * *status_dev (device int; the first error written wins, so zero it first), and
 * the kernel returns, leaving the context usable: how a lost producer is reported
 * without faulting or hanging the GPU. */
int moe_debug_wait_timeout(int* status_dev, int32_t* diag_dev, void* stream);

/* Lane-layout check of the E2M1 pair conversion used by the FFN kernels: writes
 * for every byte b (0..255) the two f16 values it decodes to (low nibble first)
 * as uint32 [256] to out_dev (device). */
int moe_debug_e2m1_pairs(uint32_t* out_dev, void* stream);

/* Test hook: both E2M1 roundings of n fp32 values |v| < 8 (already divided by their
 * block scale).  out_dev uint32 [2n]: out[2i] from the hardware pair conversion the
 * block-scaled kernels use (round to nearest, ties to the even code, saturating at
 * 6), out[2i + 1] from the comparison rule of the stand-alone quantiser; both with
 * the sign in bit 3.  Errors: MOE_ERR_INVALID_ARG, MOE_ERR_CUDA. */
int moe_debug_e2m1_round(const float* v_dev, int n, uint32_t* out_dev, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOEHOST_H */
