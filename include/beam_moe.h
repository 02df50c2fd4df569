/*
 * beam_moe.h -- C ABI of the BEAM-masked MoE layer forward pass (B200, sm_100a).
 *
 * The operation is the MoE layer of "BEAM: Binary Expert Activation Masking
 * for Dynamic Routing in MoE" (arXiv 2605.14438), §3.2, for one batch of T
 * tokens x [T, d]:
 *
 *   r = x W_gate                 main-router logits                (step 1)
 *   g = Softmax(Top-K(r))        candidate weights                 (Eq. 1/4)
 *   m = [sigmoid(x W_mask) >= 0.5] on the K candidates             (Eq. 5-6)
 *   w = g * m                    no renormalisation after the mask (Eq. 7)
 *   y = sum_k w_k E_{c_k}(x)     only kept (token, expert) pairs   (Eq. 8)
 *   E_e(x) = (SiLU(x W1_e^T) * (x W3_e^T)) W2_e^T                  (Eq. 3)
 *
 * A token whose candidates are all masked gets y = 0 (it passes the layer
 * through the residual, which stays the caller's).  A masked pair is never
 * scheduled, so an expert without kept pairs has none of its weights read.
 *
 * Conventions (all entry points):
 *  - Layouts are row-major and contiguous: x [T,d]; W_gate, W_mask [E,d]
 *    (row e = column e of the paper's d x N matrices); W1 (gate), W3 (up)
 *    [E,I,d]; W2 (down) [E,d,I]; out [T,d].
 *  - dtype BEAM_BF16: x, weights and out are bfloat16; accumulation is fp32;
 *    the SwiGLU activations H (the second GEMM's operand) are rounded to bf16
 *    once; the per-pair expert outputs stay fp32 and the weighted sum is
 *    rounded to bf16 once.  dtype BEAM_F32: everything fp32.  Logits, softmax
 *    weights and the combine are fp32 in both.
 *  - Every pointer except the host descriptor is a DEVICE pointer, 16-byte
 *    aligned.  The caller owns every buffer, including the workspace; the
 *    library allocates nothing and keeps no state between calls.
 *  - Every launch is ordered on `stream` (a cudaStream_t; NULL = the legacy
 *    default stream) and the calls never synchronise the host, except
 *    beam_moe_check.  Argument and shape errors are returned before anything
 *    is launched; a failed launch returns BEAM_ERR_CUDA.
 *  - Constraints: 1 <= K <= min(E, 16), E <= 256, T >= 0.  BEAM_BF16 needs
 *    d % 128 == 0 and I % 128 == 0; BEAM_F32 needs d % 8 == 0 and I % 8 == 0
 *    (else BEAM_ERR_UNSUPPORTED_SHAPE).  T*K and the workspace rows must fit
 *    in int32.
 *  - Top-K ties go to the lower expert index; candidates are listed by
 *    descending logit (the paper does not fix either).  The mask test is taken
 *    on the pre-sigmoid value, z >= 0 <=> sigmoid(z) >= 0.5 (Eq. 6); NaN is
 *    not kept.  Non-finite inputs are the caller's responsibility.
 */
#ifndef BEAM_MOE_H
#define BEAM_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    BEAM_OK = 0,
    BEAM_ERR_INVALID_ARG = 1,       /* NULL / misaligned pointer, bad K, E, dtype, ... */
    BEAM_ERR_UNSUPPORTED_SHAPE = 2, /* d or I not a multiple of the tile width */
    BEAM_ERR_WORKSPACE = 3,         /* workspace NULL, misaligned or too small */
    BEAM_ERR_CUDA = 4,              /* a CUDA runtime call or launch failed */
    BEAM_ERR_TIMEOUT = 5,           /* a bounded device-side wait gave up */
    BEAM_ERR_INTERNAL = 6           /* a device-side consistency check failed */
} beam_status;

typedef enum { BEAM_BF16 = 0, BEAM_F32 = 1 } beam_dtype;

/* One MoE layer call: T tokens of width d, E experts, top-K, SwiGLU width I.
 * renorm_topk = 1: softmax over the K largest logits (Eq. 4, sums to 1).
 * renorm_topk = 0: softmax over all E logits, restricted to the K largest.
 * mask_logit_threshold: the binarisation threshold tau of Eq. (6) given as
 *   its logit, ln(tau / (1 - tau)); a candidate is kept iff its mask
 *   pre-activation z >= mask_logit_threshold (i.e. sigmoid(z) >= tau).
 *   0 is the paper's tau = 0.5, so a zero-initialised descriptor keeps the
 *   method's default; other values reproduce the threshold ablation (news
 *   article on BEAM, §8); beam_moe_tau_to_logit converts a tau.  Must not
 *   be NaN.
 * n_shared, I_shared: always-on shared experts (news article on BEAM, §5:
 *   models such as Qwen1.5-MoE and DeepSeek-V2-Lite keep running them for
 *   every token, all-masked tokens included), n_shared SwiGLU experts of
 *   width I_shared, each added with weight 1 after the routed sum.  0 = none
 *   (beam_moe_forward); > 0 needs beam_moe_forward_shared, BEAM_BF16,
 *   n_shared <= 16 and I_shared % 128 == 0. */
typedef struct {
    int T, d, E, I, K;
    int dtype;       /* beam_dtype */
    int renorm_topk; /* 0 or 1 */
    float mask_logit_threshold;
    int n_shared, I_shared;
} beam_moe_desc;

/* Workspace layout chosen for a descriptor (byte offsets from the workspace
 * base).  Exposed so that tests and tools can read the intermediate arrays
 * after beam_moe_forward; none of it is needed to call the layer.
 *   err       int32      device error word (0 = ok), read by beam_moe_check
 *   meta      int32[4]   [0] tiles in the tile list, [1] padded rows,
 *                        [2] kept pairs P, [3] work counter of the fused
 *                        expert kernel (units handed out so far), or with
 *                        256-row tiles the number of 128-row sub-tiles
 *   counts    int32[E]   kept pairs per expert
 *   hist      int32[K+1] tokens by number of kept candidates
 *   partial   f32[S][T][2E] router partial logits (S = router_splits)
 *   idx       int32[T][K] candidate expert, -1 where masked
 *   w         f32[T][K]   g * m
 *   pair      int32[p_cap] permuted row -> t*K + k (-1 on padding rows);
 *             expert e owns rows [off_e, off_e + roundup(counts[e], BN)),
 *             experts in ascending order, tokens ascending inside
 *   pair_pos  int32[T][K] permuted row of a kept pair (undefined if masked)
 *   tiles     int32[tiles_cap][4] (expert, first row, valid rows, 0)
 *   tile_done int32[tiles_cap] gate/up units finished per tile (fused path)
 *   xp        [p_cap][d]  gathered token rows (dtype)
 *   h         [p_cap][I]  SiLU(x W1^T) * (x W3^T) per pair (dtype)
 *   y         f32[p_cap][d] expert output per pair
 *   hs        [n_shared*T][I_shared] shared experts' SwiGLU activations (dtype)
 *   ys        f32[sh_split2][n_shared*T][d] shared experts' outputs, one slab per
 *             split of their down reduction (the combine adds every slab)
 *   sp        f32[2][sh_split1][n_shared*T][I_shared] partial gate and up
 *             pre-activations of the shared experts' split reduction
 *   tiles_sub int32[][4] with 256-row tiles: the same rows as 128-row tiles,
 *             the gate/up GEMM's units (their count in meta[3])
 *   ctl       int32[]     one-launch path: gate/up units finished per expert,
 *                         down units finished per (token, output row block)
 * With one_launch the layer runs as one kernel that writes err, meta,
 * counts, hist, partial (one split), idx, w, pair, pair_pos, tiles, h and y
 * as above; xp, tile_done, hs, ys and tiles_sub are not used.             */
typedef struct {
    int BN;            /* token rows per expert tile; the padding unit */
    int router_bn;     /* token rows per router tile */
    int router_splits; /* router split-K factor S */
    int p_cap;         /* rows of xp / h / y / pair */
    int tiles_cap;     /* entries of the tile list */
    int sub_bn;        /* token rows of the gate/up GEMM's tiles (BN, or 128 when BN = 256) */
    int one_launch;    /* 1: beam_moe_forward runs the whole layer as one kernel */
    int sh_bn;         /* shared experts: token rows per tile */
    int sh_split1;     /* shared experts: splits of the gate/up reduction (over d) */
    int sh_split2;     /* shared experts: splits of the down reduction (over I_shared) */
    size_t off_err, off_meta, off_counts, off_hist, off_partial, off_idx, off_w,
        off_pair, off_pair_pos, off_tiles, off_xp, off_h, off_y, off_tile_done, off_hs,
        off_ys, off_tiles_sub, off_ctl, off_sp;
    size_t workspace_bytes;
} beam_moe_plan_info;

/* Stage slots of one beam_moe_forward call (router GEMM, top-K + mask,
 * grouping, gather, gate/up GEMM, down GEMM, combine).  With token tiles
 * thinner than 128 rows (decode batches, bf16) the grouping kernel copies the
 * token rows itself, so the gather slot is empty, and the two expert GEMMs run
 * as one fused launch in the gate/up slot, so the down slot is empty too; see
 * beam_moe_forward_kernel_count. */
#define BEAM_MOE_FORWARD_STAGES 7

/* Bytes of device workspace beam_moe_forward needs for `desc` (0 on a bad
 * descriptor).  Grows with T: O(T*K*(2d + I)) for the permuted activations. */
size_t beam_moe_workspace_size(const beam_moe_desc *desc);

/* Fill `info` with the workspace layout for `desc`.  Host only. */
beam_status beam_moe_plan(const beam_moe_desc *desc, beam_moe_plan_info *info);

/* Routing alone: §3.2 steps 1-3 and Eq. (7).
 *   x, W_gate [E,d], W_mask [E,d] or NULL (mask disabled: all candidates kept)
 *   topk_idx  int32 [T,K]  candidate expert id, -1 where masked      (written)
 *   topk_w    f32   [T,K]  g * m                                     (written)
 *   expert_counts int32 [E] kept pairs per expert                    (written)
 *   kept_hist int32 [K+1] tokens by kept count, or NULL              (written)
 *   logits    f32 [T,2E] or NULL: r in columns [0,E), the mask pre-activation
 *             z in [E,2E) (not written when W_mask is NULL)          (written)
 *   workspace of beam_moe_workspace_size(desc) bytes (partial logits).
 * Uses the same kernels, tiling and summation order as beam_moe_forward, so
 * both take bitwise identical routing decisions for the same inputs. */
beam_status beam_moe_route(const beam_moe_desc *desc, const void *x, const void *W_gate,
                           const void *W_mask, int32_t *topk_idx, float *topk_w,
                           int32_t *expert_counts, int32_t *kept_hist, float *logits,
                           void *workspace, size_t workspace_bytes, void *stream);

/* The whole layer, Eq. (4)-(8): out [T,d] = sum of kept experts' outputs
 * weighted by g * m.  W_mask NULL runs the same kernels with the mask test
 * off (vanilla Top-K MoE).  Launches beam_moe_forward_kernel_count(desc)
 * kernels: with 128-row token tiles (bf16 prefill batches, and BEAM_F32) all
 * seven stages -- router GEMM, top-K + mask, grouping, row gather, gate/up
 * GEMM + SwiGLU, down GEMM, weighted combine; with thinner tiles (bf16 decode
 * batches) five, because the grouping copies the token rows and both expert
 * GEMMs run as one launch.  No host synchronisation; capturable into a CUDA
 * graph. */
beam_status beam_moe_forward(const beam_moe_desc *desc, const void *x, const void *W_gate,
                             const void *W_mask, const void *W1, const void *W3,
                             const void *W2, void *out, void *workspace,
                             size_t workspace_bytes, void *stream);

/* beam_moe_forward with shared experts (desc->n_shared > 0): out = routed sum
 * (Eq. 8) + sum over the shared experts of E_s(x), the shared experts run for
 * every token.  W1s (gate), W3s (up) [n_shared, I_shared, d], W2s (down)
 * [n_shared, d, I_shared], bf16.  Two or three more launches than
 * beam_moe_forward (a gate/up GEMM, when its reduction is split a SwiGLU
 * kernel, and a down GEMM over all tokens; see beam_moe_forward_kernel_count).
 * They read no routing, so they run on a second stream that the library owns
 * (one per device, created by the first such call made outside a stream
 * capture): the call records an event on `stream` at its start, the second
 * stream waits for it, and `stream` waits for the second stream's event
 * before the combine.  Work issued on `stream` after the call therefore
 * follows all of it, as with any other call; a captured call records the
 * fork and the join as graph edges.  A first call made inside a capture runs
 * the shared experts on `stream` itself.  Calls are serialised on the host
 * from the fork to the end of their enqueue (a lock), so concurrent callers
 * never interleave their events.  With n_shared == 0 it is beam_moe_forward
 * (the shared pointers may be NULL). */
beam_status beam_moe_forward_shared(const beam_moe_desc *desc, const void *x,
                                    const void *W_gate, const void *W_mask, const void *W1,
                                    const void *W3, const void *W2, const void *W1s,
                                    const void *W3s, const void *W2s, void *out,
                                    void *workspace, size_t workspace_bytes, void *stream);

/* beam_moe_forward that also records `events[i]` (cudaEvent_t, created by the
 * caller) on `stream` before stage i and events[BEAM_MOE_FORWARD_STAGES]
 * after the last one, so the caller can time each kernel with
 * cudaEventElapsedTime.  The records are "external" (cudaEventRecordExternal):
 * captured into a CUDA graph they become event nodes that every replay
 * re-records.  A NULL entry records nothing at that point (each record costs
 * a few microseconds of device time, so time one kernel with just the two
 * events around it).  Same launches and results as beam_moe_forward. */
beam_status beam_moe_forward_profiled(const beam_moe_desc *desc, const void *x,
                                      const void *W_gate, const void *W_mask,
                                      const void *W1, const void *W3, const void *W2,
                                      void *out, void *workspace, size_t workspace_bytes,
                                      void *stream, void *const *events);

/* Bytes of the fixed device array behind beam_moe_route_noalloc (16 MiB). */
#define BEAM_MOE_ROUTE_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)

/* beam_moe_route for callers that cannot allocate device memory.  The paper
 * has no counterpart: this is a service of this library.
 *
 * Who needs it: plugins inside a host runtime whose memory pool owns all of
 * the device memory and lets its extensions allocate none (a serving engine
 * that reserves the GPU when it starts, for example), and callers inside a
 * fixed memory budget, where a new allocation may fail or fragment the pool.
 * The caller still passes every input and output exactly as for
 * beam_moe_route; the scratch (router partial logits, error words, counters)
 * lives in a file-scope device array of BEAM_MOE_ROUTE_NOALLOC_SCRATCH_BYTES
 * that every GPU loading the library holds until the process exits.  Nothing
 * here calls cudaMalloc, cudaFree or any allocating routine.
 *  - Size limit: the call needs beam_moe_plan(desc)->off_idx bytes of
 *    scratch; larger batches return BEAM_ERR_WORKSPACE before any launch (for
 *    d=2048, E=128 every T up to 8192 fits).
 *  - The first call on a device looks the array's address up on that device
 *    (cudaGetSymbolAddress, with that device current); make that first call
 *    before any stream capture.
 *  - All calls share the one array, which keeps the last call's contents:
 *    calls whose kernels may overlap on the GPU (different streams, or
 *    concurrent host threads) race on it and must be ordered by the caller.
 *    Each call clears what must start at zero.
 *  - Same kernels and results as beam_moe_route.  Its device error word is in
 *    the array: read it with beam_moe_route_noalloc_check. */
beam_status beam_moe_route_noalloc(const beam_moe_desc *desc, const void *x,
                                   const void *W_gate, const void *W_mask, int32_t *topk_idx,
                                   float *topk_w, int32_t *expert_counts, int32_t *kept_hist,
                                   float *logits, void *stream);

/* Synchronise `stream`, then read the error word of the last
 * beam_moe_route_noalloc call on the current device: BEAM_OK, or
 * BEAM_ERR_TIMEOUT when a bounded device wait of the router expired (its
 * outputs are then not valid).  Allocates nothing. */
beam_status beam_moe_route_noalloc_check(void *stream);

/* Kernel launches one forward call makes for `desc`: 5 (bf16 with
 * decode-sized token tiles) or 7, plus 2 with shared experts; 0 for T = 0 or
 * a bad descriptor. */
int beam_moe_forward_kernel_count(const beam_moe_desc *desc);

/* Tuning switch of the one-launch path (plan field one_launch): bf16 calls
 * without shared experts and with at most max_tokens tokens (and at most 16,
 * whose token rows, logits and weight stages fit one CTA's shared memory)
 * run router, top-K + mask, grouping, both expert projections and the
 * combine as ONE kernel whose phases hand off through counters in the
 * workspace.  Larger batches take the multi-kernel path.  0 turns it off.
 * Default 4: the batch sizes where it was measured faster.  Returns the
 * previous value; process-wide, not per call.  Routing at those sizes (and
 * only the routing) is the same in both paths: the router logits of every
 * bf16 call with T <= 16 come from the same router code. */
int beam_moe_set_one_launch_tokens(int max_tokens);

/* ------------------------------------------------------------ training --
 * Backward pass of the layer for training the mask router (techwalker news
 * article on BEAM, §4: the binary decision is trained through a
 * straight-through estimator, and a penalty weighted by beta on the
 * candidates' mask scores pushes towards fewer active experts).  The pages
 * give both in words; the readings taken here:
 *   objective  L = sum_t <dy_t, y_t> + beta * sum_t sum_{k<K} sigmoid(z_{t,c_k})
 *              (the penalty adds up the K candidates' scores of every token;
 *              divide beta by the token count for a mean)
 *   estimator  the forward keeps the hard mask of Eq. (6); the backward
 *              passes the gradient straight through the threshold
 *              (dm/dsigmoid = 1) and keeps the sigmoid's slope
 *   candidates every candidate's expert is evaluated, masked or not: candidate
 *              k's mask gets g_k <dy, E_k(x)> through the estimator either way
 *   weights    only kept candidates get expert-weight gradients (their
 *              weight in Eq. 7 is g_k; a masked candidate's is 0)
 * Arguments: the forward's inputs (same layouts, dtype of desc) and dy [T,d]
 * in that dtype; beta finite.  desc->n_shared must be 0.
 * Outputs, fp32, row-major like their weights:
 *   dx [T,d]                       overwritten
 *   dW_gate, dW_mask [E,d]         accumulated (+=); dW_mask NULL iff W_mask NULL
 *   dW1, dW3 [E,I,d], dW2 [E,d,I]  accumulated (+=) for experts with at least
 *                                  one kept pair; other experts' rows are not
 *                                  touched (zero them once per step)
 * Every sum runs in a fixed order: the gradients are bitwise repeatable.
 * Workspace: beam_moe_backward_workspace_size bytes, 256-byte aligned; the
 * caller owns it and every output.  Errors as for beam_moe_forward; also
 * BEAM_ERR_UNSUPPORTED_SHAPE for shared experts, and for fp32 layers with
 * d > 7168 or I > 4096 at 128-token tiles (8x larger at decode tile sizes),
 * beyond which a split of the CUDA-core kept-row products no longer fits in
 * shared memory.
 * Precision (bf16): both kept-row products (dh = dy W2_e and
 * dxp = da W1_e + db W3_e) run on the tensor cores with bf16 operands and fp32
 * accumulation; their da, db operands are da, db rounded once to bf16, while
 * dW1, dW3 use da, db in fp32. */
size_t beam_moe_backward_workspace_size(const beam_moe_desc *desc);
beam_status beam_moe_backward(const beam_moe_desc *desc, const void *x, const void *W_gate,
                              const void *W_mask, const void *W1, const void *W3, const void *W2,
                              const void *dy, float beta, float *dx, float *dW_gate,
                              float *dW_mask, float *dW1, float *dW3, float *dW2,
                              void *workspace, size_t workspace_bytes, void *stream);
/* beam_moe_backward with a further gradient of the main router's logits,
 * dlogits f32 [T,E] (beam_moe_balance_backward's), added to the layer's own
 * before both go on to x and W_gate.  NULL: beam_moe_backward itself. */
beam_status beam_moe_backward_aux(const beam_moe_desc *desc, const void *x, const void *W_gate,
                                  const void *W_mask, const void *W1, const void *W3,
                                  const void *W2, const void *dy, const float *dlogits,
                                  float beta, float *dx, float *dW_gate, float *dW_mask,
                                  float *dW1, float *dW3, float *dW2, void *workspace,
                                  size_t workspace_bytes, void *stream);
/* Kernel launches of one beam_moe_backward call: 15 for bf16 (its dh = dy W2_e
 * product runs on the tensor cores, after a launch that lists each kept
 * expert's candidate rows), 14 for fp32; 0 for T = 0 or a bad descriptor. */
int beam_moe_backward_kernel_count(const beam_moe_desc *desc);

/* ------------------------------------------------- expert parallelism --
 * G ranks (one process per GPU), rank r owning experts [r E/G, (r+1) E/G).
 * The pages describe the exchange only in general terms (the MoE tutorial
 * page on "Beam", §4.2: tokens travel to the GPU that holds their expert by
 * an all-to-all) and BEAM's own contribution to it in the news article on
 * BEAM, §5: masked entries are left out of the expert-token grouping.  Here
 * only KEPT pairs are dispatched, so the mask cuts the rows that cross the
 * interconnect by the kept fraction.  A step, per rank:
 *   beam_moe_route (own tokens) -> beam_moe_ep_dispatch -> all-to-all of the
 *   send counts, rows and local expert ids -> beam_moe_expert_rows on the
 *   received rows -> all-to-all of the fp32 rows back -> beam_moe_ep_combine.
 * The exchanges are the caller's (NCCL through torch.distributed in the
 * Python binding); these calls never touch another GPU's memory. */

/* Dispatch of the kept pairs of one routed batch (desc, topk_idx and
 * expert_counts as written by beam_moe_route on `workspace`).  Pairs are
 * listed by expert (ascending) then token (ascending) -- the order of the
 * layer's own grouping -- so the rows bound for rank r are contiguous and
 * ranks appear in order.  Writes, with P = the number of kept pairs:
 *   send_rows   [P, d] (desc dtype)  the pairs' token rows, in that order
 *   send_pair   int32 [P]    t*K + k of each row
 *   send_expert int32 [P]    the row's expert id local to its destination
 *   send_counts int32 [n_ranks]  rows per destination rank
 *   pair_pos    int32 [T,K]  send row of each kept pair (masked: unwritten)
 * Capacity: send_rows/send_pair/send_expert hold T*K entries.  Needs
 * E % n_ranks == 0, 1 <= n_ranks <= E and n_shared == 0.  A consistency
 * failure sets the workspace error word (BEAM_ERR_INTERNAL through
 * beam_moe_check), which this call never clears: check once after the step. */
beam_status beam_moe_ep_dispatch(const beam_moe_desc *desc, int n_ranks, const void *x,
                                 const int32_t *topk_idx, const int32_t *expert_counts,
                                 void *send_rows, int32_t *send_pair, int32_t *send_expert,
                                 int32_t *send_counts, int32_t *pair_pos, void *workspace,
                                 size_t workspace_bytes, void *stream);

/* Expert outputs of pre-routed rows: y_rows[i] = E_{expert_id[i]}(x_rows[i])
 * (Eq. 3), fp32, computed by the layer's own grouping and expert GEMMs, so a
 * row's value is the per-pair output the one-GPU layer combines.  desc: T =
 * number of rows, E = the experts in W1/W3/W2, K = 1, n_shared = 0; the
 * router fields are unused.  expert_id int32 [T]: an id in [0, E) or -1 (the
 * row gets zeros); any other value sets BEAM_ERR_INTERNAL and is treated as
 * -1.  Workspace: beam_moe_workspace_size(desc) bytes; errors through
 * beam_moe_check on it. */
beam_status beam_moe_expert_rows(const beam_moe_desc *desc, const void *x_rows,
                                 const int32_t *expert_id, const void *W1, const void *W3,
                                 const void *W2, float *y_rows, void *workspace,
                                 size_t workspace_bytes, void *stream);

/* Eq. (8) at the source rank: out_t = sum over kept k, in slot order, of
 * topk_w[t,k] * y_rows[pair_pos[t,k]] (fp32 sums, one rounding to the desc
 * dtype); 0 for a token with no kept candidate.  y_rows: the returned fp32
 * rows in send order (non-NULL even when no pair is kept; nothing is then
 * read).  T = 0 does nothing. */
beam_status beam_moe_ep_combine(const beam_moe_desc *desc, const float *y_rows,
                                const int32_t *topk_idx, const float *topk_w,
                                const int32_t *pair_pos, void *out, void *stream);

/* ---------------------------------------------- the residual block around --
 * What a transformer block puts around the layer, one pass over the rows
 * each.  The pages leave the residual to the caller; these calls are that
 * caller's part.  r(x) = 1 / sqrt(mean_j x_j^2 + eps) per row, in fp32.
 *   T, d       token rows of width d; d % 8 == 0, d <= 16384
 *   dtype      of the rows, the weights and the gates
 *   eps        finite and >= 1e-30
 *   res_scale, branch_scale   a and b below; finite
 *   accumulate backward: 1 adds to the gradients of the weights and of
 *              gate_c (fp32 [d]), 0 overwrites them; every other gradient is
 *              overwritten
 * Rows are contiguous, pointers 16-byte aligned.  An output may be the very
 * buffer of one input row for row: n that of x, out that of res or y, n_next
 * that of y or res (not out's), dres or dx that of dout or dskip, dy that of
 * y.  Squares are summed in fp32: rows beyond 1e19 overflow.
 * Rounding: one, to dtype, of each result; the next norm and the gradients
 * read `out` as it is stored. */
typedef struct {
    int T, d;
    int dtype; /* beam_dtype */
    float eps, res_scale, branch_scale;
    int accumulate; /* 0 or 1 */
} beam_block_desc;

/* n = x r(x) w: the rows the layer reads. */
beam_status beam_block_enter(const beam_block_desc *desc, const void *x, const void *w, void *n,
                             void *stream);

/* out = a res + b s(gate_t[t]) gate_c[j] w_out[j] y r(y), with s the logistic
 * function: the norm behind the layer, its gates and the residual;
 * n_next = out r(out) w_next: the norm in front of the next block.
 *   w_out [d] or NULL (y as it is, without r(y)), gate_c [d] or NULL (1),
 *   gate_t [T] or NULL (s = 1), w_next [d] and n_next [T,d] or both NULL */
beam_status beam_block_exit(const beam_block_desc *desc, const void *res, const void *y,
                            const void *w_out, const void *gate_c, const void *gate_t, void *out,
                            const void *w_next, void *n_next, void *stream);

/* Bytes of workspace of the two backward calls (0 on a bad descriptor); it is
 * 256-byte aligned, and calls that may overlap need one each. */
size_t beam_block_workspace_size(const beam_block_desc *desc);

/* dx = dskip + (dn through the norm), dw = sum_t dn x r(x).  dn fp32 [T,d],
 * as beam_moe_backward writes its dx; dskip [T,d] of dtype or NULL: the
 * gradient that reaches x past the block.  res_scale, branch_scale unused. */
beam_status beam_block_enter_backward(const beam_block_desc *desc, const void *x, const void *w,
                                      const float *dn, const void *dskip, void *dx, float *dw,
                                      void *workspace, size_t workspace_bytes, void *stream);

/* Gradients of beam_block_exit for dout [T,d] (dtype) and, with w_next,
 * dn_next [T,d] (fp32): dres and dy [T,d] (dtype); dw_out, dgate_c, dw_next
 * fp32 [d] and dgate_t fp32 [T], each given exactly when its weight or gate
 * is.  y: as in the forward; out: the forward's, needed with w_next.  dy is
 * the layer's upstream gradient (beam_moe_backward's dy).  Bitwise repeatable. */
beam_status beam_block_exit_backward(const beam_block_desc *desc, const void *y, const void *out,
                                     const void *w_out, const void *gate_c, const void *gate_t,
                                     const void *w_next, const void *dout, const float *dn_next,
                                     void *dres, void *dy, float *dw_out, float *dgate_c,
                                     float *dgate_t, float *dw_next, void *workspace,
                                     size_t workspace_bytes, void *stream);

/* --------------------------------------------------------- balance loss --
 * The load-balance loss on the main router (news article on BEAM, §4: one of
 * the three training losses; its form is not given, this is the usual one)
 * over n_seq sequences of tokens, L_s long, with p_t the softmax of token t's
 * logits over all E experts:
 *   f_se = E / (K L_s) #{t in s with e among its K candidates}
 *   P_se = 1 / L_s sum_{t in s} p_te
 *   loss = coef / n_seq sum_s sum_e f_se P_se          (coef: even load)
 * An empty sequence adds 0 and counts in n_seq.  Candidates are those of
 * beam_moe_route: the K largest logits, ties to the lower id, NaN last.
 * count_kept = 1 counts only the candidates the mask keeps (z >=
 * mask_logit_threshold).  A row of -inf has no softmax and counts as zeros.
 *   T tokens (< 2^30), n_seq <= 2^20, E <= 256, 1 <= K <= min(E, 16)
 *   logits_ld  floats per row of logits: >= E, and >= 2E with has_mask, whose
 *              columns [E, 2E) hold z -- beam_moe_route's logits have 2E */
typedef struct {
    int T, E, K, n_seq;
    int logits_ld;
    int has_mask, count_kept; /* 0 or 1 */
    float mask_logit_threshold, coef;
} beam_balance_desc;

/* Forward.  logits f32 [T, logits_ld]; seq_begin int32 [n_seq + 1] (device) or
 * NULL (n_seq == 1: all T): sequence s is tokens [seq_begin[s],
 * seq_begin[s + 1]); tokens outside every sequence do not count.  Boundaries
 * that decrease or leave [0, T] make the loss NaN; the counts, P and the
 * gradient are then of no use.  A NaN logit makes P and the loss NaN.
 * Written: loss f32 [1]; cand_counts int32 [n_seq, E]; kept_counts the same or
 * NULL (only with has_mask); mean_prob f32 [n_seq, E] (P) or NULL.  Sums run
 * in a fixed order.  Workspace 256-byte aligned; calls that may overlap need
 * one each. */
size_t beam_moe_balance_workspace_size(const beam_balance_desc *desc);
beam_status beam_moe_balance(const beam_balance_desc *desc, const float *logits,
                             const int32_t *seq_begin, float *loss, int32_t *cand_counts,
                             int32_t *kept_counts, float *mean_prob, void *workspace,
                             size_t workspace_bytes, void *stream);

/* dlogits f32 [T,E] (overwritten): dloss coef / (n_seq L_s) p_te (f_se -
 * sum_e' f_se' p_te'), zeros for tokens outside every sequence.  counts:
 * cand_counts, or with count_kept kept_counts, of the forward (the counts pass
 * no gradient); dloss f32 [1] (device) or NULL (1).  beam_moe_backward_aux
 * carries dlogits on to x and W_gate. */
beam_status beam_moe_balance_backward(const beam_balance_desc *desc, const float *logits,
                                      const int32_t *seq_begin, const int32_t *counts,
                                      const float *dloss, float *dlogits, void *stream);

/* ------------------------------------- experts in 4-bit floating point --
 * The layer's experts with weights and token rows in MXFP4 (OCP Microscaling
 * Formats v1.0), a quarter of the bf16 weight bytes that bound a decode step;
 * the pages have no counterpart.  Blocks of 32 consecutive values of a row
 * share one scale 2^X, X = floor(log2 max|v|) - 2 (at least -127), stored as
 * the byte X + 127; each value is v / 2^X rounded to nearest, ties to even, on
 * the E2M1 grid 0, .5, 1, 1.5, 2, 3, 4, 6 with a sign bit, saturating at 6.  A
 * block that holds an infinity or a NaN stands for NaN throughout: scale byte
 * 255, codes 0.  codes [rows, cols / 2]: value 2i of a row in the low half of
 * byte i, value 2i + 1 in the high half.  scales [rows, cols / 32], either row
 * by row (tiled = 0) or, for the product's weights, in tiles of 128 rows x 4
 * blocks (tiled = 1; rows and cols % 128 == 0): the byte of (row, block) is at
 * ((row / 128) (cols / 128) + block / 4) 512 + 16 (row % 32) +
 * 4 ((row % 128) / 32) + block % 4.
 * Pointers are 16-byte aligned, cols % 32 == 0.  Rows need no alignment. */

/* x [rows, cols] of `dtype` -> codes, scales.  n_rows (device int32, or NULL):
 * only the first min(*n_rows, rows) rows are read and written (not with
 * tiled = 1), so that rows whose number only the device knows need no copy to
 * the host. */
beam_status beam_mx4_quantize(int dtype, long long rows, int cols, const void *x,
                              const int32_t *n_rows, uint8_t *codes, uint8_t *scales, int tiled,
                              void *stream);

/* The values the codes stand for, in `dtype` (exact: every value of the
 * format with X <= 125 is a bfloat16). */
beam_status beam_mx4_dequantize(int dtype, long long rows, int cols, const uint8_t *codes,
                                const uint8_t *scales, int tiled, void *out, void *stream);

/* Grouped product of one projection: N token rows (capacity) of width k,
 * grouped by expert in ascending order as beam_moe_ep_dispatch lists them, E
 * experts (<= 256) of n weight rows; n % 128 == 0, k % 128 == 0.  out_dtype:
 * beam_dtype of out.  swiglu = 1: two weight matrices, gate and up. */
typedef struct {
    int N, E, n, k;
    int swiglu;    /* 0 or 1 */
    int out_dtype; /* beam_dtype */
} beam_mx4_desc;

/* out[i, :] = a_i w_e^T for the rows i of expert e, or with swiglu
 * SiLU(a_i w_e^T) * (a_i w3_e^T) (Eq. 3); fp32 accumulation, one rounding.
 *   a_codes [N, k/2], a_scales [N, k/32] row by row
 *   expert_counts int32 [E] (device): rows of each expert, as beam_moe_route
 *     writes them; expert e's rows follow those of the experts before it.
 *     Rows past the last expert's are neither used nor written.  Counts that
 *     are negative or add up to more than N are cut at N and reported
 *     (BEAM_ERR_INTERNAL through beam_mx4_check).
 *   w_codes [E, n, k/2] and w_scales in tiles over the E n rows (tiled = 1);
 *     w3 the same with swiglu, else NULL.  Experts without rows are not read.
 *   out [N, n] of out_dtype
 *   workspace: beam_mx4_workspace_size(desc) bytes, 256-byte aligned; calls
 *     that may overlap need one each. */
size_t beam_mx4_workspace_size(const beam_mx4_desc *desc);
beam_status beam_mx4_expert_product(const beam_mx4_desc *desc, const uint8_t *a_codes,
                                    const uint8_t *a_scales, const int32_t *expert_counts,
                                    const uint8_t *w_codes, const uint8_t *w_scales,
                                    const uint8_t *w3_codes, const uint8_t *w3_scales, void *out,
                                    void *workspace, size_t workspace_bytes, void *stream);
/* As beam_moe_check, for the workspace of the last product made on it. */
beam_status beam_mx4_check(const beam_mx4_desc *desc, void *workspace, void *stream);

/* Synchronise `stream`, then read the workspace error word written by the last
 * call: BEAM_OK, BEAM_ERR_TIMEOUT (a bounded device wait expired, the kernel
 * returned early; that call's outputs are not valid) or BEAM_ERR_INTERNAL (a
 * device consistency check failed).  Every call resets the word, so it
 * describes the last call made on the workspace.  After a timeout the
 * workspace and the context stay usable: the next call starts clean. */
beam_status beam_moe_check(const beam_moe_desc *desc, void *workspace, void *stream);

/* The descriptor's mask_logit_threshold for a threshold tau of Eq. (6):
 * ln(tau / (1 - tau)) evaluated in double and rounded once to float, so that
 * a candidate is kept iff sigmoid(z) >= tau <=> z >= the returned value.
 * tau = 0.5 gives 0 exactly; tau = 0 gives -inf, tau = 1 gives +inf; NaN for
 * tau outside [0, 1] (which beam_moe_plan rejects). */
float beam_moe_tau_to_logit(float tau);

/* Testing aid, off by default; the paper has no counterpart.  It lets a test
 * observe the bounded-wait path without faulting or hanging the GPU:
 *   mode 0  off;
 *   mode 1  in every later forward call, CTA 0 of the expert GEMM launch (the
 *           fused expert kernel at decode tile sizes, the gate/up GEMM
 *           otherwise; bf16 only) skips the first shared-memory stage of its
 *           first unit: it issues neither the copy nor the transaction count,
 *           so the MMA issuer's bounded wait on that stage expires;
 *   mode 2  the same in CTA 0 of the router GEMM of every later route or
 *           forward call (bf16 only);
 *   mode 3  the same in CTA 0 of the shared experts' gate/up GEMM of every
 *           later forward call with shared experts (bf16 only);
 *   mode 4  the same in CTA 0 of every later beam_mx4_expert_product
 *           (beam_mx4_check then reports it).
 * The kernels then record the timeout, let their own copies and MMAs land,
 * free their tensor memory and return: beam_moe_check reports
 * BEAM_ERR_TIMEOUT and the context stays usable.  wait_limit_ns replaces the
 * 1 s limit of every bounded device wait (0 restores it).  Process-wide; set
 * it while no other thread is calling the library.  BEAM_ERR_INVALID_ARG for
 * an unknown mode. */
beam_status beam_moe_set_fault_injection(int mode, unsigned long long wait_limit_ns);

/* Static, NUL-terminated name of a status code. */
const char *beam_status_str(beam_status status);

/* Name of forward stage i (0 <= i < BEAM_MOE_FORWARD_STAGES), else NULL. */
const char *beam_moe_stage_name(int stage);

#ifdef __cplusplus
}
#endif
#endif
