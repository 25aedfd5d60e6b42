/*
 * moe_layout.h -- C ABI of the MI355X (gfx950) MoE token layout / dispatch /
 * combine library (libmoe_layout.so).
 *
 * What it computes is the data-parallel hot path of expert-parallel token
 * exchange, on one GPU: the P expert-parallel ranks are P virtual partitions
 * of one receive buffer in HBM.
 *
 *   "Add an opt-in DeepEP transport for the AutoEP expert all-to-all"
 *   (DeepSpeed PR), sections "Why" and "Scope and safety": the exchange
 *   receives tokens before their top-k expansion, together with their expert
 *   ids and weights; it replicates each token to the ranks that host its
 *   experts, presents the arrivals grouped by expert, and its combine forms
 *   the weighted top-k sum in token order again.  Backward needs no entry
 *   points of its own: each backward pass is the opposite row movement, run
 *   on the handle the forward dispatch produced.  The review-fix commit on
 *   that page makes dispatch hand back the received weights and makes both
 *   backward passes return the router-weight gradient.
 *
 *   "[MoE] Apply router scores before W2 projection" (torchtitan issue),
 *   sections "Motivation" and "Implementation": when the router scores are
 *   absorbed into W2's input, dispatch also returns each receive row's score
 *   in the rows' expert-major order, the scaling is done in float32 and
 *   rounded back to the row type, and the combine is a plain sum.
 *
 * Conventions (every entry point):
 *   - All tensor pointers are DEVICE pointers; the caller owns every buffer,
 *     the workspace and the stream.  Row-major, contiguous.
 *   - Calls are stream-ordered on `stream` and never block the host, except
 *     moe_handle_check, which synchronises the stream.
 *   - Arguments are validated on the host before anything is launched; a
 *     rejected call launches nothing and returns a negative MOE_ERR_* code.
 *   - T = tokens, K = top-k, E = experts, P = partitions (virtual EP ranks),
 *     H = row width in elements, R = receive rows: T*K, or T*K + E*(m-1)
 *     for a handle whose expert segments are padded to a multiple of m
 *     (moe_handle_create_padded; moe_recv_capacity returns R).
 *   - Expert e belongs to partition e / (E/P); E must be a multiple of P.
 *   - Element types: MOE_F32 (float) or MOE_BF16 (bfloat16 bits).  Every
 *     row is a whole number of 16-byte chunks: H*sizeof(elem) % 16 == 0.
 *   - Floating-point contract: products and sums in IEEE float32, each
 *     rounded on its own (no fused multiply-add); sums over k run in k order
 *     from +0.0; bfloat16 results are rounded to nearest, ties to even.
 *     Router-weight gradients use a fixed segment-major order (see
 *     moe_combine_bwd), so results are bitwise reproducible.
 */
#ifndef MOE_LAYOUT_H
#define MOE_LAYOUT_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
#define MOE_OK                 0
#define MOE_ERR_INVALID_ARG   -1  /* null pointer, negative size, missing companion argument */
#define MOE_ERR_SHAPE         -2  /* K < 1, K > E, E % P != 0, H*elem % 16 != 0, H < 1 */
#define MOE_ERR_UNSUPPORTED   -3  /* unknown dtype/itype, P > 64, E > 1024, K > 32, T*K >= 2^31 */
#define MOE_ERR_ALIGNMENT     -4  /* row pointers not 16-byte aligned, others not elem-aligned */
#define MOE_ERR_WORKSPACE     -5  /* workspace smaller than moe_workspace_size() */
#define MOE_ERR_HANDLE        -6  /* bad handle, or a data call before moe_layout */
#define MOE_ERR_HIP           -7  /* a HIP runtime call failed */
#define MOE_ERR_SCRATCH       -8  /* moe_layout_noalloc: the histogram exceeds its static scratch */

/* ---- element and index types ------------------------------------------- */
enum moe_dtype { MOE_F32 = 0, MOE_BF16 = 1 };
enum moe_itype { MOE_I32 = 0, MOE_I64 = 1 };

/* ---- limits -------------------------------------------------------------- */
#define MOE_MAX_K 32
#define MOE_MAX_E 1024
#define MOE_MAX_P 64

/* ---- device status bits (read with moe_handle_check) --------------------- */
#define MOE_STATUS_BAD_EXPERT   1  /* a topk_idx entry outside [0, E) */
#define MOE_STATUS_BAD_POSITION 2  /* a data kernel met a receive row outside [0, R) */

/* ---- handle fields (moe_handle_field) ------------------------------------ */
enum moe_field {
  MOE_FIELD_NUM_TOKENS_PER_EXPERT = 0, /* int32 [E]   (t,k) pairs per expert               */
  MOE_FIELD_NUM_TOKENS_PER_RANK   = 1, /* int32 [P]   distinct tokens per partition         */
  MOE_FIELD_IS_TOKEN_IN_RANK      = 2, /* uint8 [T,P] 1 if any of t's experts is on r       */
  MOE_FIELD_EXPERT_OFFSET         = 3, /* int32 [E+1] exclusive prefix of expert segment
                                          rows (counts, padded to the handle's multiple) */
  MOE_FIELD_RANK_OFFSET           = 4, /* int32 [P+1] first receive row of each partition   */
  MOE_FIELD_SEND_OFFSET           = 5, /* int32 [P+1] exclusive prefix of num_tokens_per_rank */
  MOE_FIELD_TOKEN_SLOT            = 6, /* int32 [T,P] t's slot in r's send list, or -1      */
  MOE_FIELD_RECV_POS              = 7, /* int32 [T,K] receive row of pair (t,k)            */
  MOE_FIELD_RECV_TOKEN            = 8, /* int32 [R]   token of each receive row, -1 if none */
  MOE_FIELD_RECV_K                = 9, /* int32 [R]   k of each receive row, -1 if none     */
  MOE_FIELD_STATUS                = 10,/* int32 [1]   device status bits                   */
  MOE_FIELD_SEND_TOKEN            = 11 /* int32 [T*min(K,P)] token of each send row
                                          (rows >= send_offset[P] unspecified)          */
};

/* Optional launch knobs; zero means "library default" except for
 * nontemporal, whose default applies when the struct is NULL.  A row is cut
 * into 16-byte chunks and the chunks into segments of 64 (one wavefront
 * access); the row kernels run one wavefront per (token, segment group).   */
typedef struct moe_tuning {
  int chunks_per_lane;  /* consecutive segments per wavefront, i.e. chunks of one row each
                           lane keeps in flight: 0 (= 1), 1, 2 or 4                        */
  int nontemporal;      /* 0: default loads/stores; 1: receive-row loads and stores
                           marked non-temporal; 2 (default): token-row stores too    */
  int waves_per_block;  /* wavefronts per workgroup of the row kernels: 0 (= 4; the
                           LDS-staged gather takes 1 when a row is whole segments and
                           their number is not a multiple of 8), 1, 2, 4, 8              */
  int layout_pairs;     /* (t,k) pairs per layout tile: 0 (= 512), 512, 1024, 2048, 4096      */
  int gather_mode;      /* receive rows of the gathers (moe_combine, unscaled moe_dispatch_bwd):
                           0 (default) by row width: staged in LDS by direct loads for rows
                           of 4 KiB and wider, in registers otherwise; 1 always LDS-staged;
                           2 always in registers                                         */
} moe_tuning;

typedef struct moe_handle_s* moe_handle_t;

/* Bytes of device workspace a layout of this shape needs (pure host).
 * Returns MOE_ERR_* on an invalid shape (same rules as moe_layout).  The
 * _padded form is for handles created with that pad_multiple.  A workspace
 * sized for the largest T serves every smaller T: calls with a varying
 * number of tokens need no new allocation. */
int moe_workspace_size(int64_t T, int K, int E, int P, size_t* bytes);
int moe_workspace_size_padded(int64_t T, int K, int E, int P, int pad_multiple, size_t* bytes);

/* Create / destroy a handle.  `tuning` may be NULL.  Host memory only: the
 * handle records views into the caller's workspace, never owns device memory. */
int moe_handle_create(moe_handle_t* out, const moe_tuning* tuning);
int moe_handle_destroy(moe_handle_t h);

/* A handle whose layouts pad every expert's segment of receive rows to a
 * multiple of pad_multiple (1..1024; 1 = moe_handle_create), fixed for the
 * handle's life (the DiffusionGemma dispatcher page lists pad_multiple as
 * set once at construction).  Segment e holds its n_e pairs, in the usual
 * order, then pad_multiple*ceil(n_e/pad_multiple) - n_e padding rows, so
 * every expert_offset is a multiple of pad_multiple (grouped-GEMM tiles).
 * Calls that write receive rows (moe_dispatch, moe_expand, the grad_y rows
 * of moe_combine_bwd) write zero rows there, and zero scores when they write
 * scores (the zero-sentinel scores of the padded permute, "[MoE] Apply
 * router scores before W2 projection", "Implementation"); rows past
 * expert_offset[E] are not written.  Calls that read receive rows never
 * read padding.  Receive buffers hold R = T*K + E*(pad_multiple-1) rows. */
int moe_handle_create_padded(moe_handle_t* out, const moe_tuning* tuning, int pad_multiple);

/* Layout of one routing decision (method steps: counts, offsets, stable
 * positions).  Fills every handle field inside `workspace`.
 *
 *   topk_idx   [T,K] int32 (itype MOE_I32) or int64 (MOE_I64), device.
 *   workspace  device, >= moe_workspace_size(T,K,E,P) bytes (the _padded
 *              size for a padded handle), 256-byte aligned; it holds the
 *              handle's arrays and must outlive every later call on this
 *              handle.  MOE_ERR_WORKSPACE if it is smaller.
 *
 * Definitions (a stable counting sort of the (t,k) pairs by expert id):
 *   recv_pos[t,k] = expert_offset[e] + #{(t',k') < (t,k) lexicographically
 *                    with topk_idx[t',k'] == e},  e = topk_idx[t,k];
 *   expert_offset[e] = sum over e' < e of n_e' (rounded up to the handle's
 *                    pad multiple, see moe_handle_create_padded);
 *   so rows are grouped by expert in ascending id (hence by partition), and
 *   inside an expert by token, then k.  The order depends on the routing
 *   only, so an activation-checkpoint replay of the same routing reproduces
 *   every position ("perf(dllm): use the DeepEP dispatcher in the
 *   DiffusionGemma recipes", section "Why hybridep + activation
 *   checkpointing fails", shows what a replay-nondeterministic dispatch does).
 *   token_slot[t,r] numbers the tokens with is_token_in_rank[t,r] in
 *   increasing t (a token is sent once per partition, not once per expert:
 *   the deduplication of the DeepSpeed transport PR's "Why" section).
 *
 * T = 0 is valid and yields an empty layout; every data call on it returns
 * MOE_OK after its non-pointer checks, reads and writes nothing, and accepts
 * NULL for any array (an empty tensor's data pointer).  Entries of topk_idx outside
 * [0,E) are an input error detected on the device: MOE_STATUS_BAD_EXPERT is
 * set and those pairs are placed after the last expert's rows (so every
 * position stays inside [0,R)); the other fields are then unspecified.
 * Duplicate ids within a token are accepted and ordered by k.
 * The handle must not be used on two streams at once.                      */
int moe_layout(moe_handle_t h, const void* topk_idx, int itype, int64_t T, int K,
               int E, int P, void* workspace, size_t workspace_bytes,
               hipStream_t stream);

/* moe_layout for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc.  Same
 * arguments, results and handle as moe_layout; the difference is where the
 * layout's scratch lives.  moe_layout keeps its per-tile histogram in the
 * caller's workspace; this call keeps it in a static array inside the
 * library, one per GPU, held until the process ends, so the workspace only
 * has to hold the handle's arrays (moe_workspace_size() bytes always
 * suffice; the histogram section at their end is not touched).  The call
 * itself allocates nothing: no hipMalloc, hipFree or allocating library
 * routine.  Limit: the histogram, (E+1+P) * (tiles+1) * 4 bytes, must fit
 * in 2 MiB (tiles: T*K/512, at most 128 until a tile reaches its cap of
 * 2048 tokens at K = 8, then T/2048); a larger shape is refused on the host
 * with MOE_ERR_SCRATCH, before any launch.  Every call
 * on one GPU shares that GPU's array: layouts that overlap in time on one
 * GPU (two streams, or two host threads) race on it and must be ordered by
 * the caller; each call writes every histogram entry it reads, so nothing
 * has to be cleared between calls.                                        */
int moe_layout_noalloc(moe_handle_t h, const void* topk_idx, int itype, int64_t T, int K,
                       int E, int P, void* workspace, size_t workspace_bytes,
                       hipStream_t stream);

/* Forward dispatch: recv[recv_pos[t,k], :] = x[t, :].
 * Defined by "Add an opt-in DeepEP transport for the AutoEP expert
 * all-to-all", sections "What this adds" and "Scope and safety" (tokens
 * before top-k expansion in, arrivals grouped by expert out), with the
 * received weights of its review fix (recv_scores) and the float32 row
 * scaling of "[MoE] Apply router scores before W2 projection",
 * "Implementation" (scale_rows).
 *
 *   x             [T,H] dtype, 16-byte aligned.
 *   topk_weights  [T,K] float32 or NULL; required when scale_rows or
 *                 recv_scores is given.
 *   scale_rows    0: copy rows bit for bit.  1: scores absorbed before W2,
 *                 recv = round(float32(x[t]) * w[t,k]).
 *   recv          [R,H] dtype, 16-byte aligned (output).
 *   recv_scores   [R] float32 or NULL (output): recv_scores[recv_pos[t,k]] = w[t,k].
 * Each x row is read once and stored to its receive rows partition by
 * partition.                                                              */
int moe_dispatch(moe_handle_t h, const void* x, int dtype, int64_t H,
                 const float* topk_weights, int scale_rows, void* recv,
                 float* recv_scores, hipStream_t stream);

/* Forward combine: out[t] = round(sum_k w[t,k] * y[recv_pos[t,k]]), or the
 * plain sum when topk_weights is NULL (scores absorbed).  float32, k order.
 * Defined by "Add an opt-in DeepEP transport for the AutoEP expert
 * all-to-all", section "Scope and safety" (the combine reduces the weighted
 * sum back to token order), and "[MoE] Apply router scores before W2
 * projection", "Implementation" (a plain sum once the scores are absorbed).
 *   y [R,H], out [T,H] dtype, 16-byte aligned.
 * Errors: MOE_ERR_HANDLE before moe_layout; MOE_ERR_SHAPE / _ALIGNMENT /
 * _INVALID_ARG for a bad row width, pointer or missing array (checked on the
 * host, nothing launched); receive rows out of [0,R) set
 * MOE_STATUS_BAD_POSITION on the device and are skipped.                  */
int moe_combine(moe_handle_t h, const void* y, int dtype, int64_t H,
                const float* topk_weights, void* out, hipStream_t stream);

/* Backward of moe_combine (a dispatch of the output gradient), per
 * "Add an opt-in DeepEP transport for the AutoEP expert all-to-all",
 * section "Scope and safety" (the gradient of a combine is a dispatch on the
 * forward's handle) and the same page's review fix (the weight gradient is
 * returned, never dropped):
 *   grad_y[recv_pos[t,k]] = round(w[t,k] * grad_out[t])  (copy if no weights)
 *   grad_w[t,k] = <grad_out[t], y[recv_pos[t,k]]>        (if grad_w != NULL)
 * grad_w needs topk_weights and y.  The dot product is float32 in a fixed
 * order: the row is cut into 16-byte chunks and the chunks into segments of
 * 64; each chunk's partial adds its element products in order from +0.0
 * (product rounded, then sum rounded); each segment folds its 64 partials
 * L[l] += L[l xor s] for s = 32,16,8,4,2,1 (absent chunks are +0.0) and
 * takes partial 0; the result adds the segment values in order from +0.0.
 * Needs ceil(H*elem/1024) * K * 4 <= 65536 (else MOE_ERR_UNSUPPORTED).
 *   grad_out [T,H], y [R,H], grad_y [R,H] dtype; grad_w [T,K] float32.     */
/* grad_y may be NULL when grad_w is given: then only the router-weight
 * gradient is computed (the rows of a staged backward come from moe_send and
 * moe_expand). */
int moe_combine_bwd(moe_handle_t h, const void* grad_out, int dtype, int64_t H,
                    const float* topk_weights, const void* y, void* grad_y,
                    float* grad_w, hipStream_t stream);

/* Backward of moe_dispatch (a combine of the receive-row gradient), per
 * "Add an opt-in DeepEP transport for the AutoEP expert all-to-all",
 * section "Scope and safety" (the gradient of a dispatch is a combine on the
 * forward's handle); with scores absorbed, "[MoE] Apply router scores before
 * W2 projection", "Implementation" and "Tests and verifications" (the score
 * gradient flows through W2's input scaling):
 *   grad_x[t] = round(sum_k [w[t,k] *] grad_recv[recv_pos[t,k]])
 *   grad_s[t,k] = <grad_recv[recv_pos[t,k]], x[t]>        (if grad_s != NULL)
 * Pass topk_weights iff the forward dispatch scaled its rows (the scaling is
 * differentiated straight through its rounding).  grad_s needs topk_weights
 * and x; same dot order and size limit as moe_combine_bwd.
 *   grad_recv [R,H], x [T,H], grad_x [T,H] dtype; grad_s [T,K] float32.   */
/* grad_x may be NULL when grad_s is given: then only the score gradient is
 * computed (the rows of a staged backward come from moe_reduce_partitions and
 * moe_combine_partitions). */
int moe_dispatch_bwd(moe_handle_t h, const void* grad_recv, int dtype, int64_t H,
                     const float* topk_weights, const void* x, void* grad_x,
                     float* grad_s, hipStream_t stream);

/* ---- staged exchange ------------------------------------------------------
 * The payload a cross-GPU transport moves, staged in one GPU's HBM: a send
 * buffer with one row per (token, destination partition) pair, at row
 * send_offset[r] + token_slot[t,r] ("Add an opt-in DeepEP transport for the
 * AutoEP expert all-to-all", section "Why": a token is sent once per
 * destination rank, not once per selected expert; arrivals are grouped by
 * expert; the combine reduces back to token order).  send_offset[P] rows are
 * used; buffers take a capacity of at least moe_send_capacity() rows, known
 * on the host without a device sync.  Staged dispatch = moe_send +
 * moe_expand (bitwise equal to moe_dispatch); staged combine =
 * moe_reduce_partitions + moe_combine_partitions (its own summation order,
 * below).  A staged backward uses the same calls: the combine's backward is
 * moe_send + moe_expand of the output gradient (scaled), the dispatch's is
 * moe_reduce_partitions + moe_combine_partitions of the receive-row gradient;
 * the router-weight gradients come from moe_combine_bwd / moe_dispatch_bwd
 * with NULL row outputs.
 *
 * Row pointers 16-byte aligned, dtype as in the other calls; send_rows is
 * the caller's buffer capacity in rows (MOE_ERR_SHAPE if below
 * moe_send_capacity()).                                                    */

/* Rows a send buffer must hold: T * min(K, P), an upper bound of send_offset[P]. */
int moe_send_capacity(moe_handle_t h, int64_t* rows);

/* Rows a receive buffer (recv, y, grad_y, grad_recv, recv_scores) holds for
 * the current layout: T*K, plus E*(pad_multiple-1) on a padded handle.
 * Known on the host; no device sync. */
int moe_recv_capacity(moe_handle_t h, int64_t* rows);

/* Source side: send[send_offset[r] + token_slot[t,r]] = x[t] for every
 * partition r of token t (each x row is read once).  x [T,H].            */
int moe_send(moe_handle_t h, const void* x, int dtype, int64_t H, void* send, int64_t send_rows,
             hipStream_t stream);

/* Receiver side: recv[recv_pos[t,k]] = send[send_offset[r] + token_slot[t,r]]
 * for every pair whose expert is on partition r (each send row is read
 * once); scale_rows, recv_scores and padding rows as in moe_dispatch.
 * recv [R,H].                                                             */
int moe_expand(moe_handle_t h, const void* send, int dtype, int64_t H, int64_t send_rows,
               const float* topk_weights, int scale_rows, void* recv, float* recv_scores,
               hipStream_t stream);

/* Receiver side of the two-level combine: for every (token, partition) send
 * row, partial = round(sum [w[t,k] *] y[recv_pos[t,k]]) over the token's k
 * with an expert on that partition, in k order, float32 from +0.0 (product
 * and sum rounded on their own); rounded to the row type, the type a
 * transport sends.  y [R,H]; partial [send_rows,H]; weights may be NULL
 * (plain sum).                                                             */
int moe_reduce_partitions(moe_handle_t h, const void* y, int dtype, int64_t H,
                          const float* topk_weights, void* partial, int64_t send_rows,
                          hipStream_t stream);

/* Source side: out[t] = round(sum of float32(partial[send row of (t,r)]))
 * over t's partitions r in ascending order, float32 from +0.0.  out [T,H]. */
int moe_combine_partitions(moe_handle_t h, const void* partial, int dtype, int64_t H,
                           int64_t send_rows, void* out, hipStream_t stream);

/* ---- router ------------------------------------------------------------------
 * From a token's expert logits to the topk_idx and topk_weights that the other
 * calls take.  No handle: the calls stand before moe_layout.
 *
 *   s = softmax(z) over the token's E experts, or sigmoid(z) of each;
 *   c = s + bias, the value experts are chosen by (without a bias and without
 *       a group limit the choice goes by the logits themselves);
 *   with topk_groups < num_groups: experts form num_groups groups of
 *       E/num_groups neighbours, a group's value is the sum of its two largest
 *       c (its one c if it has a single expert; +inf if its largest is), and
 *       only the topk_groups groups of largest value take part;
 *   the K largest c are chosen, in descending order; equal values (experts or
 *       groups) go to the lower index;
 *   w[t,k] = scale * s of the chosen expert, divided by the sum of the token's
 *       K chosen s if renormalize.
 * Where values are compared after arithmetic (bias, groups) the choice is that
 * of 64-bit arithmetic: it is made in 32 bits only where that cannot differ.
 * Weights are computed in 32 bits; renormalised ones (and their gradient) from
 * scores relative to each other, so that they are right however small the scores
 * are.  A sigmoid below 2^-1022 counts as zero there.  A NaN logit counts as -inf
 * in the choice, as a c that is NaN does; it makes its own sigmoid weight NaN
 * (all of the token's if renormalised) and every softmax weight of its token, as
 * +inf does in a softmax.  A token whose logits are all -inf (or whose chosen
 * scores add up to zero) gets weight zero throughout and the lowest ids that may
 * take part.                                                                */
enum moe_score { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 };

typedef struct moe_route_options {
  int score;        /* MOE_SCORE_*                                             */
  int renormalize;  /* 1: the K weights of a token add up to scale; 0: not     */
  int num_groups;   /* 1..64, divides E; 1 with topk_groups 1: no group limit  */
  int topk_groups;  /* 1..num_groups; K <= topk_groups * E/num_groups          */
  float scale;      /* finite factor of every weight                           */
} moe_route_options;

/* logits [T,E] dtype (any E from 1 to 1024; rows need no alignment beyond the
 * element's), bias [E] float32 or NULL; topk_idx [T,K] int32 and topk_weights
 * [T,K] float32 are written.  MOE_ERR_INVALID_ARG for options out of range,
 * MOE_ERR_SHAPE for K > E, groups that do not divide E or hold fewer than K
 * experts in all, MOE_ERR_UNSUPPORTED beyond the limits above and for more
 * than 2^26 - 4 tokens.  T = 0 is valid.                                    */
int moe_route(const void* logits, int dtype, int64_t T, int E, int K, const moe_route_options* options,
              const float* bias, int32_t* topk_idx, float* topk_weights, hipStream_t stream);

/* Backward of moe_route: grad_logits[t,:] from the gradient of the weights,
 * for the choice topk_idx (the choice itself has no gradient, and neither has
 * the bias).  With G_k = scale * grad_weights[t,k], s the token's scores:
 *   softmax:               dz_j = s_j (sum_k [idx_k = j] G_k - sum_k s_k G_k)
 *   softmax, renormalised: dz at idx_k = q_k (G_k - sum_m q_m G_m), q = s / sum of the chosen s
 *   sigmoid:               dz at idx_k = G_k s_k (1 - s_k)
 *   sigmoid, renormalised: dz at idx_k = (G_k - sum_m q_m G_m) q_k (1 - s_k)
 * and zero elsewhere.  float32 throughout, rounded once to dtype.  Only the first
 * form reads logits that were not chosen: in the others a NaN there, which makes
 * softmax weights NaN, leaves the gradient as it is.  The same options as the
 * forward call (groups are checked, and have no other part).  An id that repeats
 * within a token adds up; an id outside [0,E) has no part.
 *   logits, grad_logits [T,E] dtype; topk_idx [T,K] int32; grad_weights [T,K]
 *   float32.                                                                 */
int moe_route_bwd(const void* logits, int dtype, int64_t T, int E, int K, const moe_route_options* options,
                  const int32_t* topk_idx, const float* grad_weights, void* grad_logits,
                  hipStream_t stream);

/* ---- balance loss ---------------------------------------------------------------
 * What a router is trained by beside its weights, and how often each expert was
 * chosen.  Tokens form S sequences: q holds tokens seq_offset[q] to
 * seq_offset[q+1] - 1 (ascending; NULL with S = 1: one sequence of all tokens).  A
 * token counts if it lies in a sequence and its token_mask is not 0 (NULL: all do);
 * logits and ids of the others are not read into any result.  With s the token's
 * softmax, or its sigmoids divided by their sum, n_q the counted tokens of q, n all
 * of them and S' the sequences with at least one:
 *   counts[q,e] = pairs (t,k) of q's counted tokens with topk_idx[t,k] = e
 *   probs[q,e]  = sum of s[t,e] over them,   tokens[q] = n_q
 *   loss[0] = 1/S' sum_q E / (K n_q^2) sum_e counts[q,e] probs[q,e]
 *   loss[1] = 1/n sum_t lse(z_t)^2       (the z loss, of the logits for both scores)
 * loss[0] is 1 where experts are chosen evenly.  Scores and lse in 32 bits, sums over
 * tokens in a fixed order (bitwise reproducible), the last of them in 64.  A sequence
 * without counted tokens has no part; with none at all both losses are 0.  Ids
 * outside [0,E) are not counted.  A token whose scores are all zero (its logits all
 * -inf, or for sigmoids below -708) has s = 0 and, if all are -inf, no part in
 * loss[1]; NaN or +inf logits spread as the formulas say (with +inf the token's softmax
 * is NaN and its lse +inf).
 *   logits [T,E] dtype (any E from 1 to 1024), topk_idx [T,K] int32 or int64,
 *   seq_offset [S+1] int32 on the device, token_mask [T] bytes; loss [2], counts
 *   [S,E], probs [S,E], tokens [S] are written; workspace 256-byte aligned,
 *   moe_balance_workspace_size bytes (one per call in flight).
 * T = 0 is valid: zeros.  MOE_ERR_UNSUPPORTED for more than 2^26 - 4 tokens or
 * MOE_MAX_SEQUENCES sequences.                                               */
#define MOE_MAX_SEQUENCES 65535
int moe_balance_workspace_size(int64_t T, int E, int64_t S, size_t* bytes);
int moe_balance(const void* logits, int dtype, int64_t T, int E, const void* topk_idx, int itype, int K,
                const int32_t* seq_offset, int64_t S, const uint8_t* token_mask, int score, float* loss,
                int32_t* counts, float* probs, int32_t* tokens, void* workspace, size_t workspace_bytes,
                hipStream_t stream);

/* Gradient of moe_balance: grad_logits[t,:] from grad_loss [2] (device), for the
 * counts and tokens that the forward call wrote.  Counts have no gradient.  With
 * a_e = grad_loss[0] E / (S' K n_q^2) counts[q,e]:
 *   softmax: dz_j = s_j (a_j - sum_m s_m a_m),   sigmoid: the same times 1 - sigmoid(z_j),
 * plus grad_loss[1] 2/n lse softmax(z)_j.  Tokens that do not count get zero.
 * grad_base [T,E] dtype or NULL is added (the gradient through the router's weights,
 * moe_route_bwd; grad_logits may be grad_base).  float32, rounded once.       */
int moe_balance_bwd(const void* logits, int dtype, int64_t T, int E, int K, const int32_t* seq_offset, int64_t S,
                    const uint8_t* token_mask, int score, const int32_t* counts, const int32_t* tokens,
                    const float* grad_loss, const void* grad_base, void* grad_logits, hipStream_t stream);

/* ---- expert layer for a few tokens ---------------------------------------------
 * The whole layer of a decode step, without a layout, a dispatch or a combine:
 *   act[t,k] = f(Wg_e x[t]) * (Wu_e x[t]),   e = topk_idx[t,k]
 *   out[t]   = round(sum_k w[t,k] * (W2_e act[t,k]))
 * with Wg the first I and Wu the last I rows of w13[e], f(g) = g / (1 +
 * exp(-g)) (MOE_ACT_SILU) or the tanh form of gelu (MOE_ACT_GELU_TANH).
 * float32 sums; act stays float32, in the second product too; the sum over k
 * runs in k order from +0.0, products and sums rounded on their own.  Results
 * are bitwise reproducible.  Only the chosen experts' weights are read.
 *
 *   x [T,H], w13 [E,2I,H], w2 [E,H,I], out [T,H] dtype, 16-byte aligned;
 *   topk_idx [T,K] int32 or int64; topk_weights [T,K] float32, or NULL for a
 *   plain sum; workspace 256-byte aligned, moe_few_workspace_size bytes (one
 *   per call in flight: calls that overlap in time must not share it).
 * An id outside [0,E) is no expert of this call and adds nothing (the ids of
 * other ranks' experts in an expert-parallel layer); a token without an
 * expert gets a zero row.  The same id may repeat within a token.
 * MOE_ERR_UNSUPPORTED above MOE_FEW_MAX_PAIRS pairs (larger batches go through
 * moe_layout, moe_dispatch and moe_combine) and for H or I above 2^18,
 * MOE_ERR_SHAPE for rows of H or I that are not whole 16-byte chunks.  T = 0
 * is valid.  K may exceed E.                                                */
#define MOE_FEW_MAX_PAIRS 512
enum moe_activation { MOE_ACT_SILU = 0, MOE_ACT_GELU_TANH = 1 };

int moe_few_workspace_size(int dtype, int64_t T, int K, int64_t I, size_t* bytes);
int moe_few(const void* x, int dtype, int64_t T, int64_t H, const void* topk_idx, int itype, int K,
            const float* topk_weights, const void* w13, const void* w2, int E, int64_t I, int activation,
            void* out, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ---- low-rank adapters -----------------------------------------------------------
 * Adapters of many requests at once, beside a projection that they share: each
 * token has one adapter, or none, and the layout groups the tokens by adapter
 * (moe_layout with K = 1, the adapter's number as the expert id and E >= the
 * number of adapters).  Tokens whose id is num_adapters or above (below E)
 * have no adapter.  One layout serves every projection of a batch.
 *   u[p]   = a_e x[t]                   p = recv_pos[t], e the token's adapter
 *   out[t] = round(base[t] + w[t] * (u[p] b_e))
 * w = topk_weights, or 1 where NULL; base, the shared projection's output, or
 * 0 where NULL; for a token without an adapter out = base and u = 0.  Sums and
 * u in float32, in the second product too, one rounding at the end; results
 * are bitwise reproducible.
 *
 *   x [T,H], a [num_adapters,r,H], b [num_adapters,r,N], base and out [T,N]
 *   dtype, 16-byte aligned (out may be base); topk_weights [T,1] float32; u
 *   [R,r] float32, written, 16-byte aligned (rows in receive order; moe_lowrank_bwd takes it).
 * MOE_ERR_SHAPE unless the layout has K = 1 and E >= num_adapters, and rows of
 * H, N and r are whole 16-byte chunks (a smaller rank is padded with zero
 * rows); MOE_ERR_UNSUPPORTED for r > MOE_MAX_RANK, H or N above 2^20 or more
 * than 2^26 receive rows.  A token whose id the layout found outside [0, E) is
 * an input error there; its rows of out (and of grad_x and grad_w below) are
 * not written, and the other tokens' are what they would be without it.  Rows
 * of u past expert_offset[E] are not written.                               */
#define MOE_MAX_RANK 128
int moe_lowrank(moe_handle_t h, const void* x, int dtype, int64_t H, const void* a, const void* b,
                int num_adapters, int rank, int64_t N, const float* topk_weights, const void* base, void* out,
                float* u, hipStream_t stream);

/* Backward of moe_lowrank, on the forward's layout and u.  With g = grad_out,
 * raw[p] = b_e g[t] and gu[p] = w[t] * raw[p]:
 *   grad_x[t] = round(grad_base[t] + gu[p] a_e)     (grad_base: 0 where NULL)
 *   grad_a[e] = round(sum_p gu[p]^T x[t]),  grad_b[e] = round(sum_p w[t] u[p]^T g[t])
 *   grad_w[t] = <raw[p], u[p]>
 * Any of the four outputs may be NULL, not all (grad_w needs no topk_weights:
 * it is then the gradient at w = 1).  An adapter without tokens gets zero
 * gradients, a token without an adapter grad_x = grad_base and grad_w = 0.
 * grad_base, added to grad_x, is the gradient that reaches x through the
 * shared projection; grad_x may be grad_base.  (The gradient of base is
 * grad_out itself.)
 *   grad_out [T,N], x [T,H], a, b as above, grad_x, grad_base [T,H], grad_a
 *   [num_adapters,r,H], grad_b [num_adapters,r,N] dtype; u as the forward call
 *   wrote it; grad_w [T,1] float32; workspace 16-byte aligned, at
 *   least R * r * 4 bytes (not needed for grad_b alone; one per call in
 *   flight).  With T = 0 grad_a and grad_b are set to zero.
 * moe_lowrank_bwd_workspace_size gives the size at which few adapters with
 * many tokens each have their gradients summed in parts, which is faster (the
 * order of the sum then depends on the shapes, not on timing); with a smaller
 * workspace they are summed in one.  A function of the shapes only.         */
int moe_lowrank_bwd_workspace_size(moe_handle_t h, int dtype, int64_t H, int64_t N, int num_adapters, int rank,
                                   size_t* bytes);
int moe_lowrank_bwd(moe_handle_t h, const void* grad_out, int dtype, int64_t H, const void* x, const void* a,
                    const void* b, int num_adapters, int rank, int64_t N, const float* topk_weights,
                    const float* u, const void* grad_base, void* grad_x, void* grad_a, void* grad_b,
                    float* grad_w, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ---- products in 8-bit integers -----------------------------------------------------
 * The experts' products for more than a few tokens, between the layout and the
 * combine, in 8-bit integers with a scale for each row and each channel.
 *
 * moe_quant_rows: scale[m] = max(amax |x[m,:]| / 127, 2^-126) in float32, q[m,k] =
 * the integer nearest to x[m,k] / scale[m], ties to even, within [-127, 127].  A row
 * with an infinity or NaN gets that as its scale and zeros in q, so that products
 * with it are NaN.  x [rows,width] dtype, q [rows,width] int8, 16-byte aligned;
 * scale [rows] float32.  Weights are laid out the same way: a bank [E,N,width] is
 * E*N rows.  MOE_ERR_SHAPE unless width is a multiple of 16, MOE_ERR_UNSUPPORTED
 * above MOE_MAX_I8_WIDTH (where 32-bit sums could overflow) and for more than
 * 2^26 - 4 rows.
 *
 * moe_matmul_i8: with acc the exact integer sum, for the receive rows p of the
 * experts first_expert .. first_expert + num_experts - 1 of the layout,
 *   y[p,n] = float(acc) * scale[r] * w_scale[e,n],   acc = sum_k q[r,k] w[e,n,k]
 *   out[p] = round(y[p])                             (MOE_ACT_NONE: N columns)
 *   out[p] = round(f(y[p,:N/2]) * y[p,N/2:])         (MOE_ACT_SILU, MOE_ACT_GELU_TANH)
 * in float32.  tokens 1: q and scale hold token rows [T,width], and r is the token
 * of p (no dispatch is needed; a row of a padded layout without a token gives
 * zeros).  tokens 0: they hold receive rows [R,width], r = p.  Rows of other experts
 * and past the layout's last are not written; out has R rows.  h NULL: one expert
 * on all `rows` rows, q [rows,width], out [rows, ..] (a shared expert).
 *   q [rows,width], w [num_experts,N,width] int8 (any values), out 16-byte aligned;
 *   scale [rows], w_scale [num_experts,N] float32; out_dtype MOE_F32 or MOE_BF16.
 * rows must be T or R of the layout; T = 0 is valid.  MOE_ERR_SHAPE for a width that
 * is not a multiple of 16 or rows of out that are not whole 16-byte chunks;
 * MOE_ERR_UNSUPPORTED above MOE_MAX_I8_WIDTH, for N above 2^20, an expert's weights
 * of 2 GiB, token rows of nearly 4 GiB and more than 2^26 receive rows.  Results
 * are bitwise reproducible.  Neither call has a gradient.                       */
#define MOE_MAX_I8_WIDTH 131056
#define MOE_ACT_NONE (-1)
int moe_quant_rows(const void* x, int dtype, int64_t rows, int64_t width, int8_t* q, float* scale, hipStream_t stream);
int moe_matmul_i8(moe_handle_t h, const int8_t* q, const float* scale, int64_t rows, int64_t width, int tokens,
                  const int8_t* w, const float* w_scale, int num_experts, int first_expert, int64_t N, int activation,
                  void* out, int out_dtype, hipStream_t stream);

/* ---- norms before and after a block --------------------------------------------------
 * With rms(v) = v / sqrt(mean(v^2) + eps) over the row and w' = w + offset (offset 1
 * for weights stored as their distance from 1, else 0):
 *   moe_prenorm:   n = round(rms(x) w')
 *   moe_postnorm:  z = residual_scale x + gate * (rms(y) weight'),   out = round(z)
 *                  n = round(rms(z) next_weight')      (the next block's norm)
 * weight NULL: no norm after the block (y as it is); next_weight and n NULL: none of
 * the next block.  gate [gates,H]: gate g belongs to tokens g*T/gates to
 * (g+1)*T/gates - 1 (gates divides T; one for all, one for each sequence or one for
 * each token); NULL with gates 0: 1.  float32, each output rounded once; n is formed
 * from z before its rounding.  moe_prenorm leaves 8-bit rows instead where q is given
 * (then n is NULL, H a multiple of 16): q and scale as moe_quant_rows makes them of
 * the rows before rounding.
 * With a handle moe_postnorm combines on the way: y holds receive rows [R,H], and
 * sum_k [topk_weights[t,k] *] y[recv_pos[t,k]] takes their place, in float32, in k
 * order, not rounded.  T must be the layout's.
 *   x, y, out, n, gate, weights dtype, 16-byte aligned, rows whole 16-byte chunks of
 *   at most MOE_MAX_NORM_BYTES; out may be x (and y without a handle), n neither;
 *   rstd float32 or NULL: 1 / sqrt(mean + eps), [T] of x for moe_prenorm, [T,2]
 *   (8-byte aligned) of y and z for moe_postnorm (1 where there is no norm), what the
 *   backward passes take.  eps > 0.  T = 0 is valid; MOE_ERR_UNSUPPORTED above 2^26. */
#define MOE_MAX_NORM_BYTES 65536
#define MOE_NORM_WIDE 8192 /* moe_postnorm_bwd needs its workspace for every row wider than this */
int moe_prenorm(const void* x, int dtype, int64_t T, int64_t H, const void* weight, float offset, float eps, void* n,
                int8_t* q, float* scale, float* rstd, hipStream_t stream);
int moe_postnorm(moe_handle_t h, const void* x, const void* y, int dtype, int64_t T, int64_t H,
                 const float* topk_weights, const void* weight, const void* gate, int64_t gates, float residual_scale,
                 const void* next_weight, float offset, float eps, void* out, void* n, float* rstd,
                 hipStream_t stream);

/* Backward of the norms.  With v^ = v * rstd:
 *   moe_prenorm_bwd:   grad_x = grad_base + rstd (w' grad_n - x^ mean(w' grad_n x^)),
 *                      grad_weight = sum_t grad_n x^   (grad_base NULL: 0)
 *   moe_postnorm_bwd:  d = grad_out + rstd_z (next' grad_n - z^ mean(next' grad_n z^)),
 *     grad_x = residual_scale d,   grad_next_weight = sum_t grad_n z^,   u = gate d,
 *     grad_gate[g] = sum over its tokens of d rms(y) weight',
 *     grad_y = rstd_y (weight' u - y^ mean(weight' u y^)),  grad_weight = sum_t u y^
 * in float32, rounded once, z formed again from x and y; sums over tokens in a fixed
 * order that depends on the shapes alone.  y is the rows of tokens (after moe_combine
 * where there is a layout; its own backward pass takes grad_y).  Any output may be
 * NULL, not all; grad_out or grad_n may be NULL (0), not both; x is read only with
 * grad_n, y only with grad_n, a norm of it or grad_gate.  grad_x may be grad_out.
 * workspace (16-byte aligned, moe_norm_bwd_workspace_size bytes; one per call in flight)
 * is not needed without a sum over tokens, of rows after a block of at most MOE_NORM_WIDE
 * elements.  With T = 0 those sums are set to zero.                               */
int moe_norm_bwd_workspace_size(int dtype, int64_t T, int64_t H, int64_t gates, size_t* bytes);
int moe_prenorm_bwd(const void* grad_n, const void* x, int dtype, int64_t T, int64_t H, const void* weight, float offset,
                    const float* rstd, const void* grad_base, void* grad_x, void* grad_weight, void* workspace,
                    size_t workspace_bytes, hipStream_t stream);
int moe_postnorm_bwd(const void* grad_out, const void* grad_n, const void* x, const void* y, int dtype, int64_t T,
                     int64_t H, const float* rstd, const void* weight, const void* gate, int64_t gates,
                     float residual_scale, const void* next_weight, float offset, void* grad_x, void* grad_y,
                     void* grad_weight, void* grad_gate, void* grad_next_weight, void* workspace,
                     size_t workspace_bytes, hipStream_t stream);

/* Device pointer and byte size of one handle field (no synchronisation). */
int moe_handle_field(moe_handle_t h, int field, void** dev_ptr, size_t* bytes);

/* Shape recorded by the last moe_layout on this handle. */
int moe_handle_dims(moe_handle_t h, int64_t* T, int* K, int* E, int* P);

/* Synchronises `stream`, then reads the device status word (MOE_STATUS_* bits). */
int moe_handle_check(moe_handle_t h, hipStream_t stream, int* device_status);

/* ---- CU budget -------------------------------------------------------------
 * A stream whose kernels may run only on compute units [cu_first, cu_first +
 * cu_count) of the current device (a hardware CU mask; default priority).
 * The exchange calls issued on it use at most that many CUs, and a GEMM on a
 * stream with the other CUs runs beside them: the analogue of the SM budget
 * of the pages' transport kernels ("Add an opt-in DeepEP transport for the
 * AutoEP expert all-to-all", section "Choosing the SM budget": too few SMs
 * slow the exchange itself and too many slow the GEMMs beside it, so the
 * budget is a whole-step trade-off; the page's follow-up work lists
 * overlapping the exchange with compute).  CU
 * indices are the HIP runtime's, numbered round-robin over the XCDs, so a
 * range of consecutive indices spreads evenly over them; the runtime refuses
 * a mask that leaves an XCD without a CU, so cu_count is at least the XCD
 * count (8 on MI355X).  MOE_ERR_INVALID_ARG for a NULL out, cu_first < 0 or
 * cu_count < 1; MOE_ERR_SHAPE if the range passes the device's CU count or
 * holds fewer CUs than XCDs; MOE_ERR_HIP if the runtime refuses.  Destroy
 * with moe_stream_destroy.                                                 */
int moe_stream_create_cu_budget(int cu_first, int cu_count, hipStream_t* out);
int moe_stream_destroy(hipStream_t stream);

/* Message for a status code (static string). */
const char* moe_strerror(int status);

/* Library version string. */
const char* moe_version(void);

#ifdef __cplusplus
}
#endif
#endif /* MOE_LAYOUT_H */
