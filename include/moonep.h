/*
 * moonep.h -- C-ABI of the MI355X (gfx950) balanced expert-parallel hot path.
 *
 * What is computed follows these pages:
 *   [NCIJ]  "Moonshot AI Open-Sources MoonEP: A Perfectly Balanced Expert
 *           Parallelism Library for MoE Training" (ncijnetwork.com), sections
 *           "The problem MoonEP targets" and "The core idea: dynamic redundant
 *           experts", the three-property list, and the interactive explainer
 *           (panels "invariant", "memory", "maxvio", "pillars").
 *   [AIPDB] "Moonshot AI open-sources MoonEP for distributed MoE
 *           communication" (aipricedb.com), the README excerpt on zero copy.
 *
 * Model.  R ranks hold E experts, L = E/R each; expert e lives on rank
 * home(e) = e div L.  Each rank has S tokens and each token is routed to K
 * experts, so rank r's routed entries are n = (r*S + t)*K + k.  Every rank
 * receives exactly C = S*K rows whatever the routing skew [NCIJ "The core
 * idea"]: overfull ranks hand whole-expert amounts (lowest expert id first)
 * to redundant copies ("replicas") of those experts hosted on underfull ranks,
 * matched two-pointer in expert order against the deficits in rank order.
 * The R ranks are logical: rank r's [C, H] bf16 buffer is rows [r*C, (r+1)*C)
 * of one device allocation.
 *
 * A step.  Forward: moonep_router (ids and gates from the router's logits, and
 * the balance loss), moonep_route_stats, moonep_plan, moonep_weight_slots and
 * moonep_prefetch_weights (the replicas' weights), moonep_dispatch, the expert
 * computation over the buffer (moonep_expert_gemm per projection, with the
 * caller's activation between projections), moonep_combine.  Backward:
 * moonep_combine_bwd, the expert's backward (moonep_expert_gemm_dx and
 * moonep_expert_gemm_dw per projection, with the caller's backward of the
 * activation in between), moonep_dispatch_bwd, moonep_router_bwd (d_gates and the
 * loss to the logits), moonep_replica_grad_reduce for the replicas'
 * weight-gradients, and moonep_grad_clip over all gradients.
 *
 * Low-rank adapters of many requests or tenants stand beside any projection that
 * all rows share: moonep_adapter adds them to its output, moonep_adapter_bwd
 * gives their gradients.
 *
 * An 8-bit forward, for serving: moonep_rmsnorm_quant (the residual stream to
 * 8-bit token rows, with the bf16 rows for the router), moonep_router,
 * moonep_plan, moonep_prefetch_weights over 8-bit weight rows
 * (moonep_quant_weights wrote them once), moonep_dispatch_quant,
 * moonep_expert_glu_quant (gate, up and the activation), moonep_expert_gemm_quant
 * (down), moonep_combine.
 *
 * Conventions shared by every call:
 *  - All array arguments are DEVICE pointers owned by the caller; the library
 *    allocates nothing.  Between calls it keeps only the CU's LDS size (read
 *    once per process) and, per device, whether a kernel's dynamic-LDS limit has
 *    been raised (one forward product's for large E and R, the 8-bit ones', the
 *    experts' gradients', the adapters' gradients' above rank 32).
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream).  Every
 *    call only enqueues work; none waits for the device, except
 *    moonep_read_error.  Output sizes depend on the shape alone, so no call
 *    needs to read device results on the host [NCIJ explainer "invariant"
 *    panel: static shapes, no per-layer host synchronisation].
 *  - Return value: MOONEP_OK, or a negative MOONEP_ERR_* found on the host
 *    before anything is enqueued (or MOONEP_ERR_HIP if a launch fails).
 *  - Device-side faults in the data (an expert id outside [0, E)) set a sticky
 *    error word in the workspace; read it with moonep_read_error.  Outputs of a
 *    call that saw bad data are unspecified, but every access stays in bounds.
 *  - bf16 arrays are raw 16-bit patterns (uint16_t) and must be 16-byte aligned;
 *    int32/fp32 arrays must be 4-byte aligned.
 */
#ifndef MOONEP_H
#define MOONEP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct moonep_shape {
    int32_t R; /* ranks (logical), >= 1 */
    int32_t E; /* experts, E % R == 0 [NCIJ explainer warns otherwise], E <= 1024 */
    int32_t S; /* tokens per rank, >= 0 */
    int32_t K; /* experts per token, 1 <= K <= E */
    int32_t H; /* hidden size; H % 8 == 0, H >= 8 */
} moonep_shape;

enum {
    MOONEP_OK = 0,
    MOONEP_ERR_INVALID_SHAPE = -1, /* a shape rule above, or R*S*K >= 2^31 */
    MOONEP_ERR_NULL_PTR = -2,      /* a required pointer is NULL */
    MOONEP_ERR_MISALIGNED = -3,    /* alignment rule above */
    MOONEP_ERR_WORKSPACE = -4,     /* workspace smaller than moonep_workspace_bytes */
    MOONEP_ERR_HIP = -5,           /* a HIP launch or copy failed */
    MOONEP_ERR_ALIAS = -6,         /* forbidden aliasing between arguments */
    MOONEP_ERR_ARG = -7            /* other invalid argument (e.g. G < 0) */
};

/* Device error word values (moonep_read_error). */
enum { MOONEP_DEV_OK = 0, MOONEP_DEV_BAD_EXPERT_ID = 1 };

/* Returns MOONEP_OK if the shape satisfies every rule above. */
int moonep_check_shape(const moonep_shape *shape);

/*
 * Bytes of scratch the caller provides to moonep_route_stats and moonep_plan
 * (the same buffer to both, in that order).  It holds per-segment expert counts
 * and the device error word.  Zero it once when it is allocated; the calls
 * keep it consistent afterwards.  One workspace serves one route_stats ->
 * plan sequence at a time: sequences that may overlap (on different streams)
 * need workspaces of their own, since they would share its counts.  Returns 0
 * for an invalid shape.
 */
size_t moonep_workspace_bytes(const moonep_shape *shape);

/*
 * The replica plan: a fixed-capacity int32 table, cap = E + R replicas (the
 * greedy never needs more than E - L).  Word offsets of its fields:
 */
typedef struct moonep_plan_layout {
    int32_t words;          /* total int32 words of the plan */
    int32_t cap;            /* replica capacity, E + R */
    int32_t header;         /* [16]: see MOONEP_PLAN_H_* */
    int32_t rep_expert;     /* [cap] expert of replica j (plan order) */
    int32_t rep_host;       /* [cap] rank that hosts replica j */
    int32_t rep_count;      /* [cap] rows replica j receives (> 0 for j < n_rep) */
    int32_t rep_spill_off;  /* [cap] offset of j's first entry among its expert's spilled ones */
    int32_t rep_row_off;    /* [cap] first row of replica j in its host's buffer */
    int32_t spill;          /* [E] entries expert e hands to replicas */
    int32_t keep;           /* [E] entries expert e keeps at home = T_e - spill_e */
    int32_t home_row_off;   /* [E] first row of expert e in its home rank's buffer */
    int32_t rep_first;      /* [E] first replica id of expert e (0 if none) */
    int32_t rep_cnt;        /* [E] number of replicas of expert e */
    int32_t exp_rep_list;   /* [E] experts with replicas, ascending (first header[N_SPILL]) */
    int32_t load;           /* [R] rows routed to rank r's home experts before balancing */
    int32_t rank_rep_first; /* [R] first replica id hosted by rank r (0 if none) */
    int32_t rank_rep_cnt;   /* [R] replicas hosted by rank r */
} moonep_plan_layout;

enum {
    MOONEP_PLAN_H_N_REP = 0,     /* replicas in this plan */
    MOONEP_PLAN_H_N_SPILL = 1,   /* experts with replicas */
    MOONEP_PLAN_H_N_DEFICIT = 2, /* ranks below C before balancing */
    MOONEP_PLAN_H_MAX_REP_RANK = 3, /* most replicas hosted by one rank */
    MOONEP_PLAN_H_TMAX = 4,      /* largest expert count */
    MOONEP_PLAN_H_C = 5,         /* rows per rank, S*K */
    MOONEP_PLAN_H_L = 6,         /* experts per rank, E/R */
    MOONEP_PLAN_H_CAP = 7        /* E + R */
};

int moonep_plan_layout_of(const moonep_shape *shape, moonep_plan_layout *layout);
size_t moonep_plan_bytes(const moonep_shape *shape); /* layout.words * 4, 0 if invalid */

/*
 * Route statistics [NCIJ "The problem MoonEP targets"; explainer "maxvio"
 * panel].  topk_idx: int32 [R*S*K], entry n = (r*S + t)*K + k, each in [0, E).
 * Writes expert_counts[e] = T_e (int32 [E]) and maxvio[0] =
 * fp32((Tmax*E)/(R*S*K) - 1) computed in IEEE double (0 when R*S*K == 0), and
 * per-segment counts into the workspace for moonep_plan.
 */
int moonep_route_stats(const moonep_shape *shape, const int32_t *topk_idx, int32_t *expert_counts,
                       float *maxvio, void *workspace, size_t workspace_bytes, void *stream);

/*
 * The replica plan and the slot maps [NCIJ "The core idea" and the
 * three-property list: exactly S*K rows per rank, tokens written straight
 * into expert-grouped rows; explainer "memory" panel: home rows precede
 * prefetch rows].  Must follow moonep_route_stats on the same topk_idx,
 * expert_counts and workspace (stream order).  Writes:
 *   plan        int32 [moonep_plan_bytes/4], layout above; unused replica
 *               entries are 0;
 *   slot_of     int32 [R*S*K]: destination row of entry n, rank*C + row.
 *               Within an expert, entries keep (src rank, token, k) order: the
 *               first keep_e rows stay home, the rest fill its replicas in plan
 *               order.  Rank d's buffer holds its home experts ascending (each
 *               keep_e rows), then the replicas it hosts in plan order;
 *   src_of_slot int32 [R*S*K]: the inverse map, entry placed at each row.
 * With a bad expert id (see the workspace error word) affected entries get
 * slot_of = -1.
 */
int moonep_plan(const moonep_shape *shape, const int32_t *topk_idx, const int32_t *expert_counts,
                void *workspace, size_t workspace_bytes, int32_t *plan, int32_t *slot_of,
                int32_t *src_of_slot, void *stream);

/*
 * The same plan and slot maps with fewer replicas [NCIJ three-property list:
 * a "near-optimal" planning kernel; the pages give no algorithm].  Identical
 * to moonep_plan (arguments, layouts, errors, and the route_stats call that
 * must precede it) except for which entries an overfull rank gives up: it
 * takes whole-expert amounts starting at its LARGEST expert count (ties to the
 * lower expert id) rather than its lowest id, which sheds the excess through
 * the fewest experts.  Each spilling expert is one entry of the spill list
 * that the two-pointer walk matches, so the plan needs fewer replicas: 32
 * instead of 61 on a DeepSeek-V3-like routing (R = 32, E = 256, Zipf 1.2),
 * each replica being one expert's weights to prefetch and one gradient to
 * reduce.  Entry order is as in moonep_plan: an expert's first keep_e
 * entries stay home, the rest fill its replicas in plan order.
 */
int moonep_plan_largest_first(const moonep_shape *shape, const int32_t *topk_idx,
                              const int32_t *expert_counts, void *workspace,
                              size_t workspace_bytes, int32_t *plan, int32_t *slot_of,
                              int32_t *src_of_slot, void *stream);

/*
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the work of
 * moonep_route_stats followed by moonep_plan, with the workspace replaced by a
 * scratch array inside the library, MOONEP_NOALLOC_SCRATCH_BYTES per device
 * (enough for every valid shape), held until the process ends.  Allocates
 * nothing.  Writes expert_counts, maxvio, plan, slot_of and src_of_slot
 * exactly as those two calls do.  Every call on one device shares that
 * device's scratch and leaves its contents behind (nothing in it must start
 * at zero between calls), so calls that overlap on one device -- other
 * streams, other host threads -- race and must be ordered by the caller.  An
 * expert id outside [0, E) gives its entries slot_of = -1 as in moonep_plan;
 * the scratch's error word cannot be read with moonep_read_error.  Returns
 * MOONEP_ERR_WORKSPACE if a shape needed more scratch than the array holds,
 * MOONEP_ERR_HIP if the scratch's device address cannot be obtained.
 */
enum { MOONEP_NOALLOC_SCRATCH_BYTES = 256 + 4 * 1024 * 2048 };
int moonep_plan_noalloc(const moonep_shape *shape, const int32_t *topk_idx, int32_t *expert_counts,
                        float *maxvio, int32_t *plan, int32_t *slot_of, int32_t *src_of_slot,
                        void *stream);

/*
 * Dispatch, the fused permute [NCIJ three-property list, zero copy; AIPDB].
 * x: bf16 [R*S, H] token rows.  buf: bf16 [R*S*K, H], the R static [S*K, H]
 * per-rank buffers [NCIJ explainer "invariant" panel] back to back.
 * buf[slot_of[n]] = x[n div K], a bit copy.  Rows whose slot_of is outside
 * [0, R*S*K) are skipped.  buf must not overlap x.
 */
int moonep_dispatch(const moonep_shape *shape, const uint16_t *x, const int32_t *slot_of,
                    uint16_t *buf, void *stream);

/*
 * Combine, the fused weighted unpermute [NCIJ three-property list and
 * explainer "pillars" panel].  expert_out: bf16 [R*S*K, H] rows in buffer
 * order (may be the dispatch buffer itself); gates: fp32 [R*S*K].
 * y[t] = bf16(sum over k ascending of gates[t*K+k] * expert_out[slot_of[t*K+k]]).
 * Each fp32 x bf16 product is exact in fp64; the products are summed in fp64
 * in ascending k from +0 and the sum is rounded once to bf16 (to nearest
 * even), for terms of any sign.  Out-of-range slots contribute nothing.
 * y: bf16 [R*S, H], must not overlap expert_out.
 */
int moonep_combine(const moonep_shape *shape, const uint16_t *expert_out, const float *gates,
                   const int32_t *slot_of, uint16_t *y, void *stream);

/*
 * Combine backward (the training backward of combine; [NCIJ "The core idea"]).
 * dy: bf16 [R*S, H].  Writes
 *   d_out[slot_of[n]] = bf16(gates[n] * dy[n div K])  (one correct rounding of
 *                       the exact product), bf16 [R*S*K, H];
 *   d_gates[n] = sum_h dy[n div K, h] * expert_out[slot_of[n], h]  (fp32
 *                       accumulation), fp32 [R*S*K].
 * d_out must not overlap dy or expert_out.
 */
int moonep_combine_bwd(const moonep_shape *shape, const uint16_t *dy, const uint16_t *expert_out,
                       const float *gates, const int32_t *slot_of, uint16_t *d_out,
                       float *d_gates, void *stream);

/*
 * Dispatch backward (the training backward of dispatch; [NCIJ "The core
 * idea"]).  d_buf: bf16 [R*S*K, H], the gradient of the dispatch buffer rows.
 * dx[t] = bf16(sum over k ascending of d_buf[slot_of[t*K+k]]), the sum taken in
 * fp64 and rounded once (to nearest even).  dx: bf16 [R*S, H], must not overlap
 * d_buf.  Out-of-range slots contribute nothing.
 */
int moonep_dispatch_bwd(const moonep_shape *shape, const uint16_t *d_buf, const int32_t *slot_of,
                        uint16_t *dx, void *stream);

/*
 * Replica-gradient reduction [NCIJ "The core idea": replica gradients return
 * to their home experts; explainer "memory" panel: they sit in an fp32 reduce
 * buffer that is pulled home and then zeroed for the next microbatch].
 * home_grads: fp32 [E, G]; replica_grads: fp32 [E + R, G], row j = replica j of
 * `plan` (plan order).  For every expert e with replicas:
 *   home[e] = fp32(home[e] + rep[j1] + rep[j2] + ...)  (fp64 sum, plan order),
 * then rep[j] = +0 for every j < n_rep.  Other rows are not touched.  G >= 0;
 * the two arrays must not overlap.
 */
int moonep_replica_grad_reduce(const moonep_shape *shape, const int32_t *plan, int64_t G,
                               float *home_grads, float *replica_grads, void *stream);

/*
 * Replica weight slots [NCIJ "The core idea": redundant experts are
 * prefetched before expert compute; explainer "memory" panel: each rank owns B
 * prefetch slots, the rows that follow the expert rows of its weight tensor;
 * training needs B = E/R, inference may use fewer (3-4 suggested), and a rank
 * that hosts more than B replicas reads the extra ones from their home rank].
 * Writes wslot: int32 [E + R], for replica j < n_rep of `plan` hosted on rank
 * d as its b-th in plan order: wslot[j] = d*B + b when b < B, else -1
 * (overflow: that replica's weights are read at the home expert's row).
 * Entries j >= n_rep are -1.  The plan is not changed.  B >= 0 and
 * R*B < 2^31, else MOONEP_ERR_ARG.
 */
int moonep_weight_slots(const moonep_shape *shape, const int32_t *plan, int32_t B, int32_t *wslot,
                        void *stream);

/*
 * Replica weight prefetch [same passages].  w_home: [E, wbytes] bytes, row e =
 * every weight of expert e (e.g. its gate, up and down projections, in any
 * layout the caller chooses); pool: [R*B, wbytes] bytes, row d*B + b = slot b
 * of rank d.  For every j < n_rep with 0 <= wslot[j] < R*B:
 *   pool[wslot[j]] = w_home[rep_expert[j]]  (a bit copy).
 * Other pool rows are not touched.  wbytes % 16 == 0 (MOONEP_ERR_ARG);
 * w_home and pool 16-byte aligned; they must not overlap.  wslot normally
 * comes from moonep_weight_slots with the same B; slots that two replicas
 * share would race.
 */
int moonep_prefetch_weights(const moonep_shape *shape, const int32_t *plan, const int32_t *wslot,
                            int32_t B, int64_t wbytes, const void *w_home, void *pool,
                            void *stream);

/*
 * Expert compute over the expert-grouped buffer: one projection, a grouped
 * GEMM [NCIJ three-property list: buffer views go straight to the
 * computation, each rank's rows grouped by expert; explainer "memory" panel:
 * replicas read their prefetch slot, or the home expert past B slots].
 * x: bf16 [R*S*K, in_dim], the buffer rows (e.g. the dispatch buffer);
 * y: bf16 [R*S*K, out_dim].  For buffer row r of rank d = r div (S*K):
 *   y[r, n] = bf16( sum_k x[r, k] * W[n, k] )  (fp32 accumulation on the
 *             matrix cores, one rounding to nearest even),
 * where W is the [out_dim, in_dim] row-major matrix starting at element
 * w_offset of the weight row of r's segment: w_home + e*w_stride for a home
 * expert e; for replica j, pool + wslot[j]*w_stride when 0 <= wslot[j] < R*B,
 * else w_home + rep_expert[j]*w_stride.  w_home holds E weight rows, pool R*B
 * (the layouts of moonep_prefetch_weights, counted in bf16 elements here).
 * Limits (else MOONEP_ERR_ARG): in_dim % 64 == 0, in_dim <= 2^22, out_dim % 128 == 0,
 * w_stride and w_offset multiples of 8, w_offset + out_dim*in_dim <= w_stride.
 * x, y, w_home, pool 16-byte aligned; y must not overlap x, w_home or pool.
 */
int moonep_expert_gemm(const moonep_shape *shape, const int32_t *plan, const int32_t *wslot,
                       int32_t B, int32_t in_dim, int32_t out_dim, const uint16_t *x,
                       const uint16_t *w_home, const uint16_t *pool, int64_t w_stride,
                       int64_t w_offset, uint16_t *y, void *stream);

/*
 * The router: scores of the experts, the K experts and gates of every token,
 * and a balance loss that keeps maxvio low in training.
 *
 * logits: [R*S, E], fp32 or bf16 by opts->logits_type; computed in fp32, scores
 * s_e to (2.5 |x| + 8) 2^-24 relative, x = l_e - max l (softmax) or l_e (sigmoid),
 * and to 0 below 2^-126.  With l the logits of one token,
 *   softmax (MOONEP_SCORE_SOFTMAX): s_e = exp(l_e - max l), Z = sum_e s_e;
 *   sigmoid (MOONEP_SCORE_SIGMOID): s_e = 1 / (1 + exp(-l_e)),
 *                                   Z = sum_e s_e + 1e-20;
 *   p_e = s_e / Z, the token's share of every expert.
 * topk_idx: int32 [R*S*K], the K largest logits of each token, descending, ties
 * to the lower expert id (-0 equals +0), so what moonep_route_stats takes.
 * gates: fp32 [R*S*K], in the same order: scale * s_k / W with
 * W = sum of the K chosen scores (+ 1e-20 with sigmoid) if opts->normalize, else
 * scale * p_k (softmax) or scale * s_k (sigmoid).
 * An expert masked by a logit of -inf has score 0; it is chosen only after all
 * others, with gate 0, and a token whose logits are all -inf has gates and
 * shares 0.  A NaN logit ranks below -inf, and the ids stay distinct and valid;
 * NaN (and, with softmax, +inf) goes through the formulas, where a maximum
 * leaves a NaN out, into the token's shares and gates.
 *
 * Balance loss (all of counts, prob_sum, loss and workspace given; for serving
 * pass NULL for each and it is left out).  The tokens are cut into
 * opts->groups equal runs of n = R*S / groups (1: all tokens; R: the tokens of
 * each rank; R*S / length: each sequence).  For group g,
 *   counts[g, e] = T_ge, int32 [groups, E]: entries routed to e;
 *   prob_sum[g, e] = P_ge = sum of p_e over its tokens, fp32 [groups, E];
 *   loss[0] = mean over g of E / (K n^2) * sum_e T_ge P_ge, fp32: 1 when
 *             counts or shares are uniform.  0 when there are no tokens.
 * Sums over tokens are fp32 within a workgroup's (2048 at most, 128 of them one
 * after the other) and fp64 beyond, in an order that the shape fixes: the same
 * inputs give the same bits.
 *
 * workspace: moonep_router_workspace_bytes, 16-byte aligned, no initial
 * contents needed; one call at a time uses it.  The outputs and the workspace
 * must not overlap the logits or each other.  Limits (MOONEP_ERR_ARG): an
 * unknown score or logits type, groups < 1, R*S % groups != 0,
 * groups > 2^20 or groups * E > 2^24, a scale that is not finite.
 */
enum { MOONEP_SCORE_SOFTMAX = 0, MOONEP_SCORE_SIGMOID = 1 };
enum { MOONEP_F32 = 0, MOONEP_BF16 = 1 };

typedef struct moonep_router_opts {
    int32_t score;       /* MOONEP_SCORE_* */
    int32_t normalize;   /* nonzero: gates of a token sum to scale */
    int32_t groups;      /* runs of tokens the loss is taken over */
    int32_t logits_type; /* MOONEP_F32 or MOONEP_BF16, of logits and d_logits */
    float scale;         /* factor of the gates */
} moonep_router_opts;

/* Bytes of scratch for the balance loss; 0 for an invalid shape or options. */
size_t moonep_router_workspace_bytes(const moonep_shape *shape, const moonep_router_opts *opts);

int moonep_router(const moonep_shape *shape, const moonep_router_opts *opts, const void *logits,
                  int32_t *topk_idx, float *gates, int32_t *counts, float *prob_sum, float *loss,
                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * Router backward: the gradient of the gates (moonep_combine_bwd's d_gates) and
 * of the balance loss with respect to the logits.  topk_idx, counts: as
 * moonep_router wrote them (the ids of one token are distinct; one outside
 * [0, E) contributes nothing).  d_gates: fp32 [R*S*K] or NULL for 0; d_loss:
 * fp32 [1], the gradient of loss[0] (the loss's weight), or NULL with counts
 * NULL for no loss.  With a_e = d_loss E / (K n^2 groups) T_ge and dg the
 * token's d_gates at their experts (0 elsewhere),
 *   ds_e = (a_e - sum_j a_j p_j) / Z
 *          + scale (dg_e - sum_j dg_j s_j / W) / W  for chosen e, normalised;
 *          + scale (dg_e - sum_j dg_j p_j) / Z      softmax, every e;
 *          + scale dg_e                             sigmoid;
 *   d_logits_e = ds_e s_e (softmax) or ds_e s_e (1 - s_e) (sigmoid),
 * rounded once to the logits' type.  The differences of a and of the normalised
 * gates are taken with the mean count and the token's first d_gates off every
 * term, so that what cancels in them (one chosen expert, one that dominates, even
 * counts) leaves no rounding noise.  The counts are constants: choosing has no
 * gradient.  Masked experts and all-masked tokens get 0.  d_logits must not
 * overlap an input.
 */
int moonep_router_bwd(const moonep_shape *shape, const moonep_router_opts *opts,
                      const void *logits, const int32_t *topk_idx, const int32_t *counts,
                      const float *d_gates, const float *d_loss, void *d_logits, void *stream);

/*
 * 8-bit rows.  A value is an OCP e4m3 code (1 byte) times the scale of its
 * block, 128 consecutive columns of one row (fewer at the end of the row).  A
 * scale is a power of two in the E8M0 form: byte b stands for 2^(b - 127).
 * These are the block scales that gfx950's matrix instructions multiply by
 * themselves, so they cost the products no vector work.
 * codes: [rows, cols] bytes; scales: [rows, moonep_scale_bytes(cols)] bytes,
 * where the bytes past ceil(cols / 128) are 127 (1.0).
 * Every call that writes scales takes the least power of two for which the
 * block's largest magnitude is at most 448 times it, not below 2^-126; a block
 * of zeros has the scale 1.  The codes are the values over their scale, rounded
 * to the nearest e4m3 value, ties to even.  A block that holds an infinity or a
 * NaN gets the scale 255 and the codes 0x7F, both NaN.
 * Codes are 16-byte aligned, scales 4-byte aligned, and cols % 16 == 0
 * (MOONEP_ERR_ARG).
 */
size_t moonep_scale_bytes(int32_t cols); /* 4 * ceil(cols / 512); 0 if cols < 1 */

/*
 * The residual's addition, RMS norm and its 8-bit output: what a layer does to
 * its token rows before the router and the dispatch.  x, res: bf16 [R*S, H];
 * weight: bf16 [H]; H % 16 == 0, H <= 65536 (MOONEP_ERR_ARG).
 *   r = bf16(x + res) (x itself if res is NULL), written to res_out;
 *   y = r * (1 / sqrt(mean over the row of r^2 + eps)) * weight, in fp32 (a row
 *       whose sum of squares is beyond fp32 becomes 0; with eps = 0 a row of
 *       zeros, or of values whose squares are all 0 in fp32, is not finite);
 *   y8, ys = the 8-bit row of y: codes [R*S, H], scales
 *            [R*S, moonep_scale_bytes(H)];
 *   y_out  = bf16(y), [R*S, H], for the router and a shared expert; NULL to
 *            leave it out.
 * res and res_out are both given or both NULL.  res_out may be res or x (the
 * row is read before it is written); otherwise outputs must not overlap inputs
 * or each other.  eps is finite and >= 0 (MOONEP_ERR_ARG).
 */
int moonep_rmsnorm_quant(const moonep_shape *shape, const uint16_t *x, const uint16_t *res,
                         const uint16_t *weight, float eps, uint16_t *res_out, uint16_t *y_out,
                         uint8_t *y8, uint8_t *ys, void *stream);

/*
 * moonep_dispatch for 8-bit rows: buf8[slot_of[n]] = x8[n div K] and
 * bufs[slot_of[n]] = xs[n div K], bit copies of H codes and
 * moonep_scale_bytes(H) scale bytes; x8 [R*S, H], buf8 [R*S*K, H].  Rows whose
 * slot_of is outside [0, R*S*K) are skipped.  H % 16 == 0.  The buffers must
 * not overlap the rows, or each other.
 */
int moonep_dispatch_quant(const moonep_shape *shape, const uint8_t *x8, const uint8_t *xs,
                          const int32_t *slot_of, uint8_t *buf8, uint8_t *bufs, void *stream);

/*
 * Expert weights in 8 bits, once when they are loaded: for every expert e of
 * E, the bf16 matrix [out_dim, in_dim] at element w_offset of row e of w
 * [E, w_stride] becomes codes [out_dim, in_dim] at byte code_offset and scales
 * [ceil(out_dim / 128), moonep_scale_bytes(in_dim)] at byte scale_offset of row
 * e of w8 [E, w8_stride], one scale for each 128 x 128 block (smaller at the
 * edges).  A row of w8 holds every matrix of an expert, so that
 * moonep_prefetch_weights moves it as it is.  Bytes outside the two windows are
 * not touched.
 * Limits (MOONEP_ERR_ARG): in_dim % 16 == 0, out_dim > 0, both at most 2^30, w_stride and w_offset
 * multiples of 8, w8_stride and code_offset multiples of 16, scale_offset of 4;
 * windows inside their rows, and apart from each other.  w and w8 16-byte
 * aligned and not overlapping.
 */
int moonep_quant_weights(const moonep_shape *shape, int32_t in_dim, int32_t out_dim,
                         const uint16_t *w, int64_t w_stride, int64_t w_offset, uint8_t *w8,
                         int64_t w8_stride, int64_t code_offset, int64_t scale_offset,
                         void *stream);

/*
 * moonep_expert_gemm in 8 bits: one projection of the expert-grouped buffer.
 * x8 [R*S*K, in_dim] codes and xs [R*S*K, moonep_scale_bytes(in_dim)] scales
 * (e.g. what moonep_dispatch_quant wrote); the weights of row r's segment are
 * the codes and scales at code_offset and scale_offset of its 8-bit weight row
 * (w_home [E, w_stride] or pool [R*B, w_stride] bytes, chosen as in
 * moonep_expert_gemm):
 *   y[r, n] = bf16( sum_k x[r, k] * W[n, k] )  (fp32 accumulation on the matrix
 *             cores, one rounding to nearest even), y: bf16 [R*S*K, out_dim].
 *             The 8-bit matrix instructions add products in groups of 8 (k to
 *             k + 7) and cut each, towards zero, to a multiple of 2^-13 of the
 *             group's largest power of two (in codes; one below 2^-6 counts as
 *             2^-6).  On normally distributed codes that is 2^-19 of sum |x| |W|
 *             (rms), 2^-14 at most; where one product of a group is 128 times the
 *             others and more, up to 7 2^-13 of it.
 * Limits (MOONEP_ERR_ARG): in_dim and out_dim multiples of 16 and at most 2^22,
 * w_stride and code_offset multiples of 16, scale_offset of 4, windows inside
 * the weight row.  x8, y, w_home, pool 16-byte aligned; y must not overlap an
 * input.
 */
int moonep_expert_gemm_quant(const moonep_shape *shape, const int32_t *plan, const int32_t *wslot,
                             int32_t B, int32_t in_dim, int32_t out_dim, const uint8_t *x8,
                             const uint8_t *xs, const uint8_t *w_home, const uint8_t *pool,
                             int64_t w_stride, int64_t code_offset, int64_t scale_offset,
                             uint16_t *y, void *stream);

/*
 * Gate and up projections with the activation and its 8-bit output in one
 * call: with g and u the two products of row r (fp32, not rounded in between),
 *   h[r, n] = g[r, n] / (1 + exp(-g[r, n])) * u[r, n]
 * (within (|g| + 4) 2^-22 of it, for the products as they are) and h8 [R*S*K, mid_dim], hs [R*S*K, moonep_scale_bytes(mid_dim)] its 8-bit
 * rows, ready for the down projection.  gate_* and up_* are the windows of the
 * two [mid_dim, in_dim] matrices; the limits are those of
 * moonep_expert_gemm_quant with out_dim = mid_dim.  h8 and hs must not overlap
 * an input or each other.
 */
int moonep_expert_glu_quant(const moonep_shape *shape, const int32_t *plan, const int32_t *wslot,
                            int32_t B, int32_t in_dim, int32_t mid_dim, const uint8_t *x8,
                            const uint8_t *xs, const uint8_t *w_home, const uint8_t *pool,
                            int64_t w_stride, int64_t gate_code_offset, int64_t gate_scale_offset,
                            int64_t up_code_offset, int64_t up_scale_offset, uint8_t *h8,
                            uint8_t *hs, void *stream);

/*
 * Backward of moonep_expert_gemm for the rows: with W as there (the same
 * arguments and limits),
 *   d_x[r, k] = bf16( sum_n d_y[r, n] * W[n, k] )  (fp32 accumulation on the
 *               matrix cores, one rounding to nearest even).
 * d_y: bf16 [R*S*K, out_dim]; d_x: bf16 [R*S*K, in_dim], must not overlap d_y,
 * w_home or pool.  out_dim is at most 2^22 as well, w_stride 2^37.
 */
int moonep_expert_gemm_dx(const moonep_shape *shape, const int32_t *plan, const int32_t *wslot,
                          int32_t B, int32_t in_dim, int32_t out_dim, const uint16_t *d_y,
                          const uint16_t *w_home, const uint16_t *pool, int64_t w_stride,
                          int64_t w_offset, uint16_t *d_x, void *stream);

/*
 * Backward of moonep_expert_gemm for the weights, into the rows that
 * moonep_replica_grad_reduce reduces.  home_grads: fp32 [E, G]; replica_grads:
 * fp32 [E + R, G], row j = replica j of `plan`.  With g the [out_dim, in_dim]
 * window at element g_offset of the row of home expert e or of replica j < n_rep,
 *   g[n, k] = sum over the buffer rows r of that expert's or replica's segment of
 *             d_y[r, n] * x[r, k]
 * in fp32 on the matrix cores, added to what g holds if accumulate is nonzero.
 * A segment without rows gives zeros (or leaves g as it is).  Nothing else of the
 * rows is touched, nor rows j >= n_rep.  x: bf16 [R*S*K, in_dim], d_y: bf16
 * [R*S*K, out_dim].
 * Limits (MOONEP_ERR_ARG): in_dim % 64 == 0, out_dim % 128 == 0, both at most
 * 2^22, g_offset >= 0, g_offset + out_dim*in_dim <= G.  x and d_y 16-byte
 * aligned, the gradients 4-byte; they must not overlap x, d_y or each other.
 */
int moonep_expert_gemm_dw(const moonep_shape *shape, const int32_t *plan, int32_t in_dim,
                          int32_t out_dim, const uint16_t *x, const uint16_t *d_y,
                          int32_t accumulate, int64_t G, int64_t g_offset, float *home_grads,
                          float *replica_grads, void *stream);

/*
 * Low-rank adapters of many requests at once, beside a projection that all rows
 * share.  Rows r < R*S*K of `shape`, where R = K = 1 (MOONEP_ERR_ARG): S rows, and
 * adapters take the place of experts, so that moonep_route_stats and moonep_plan
 * on `ids` group the rows by adapter (E - 1 adapters, say, and id E - 1 for rows
 * without one).  H is not used.
 *
 * A bank holds the adapters: row m of bank [n, stride] (bf16) is adapter m, its
 * matrices A [rank, in_dim] at element a_offset and B [out_dim, rank] at
 * b_offset, row-major, so that one row may hold the adapter's matrices of every
 * layer.  scale: fp32 [n].  ids: int32 [S]; a row whose id is outside [0, n) has no
 * adapter.  An adapter of a lower rank has zeros in the rows of A and the columns
 * of B past it; their gradients are then zeros too.
 *   u[r] = x[r] A^T,  y[r] = bf16(base[r] + scale * u[r] B^T)
 * x: bf16 [S, in_dim]; base, y: bf16 [S, out_dim], base being the shared
 * projection's output and y possibly the same array; u: fp32 [S, rank], which
 * moonep_adapter_bwd takes.  u is summed in fp32 on the matrix cores; scale * u
 * enters the second product with 16 bits (2^-17 relative), and y is rounded once.
 * A row without an adapter has u = 0 and y = base, bit for bit.
 * order: int32 [S] or NULL, the rows in the order to work in, each once:
 * moonep_plan's src_of_slot.  Rows of one adapter that stand together share its
 * loads, so NULL (the rows as they are) is right for few rows or whole prompts one
 * after the other.  The results depend on it in the order of u's fp32 sums only; a
 * row that is not in it is left out.
 *
 * workspace: moonep_adapter_workspace_bytes (64 rank bytes a row, what the call in most
 * parts takes), 16-byte aligned, no initial contents needed; one call at a time uses it.
 * Infinities and NaN come out where the formulas have them, and reach no other row.
 * Limits (MOONEP_ERR_ARG): 1 <= n <= E, rank, in_dim and out_dim multiples of 8,
 * rank at most 128, in_dim and out_dim at most 2^22, stride and offsets multiples
 * of 8, windows inside the row and apart.  bf16 arrays, u and workspace 16-byte
 * aligned.  Outputs and the workspace must not overlap inputs or each other,
 * except y = base.
 */
typedef struct moonep_adapters {
    int32_t n;        /* adapters in the bank */
    int32_t rank;     /* the largest rank */
    int32_t in_dim, out_dim;
    int64_t stride;   /* elements of a bank row */
    int64_t a_offset; /* A [rank, in_dim] in it */
    int64_t b_offset; /* B [out_dim, rank] in it */
} moonep_adapters;

/* Bytes of scratch; 0 for an invalid shape or adapters. */
size_t moonep_adapter_workspace_bytes(const moonep_shape *shape, const moonep_adapters *ad);
size_t moonep_adapter_bwd_workspace_bytes(const moonep_shape *shape, const moonep_adapters *ad);

int moonep_adapter(const moonep_shape *shape, const moonep_adapters *ad, const int32_t *ids,
                   const int32_t *order, const uint16_t *x, const uint16_t *bank,
                   const float *scale, const uint16_t *base, float *u, uint16_t *y,
                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * Adapter backward.  With u as moonep_adapter wrote it, d_y: bf16 [S, out_dim],
 *   du[r]  = scale * d_y[r] B                       (fp32)
 *   d_x[r] = bf16(dx_base[r] + du[r] A)
 *   dA     = sum over the adapter's rows of du[r]^T x[r]
 *   dB     = sum over the adapter's rows of scale * d_y[r]^T u[r]
 * dx_base, d_x: bf16 [S, in_dim], dx_base being the shared projection's part and
 * d_x possibly the same array; d_x = dx_base, bit for bit, without an adapter.  Both
 * NULL: not computed.  d_bank: fp32 [n, stride], its windows laid out as bank's;
 * the sums are written there, or added to what it holds if accumulate is nonzero;
 * an adapter without rows gets zeros (or stays as it is), and the rest of a row is
 * not touched.  d_bank NULL: not computed, and plan, x and u may be NULL too.
 * Every product is summed in fp32, du and u entering the gradients' with all their
 * bits; sums over rows are taken in an order that the shape and the plan fix.
 * order and plan: moonep_plan's src_of_slot and plan for `shape` and ids (order
 * may be NULL where d_bank is).  With another plan's tables d_bank is unspecified,
 * but every access stays in bounds.  The other arguments and the limits are
 * moonep_adapter's; workspace: moonep_adapter_bwd_workspace_bytes (68 rank bytes a row
 * and n + 64 fp32 windows, whatever is computed); d_bank 16-byte aligned.
 */
int moonep_adapter_bwd(const moonep_shape *shape, const moonep_adapters *ad, const int32_t *ids,
                       const int32_t *order, const int32_t *plan, const uint16_t *x, const float *u,
                       const uint16_t *d_y, const uint16_t *bank, const float *scale,
                       const uint16_t *dx_base, uint16_t *d_x, int32_t accumulate, float *d_bank,
                       void *workspace, size_t workspace_bytes, void *stream);

/*
 * The norm over many gradient tensors, and their clipping.  The tensors are named
 * by a device table of runs, int64 [entries, 4]: address of the gradient, address
 * of the clipped one (may be the same), elements, type (MOONEP_F32 or MOONEP_BF16,
 * of both).  moonep_grad_table writes it, on the host, for the caller to copy to
 * the device: tensor i, counts[i] elements at src[i], in runs of at most
 * MOONEP_GRAD_RUN (a run is one workgroup's work; longer ones are right as well);
 * entries past the last run get no elements and add nothing.
 * dst NULL: dst[i] = src[i].  It refuses (MOONEP_ERR_ARG) a negative count or an unknown
 * type, (MOONEP_ERR_MISALIGNED) an address that is no multiple of the element,
 * (MOONEP_ERR_NULL_PTR) a NULL address of a tensor with elements,
 * (MOONEP_ERR_WORKSPACE) more entries than `entries`, and (MOONEP_ERR_ALIAS)
 * tensors that overlap each other, or an output that overlaps a gradient other than
 * by being it.  The table holds addresses: the tensors have to live as long as it
 * is used.
 */
enum { MOONEP_GRAD_RUN = 16384, MOONEP_GRAD_WORKSPACE_BYTES = 16384 };

/* Entries of the table; -1 for a negative n or count. */
int64_t moonep_grad_entries(int64_t n, const int64_t *counts);
int moonep_grad_table(int64_t n, const uint64_t *src, const uint64_t *dst, const int64_t *counts,
                      const int32_t *types, int64_t entries, int64_t *table);

/*
 * norm[0] = fp32(sqrt(sum of g^2)) over every element of the table; sumsq[0], if
 * given, the sum itself in fp64 (to be added up over ranks).  Squares and sums are
 * fp64, in an order that the table fixes: not finite only if an element is not
 * (or, for norm, beyond fp32).  workspace: MOONEP_GRAD_WORKSPACE_BYTES, 8-byte
 * aligned, no initial contents needed; one call at a time uses it.
 */
int moonep_grad_norm(int64_t entries, const int64_t *table, double *sumsq, float *norm,
                     void *workspace, size_t workspace_bytes, void *stream);

/*
 * The same norm (of sumsq[0] if it is given: the sum over all ranks), and, with
 * the fp64 root in the place of norm,
 *   dst = g * fp32(max_norm / norm)   if norm > max_norm and norm is finite,
 *   dst = g                           otherwise (nothing is written where dst is
 *                                     the gradient itself),
 * the exact product rounded once to the gradient's type.  An infinity or a NaN among
 * the gradients leaves them all as they are, and norm says so; finite ones whose
 * norm is beyond fp32 are scaled as above, norm[0] being an infinity.  max_norm is
 * finite and >= 0 (MOONEP_ERR_ARG).  workspace may be NULL where sumsq is given.
 */
int moonep_grad_clip(int64_t entries, const int64_t *table, double max_norm, const double *sumsq,
                     float *norm, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Reads the sticky device error word of a workspace into *host_code, then
 * clears it.  Synchronises `stream`.  The only call that waits for the device.
 */
int moonep_read_error(void *workspace, size_t workspace_bytes, int32_t *host_code, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOONEP_H */
