/*
 * moe_async.h -- C ABI of the asynchronous MoE expert-execution library (GB300, sm_103a).
 *
 * What the library computes.  One or more MoE layers executed asynchronously:
 * routed token vectors arrive in waves tagged (RequestID, LayerID, expert,
 * top-k weight) and are appended to per-expert micro-queues; a scheduling step
 * picks ready queues (most-tokens-first or a minimum batch), gathers each
 * picked queue's tokens into one contiguous batch, runs the expert SwiGLU FFN
 * as a grouped GEMM, and scatters w * E(x) into per-(request, k) combine slots;
 * a token's output y = sum_j w_j E_j(x) is released only once all K results
 * (plus the shared expert's, if any) have landed.
 *   - Metadata, token pool, micro-queues, scheduler, gather + top-k merge:
 *     "SOSP'26 StreamEP" (marsggbo.github.io), sections 3 and 4.
 *   - Minimum-batch streaming of ready tokens (streamFFN) and starting expert
 *     work before every replica's tokens are ready: "CascadeEP: Asynchronous
 *     Expert Execution for MoE Prefill under Attention Imbalance", abstract.
 *   - Readiness published after the payload, exactly-once acceptance, reclaim
 *     after the last read, generation-tagged slots: "asynchronous MoE serving"
 *     notes, sections "recent work that narrows the proposals" (CascadeEP,
 *     Appendix C) and "inferred obligations for a concrete protocol".
 *
 * Conventions for every call.
 *   - Pointers named d_* are DEVICE pointers on the current CUDA device; h_*
 *     are host pointers.  `stream` is a cudaStream_t passed as void* (NULL =
 *     the legacy default stream).  Calls are stream-ordered and asynchronous
 *     unless stated otherwise; a handle must be used from one stream at a time.
 *   - Host-detectable errors (bad arguments) return immediately and launch
 *     nothing.  Errors found on the device (duplicate pair, stale generation,
 *     bucket overflow, out-of-range id) set a sticky device error word; it is
 *     returned by the next synchronising call (moe_async_sync, _wait,
 *     _get_stats) and stays set until moe_async_destroy.
 *   - No call blocks without bound: moe_async_wait is limited by a step count.
 *   - Thread safety: a handle is not thread-safe; distinct handles are.
 *   - Kernels are launched as programmatic dependents of the kernel before them
 *     in the stream (they may start early and wait on the device for it to
 *     finish), so every call still sees all earlier work of the stream; the
 *     caller's own kernels, copies and events order as usual.
 */
#ifndef MOE_ASYNC_H
#define MOE_ASYNC_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct moe_async_s* moe_async_t;

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID = 1,      /* bad argument (host) or out-of-range id (device)          */
  MOE_ERR_CAPACITY = 2,     /* a per-expert bucket or the ready ring overflowed          */
  MOE_ERR_DUPLICATE = 3,    /* a (slot, k) pair was delivered twice; the copy is dropped */
  MOE_ERR_STALE = 4,        /* a pair carried an out-of-date slot generation; dropped    */
  MOE_ERR_TIMEOUT = 5,      /* moe_async_wait ran out of steps with tokens still open;   */
                            /* or (sticky) a device wait in the tensor-core kernels     */
                            /* exceeded its 2 s bound -- the handle's state is then     */
                            /* undefined and it should be destroyed                     */
  MOE_ERR_CUDA = 6,         /* a CUDA runtime call failed                                */
  MOE_ERR_UNSUPPORTED = 7,  /* shape/dtype combination not supported by the kernels      */
  MOE_ERR_BOUNDS = 8        /* (bounds-checked build only) an index read back from device
                               state was out of range; the access was skipped           */
} moe_status;

/* MOE_E4M3: operands of moe_async_linear and the 8-bit output of moe_async_add_rms_norm only */
typedef enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_E4M3 = 2 } moe_dtype;

typedef enum {
  MOE_POLICY_MTFS = 0,       /* most tokens first: deepest buckets first (StreamEP, section 4) */
  MOE_POLICY_THRESHOLD = 1,  /* buckets holding >= min_batch tokens; else MTFS fallback         */
  MOE_POLICY_RANKS = 2       /* simulated expert-parallel ranks with work stealing: expert e
                              * belongs to rank e mod max_groups; each rank runs its deepest
                              * bucket; with fallback_groups != 0 a rank owning no non-empty
                              * bucket takes the deepest bucket no rank picked (unstarted work
                              * reassigned to an idle helper: "asynchronous MoE serving" notes,
                              * CascadeEP v1).  Picks are planned in rank order.              */
} moe_policy_kind;

typedef enum {
  MOE_EXPERT_SWIGLU = 0,     /* E(x) = (silu(x W1) * (x W3)) W2                               */
  MOE_EXPERT_IDENTITY = 1    /* E(x) = x; exercises queues/readiness/combine without a GEMM    */
} moe_expert_kind;

typedef struct {
  int32_t num_layers;       /* L >= 1                                                          */
  int32_t num_experts;      /* E routed experts per layer, 1..1024                             */
  int32_t top_k;            /* K, 1..30                                                        */
  int32_t hidden;           /* H, multiple of 8                                                */
  int32_t inter;            /* I, multiple of 16                                               */
  int32_t dtype;            /* moe_dtype of x, weights and y (accumulation is always fp32)     */
  int32_t has_shared;       /* 1: one always-on shared expert per layer, weight 1, I_s == I   */
  int32_t max_slots;        /* combine slots (RequestIDs 0..max_slots-1) per layer             */
  int32_t bucket_capacity;  /* pairs per expert bucket; 0 = max_slots (cannot overflow)        */
  int32_t expert_kind;      /* moe_expert_kind                                                 */
  int32_t trace_capacity;   /* >0: record up to this many (step, layer, expert, count) picks   */
} moe_async_config;

typedef struct {
  int32_t kind;             /* moe_policy_kind                                                 */
  int32_t max_groups;       /* at most this many buckets per step; 0 = no limit;
                             * RANKS: the number of ranks, >= 1                                */
  int32_t min_batch;        /* THRESHOLD: minimum bucket depth to run                          */
  int32_t fallback_groups;  /* THRESHOLD: buckets taken (deepest first) when none qualifies;
                             * RANKS: nonzero = idle ranks steal                               */
} moe_async_policy;

typedef struct {
  int64_t steps;            /* scheduling steps executed                                       */
  int64_t pairs_executed;   /* routed (token, expert) pairs run through an expert              */
  int64_t expert_runs;      /* sum over steps of the number of buckets picked                  */
  int64_t weight_bytes;     /* expert weight bytes streamed, as scheduled (3*H*I*elem per run) */
  int64_t tokens_combined;  /* tokens whose merge completed                                    */
  int64_t duplicates;       /* pairs rejected as duplicates                                    */
  int64_t stale;            /* pairs rejected for a stale generation                           */
  int32_t open_tokens;      /* tokens with >= 1 accepted pair not yet combined (all layers)    */
  int32_t pending_pairs;    /* accepted pairs not yet picked (all layers)                      */
  int32_t ready;            /* combined tokens not yet collected (all layers)                  */
  int32_t error;            /* sticky device error (moe_status)                                */
  int64_t packed_weight_bytes; /* library-owned packed weight copy made at create              */
  int64_t kernel_launches;  /* kernels this handle has launched since create                   */
  int64_t cancelled;        /* requests retired by moe_async_cancel                            */
} moe_async_stats;

/* Kernel kinds timed by moe_async_profile (index into the arrays of moe_async_profile_read). */
typedef enum {
  MOE_KERNEL_ENQUEUE = 0,    /* Receptor: pairs into buckets, token rows into the pool          */
  MOE_KERNEL_SCHEDULE = 1,   /* device-side policy + work list                                  */
  MOE_KERNEL_FFN1 = 2,       /* gather + GEMM1 (gate/up) + SwiGLU   (identity: scatter)         */
  MOE_KERNEL_FFN2 = 3,       /* GEMM2 (down) + scatter of the results + readiness               */
  MOE_KERNEL_COLLECT = 4,    /* top-k merge of ready tokens, rows to the caller, slot reclaim   */
  MOE_KERNEL_TICK = 5,       /* moe_async_tick's control kernel: collect + Receptor + reclaim   */
  MOE_KERNEL_KINDS = 6
} moe_kernel_kind;

/* Create a handle.  Weights are given per layer as arrays of L device pointers:
 *   w1[l], w3[l] : [E, H, I] (expert e computes x @ W1[e]),  w2[l] : [E, I, H]
 *   shared_w1[l], shared_w3[l] : [H, I], shared_w2[l] : [I, H]  (NULL arrays when has_shared = 0)
 * all in cfg->dtype, row-major, contiguous.  The library packs them into its own K-major
 * copy (gate/up rows interleaved) before returning (it synchronises `stream`), so the
 * caller's weight buffers may be freed afterwards.  All state (token pool, buckets, combine
 * slots, outputs, work lists) is allocated here; no later call allocates device memory.
 * Returns MOE_ERR_INVALID / MOE_ERR_UNSUPPORTED for bad configs, MOE_ERR_CUDA on allocation
 * failure (nothing leaks).  *out is set only on MOE_OK. */
moe_status moe_async_create(const moe_async_config* cfg,
                            const void* const* w1, const void* const* w3, const void* const* w2,
                            const void* const* shared_w1, const void* const* shared_w3,
                            const void* const* shared_w2,
                            void* stream, moe_async_t* out);

/* Router: top-K experts per token with renormalised softmax weights.
 * StreamEP section 3 (each token selects its K highest-scoring experts); the rule is softmax
 * over the E logits, keep the K largest, renormalise them to sum to one.  Equal logits go to
 * the lower expert index; k = 0 is the highest score.
 *   d_logits : [T, E] fp32      d_idx : [T, K] int32 (out)      d_w : [T, K] fp32 (out)
 * Stateless (no handle).  1 <= K <= E <= 1024, K <= 32. */
moe_status moe_async_route(const float* d_logits, int32_t T, int32_t E, int32_t K,
                           int32_t* d_idx, float* d_w, void* stream);

/* Receptor: deliver one wave of routed pairs into layer `layer`'s expert queue.
 * StreamEP section 3, steps 1-2: each carried token is stored in the token pool under its
 * combine slot, and each delivered (expert, k, w) pair is appended to that expert's bucket
 * (warp-aggregated atomics).  A token's first accepted pair also enqueues the shared expert.
 *   n        : tokens carried (0 is a no-op)
 *   d_rows   : [n] row of d_x / d_expert / d_w for each carried token; NULL = rows 0..n-1
 *   d_slot   : [n] combine slot (RequestID) per token, < max_slots; NULL = the row index
 *   d_x      : [*, H] token vectors in cfg dtype (row-indexed)
 *   d_expert : [*, K] int32 expert ids (row-indexed), 0 <= id < E
 *   d_w      : [*, K] fp32 routing weights (row-indexed)
 *   d_kmask  : [n] uint32, bit k set = pair k is delivered by this wave; NULL = all K
 *   d_gen    : [n] uint32 expected slot generation; NULL = unchecked.  Mismatch -> the
 *              token's pairs are dropped and MOE_ERR_STALE is latched.
 * A pair already accepted for this slot generation is dropped and MOE_ERR_DUPLICATE latched.
 * The caller's buffers may be reused once the stream reaches this point. */
moe_status moe_async_enqueue(moe_async_t h, int32_t layer, int32_t n,
                             const int32_t* d_rows, const int32_t* d_slot, const void* d_x,
                             const int32_t* d_expert, const float* d_w,
                             const uint32_t* d_kmask, const uint32_t* d_gen, void* stream);

/* One scheduling step of layer `layer`, decided on the device from the bucket depths
 * (no host synchronisation): the policy picks buckets, each picked bucket is drained whole,
 * its tokens are gathered and run through the expert (grouped GEMM over all picks), the
 * results E_k(x) are written to their combine slots in the activation dtype, and every
 * token whose K (+shared) results are now complete is appended to the ready list (its
 * merge runs in moe_async_collect).  A step with nothing to pick launches kernels that exit
 * at once. */
moe_status moe_async_schedule_step(moe_async_t h, int32_t layer, const moe_async_policy* policy,
                                   void* stream);

/* Up to max_steps (>= 1) consecutive scheduling steps of layer `layer` in one device plan,
 * with the same picks, values and emission steps as that many moe_async_schedule_step calls
 * with nothing enqueued between them.  StreamEP section 4 (MTFS) and the CascadeEP abstract
 * (streamFFN): with no arrival between steps the queue depths only shrink, so the picks of
 * consecutive steps are one deepest-first order of the non-empty buckets cut into steps --
 * MTFS max_groups buckets a step (0 = all in one); THRESHOLD up to max_groups buckets of at
 * least min_batch a step while any remain, then fallback_groups a step.  All picked buckets
 * run in one grouped GEMM launch pair, each work item tagged with its step, so a drain of
 * many one-expert fallback steps streams weights on every SM instead of one expert per
 * launch.  The steps counter and the pick trace advance by the steps up to the last
 * non-empty one (a call that finds every bucket empty counts none).  MTFS and THRESHOLD
 * only: RANKS returns MOE_ERR_UNSUPPORTED for max_steps > 1.  Asynchronous, no host
 * synchronisation. */
moe_status moe_async_schedule_steps(moe_async_t h, int32_t layer, const moe_async_policy* policy,
                                    int32_t max_steps, void* stream);

/* One tick of a serving loop: one control launch, then the step's launches (plan, GEMM1,
 * GEMM2).  The control launch runs, side by side, the collect of the tokens that were ready
 * when the call was made (outputs as moe_async_collect, with max_out, d_y_out .. d_n_out and
 * append meaning the same; max_out = 0 collects nothing and d_n_out may then be NULL) and the
 * Receptor for a wave of n arriving tokens (arguments as moe_async_enqueue; n = 0 for none);
 * then one scheduling step runs under `policy` (as moe_async_schedule_step).  StreamEP section 3 (the Receptor feeds the per-expert queues,
 * ready tokens leave after their K results) and section 4 (the scheduler then picks).
 *   Equivalent to moe_async_collect, moe_async_enqueue and moe_async_schedule_step in that
 * order, with one difference: the collected slots are reclaimed after the wave's pairs have
 * been judged, so a pair of this wave for a slot collected by this call is judged against the
 * request it completed (a duplicate) rather than against the slot's next generation.  A
 * caller learns which slots are free only from a collect's outputs, so it never assigns a new
 * request to a slot collected by the same call.
 *   Asynchronous, no host synchronisation.  Errors as the three calls; MOE_ERR_INVALID for a
 * bad argument of any of them. */
moe_status moe_async_tick(moe_async_t h, int32_t layer, int32_t n, const int32_t* d_rows, const int32_t* d_slot,
                          const void* d_x, const int32_t* d_expert, const float* d_w, const uint32_t* d_kmask,
                          const uint32_t* d_gen, const moe_async_policy* policy, int32_t max_out, void* d_y_out,
                          int32_t* d_slot_out, uint32_t* d_gen_out, uint32_t* d_step_out, int32_t* d_n_out,
                          int32_t append, void* stream);

/* Collect ready tokens of layer `layer` in completion order, each merged on the way out:
 * y = sum_k w_k E_k(x) in fp32, ascending k (k = K is the shared expert, weight 1), each
 * product and sum rounded (no fused multiply-add), stored in the cfg dtype:
 *   d_y_out    : [max_out, H] cfg dtype     d_slot_out : [max_out] int32
 *   d_gen_out  : [max_out] uint32 (generation the result belongs to; may be NULL)
 *   d_step_out : [max_out] uint32 (emission step: the scheduling step, counted from 1 over
 *                the handle's life, in which the token's last result landed; may be NULL)
 *   d_n_out    : [1] int32 on the device
 *   append = 0 : rows are written from index 0 and *d_n_out = number written (<= max_out)
 *   append = 1 : rows are written from index *d_n_out (read on the device) and *d_n_out is
 *                advanced by the number written (total <= max_out), so a caller can collect
 *                after every step into one buffer without reading anything back
 * Each collected slot is reclaimed (its generation advances) after its output row is copied,
 * so it may carry a new request from then on. */
moe_status moe_async_collect(moe_async_t h, int32_t layer, int32_t max_out, void* d_y_out,
                             int32_t* d_slot_out, uint32_t* d_gen_out, uint32_t* d_step_out,
                             int32_t* d_n_out, int32_t append, void* stream);

/* Cancel the current request of each slot in d_slots[0..n) (int32, device) of `layer`.
 * "asynchronous MoE serving" notes: an abandoned operation retires its buffer until a quiescent
 * point, and output readiness is tracked separately from buffer reclamation (CascadeEP).  The
 * slot is retired: later pairs for it are dropped on arrival, pairs already queued still run
 * but their results are neither merged nor published, and the slot is freed (generation
 * advanced, reusable) when its last queued result has landed -- at once if nothing is queued.
 * Free slots and slots whose output is already merged are left unchanged.  Not available on a
 * handle running the streaming runtime (MOE_ERR_UNSUPPORTED). */
moe_status moe_async_cancel(moe_async_t h, int32_t layer, int32_t n, const int32_t* d_slots,
                            void* stream);

/* Run scheduling steps of `layer` under `policy` until no token of the handle is open
 * (accepted but not yet combined, in any layer); at most max_steps steps.  Under MTFS and
 * THRESHOLD the layer's queued buckets are drained as one plan of consecutive steps
 * (moe_async_schedule_steps), re-planned while the last plan left buckets behind.  Once the
 * queues are empty while tokens are still open, and under RANKS, single steps run: between
 * reads of the device counters as many as the layer's queues certainly still need (each step
 * drains its picks whole and takes at most max_groups buckets under RANKS), else
 * `check_every` steps.  Synchronises `stream`.  Returns MOE_ERR_TIMEOUT when tokens are still open after
 * max_steps (e.g. a withheld pair), else the sticky device error. */
moe_status moe_async_wait(moe_async_t h, int32_t layer, const moe_async_policy* policy,
                          int32_t max_steps, int32_t check_every, void* stream);

/* Synchronise `stream` and return the sticky device error (MOE_OK if none). */
moe_status moe_async_sync(moe_async_t h, void* stream);

/* Synchronise `stream` and copy the counters into *h_stats. */
moe_status moe_async_get_stats(moe_async_t h, void* stream, moe_async_stats* h_stats);

/* Synchronise and copy the pick trace: h_buf receives up to cap records of 4 int32
 * (step, layer, expert, count) in step order, *h_n the number of records written. */
moe_status moe_async_get_trace(moe_async_t h, void* stream, int32_t* h_buf, int32_t cap,
                               int32_t* h_n);

/* Synchronise and copy layer `layer`'s queue contents: h_depth[b] (b < E + has_shared) gets
 * bucket b's depth, and h_records the pending records of every bucket in bucket order, each
 * as (slot, k) int32 pairs (bucket-internal order is arrival order, which concurrent appends
 * make nondeterministic).  cap = capacity of h_records in pairs; *h_n = pairs written. */
moe_status moe_async_snapshot(moe_async_t h, int32_t layer, void* stream, int32_t* h_depth,
                              int32_t* h_records, int32_t cap, int32_t* h_n);

/* ---- Streaming multi-layer decode on the 2L micro-queues --------------------------------
 * "SOSP'26 StreamEP" section 3: each layer has an attention queue and an expert queue; a
 * request's token is served by its layer's attention stage, routed, dispatched to the expert
 * queue, merged back and queued for the next layer's attention -- each request advances at
 * its own pace, with no barrier across requests.  Section 4: one queue is served per
 * scheduling decision, the one holding the most tokens (MTFS; equal counts -> lower layer,
 * attention before expert).  The attention stage is a stub: a = RMSNorm(x) P_l (eps 1e-6,
 * no gain), x^(n+1) = MoE_l(a) with l = n mod L.  All state lives on the device and one
 * scheduling decision ("tick") runs as a CUDA graph with no host round trip. */
typedef enum {
  MOE_STREAM_MTFS = 0,      /* most tokens first (StreamEP section 4)                             */
  MOE_STREAM_FLFS = 1,      /* first layer first: earliest non-empty queue of the chain           */
  MOE_STREAM_DEFRAG = 2,    /* S(s) = Q(s) + sum_{j=1..W} decay^j [Q(s_j) + H(s_j)] (section 4)   */
  MOE_STREAM_BARRIER = 3,   /* synchronous baseline: nothing served while a dispatch is in flight */
  MOE_STREAM_DEFRAG_SRC = 4 /* the same score as section 4 describes the source implementation:
                               H(s) = average of s's depth snapshots over the last history_window
                               ticks, lookahead continued cyclically along the chain              */
} moe_stream_policy;

typedef struct {
  int32_t num_requests;     /* R <= max_slots; request r uses combine slot r in every layer    */
  int32_t max_steps;        /* steps per request at most (history depth)                       */
  int32_t stop_combines;    /* attention queues are closed once this many merges are done      */
  int32_t policy;           /* moe_stream_policy                                               */
  int32_t defrag_window;    /* DEFRAG(_SRC): W, queues looked ahead along att_0, exp_0, att_1, ... */
  int32_t history_window;   /* DEFRAG: H(s) = tokens drained from s over the last N ticks, <=16;
                               DEFRAG_SRC: the window of depth snapshots H(s) averages         */
  double defrag_decay;      /* DEFRAG: decay per lookahead step (scores in fp64)               */
} moe_stream_config;

/* Set up the streaming runtime on a bf16 SwiGLU handle (its merges then feed the runtime,
 * not the collect ring).  Synchronises `stream`.
 *   d_proj[l]   : [H, H] bf16 projection of layer l's attention stub (x @ P); packed, may be freed
 *   d_x0        : [R, H] bf16 initial states (copied into the history)
 *   d_logits    : [R, max_steps, E] fp32 router logits of (request, step)   (borrowed)
 *   d_delay     : [R, max_steps] int32 dispatch delay in ticks, >= 1       (borrowed)
 *   d_admit     : [R] int32 tick at which each request enters layer 0's attention queue
 *                 (<= 0: at the start); NULL = every request at the start   (borrowed)
 *   d_history   : [R, max_steps + 1, H] bf16 out: x^(n) of every request, x^(0) at n = 0
 *   d_done_tick : [R, max_steps + 1] int32 out: tick at which step n completed (-1 = not)
 * Requests admitted later join the attention queue at the start of their tick, after that
 * tick's dispatches are delivered; while attention is open, requests still to be admitted
 * keep the stream running (idle ticks).  MOE_ERR_UNSUPPORTED for fp32 or identity handles or
 * more than 8 layers. */
moe_status moe_async_stream_setup(moe_async_t h, const moe_stream_config* sc,
                                  const void* const* d_proj, const void* d_x0,
                                  const float* d_logits, const int32_t* d_delay,
                                  const int32_t* d_admit, void* d_history, int32_t* d_done_tick,
                                  void* stream);

/* Queue occupancy of the streaming runtime so far (for latency studies; StreamEP section 4:
 * queue depths are what the scheduler acts on).  Depths are in tokens (requests), seen at
 * each tick's decision after that tick's arrivals and admissions. */
typedef struct {
  int32_t ticks;                 /* ticks run                                                    */
  int32_t combined;              /* merges completed (token-layer steps)                         */
  int32_t peak_transit;          /* most requests in transit (dispatched, not yet arrived)       */
  int32_t peak_bucket;           /* deepest expert bucket at the moment its layer was served     */
  int32_t num_queues;            /* 2L: the queues below in chain order att_0, exp_0, att_1, ... */
  int32_t peak_queue[16];        /* deepest each queue was at a decision (closed attention: 0)   */
  int64_t occupancy_sum[16];     /* each queue's depth summed over the ticks (mean = / ticks)    */
} moe_stream_stats;

/* Synchronise `stream` and read the streaming runtime's occupancy figures. */
moe_status moe_async_stream_stats(moe_async_t h, void* stream, moe_stream_stats* out);

/* Run ticks until nothing is left (no dispatch in transit, expert queues empty, attention
 * queues closed or empty), reading the control block every `check_every` ticks; at most
 * max_ticks ticks (then MOE_ERR_TIMEOUT).  Synchronises; *h_ticks = ticks run,
 * *h_combined = merges completed. */
moe_status moe_async_stream_run(moe_async_t h, int32_t max_ticks, int32_t check_every,
                                int32_t* h_ticks, int32_t* h_combined, void* stream);

/* Synchronise and copy the tick trace: 4 int32 per tick (tick, kind, layer, count), kind
 * 1 = attention queue, 2 = expert queue, 0 = idle (only dispatches in transit). */
moe_status moe_async_stream_trace(moe_async_t h, void* stream, int32_t* h_buf, int32_t cap,
                                  int32_t* h_n);

/* Per-kernel timing (tracing).  enable = 1 brackets every later kernel launch of the handle
 * with a pair of CUDA events on its stream (up to 65536 launches are kept); enable = 0 stops.
 * Host-side events only: no device memory is allocated. */
moe_status moe_async_profile(moe_async_t h, int32_t enable);

/* Synchronise `stream`, then for each kernel kind k < n_kinds add the summed event time of its
 * recorded launches to h_ms[k] (milliseconds) and their number to h_launches[k]; the record
 * is cleared afterwards. */
moe_status moe_async_profile_read(moe_async_t h, void* stream, double* h_ms, int64_t* h_launches,
                                  int32_t n_kinds);

/* Free every device allocation of the handle.  Synchronises `stream` first. */
moe_status moe_async_destroy(moe_async_t h, void* stream);

/* One routed MoE layer forward that allocates no device memory.  The pages have no
 * counterpart: this is for callers that cannot call cudaMalloc where they run the layer
 * (a memory pool owns the device, an allocation-free runtime, a plugin that is handed only
 * its input and output buffers).
 *   y[t] = sum_{k=0..K-1, ascending} w[t,k] * E_{expert[t,k]}(x[t]),
 *   E(x) = (silu(x W1) * (x W3)) W2, fp32 accumulation, no shared expert.
 *   d_x [T,H], d_y [T,H] in dtype (moe_dtype); d_expert [T,K] int32 in [0,E); d_w [T,K]
 *   fp32; d_w1, d_w3 [E,H,I] and d_w2 [E,I,H] in dtype -- the caller's own weight layout,
 *   no packing.  All device pointers, all caller-owned.
 * Expert ids outside [0,E) contribute nothing, silently: unlike moe_async_enqueue, which
 * latches MOE_ERR_INVALID in its handle's sticky error, this call has no handle to hold an
 * error, and the ids live in device memory where the host cannot check them without a sync.
 * Scratch: a fixed 16 MiB array compiled into the library (held on every GPU that loads
 * it, until the process exits) holds the T*K*I fp32 SwiGLU activations, so T*K*I*4 bytes
 * may not exceed 16 MiB: larger calls return MOE_ERR_CAPACITY and launch nothing.  Every
 * call looks up the array's device address in the current context (no allocation); the
 * first call in a context may load the library's device code, so make it before any stream
 * capture.  Work: each (token, k) pair reads its expert's W1 and W3 columns on its own (no
 * weight reuse between pairs of one expert), so this path is far slower than the grouped
 * GEMMs of the handle-based calls.  Every call shares the one array and each call
 * overwrites every element it reads, so nothing has to be cleared, but calls whose kernels
 * overlap on the GPU (different streams, or different host threads) race on it: order them.
 * Calls no cudaMalloc/cudaFree.  Asynchronous on `stream`. */
moe_status moe_async_forward_noalloc(int32_t T, int32_t E, int32_t K, int32_t H, int32_t I,
                                     int32_t dtype, const void* d_x, const int32_t* d_expert,
                                     const float* d_w, const void* d_w1, const void* d_w3,
                                     const void* d_w2, void* d_y, void* stream);

/* ---------------------------------------------------------------- stateless operators
 * The synchronous form of the path for callers that hold a whole routed batch: norm, products,
 * tokens sorted by expert and merged back, and the gradients a training step needs.  No handle,
 * no allocation, nothing kept between calls; any number of calls may run at once on streams of
 * their own, and every call can be captured into a graph.
 *   - Row operands are [rows, width] with a row stride in elements (>= width); columns are
 *     adjacent.  Rows whose base and stride are multiples of 16 bytes, and whose width is a
 *     whole number of 16-byte units, move in such units; others element by element.
 *   - Parameter vectors (gain, bias, scales, routing weights) are fp32.
 *   - Sizes are at least 1, but 0 rows (or tokens) are a call that does nothing; widths are at most
 *     2^31 - 65537 (moe_async_linear: 2^31 - 1025).
 *   - Sums are fp32 in an order fixed by the sizes and the alignment (no atomics): equal calls
 *     give equal bits.
 *   - An output may share memory with an input only where stated. */

/* Sorted order of the pairs of a routed batch: by expert, pairs of one expert in pair order
 * (pair i = t * K + k).
 *   d_expert  : [T, K] int32; an id outside [0, E) belongs to no expert here (another rank's,
 *               or a padded token's): its pair gets no row
 *   d_offsets : [E + 1] int32 out: rows of expert e are offsets[e] .. offsets[e + 1]
 *   d_pos     : [T, K] int32 out: the pair's row, -1 without one
 *   d_pair    : [T * K] int32 out: the pair of each row; behind offsets[E], the pairs without
 *               a row in pair order
 * E <= 1024, K <= 32, T * K < 2^31 - 1024.  Asynchronous. */
moe_status moe_async_sort_experts(const int32_t* d_expert, int32_t T, int32_t K, int32_t E, int32_t* d_offsets,
                                  int32_t* d_pos, int32_t* d_pair, void* stream);

/* rows[pos[t, k]] = x[t] for every pair whose pos lies in [0, n_rows); other rows are left as
 * they were.  Each row is named by at most one pair.  dtype: MOE_F32 or MOE_BF16. */
moe_status moe_async_sort_rows(int32_t dtype, const void* d_x, int64_t x_stride, const int32_t* d_pos, int32_t T,
                               int32_t K, int32_t H, void* d_rows, int64_t rows_stride, int64_t n_rows, void* stream);

/* y[t] = sum_k w[t, k] rows[pos[t, k]] + residual[t]: products and sums rounded in fp32 in
 * ascending k, the residual last, as moe_async_collect merges.  Pairs whose pos lies outside
 * [0, n_rows) add nothing and their weights are not looked at: a token without any gets its
 * residual, or zeros.  d_w NULL: plain sums (the gradient of moe_async_sort_rows).  d_residual
 * may be NULL, or y itself. */
moe_status moe_async_merge_rows(int32_t dtype, const void* d_rows, int64_t rows_stride, int64_t n_rows,
                                const int32_t* d_pos, const float* d_w, int32_t T, int32_t K, int32_t H,
                                const void* d_residual, int64_t residual_stride, void* d_y, int64_t y_stride,
                                void* stream);

/* Gradients of moe_async_merge_rows: grad_rows[pos[t, k]] = w[t, k] grad[t] (other rows are left
 * as they were) and grad_w[t, k] = <rows[pos[t, k]], grad[t]> (0 for a pair without a row); the
 * residual's gradient is `grad` itself.  Each row is named by at most one pair. */
moe_status moe_async_merge_rows_backward(int32_t dtype, const void* d_grad, int64_t grad_stride, const void* d_rows,
                                         int64_t rows_stride, int64_t n_rows, const int32_t* d_pos, const float* d_w,
                                         int32_t T, int32_t K, int32_t H, void* d_grad_rows, int64_t grad_rows_stride,
                                         float* d_grad_w, void* stream);

/* Gradient of moe_async_route's weights: grad_logits[t, idx[t, k]] = w_k (grad_w_k - sum_j w_j
 * grad_w_j), 0 at the experts not chosen; all of [T, E] is written.  d_idx and d_w are what
 * moe_async_route returned. */
moe_status moe_async_route_backward(const int32_t* d_idx, const float* d_w, const float* d_grad_w, int32_t T, int32_t E,
                                    int32_t K, float* d_grad_logits, void* stream);

/* h = x + residual, rounded to dtype; y = h / sqrt(mean(h^2) + eps) * gain per row.
 *   d_residual : [T, H] or NULL (then h = x, and d_h must be NULL)
 *   d_gain     : [H] fp32 or NULL (all ones)
 *   d_h        : [T, H] out, the sum; may be NULL, d_x or d_residual
 *   d_scale    : NULL: y is [T, H] in dtype.  Else [T] fp32 out and y is [T, H] e4m3:
 *                scale = max(max|y| / 448, 2^-126), stored value y / scale, round to nearest
 * A NaN makes its row NaN, an infinity makes finite columns 0 and itself NaN, and a row of finite
 * values whose sum of squares is beyond fp32 becomes zeros; in e4m3 each of them, and an h * gain
 * or a y beyond fp32, makes the whole row and its scale NaN.  dtype: MOE_F32 or MOE_BF16. */
moe_status moe_async_add_rms_norm(int32_t dtype, const void* d_x, int64_t x_stride, const void* d_residual,
                                  int64_t residual_stride, const float* d_gain, float eps, int32_t T, int32_t H,
                                  void* d_h, int64_t h_stride, void* d_y, int64_t y_stride, float* d_scale,
                                  void* stream);

/* Gradients of moe_async_add_rms_norm's y at h (its output h, or x): with u = grad * gain and
 * n = h / sqrt(mean(h^2) + eps), grad_x = (u - n mean(u n)) / sqrt(mean(h^2) + eps) + grad_h,
 * the gradient of x and of the residual alike, and grad_gain[c] = sum_t grad[t, c] n[t, c].
 *   d_grad_h    : [T, H] gradient that arrives at h itself, or NULL; may be d_grad_x
 *   d_grad_gain : [H] fp32 out or NULL; it needs a workspace (16-byte aligned) of at least
 *                 moe_async_add_rms_norm_backward_workspace(T, H) bytes, the caller's until the
 *                 call has run; calls that may run at once need one each.  Smaller:
 *                 MOE_ERR_CAPACITY */
int64_t moe_async_add_rms_norm_backward_workspace(int32_t T, int32_t H);
moe_status moe_async_add_rms_norm_backward(int32_t dtype, const void* d_grad, int64_t grad_stride, const void* d_h,
                                           int64_t h_stride, const float* d_gain, float eps, int32_t T, int32_t H,
                                           const void* d_grad_h, int64_t grad_h_stride, void* d_grad_x,
                                           int64_t grad_x_stride, float* d_grad_gain, void* d_workspace,
                                           int64_t workspace_bytes, void* stream);

/* silu is computed to within 10 * 2^-24 of its value for fp32 results, gelu (x times the normal
 * distribution's integral) to within 20 * 2^-24; for bf16 ones, whose own rounding is up to 2^-8,
 * both to within 2^-15. */
typedef enum { MOE_ACT_NONE = 0, MOE_ACT_SILU = 1, MOE_ACT_GELU = 2, MOE_ACT_RELU = 3 } moe_act;

/* y[t, n] = act(sx[t] sw[n] sum_k x[t, k] w[n, k] + bias[n]) * mul[t, n] + residual[t, n]
 *   dtype     : MOE_BF16, or MOE_E4M3 with d_x_scale [rows] and d_w_scale [fan_out] fp32 (NULL
 *               for MOE_BF16); MOE_F32 operands return MOE_ERR_UNSUPPORTED
 *   d_x       : [rows, fan_in]    d_w : [fan_out, fan_in]    fp32 accumulation
 *   d_y       : [rows, fan_out] in out_dtype (MOE_BF16 or MOE_F32), rounded once
 *   d_bias    : [fan_out] fp32 or NULL
 *   d_mul, d_residual : [rows, fan_out] in out_dtype or NULL; either may be y itself
 *   groups = 0: dense.  groups = G > 0: one weight matrix per expert on sorted rows: d_w is
 *   [G, fan_out, fan_in] (each matrix fan_out * w_stride elements), d_bias and d_w_scale are
 *   [G, fan_out], and rows d_offsets[g] .. d_offsets[g + 1] (device, int32, ascending, clipped to
 *   [0, rows]) meet matrix g; rows of no group are left as they were.
 * The same d_x and d_w of the same sizes give the same sums whatever the epilogue and the strides.
 * fan_in, the bases and the strides of x and w are multiples of 16 bytes, else
 * MOE_ERR_UNSUPPORTED; fan_out and the other strides are free.  Asynchronous. */
typedef struct {
  int32_t dtype, out_dtype, act, rows, fan_in, fan_out, groups;
  const void* d_x;
  const void* d_w;
  const float* d_bias;
  const float* d_x_scale;
  const float* d_w_scale;
  const void* d_mul;
  const void* d_residual;
  const int32_t* d_offsets;
  void* d_y;
  int64_t x_stride, w_stride, mul_stride, residual_stride, y_stride;
} moe_async_linear_args;
moe_status moe_async_linear(const moe_async_linear_args* args, void* stream);

/* moe_async_linear with a scale per block of 128 (MOE_E4M3 only; anything else returns MOE_ERR_UNSUPPORTED):
 *   v[t, n] = sum_k (x[t, k] sx[t, k / 128]) (w[n, k] sw[n / 128, k / 128]), then act(v + bias) * mul + residual
 *   d_x_scale : fp32, element (t, b) at t * x_scale_row + b * x_scale_block (tokens adjacent, x_scale_row = 1, is read
 *               fastest), b < ceil(fan_in / 128)
 *   d_w_scale : [ceil(fan_out / 128), ceil(fan_in / 128)] fp32, with groups [G, ..]
 * Each block's products are summed on their own and added, scaled, with rounding in fp32.  Everything else as there. */
moe_status moe_async_linear_blocks(const moe_async_linear_args* args, int64_t x_scale_row, int64_t x_scale_block, void* stream);

/* The operands of moe_async_linear_blocks: each block's scale = max(max|x| / 448, 2^-126), stored value x / scale, the
 * quotient's fp32 rounding rounded to nearest (as dividing in fp32 gives it).  A block with an infinity or a NaN becomes NaN, and its
 * scale.
 *   block_rows = 1   : blocks of 1 x 128; x [rows, width] (G = 1), scale of (t, b) at t * scale_row + b * scale_block
 *   block_rows = 128 : blocks of 128 x 128 of G matrices [rows, width], one behind another (rows * stride elements each), scale
 *                      [G, ceil(rows / 128), ceil(width / 128)] contiguous (scale_row and scale_block are not looked at); G and
 *                      rows / 128 at most 65,535, else MOE_ERR_UNSUPPORTED
 * dtype: MOE_F32 or MOE_BF16; blocks at an edge are as wide or high as the matrix lets them. */
moe_status moe_async_quantize_blocks(int32_t dtype, const void* d_x, int64_t x_stride, int32_t G, int32_t rows, int32_t width, int32_t block_rows,
                                     void* d_q, int64_t q_stride, float* d_scale, int64_t scale_row, int64_t scale_block, void* stream);

/* Gradients of moe_async_linear without its epilogue, y[t, n] = sum_k x[t, k] w[n, k] + bias[n], from
 * grad = dL/dy:
 *   grad_x[t, k]    = sum_n grad[t, n] w[n, k] + residual[t, k]
 *   grad_w[n, k]    = sum_t grad[t, n] x[t, k]
 *   grad_bias[n]    = sum_t grad[t, n]
 * (an epilogue's gradient comes first: moe_async_act_mul_backward).  Operands are bf16, sums fp32, results rounded
 * once.  Each of the three is computed if its pointer is given, and lies apart from the others and from the operands (where one
 * is another, MOE_ERR_INVALID); accumulate != 0 adds grad_w and grad_bias to what they hold.
 *   d_grad : [rows, fan_out]     d_x : [rows, fan_in], for grad_w     d_w : [fan_out, fan_in], for grad_x
 *   d_grad_x : [rows, fan_in] in x_dtype, d_residual in the same or NULL; it may be grad_x itself
 *   d_grad_w : [fan_out, fan_in] in w_dtype           d_grad_bias : [fan_out] fp32
 *   groups = G > 0: as in moe_async_linear; d_w and d_grad_w are [G, fan_out, fan_in] (matrices of fan_out * stride elements
 *   one behind another), d_grad_bias [G, fan_out]; rows of no group count nowhere, whatever they hold, and their grad_x is
 *   left as it was; a group without rows has a gradient of zeros.  Added to in fp32, values below 2^-126 are taken as 0.
 * rows are at most 2^31 - 4097.  fan_in is a multiple of 8, the bases and strides of x and w of 16 bytes, else MOE_ERR_UNSUPPORTED; fan_out and the other strides
 * are free, but rows of grad that do not start on 16-byte boundaries are copied first, into a workspace (16-byte aligned) of
 * moe_async_linear_backward_workspace(args) bytes (0 if they do), the caller's until the call has run; calls that may run at
 * once need one each.  Smaller: MOE_ERR_CAPACITY.  0 rows: grad_w and grad_bias are set to zeros, or left.  Asynchronous. */
typedef struct {
  int32_t x_dtype, w_dtype, rows, fan_in, fan_out, groups, accumulate, reserved;
  const void* d_grad;
  const void* d_x;
  const void* d_w;
  const void* d_residual;
  const int32_t* d_offsets;
  void* d_grad_x;
  void* d_grad_w;
  float* d_grad_bias;
  void* d_workspace;
  int64_t grad_stride, x_stride, w_stride, residual_stride, grad_x_stride, grad_w_stride, workspace_bytes;
} moe_async_linear_backward_args;
int64_t moe_async_linear_backward_workspace(const moe_async_linear_backward_args* args);
moe_status moe_async_linear_backward(const moe_async_linear_backward_args* args, void* stream);

/* Gradients of y = act(z) * mul (of y = act(z): d_mul and d_grad_mul NULL) from grad = dL/dy:
 *   grad_z = grad * mul * act'(z), grad_mul = grad * act(z), each [T, H] in dtype (MOE_F32 or MOE_BF16), rounded once (finite where
 *   the result is: grad * mul alone may lie outside fp32)
 * relu's slope is 0 at 0.  An output may be any of the inputs, in the same layout, but not the other output.  fp32 slopes of silu and gelu are within
 * 24 * 2^-24 of the sum of their terms' absolute values (s + |z| s (1 - s), and Phi + |z| phi); for bf16 results within 2^-14.
 * Asynchronous. */
moe_status moe_async_act_mul_backward(int32_t dtype, int32_t act, const void* d_grad, int64_t grad_stride, const void* d_z, int64_t z_stride,
                                      const void* d_mul, int64_t mul_stride, int32_t T, int32_t H, void* d_grad_z, int64_t grad_z_stride,
                                      void* d_grad_mul, int64_t grad_mul_stride, void* stream);

/* Synchronise `stream`, return the error of the stateless operators on the current device and clear
 * it: MOE_OK, or MOE_ERR_TIMEOUT if a device wait in a product exceeded its 2 s bound since
 * the last report, on any stream (that call's output is then undefined). */
moe_status moe_async_ops_status(void* stream);

/* Bounds-checked build (libmoe_async_debug.so, compiled with MOE_DEBUG_BOUNDS): every bucket,
 * slot and k index the kernels read back from device state is checked before use, and an
 * index out of range latches MOE_ERR_BOUNDS (the access is skipped, the scheduler halts).  This
 * call appends the raw value `record` (slot << 5 | k, unchecked) to bucket `bucket` of `layer`,
 * so a test can plant an out-of-range record and see it rejected without touching memory
 * out of range.  Release builds return MOE_ERR_UNSUPPORTED and write nothing.  Asynchronous. */
moe_status moe_async_debug_append_record(moe_async_t h, int32_t layer, int32_t bucket, int32_t record,
                                        void* stream);

/* The bounds-checked build sets the error of moe_async_ops_status to MOE_ERR_TIMEOUT, so a test can see
 * it reported without a wait that runs out.  Release builds return MOE_ERR_UNSUPPORTED. */
moe_status moe_async_debug_latch_ops_error(void* stream);

/* The same for one of the words behind it: 0 the product's (the call above), 1 its gradients', 2 the block-scaled product's; another
 * word is MOE_ERR_INVALID. */
moe_status moe_async_debug_latch_ops_word(int32_t word, void* stream);

/* 1 if the kernels can write `n` bytes at host address `p` directly (pinned host memory
 * mapped into the device's address space at the same address), else 0.  A caller may then
 * pass such a buffer as a collect output (d_y_out, d_slot_out, ...), so each merged row goes
 * to host memory as it is produced instead of by a copy after the step.  Host-side query, no
 * device work. */
int32_t moe_async_host_writable(const void* p, int64_t n);

/* Human-readable name of a status code (static string). */
const char* moe_async_status_string(moe_status s);

#ifdef __cplusplus
}
#endif
#endif /* MOE_ASYNC_H */
