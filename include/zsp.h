/*
 * zsp.h -- C ABI of libzsp, the per-rank hot path of ZeRO-3 intra-layer
 * partitioning on one MI355X (gfx950): N_d data-parallel ranks live as
 * "virtual ranks" in one GPU's memory and every exchange between them is a
 * local HIP kernel.
 *
 * Pages the operations follow (cited by title and section):
 *   [ZD]  "The ZeRO-3 Diagram Most People Remember Is Wrong"
 *         section 2 (flatten, pad, contiguous slice per rank) and section 3
 *         (AllGather before compute, ReduceScatter of gradients, optimizer
 *         updates the local shard)
 *   [ZS3] "ZeRO Stage 3: Parameter Partitioning" (on-demand fetch steps,
 *         equation M_Stage3 and its 7B / 64-GPU example)
 *   [ZST] "ZeRO Stages: Sharding Optimizer State, Gradients, and Parameters"
 *         ("What stage 1 partitions": rank i owns [i*N/P, (i+1)*N/P);
 *          "Stage 2 also partitions gradients": reduce-scatter, shard-sized
 *          gradient buffer, each micro-batch's reduced shard summed into a
 *          running one)
 * The Adam update is the textbook one (Kingma & Ba, Algorithm 1), which the
 * pages name without printing.
 *
 * Terms
 *   nd            number of data-parallel ranks (N_d), 1..ZSP_MAX_RANKS
 *   numel[t]      element count of parameter t, flattened row-major
 *   pad[t]        (nd - numel[t] % nd) % nd
 *   shard_len[t]  (numel[t] + pad[t]) / nd   -- s_t
 *   S             sum of shard_len over all parameters: elements one rank owns
 *   full_off[t]   sum_{u<t} (numel[u] + pad[u])   (full padded layout)
 *   shard_off[t]  sum_{u<t} shard_len[u]          (a rank's shard layout)
 *   flat_off[t]   sum_{u<t} numel[u]              (unpadded concatenation)
 *   total_numel   sum of numel over all parameters
 *   Rank r owns elements [r*s_t, (r+1)*s_t) of padded parameter t and stores
 *   them at shard_off[t] of its shard; positions >= numel[t] are pad.
 *
 * Memory and ownership
 *   The caller allocates and owns every device buffer (parameters, gradients,
 *   optimizer state, accumulator, gather outputs, schedule arenas). A plan
 *   owns its host tables, the device copies of its offset tables (allocated
 *   in zsp_bind_state), the staging slots of long zsp_gather_many lists
 *   (allocated when such a list first needs them; prepared lists,
 *   zsp_gather_list_create and zsp_tensor_list_create, own memory of their
 *   own) and, from its first checkpoint save or load, the checkpoint staging
 *   (pinned host chunks, streams, events); zsp_destroy frees them. The other
 *   hot-path calls (reduce, norm, clip, Adam, the range and single gathers,
 *   schedule acquire and release) allocate nothing on the device; checkpoint
 *   calls also use host memory for their own duration. The reduce, norm, clip,
 *   Adam, range and single gather calls, zsp_gather_list_run, and
 *   zsp_gather_many on lists of at most 64 parameters, only check arguments
 *   and launch kernels (no host wait, no copy, no memset), so they can be
 *   captured into a HIP graph; Adam's scalars (lr, betas, eps and the step's
 *   bias corrections) are kernel arguments, so a replay repeats the step it
 *   was captured with (a clipped step reads its coefficient from device
 *   memory, so a replay uses the one that is there then).
 *   Every device pointer must be 16-byte aligned (torch allocations are),
 *   but for the tensors of a list to clip or to take the norm of.
 *   State arrays bound for all ranks hold nd*S elements, rank r at
 *   [r*S, (r+1)*S); bound for one rank j they hold that rank's S elements.
 *
 * Streams
 *   Every call that touches the device enqueues its kernels on `stream` (a
 *   hipStream_t; NULL is the default stream) and returns without waiting,
 *   unless its own comment says that it waits.
 *   The caller keeps buffers alive until the stream has run them. The plan is
 *   tied to the device that was current at zsp_bind_state; calls made with
 *   another device current fail with ZSP_ESTATE.
 *
 * Errors
 *   Arguments are checked before anything is enqueued; a bad argument returns
 *   a negative zsp_status and enqueues nothing. A failed kernel launch returns
 *   ZSP_EHIP. zsp_last_error() gives a message for the calling thread's most
 *   recent failure. Values are not checked: NaN and Inf propagate.
 *
 * Threads
 *   The reduce, norm, Adam and gather calls (whole-model and _params forms,
 *   list gathers, prepared-list create and run) and zsp_load_params only read
 *   the plan (zsp_gather_many takes the plan's staging slots under a lock
 *   of their own): several threads may issue them on one plan at once, e.g.
 *   one thread per rank, each on its own stream (work that writes the same
 *   state at the same time is the caller's race, as for any two kernels).
 *   zsp_bind_state, the checkpoint calls and zsp_destroy change the plan
 *   and must not overlap any other call on it.
 *   A schedule's calls must not overlap one another; other schedules and
 *   the read-only calls above may run beside them. Different plans are
 *   independent.
 */
#ifndef ZSP_H
#define ZSP_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct zsp_plan zsp_plan;
typedef struct zsp_sched zsp_sched;
typedef struct zsp_gather_list zsp_gather_list;
typedef struct zsp_tensor_list zsp_tensor_list;

typedef enum {
    ZSP_OK = 0,
    ZSP_EINVAL = -1, /* bad argument: null/misaligned pointer, bad rank, dtype, ... */
    ZSP_ERANGE = -2, /* index or size out of the supported range */
    ZSP_ENOMEM = -3, /* host or device allocation for the plan's tables failed */
    ZSP_EHIP = -4,   /* a HIP runtime call or kernel launch failed */
    ZSP_ESTATE = -5, /* call not valid in the plan's current binding/device */
    ZSP_EIO = -6     /* checkpoint file missing, unreadable, corrupt or of another model */
} zsp_status;

typedef enum { ZSP_F32 = 0, ZSP_BF16 = 1 } zsp_dtype;

typedef enum {
    ZSP_GRADS_FULL = 0,  /* grads[r]: rank r's full padded gradient, tensor t at full_off[t] */
    ZSP_GRADS_SHARD = 1  /* grads[r]: indexed like the bound state arrays (see below) */
} zsp_grad_layout;

typedef enum {
    ZSP_SRC_WORK = 0,    /* bf16 working copy of the parameters */
    ZSP_SRC_MASTER = 1,  /* fp32 master parameters */
    ZSP_SRC_ACC = 2      /* fp32 gradient accumulator: each rank's reduced slice */
} zsp_source;

typedef enum {
    ZSP_NORM_L2 = 0, /* square root of the sum of squares */
    ZSP_NORM_MAX = 1 /* largest absolute value */
} zsp_norm_kind;

/* What a norm call leaves in device memory (see "Gradient norm and clipping"). */
typedef struct zsp_clip {
    double total; /* ZSP_NORM_L2: the sum of squares; ZSP_NORM_MAX: the largest |g| */
    float norm;   /* infinity where it is beyond fp32; total and coef still hold */
    float coef;   /* 1, or max_norm / norm where norm > max_norm; NaN: norm not finite */
} zsp_clip;

#define ZSP_ALL_RANKS (-1)
#define ZSP_MAX_RANKS 256

/* partition(param list, N_d) -- [ZD] section 2; [ZST] "What stage 1
 * partitions". Builds the per-parameter layout tables for n_params
 * parameters of numel[0..n_params) elements split over n_d ranks. Host only:
 * touches no device. n_params >= 1, numel[t] >= 0, 1 <= n_d <= ZSP_MAX_RANKS.
 * On success *out receives a new plan (free with zsp_destroy). */
zsp_status zsp_partition(const int64_t* numel, int32_t n_params, int32_t n_d,
                         zsp_plan** out);

/* Release the plan, its host tables and its device tables. NULL is ignored.
 * The caller must make sure no enqueued work still reads the tables. */
void zsp_destroy(zsp_plan* plan);

/* Sizes of the plan. Any output pointer may be NULL.
 *   shard_elems  S
 *   total_padded sum of numel+pad (elements of one full-layout gradient)
 *   model_state_bytes_per_rank  16*S: 16-bit param + 16-bit grad + fp32
 *     master + fp32 m + fp32 v per owned element ([ZS3] equation M_Stage3).
 * total_numel and flat_off[t] (see Terms) follow from the numel list. */
zsp_status zsp_plan_info(const zsp_plan* plan, int64_t* shard_elems, int64_t* total_padded,
                         int64_t* model_state_bytes_per_rank);

/* Layout of parameter t (0 <= t < n_params). Any output pointer may be NULL.
 * full_off: its offset in a full-layout gradient; shard_off: its slot's
 * offset in each rank's shard. */
zsp_status zsp_plan_tensor(const zsp_plan* plan, int32_t t, int64_t* numel, int64_t* pad,
                           int64_t* shard_len, int64_t* full_off, int64_t* shard_off);

/* Bind the caller-owned optimizer state and build the device tables.
 *   rank_or_all = ZSP_ALL_RANKS: every array holds n_d*S elements (all ranks
 *     resident on this GPU); every rank-taking call may name any rank or all.
 *   rank_or_all = j: every array holds rank j's S elements only; calls must
 *     name rank j, and gathers are not possible (ZSP_ESTATE).
 *   master, m, v: fp32; work: bf16 bit patterns; grad_acc: fp32 accumulator
 *     or NULL (then accumulate/use_acc calls fail with ZSP_ESTATE).
 * Allocates the device tables (setup path): 40 bytes per bound piece (one
 * rank's slice of one parameter) and 4 bytes per 512 elements of the bound
 * state; an all-rank binding adds the gather's 16 bytes per piece, 36 bytes
 * per 512 elements of the unpadded parameters and 32 bytes per parameter.
 * Rebinding replaces the previous binding. */
zsp_status zsp_bind_state(zsp_plan* plan, int32_t rank_or_all, float* master, float* m,
                          float* v, uint16_t* work, float* grad_acc);

/* Copy-in ([ZD] section 2, steps 1-4): split the unpadded parameters into the
 * bound ranks' shards. flat_params holds total_numel elements of `dtype`,
 * parameter t at flat_off[t]. Writes master = fp32(x), work = x (bf16 input)
 * or its round-to-nearest-even bf16 (fp32 input), m = v = 0, and +0 at every
 * pad position of all four arrays. */
zsp_status zsp_load_params(zsp_plan* plan, const void* flat_params, zsp_dtype dtype,
                           void* stream);

/* reduce_shard(rank, grads[N_d]) -- ReduceScatter restricted to the owned
 * slice ([ZD] section 3; [ZST] "Stage 2 also partitions gradients").
 * For each owned non-pad element: red = sum over r = 0..n_d-1, in rank
 * order, of fp32(grads[r][...]), one fp32 addition at a time starting from
 * rank 0's value. Writes grad_acc = red (accumulate = 0) or
 * grad_acc = grad_acc + red (accumulate = 1); pad positions of grad_acc are
 * set to +0. grads: n_d device pointers (host array) of `dtype`.
 *   ZSP_GRADS_FULL : grads[r] holds total_padded elements; the element of
 *                    parameter t at padded index k is at full_off[t] + k.
 *   ZSP_GRADS_SHARD: grads[r] is the chunk rank r sends to the owners, in the
 *                    bound arrays' indexing: S elements for a one-rank
 *                    binding, n_d*S (owner j at j*S) for an all-rank one.
 * Pad positions of grads are never read. rank_or_all: a rank or
 * ZSP_ALL_RANKS (all-rank binding only). */
zsp_status zsp_reduce_shard(zsp_plan* plan, int32_t rank_or_all, const void* const* grads,
                            zsp_dtype dtype, zsp_grad_layout layout, int32_t accumulate,
                            void* stream);

/* adam_step(shard, lr, beta1, beta2, eps, step) -- the optimizer updates the
 * local shard ([ZD] section 3; [ZS3] on-demand fetch, last step; [ZST]).
 * Uses grad_acc as the gradient. For each owned non-pad element, in fp32 with
 * one rounding per operation, in this order:
 *   m = beta1*m + (1-beta1)*g ;  v = beta2*v + (1-beta2)*(g*g)
 *   mh = m/(1-beta1^step) ;  vh = v/(1-beta2^step)
 *   master = master - (lr*mh)/(sqrt(vh) + eps) ;  work = bf16_rne(master)
 * 1-beta is computed in fp32; 1-beta^step in double and rounded once to
 * fp32. Pad positions are not touched. step >= 1. */
zsp_status zsp_adam_step(zsp_plan* plan, int32_t rank_or_all, float lr, float beta1,
                         float beta2, float eps, int64_t step, void* stream);

/* The hot path: reduce_shard and adam_step fused in one pass. g = red
 * (use_acc = 0) or g = grad_acc + red (use_acc = 1, the last micro-batch of
 * an accumulation window); the reduced gradient stays in registers and
 * grad_acc is not written. Same arithmetic, bit for bit, as reduce_shard
 * followed by adam_step. */
zsp_status zsp_reduce_adam_step(zsp_plan* plan, int32_t rank_or_all,
                                const void* const* grads, zsp_dtype dtype,
                                zsp_grad_layout layout, int32_t use_acc, float lr,
                                float beta1, float beta2, float eps, int64_t step,
                                void* stream);

/* The three calls above restricted to the parameters [first_param,
 * first_param + n_params): only those parameters' slots of each rank the
 * call names are read or written; every other slot, the accumulator's
 * included, is untouched. This is the reduce-scatter of one layer during
 * backward ([ZD] section 6: gradient reduce-scatters appear during backward;
 * [ZS3]: after a layer's backward its gradients go to the ranks owning
 * them), or the update of one layer. grads[] are the same whole-model
 * buffers as above. Each rank's slots of a parameter range are one
 * contiguous span, so the call is one launch per rank (one launch for every
 * parameter). ZSP_ERANGE if the range is empty or outside [0, n_params). */
zsp_status zsp_reduce_shard_params(zsp_plan* plan, int32_t rank_or_all, int32_t first_param,
                                   int32_t n_params, const void* const* grads, zsp_dtype dtype,
                                   zsp_grad_layout layout, int32_t accumulate, void* stream);
zsp_status zsp_adam_step_params(zsp_plan* plan, int32_t rank_or_all, int32_t first_param,
                                int32_t n_params, float lr, float beta1, float beta2, float eps,
                                int64_t step, void* stream);
zsp_status zsp_reduce_adam_step_params(zsp_plan* plan, int32_t rank_or_all, int32_t first_param,
                                       int32_t n_params, const void* const* grads,
                                       zsp_dtype dtype, zsp_grad_layout layout, int32_t use_acc,
                                       float lr, float beta1, float beta2, float eps,
                                       int64_t step, void* stream);

/* gather(param_id) -- AllGather of a full parameter just before compute
 * ([ZD] section 3; [ZS3] on-demand fetch, step 2; [ZST] "Stage 3
 * partitions parameters"). Writes numel[param_id] elements to `out`, pad
 * dropped: out[k] = src_r[shard_off[t] + k - r*s_t] with r = k / s_t.
 * src = ZSP_SRC_WORK (bf16 out), ZSP_SRC_MASTER (fp32 out) or ZSP_SRC_ACC
 * (fp32 out, needs an accumulator bound): gathering the reduced gradient
 * slices completes an all-reduce of the gradients, the reduction stage 1
 * keeps ([ZST] "What stage 1 partitions": gradients arrive complete on
 * every rank, each rank updates its own slice); pad slots are dropped as
 * for parameters. Needs an all-rank binding. */
zsp_status zsp_gather(zsp_plan* plan, int32_t param_id, zsp_source src, void* out,
                      void* stream);

/* Gather of the consecutive parameters [first_param, first_param +
 * n_params) -- one layer's worth, e.g. -- in one launch ([ZD] section 3:
 * each layer's parameters are all-gathered just before it runs). `out`
 * receives them back to back, unpadded: parameter t at flat_off[t] -
 * flat_off[first_param]. ZSP_ERANGE if the range is empty or outside
 * [0, n_params). The per-layer schedule below uses this gather. */
zsp_status zsp_gather_range(zsp_plan* plan, int32_t first_param, int32_t n_params,
                            zsp_source src, void* out, void* stream);

/* gather(param_id) for a list of parameters: ids[0..n) in any order
 * (repeats allowed), parameter ids[i] into its own output outs[i]
 * (numel[ids[i]] elements, unpadded, as zsp_gather writes them). This is
 * the all-gather of a bucket of parameters, e.g. the module about to run
 * ([ZD] section 3: a module's full parameters are gathered just before its
 * forward and again before its backward; section 8: gathers go out in
 * buckets of parameters). ids and outs are host arrays, read during the
 * call; every outs[i] of a non-empty parameter must be a 16-byte aligned
 * device pointer (NULL is allowed for empty ones); outputs must not
 * overlap one another or the bound state. n = 0 does nothing.
 *   Lists of at most 64 non-empty parameters: one launch, nothing staged.
 *   Longer lists: their entries (16 bytes per parameter plus 4 bytes per
 *   32768 output elements) go to the device through one of four staging
 *   slots the plan keeps (a copy kernel reads them from the slot's pinned
 *   host buffer), then two launches per chunk of records. A slot is allocated
 *   (pinned host and device memory) the first time a list needs more room
 *   than it has -- the only allocation of any gather call -- and is refilled
 *   only after the gathers of its previous use have run: the call waits on
 *   the host when four staged gathers are still in flight. Each slot holds
 *   the records of at most 2^19 tiles of 512 elements (16 MiB); longer
 *   lists go in several pairs of launches.
 * Errors: ZSP_ERANGE for an id outside [0, n_params) or a list of 2^31
 * tiles or more; ZSP_EINVAL for NULL arrays with n > 0, a NULL or
 * misaligned output, or n < 0; ZSP_ESTATE without an all-rank binding;
 * ZSP_ENOMEM if a staging slot cannot grow. Needs an all-rank binding. */
zsp_status zsp_gather_many(zsp_plan* plan, const int32_t* ids, int32_t n, zsp_source src,
                           void* const* outs, void* stream);

/* zsp_gather_many for callers that cannot allocate (tight serving loops,
 * harnesses that forbid allocation, and code under HIP graph capture for
 * lists of at most 64 non-empty parameters, which are one kernel launch):
 * the same arguments, checks and results, but nothing is allocated, on the
 * device or the host. A longer list's staging copy reads a host buffer that
 * the next call refills, so a captured copy would replay stale entries:
 * capture such lists as a prepared list (zsp_gather_list_run) instead.
 * A long list (more than 64 non-empty parameters) is staged
 * in a fixed device array the library holds on every GPU it runs on from
 * load to process end (9.25 MiB): its entries and coarse index are copied
 * there from a static host buffer, then the same two kernels run. Limits:
 * at most 65536 non-empty parameters and 2^22 tiles of 512 elements (2^31
 * elements) per call, else ZSP_ERANGE; longer lists than 2^18 tiles run in
 * several pairs of launches. The array keeps the last call's contents and
 * every call on a GPU shares it: calls on one stream run in order, but
 * calls that overlap on one GPU (other streams or threads) race. The array's
 * address is taken at an all-rank zsp_bind_state (or the first call) on
 * each device. Lists of at most 64 non-empty parameters touch no staging
 * at all, as in zsp_gather_many. */
zsp_status zsp_gather_many_noalloc(zsp_plan* plan, const int32_t* ids, int32_t n,
                                   zsp_source src, void* const* outs, void* stream);

/* A list gather prepared once and run many times: the same bucket into the
 * same outputs every step ([ZD] section 3: a module's parameters are
 * gathered before its forward and again before its backward, every step;
 * section 8: gathers go out in buckets). zsp_gather_list_create takes the
 * arguments of zsp_gather_many, with the same checks and errors, and keeps
 * what a run needs: for a list of more than 64 non-empty parameters, its
 * per-tile records (32 bytes per 512 output elements, plus 16 bytes per
 * parameter), built on the device once -- create allocates that memory,
 * enqueues the build on `stream` and waits for it before returning
 * (ZSP_ENOMEM if the allocation fails). Lists of at most 64 keep their
 * entries on the host and run as zsp_gather_many's one launch.
 *   zsp_gather_list_run enqueues the gather on `stream`: one launch, no
 * copy, no allocation, no host wait (capturable into a HIP graph). It reads
 * the source named at create from the plan's current binding, so the list
 * stays valid when state is bound again on the same device; the outputs
 * named at create must stay allocated while runs may be in flight.
 * ZSP_ESTATE if the plan has no all-rank binding now, is bound on another
 * device than at create, or the source is the accumulator and none is
 * bound; ZSP_EINVAL for a NULL list.
 *   zsp_gather_list_destroy frees the list (NULL is a no-op); runs must have
 * finished. A list refers to its plan, which must outlive it. */
zsp_status zsp_gather_list_create(zsp_plan* plan, const int32_t* ids, int32_t n,
                                  zsp_source src, void* const* outs, void* stream,
                                  zsp_gather_list** list);
zsp_status zsp_gather_list_run(zsp_gather_list* list, void* stream);
void zsp_gather_list_destroy(zsp_gather_list* list);

/* ---- Gradient norm and clipping --------------------------------------------
 * The global norm of the gradients, and the step with gradients scaled down
 * to a largest norm:
 *   ZSP_NORM_L2   total = sum of g*g, norm = sqrt(total)
 *   ZSP_NORM_MAX  total = largest |g|, norm = total
 *   coef = 1 if norm <= max_norm, else max_norm / norm
 * Squares are summed in 64 bits, so no finite gradient's square is lost or
 * overflows; coef is computed in 64 bits and rounded once to fp32. If the
 * total is infinite or NaN, coef is NaN, and a call that takes the record
 * then changes nothing: the update of a step whose gradients are not finite
 * is skipped. max_norm >= 0 (INFINITY: only the norm is wanted, coef is 1
 * for every finite norm). Nothing here brings a value to the host, and only
 * zsp_tensor_list_create waits for the device: the record (zsp_clip) stays in
 * device memory, from where the clipped calls read the coefficient.
 *   Every call that makes a norm writes one record to `out` (device memory,
 * 16-byte aligned) and uses a workspace `ws` (device memory, 16-byte aligned,
 * ws_bytes >= what zsp_norm_workspace says; its contents mean nothing between
 * calls). Calls in one stream's order may share a workspace; calls that may
 * run at the same time, replays of captured graphs among them, each need
 * their own. Equal inputs give equal bits.
 *   Errors beside each call's own: ZSP_EINVAL for a bad kind, a negative or
 * NaN max_norm, a NULL or misaligned ws, out or clip; ZSP_ERANGE if ws_bytes
 * is too small. */

/* Workspace bytes for the norm calls on `plan` as it is bound now (before
 * it is bound: as for all ranks): the larger of 35,856 bytes and
 * 16 * (E / 512) + 32 * nd + 1072, E the elements of the bound state and the
 * quotient rounded down. With plan NULL, for norms of lists of tensors:
 * 35,856. Host only. A plan's workspace also serves lists. */
zsp_status zsp_norm_workspace(const zsp_plan* plan, int64_t* bytes);

/* Norm of the bound accumulator's real elements (pad slots are left out,
 * whatever they hold), of one rank or all, whole-model or parameters
 * [first_param, first_param + n_params). Needs an accumulator bound. */
zsp_status zsp_grad_norm(zsp_plan* plan, int32_t rank_or_all, zsp_norm_kind kind, double max_norm,
                         void* ws, int64_t ws_bytes, zsp_clip* out, void* stream);
zsp_status zsp_grad_norm_params(zsp_plan* plan, int32_t rank_or_all, int32_t first_param,
                                int32_t n_params, zsp_norm_kind kind, double max_norm, void* ws,
                                int64_t ws_bytes, zsp_clip* out, void* stream);

/* zsp_reduce_shard (_params) with the norm of the accumulator elements it
 * writes, in the same pass over the gradients: grad_acc is what
 * zsp_reduce_shard leaves, bit for bit. */
zsp_status zsp_reduce_shard_norm(zsp_plan* plan, int32_t rank_or_all, const void* const* grads,
                                 zsp_dtype dtype, zsp_grad_layout layout, int32_t accumulate,
                                 zsp_norm_kind kind, double max_norm, void* ws, int64_t ws_bytes,
                                 zsp_clip* out, void* stream);
zsp_status zsp_reduce_shard_norm_params(zsp_plan* plan, int32_t rank_or_all, int32_t first_param,
                                        int32_t n_params, const void* const* grads,
                                        zsp_dtype dtype, zsp_grad_layout layout,
                                        int32_t accumulate, zsp_norm_kind kind, double max_norm,
                                        void* ws, int64_t ws_bytes, zsp_clip* out, void* stream);

/* The norm of the gradient that zsp_reduce_adam_step (use_acc likewise) would
 * use, whole-model, writing nothing but the record: with
 * zsp_reduce_adam_step_clip, the clipped step of a caller that keeps no
 * accumulator. Reads the gradients once more than an unclipped step. */
zsp_status zsp_reduce_norm(zsp_plan* plan, int32_t rank_or_all, const void* const* grads,
                           zsp_dtype dtype, zsp_grad_layout layout, int32_t use_acc,
                           zsp_norm_kind kind, double max_norm, void* ws, int64_t ws_bytes,
                           zsp_clip* out, void* stream);

/* Joins the totals of n >= 0 records into one: the layers' records of a
 * backward pass that reduced layer by layer, or one record whose total was
 * summed (ZSP_NORM_MAX: maximised) over the processes of a data-parallel
 * group. parts: n records in device memory, 16-byte aligned; only their
 * totals are read. out may be one of them. No records: norm 0. */
zsp_status zsp_clip_combine(const zsp_clip* parts, int32_t n, zsp_norm_kind kind, double max_norm,
                            zsp_clip* out, void* stream);

/* zsp_adam_step and zsp_reduce_adam_step (_params) with the gradient g
 * replaced by g * coef (one fp32 rounding), coef read from *clip in device
 * memory when the kernel runs. coef NaN: no state of the named slots
 * changes. The accumulator keeps the gradient as it was. A record of the
 * whole model's norm clips every call of a step, layer by layer or whole. */
zsp_status zsp_adam_step_clip(zsp_plan* plan, int32_t rank_or_all, const zsp_clip* clip, float lr,
                              float beta1, float beta2, float eps, int64_t step, void* stream);
zsp_status zsp_adam_step_clip_params(zsp_plan* plan, int32_t rank_or_all, int32_t first_param,
                                     int32_t n_params, const zsp_clip* clip, float lr,
                                     float beta1, float beta2, float eps, int64_t step,
                                     void* stream);
zsp_status zsp_reduce_adam_step_clip(zsp_plan* plan, int32_t rank_or_all,
                                     const void* const* grads, zsp_dtype dtype,
                                     zsp_grad_layout layout, int32_t use_acc,
                                     const zsp_clip* clip, float lr, float beta1, float beta2,
                                     float eps, int64_t step, void* stream);
zsp_status zsp_reduce_adam_step_clip_params(zsp_plan* plan, int32_t rank_or_all,
                                            int32_t first_param, int32_t n_params,
                                            const void* const* grads, zsp_dtype dtype,
                                            zsp_grad_layout layout, int32_t use_acc,
                                            const zsp_clip* clip, float lr, float beta1,
                                            float beta2, float eps, int64_t step, void* stream);

/* The same for gradients that are not sharded (stages 0 and 1): the norm of
 * n tensors taken together, and their scaling in place by a record's coef
 * (x = x * coef in fp32, rounded once more to bf16 for a bf16 tensor; coef 1
 * or NaN: nothing is written). Tensor i is numel[i] contiguous elements of
 * type dtype[i] (a zsp_dtype) at x[i], which needs the alignment of its
 * element type only; NULL is allowed for empty ones. The three arrays are
 * host arrays, read during the call. The same tensor twice counts twice in a
 * norm; a clip refuses tensors that overlap (ZSP_EINVAL). Tensors travel in
 * kernel arguments, 128 per launch (launches follow one another on the
 * stream); a list that is used again and again is better prepared.
 * ZSP_EINVAL: n < 0, NULL arrays with n > 0, a negative numel, a bad dtype, a
 * NULL or misaligned tensor; ZSP_ERANGE: 2^31 chunks of 8 KiB or more,
 * counted per tensor. No plan is involved: all tensors, ws, out and
 * clip are on the current device. */
zsp_status zsp_norm_many(const void* const* x, const int64_t* numel, const int32_t* dtype,
                         int32_t n, zsp_norm_kind kind, double max_norm, void* ws,
                         int64_t ws_bytes, zsp_clip* out, void* stream);
zsp_status zsp_clip_many(void* const* x, const int64_t* numel, const int32_t* dtype, int32_t n,
                         const zsp_clip* clip, void* stream);

/* A list of tensors prepared once: zsp_tensor_list_create takes the arrays of
 * zsp_norm_many, with the same checks, and keeps on the current device a
 * record of 16 bytes per 8 KiB of each tensor (allocated, filled on
 * `stream` and waited for before it returns). _norm and _clip are then as
 * zsp_norm_many and zsp_clip_many, each over the whole list in one pass, and
 * need that device current (ZSP_ESTATE). The tensors must stay allocated.
 * Calls only read the list: several threads and streams may use it at once,
 * each norm with a workspace of its own. _destroy frees it (NULL is a no-op);
 * calls on it must have finished. */
zsp_status zsp_tensor_list_create(void* const* x, const int64_t* numel, const int32_t* dtype,
                                  int32_t n, void* stream, zsp_tensor_list** list);
zsp_status zsp_tensor_list_norm(const zsp_tensor_list* list, zsp_norm_kind kind, double max_norm,
                                void* ws, int64_t ws_bytes, zsp_clip* out, void* stream);
zsp_status zsp_tensor_list_clip(const zsp_tensor_list* list, const zsp_clip* clip, void* stream);
void zsp_tensor_list_destroy(zsp_tensor_list* list);

/* ---- Losses over the head ----------------------------------------------------
 * Where a step turns from forward to backward: the loss over the model's
 * output matrix (the head, a parameter of v rows of d elements, e.g. as a
 * gather or the schedule below leaves it) and the gradients that the backward
 * starts with. grad_head is a rank's gradient of that parameter, in the type
 * and order that zsp_reduce_shard reads: it may lie in grads[r] at full_off.
 *   l_iv = (hidden_i . head_v) / T     lse_i = log(sum over v of exp(l_iv))
 *   p_iv = exp(l_iv - lse_i)
 * zsp_head_loss    softmax cross entropy with one target per token, T = 1:
 *     loss_i = lse_i - l_i,target        g_iv = p_iv - [v = target_i]
 * zsp_head_distill distillation from the teacher's `top` largest logits per
 *     token, logit[i, k] at index[i, k]; q_ik = softmax over the token's k of
 *     logit[i, k] / T:
 *     loss_i = T^2 * sum over k of q_ik * (log q_ik - log p_i,index[i,k])
 *     g_iv = T * (p_iv - sum of q_ik over the k with index[i, k] = v)
 * Both leave loss [n] and, unless NULL, lse [n] (fp32) and the gradients of
 *     scale * sum over i of token_weight_i * loss_i
 * with regard to hidden, sum over v of scale * token_weight_i * g_iv *
 * head_v, in grad_hidden [n, d], and with regard to head, sum over i of
 * scale * token_weight_i * g_iv * hidden_i, in grad_head [v, d]. A NULL
 * gradient is not computed; token_weight NULL is 1 for every token.
 *   A token counts if its target (one of its indices) lies in [0, v) and its
 * weight is not 0. Of a token that does not count, loss, lse and its row of
 * grad_hidden are 0 and nothing reaches grad_head, whatever its row of
 * hidden holds; the batch costs what the tokens that count cost. Of a
 * token's entries those with an index outside [0, v) or a logit of -infinity
 * are left out; a token without any other does not count. An index that
 * occurs twice is two entries. The logits are not kept: a call with
 * gradients keeps the softmax of some of its tokens at a time in the
 * workspace, up to 4 GiB, or of 256 tokens (64, of a call with no more) where
 * those take more.
 *   hidden, head and the gradients are all of `dtype`. Products are summed
 * in fp32 (operands of fp32 type are split into three bf16 values, exactly,
 * and products below 2^-23 of a term left out). Of an infinity in hidden or
 * head, and in fp32 of a value beyond bf16's largest, a NaN may come. The
 * softmax is taken in fp32, its sums too within 64 columns (where the logits
 * are summed in parts, of a vocabulary up to 8192, within a thread's columns of
 * a row) and in 64 bits over them; the losses, a target's own g and logits'
 * differences from lse are taken in 64 bits. For bf16, token_weight_i * g_iv / T
 * is rounded to bf16 once before the two products that make the gradients (p
 * comes to it within 2^-11 of itself, as 0 below 2^-63.9 of the largest of its
 * 64 columns); calls with fp32 copies of hidden and head round nothing to bf16.
 * scale * T comes to the products' sums in fp32. Equal inputs give equal bits.
 *   0 <= n <= 2^23 tokens, 1 <= v <= 2^22, 1 <= d <= 65536, top <= 1024, n *
 * d below about 2^34. Pointers need the alignment of their element type
 * only, ws 16 bytes; a head on 16 bytes whose d is a multiple of 8 is read
 * in place (fp32: of 4, by up to 64 tokens), any other is copied into the
 * workspace first. No plan is involved: all tensors are on the current
 * device. Nothing is waited for, copied by the host or allocated, so calls
 * can be captured into a HIP graph. A workspace's contents mean nothing
 * between calls; calls that may run at the same time, replays of captured
 * graphs among them, each need their own.
 *   ZSP_EINVAL: a bad dtype, a negative size, v or d of 0, a NULL or
 * misaligned argument, scale, temperature, their product or log2(e) /
 * temperature not finite, temperature <= 0, an output that overlaps another
 * argument; ZSP_ERANGE: a size beyond the limits, ws_bytes too small. n = 0:
 * grad_head is set to 0. */
#define ZSP_HEAD_GRAD_HIDDEN 1 /* grad_hidden is wanted */
#define ZSP_HEAD_GRAD_HEAD 2   /* grad_head is wanted */
#define ZSP_HEAD_UNALIGNED 4   /* head may start off a 16-byte boundary */

/* Workspace bytes of calls of up to n tokens and `top` entries (0 for
 * zsp_head_loss alone), with any of the gradients that flags (of the above)
 * name. (A call of fewer tokens may cut its sums into more parts, or its tokens
 * into larger chunks; the answer holds all of them.) Host only. */
zsp_status zsp_head_workspace(int64_t n, int64_t v, int64_t d, zsp_dtype dtype, int32_t top,
                              int32_t flags, int64_t* bytes);
zsp_status zsp_head_loss(const void* hidden, const void* head, zsp_dtype dtype, int64_t n,
                         int64_t v, int64_t d, const int64_t* target, const float* token_weight,
                         float scale, float* loss, float* lse, void* grad_hidden, void* grad_head,
                         void* ws, int64_t ws_bytes, void* stream);
zsp_status zsp_head_distill(const void* hidden, const void* head, zsp_dtype dtype, int64_t n,
                            int64_t v, int64_t d, const int64_t* index, const float* logit,
                            int32_t top, float temperature, const float* token_weight, float scale,
                            float* loss, float* lse, void* grad_hidden, void* grad_head, void* ws,
                            int64_t ws_bytes, void* stream);

/* ---- Per-layer gather schedule with prefetch ------------------------------
 * [ZS3] on-demand fetch list (gather layer l before its computation, discard
 * after) and prefetch paragraph (gather layer l+1 while layer l computes);
 * [ZST] "Stage 3 partitions parameters" (gather before forward, again before
 * backward, release after use; prefetch depth trades memory for latency).
 * A schedule visits groups of consecutive parameters (one layer each) in a
 * fixed order of positions. Position p is gathered into slot p mod (D+1) of
 * a caller-owned device arena, D = prefetch depth; with D > 0 the gathers of
 * positions up to p+D run on a gather stream of the caller's while the
 * compute stream works on p. All ordering is by HIP events (no host waits):
 * a gather into a slot follows the release of the slot's previous position,
 * a pass's first gathers follow what the compute stream did before position
 * 0's acquire (e.g. the optimizer step), and the compute stream's work after
 * an acquire follows that position's gather. D = 0 gathers on the compute
 * stream in line. The plan must outlive the schedule. */

/* Build a schedule over `plan` (host only). Group g is the parameters
 * [group_first[g], group_first[g] + group_count[g]); order[p] is the group
 * of position p, 0 <= p < n_steps. 0 <= depth <= 64 (depths beyond
 * n_steps - 1 act as n_steps - 1). *arena_bytes receives the device bytes
 * zsp_sched_bind needs: (D+1) slots, each the largest group's gathered size
 * (2 B per element for ZSP_SRC_WORK, 4 for ZSP_SRC_MASTER) rounded up to
 * 256 B. Every gather is zsp_gather_range's kernel. */
zsp_status zsp_sched_create(zsp_plan* plan, int32_t n_groups, const int32_t* group_first,
                            const int32_t* group_count, int32_t n_steps, const int32_t* order,
                            int32_t depth, zsp_source src, int64_t* arena_bytes,
                            zsp_sched** out);

/* Attach the arena (caller-owned device memory of at least *arena_bytes,
 * 256-byte aligned) and the gather stream (required when D > 0; a stream
 * other than the compute stream, at default priority). Needs an all-rank
 * binding of the plan, on the current device. Creates the schedule's HIP
 * events; a later bind replaces them and restarts at position 0. */
zsp_status zsp_sched_bind(zsp_sched* sched, void* arena, int64_t arena_bytes,
                          void* gather_stream);

/* Acquire position `position` for work on `compute_stream`: issue any
 * gathers not yet issued up to position + D, order the compute stream after
 * this position's gather, and return in *params the device address of its
 * group: parameter t at flat_off[t] - flat_off[first] elements, unpadded.
 * Positions are acquired in order 0..n_steps-1, each released before the
 * next is acquired; after the last, the next pass starts at 0. Otherwise
 * ZSP_ESTATE. */
zsp_status zsp_sched_acquire(zsp_sched* sched, int32_t position, void* compute_stream,
                             void** params);

/* Release the held position: every use of its slot must already be enqueued
 * on `compute_stream`; the slot may be overwritten once that work is done. */
zsp_status zsp_sched_release(zsp_sched* sched, int32_t position, void* compute_stream);

typedef enum {
    ZSP_ENGINE_KERNEL = 0, /* the gather kernel (zsp_gather_range's), on the CUs */
    ZSP_ENGINE_COPY = 1    /* the DMA copy engines: no compute units */
} zsp_gather_engine;

/* What runs the schedule's gathers ([ZS3] prefetch paragraph: the next
 * layer's gather should overlap the current layer's computation; a gather
 * kernel competes with that computation for the CUs, the copy engines do
 * not). ZSP_ENGINE_COPY issues one device-to-device copy per rank's slice
 * of each parameter (n_d per parameter) on the stream the kernel would run
 * on, ordered by the same events. Takes effect at the next zsp_sched_bind:
 * a bound schedule is unbound (ZSP_ESTATE until bound again); ZSP_ESTATE
 * while a position is held. */
zsp_status zsp_sched_set_engine(zsp_sched* sched, zsp_gather_engine engine);

/* Abandon the current pass; the next acquire is position 0. Gathers already
 * issued still complete in stream order before any later one. */
zsp_status zsp_sched_reset(zsp_sched* sched);

/* Effective depth, slot count and slot stride in bytes. Host only. */
zsp_status zsp_sched_info(const zsp_sched* sched, int32_t* depth, int32_t* slots,
                          int64_t* slot_bytes);

/* Free the schedule and its events (the arena stays the caller's). Work
 * already enqueued is unaffected. NULL is a no-op. */
void zsp_sched_destroy(zsp_sched* sched);

/* ---- Sharded checkpoint, resume and reshard ------------------------------
 * [ZST] "Where the shards live and what happens on failure": each rank
 * writes its own shard set together with the layout it was cut with; loading
 * under a different rank count reshuffles the shards; the consistent point is
 * between steps (the gradient accumulator is not saved).
 * A checkpoint is a directory holding one file per rank,
 * "rank-<r>-of-<n_d>.zsp": a header (magic "ZSPCKPT1", n_d, rank, number of
 * parameters, S, step), the numel list, master[S], m[S], v[S] (fp32), work[S]
 * (bf16 bits), and the XXH64 hash (seed 0) of all of it, all little-endian.
 * The directory must exist. */

/* Write rank `rank`'s shard set from host arrays of S elements each. Host
 * only. Files are written under a temporary name and renamed. */
zsp_status zsp_checkpoint_write_host(const zsp_plan* plan, int32_t rank, const char* dir,
                                     int64_t step, const float* master, const float* m,
                                     const float* v, const uint16_t* work);

/* Read rank `rank`'s shard set for this plan's layout into host arrays of S
 * elements each; *step receives the saved step. If the checkpoint was written
 * with another rank count, every one of its rank files is read and the shard
 * is rebuilt for this plan (element k of parameter t comes from old rank
 * k / s_old, pads are +0): a reshard, bit-exact. The saved numel list must
 * equal the plan's, else ZSP_EIO; a file whose S differs is refused before
 * anything is written to the arrays, otherwise on error their contents are
 * unspecified. Host only. */
zsp_status zsp_checkpoint_read_host(const zsp_plan* plan, int32_t rank, const char* dir,
                                    int64_t* step, float* master, float* m, float* v,
                                    uint16_t* work);

/* Save the bound state of one rank or of every bound rank
 * (ZSP_ALL_RANKS) to `dir`. The copies follow everything already enqueued
 * on `stream` (an event taken on it orders the library's own copy streams);
 * returns after the files are written. Up to 16 files are written at once,
 * through pinned host chunks the plan keeps until zsp_destroy (32 MiB per
 * file in flight, 512 MiB at most). */
zsp_status zsp_checkpoint_save(zsp_plan* plan, int32_t rank_or_all, const char* dir,
                               int64_t step, void* stream);

/* Load one rank or every bound rank from `dir` into the bound state,
 * resharding if the checkpoint has another rank count; *step receives the
 * saved step. Every file involved is read and checked (header, parameter
 * list, checksum, one common step) before any device write, so a failed
 * load leaves the state untouched. The copies follow everything already
 * enqueued on `stream` and complete before the call returns. Restoring only
 * rank r (e.g. after losing it) leaves the other ranks' state untouched. */
zsp_status zsp_checkpoint_load(zsp_plan* plan, int32_t rank_or_all, const char* dir,
                               int64_t* step, void* stream);

/* Message for the calling thread's most recent failed call ("" if none). */
const char* zsp_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* ZSP_H */
