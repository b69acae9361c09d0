/*
 * zero_shard.h -- C ABI of the MI355X sharded optimizer step.
 *
 * One GPU's share of the ZeRO-1/2/3 and FSDP optimizer step: the local
 * reduction of the reduce-scatter (N_d ranks' bf16 gradient slices of this
 * rank's shard into an fp32 mean), the squared gradient norm for a global
 * clip, the elementwise mixed-precision AdamW update of the shard's fp32
 * master weights and moments, and the bf16 cast and pack of the new shard
 * into the buffer the all-gather fills.
 *
 * Sources (page title, then section):
 *  - "Data parallelism, ZeRO and FSDP" (ML Systems, Lesson 8): section 2
 *    "What is redundant" (AdamW is elementwise, so rank k owns and updates
 *    slice k) and "The communication is already there" (reduce-scatter, the
 *    update of slice k, then the all-gather of the new weights); section 3
 *    Theorem "ZeRO memory and communication" (12 optimizer bytes per
 *    parameter, the stages); "How FSDP implements ZeRO-3" step 1 (a unit's
 *    flat parameter cut into N_d equal chunks) and step 4 (a normal
 *    optimizer on the local shards); section 5 "In code" (the adamw of the
 *    simulator, whose expression order this library follows); section 7
 *    "Common mistakes" (a global clip needs the squared shard norms summed).
 *  - "Distributed Training Basics -- DDP and FSDP": the clip at the update
 *    boundary in its DDP reference program; the errors raised by its
 *    state_bytes helper.
 *
 * Conventions for every call:
 *  - All tensor pointers are DEVICE pointers (HBM of the current HIP device),
 *    16-byte aligned, owned by the caller.  The library allocates nothing at
 *    run time.  The only state it keeps is, per device, the LDS size it
 *    queried, the kernels' dynamic-LDS limits it raised and the address of its
 *    static scratch array (see shard_grad_sqnorm_noalloc), all set once,
 *    thread-safely, by zs_init or by the first call that needs them; calls
 *    may come from several host threads at once.
 *  - HIP graphs: every entry point enqueues kernels only (no memset, no
 *    allocation, no synchronisation), so its calls may be captured into a
 *    HIP graph.  The per-device set-up above is not a stream operation and
 *    must not happen inside a capture: call zs_init on each device (or make
 *    one call of each kind eagerly) before capturing.
 *  - bf16 values are passed as their uint16_t bit patterns.
 *  - `stream` is a hipStream_t (NULL: the null stream).  Calls only enqueue
 *    work and return; results are ready after the caller synchronises the
 *    stream.  A device fault surfaces at that synchronisation.
 *  - Arguments are validated on the host before anything is enqueued; a call
 *    that returns an error other than ZS_ELAUNCH has enqueued nothing and
 *    written nothing.  ZS_ELAUNCH reports a launch the runtime refused; the
 *    call's earlier launches (a long shard takes several) may have run.
 *  - Return value: ZS_OK (0) or one of the negative codes below.  Nothing is
 *    thrown across the ABI.
 *  - Arithmetic: IEEE-754 fp32, round to nearest even, no fused
 *    multiply-add, correctly rounded division and square root, subnormals
 *    kept; the squared norm in fp64.  NaN and Inf propagate (no skipping).
 *  - Outputs must not overlap inputs, except master/exp_avg/exp_avg_sq which
 *    are updated in place.  Calls that write the same buffers must not run
 *    concurrently on different streams.
 *
 * The calls on the vocabulary table (embed_*, distill_*) state their own
 * conventions where they differ.
 */
#ifndef ZERO_SHARD_H
#define ZERO_SHARD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Error codes. */
#define ZS_OK               0
#define ZS_EINVAL_PSI     (-1)   /* psi <= 0 */
#define ZS_EINVAL_ND      (-2)   /* n_d < 1 */
#define ZS_EINVAL_RANK    (-3)   /* rank outside [0, n_d) */
#define ZS_EINVAL_LAYOUT  (-4)   /* align < 1, or shard_len / shard_offset /
                                    valid_len not those zs_layout gives */
#define ZS_EALIGN         (-5)   /* a pointer not 16-byte aligned, or
                                    shard_len not a multiple of 8 */
#define ZS_EINVAL_HPARAM  (-6)   /* lr < 0, beta outside [0,1), eps <= 0,
                                    weight_decay < 0, step < 1, or any
                                    hyperparameter not finite */
#define ZS_EINVAL_STAGE   (-7)   /* stage outside 0..3 or unknown out_mode */
#define ZS_ENULL          (-8)   /* a required pointer is NULL, or both /
                                    neither of grad_slices and mean_in */
#define ZS_EUNSUPPORTED   (-9)   /* n_d > ZS_MAX_RANKS */
#define ZS_EWORKSPACE    (-10)   /* workspace smaller than zs_workspace_bytes */
#define ZS_ELAUNCH       (-11)   /* the HIP runtime rejected a kernel launch
                                    or a set-up call (device query, kernel
                                    attribute, symbol address) */
#define ZS_EINVAL_REDUCE (-12)   /* zs_reduce: unknown grad_dtype, reserved != 0,
                                    micro outside [0, micro_count), micro_count
                                    < 1, or a negative token count */
#define ZS_EZERO_TOKENS  (-13)   /* every rank_tokens entry is 0: the update is
                                    rejected on every rank; nothing is written */
#define ZS_EINVAL_UNITS  (-14)   /* units < 1 */
#define ZS_ESCRATCH      (-15)   /* shard_grad_sqnorm_noalloc: the shard needs
                                    more than ZS_SCRATCH_BYTES of workspace */
#define ZS_EINVAL_EMBED  (-16)   /* zs_embed: a size, pitch, type or scale out of
                                    range, or reserved != 0 */
#define ZS_EINVAL_DISTILL (-17)  /* zs_distill: a size, pitch, type, temperature,
                                    alpha or scale out of range */

#define ZS_MAX_RANKS 64          /* gradient slices one call can reduce */
/* Bytes of the per-device static scratch array of shard_grad_sqnorm_noalloc:
 * the workspace of shards of up to 2,146,959,360 parameters. */
#define ZS_SCRATCH_BYTES ((size_t)16 << 20)

/* Where the new bf16 shard goes. */
#define ZS_OUT_GATHER 0  /* param_out is the bf16[n_d * shard_len] all-gather
                            buffer; this rank writes at shard_offset (stage 0:
                            offset 0, the whole vector) */
#define ZS_OUT_SHARD  1  /* param_out is this rank's own bf16[shard_len] */

/* One rank's shard of a flat parameter vector of psi elements.
 * Stages: 0 = DDP (nothing sharded: the rank owns the whole vector),
 * 1 = ZeRO-1, 2 = ZeRO-2, 3 = ZeRO-3 / FSDP.  The stage does not change the
 * arithmetic, only the layout (stage 0) and which out_mode is natural. */
typedef struct zs_shard {
    int64_t psi;           /* parameters in the flat vector (or FSDP unit) */
    int32_t n_d;           /* data-parallel ranks */
    int32_t rank;          /* k, the owner of this shard */
    int64_t align;         /* shard_len is a multiple of this */
    int64_t shard_len;     /* S: padded slice length */
    int64_t shard_offset;  /* k*S (0 at stage 0) */
    int64_t valid_len;     /* V = clamp(psi - k*S, 0, S): real parameters */
    int32_t stage;         /* 0..3 */
    int32_t out_mode;      /* ZS_OUT_GATHER or ZS_OUT_SHARD */
} zs_shard;

/* AdamW hyperparameters (decoupled weight decay inside the step, on every
 * element), in double; rounded once to fp32 by the library. */
typedef struct zs_adamw {
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;          /* t >= 1, the bias-correction step; the caller
                              increments it between calls */
    double max_grad_norm;  /* > 0: clip the gradient to this global L2 norm;
                              <= 0: no clip */
} zs_adamw;

/* Fill *out with the shard of `rank`.  "Data parallelism, ZeRO and FSDP",
 * section 2 "What is redundant" (GPU k owns slice k of the parameters) and
 * "How FSDP implements ZeRO-3" step 1 (FSDP1 cuts a unit's flat parameter
 * into N_d equal chunks).  The flat vector is padded at its tail
 * to n_d*S with S = roundup(ceil(psi/n_d), align) (stage 0: S =
 * roundup(psi, align), offset 0, valid_len psi); slot k is [k*S, (k+1)*S).
 * Host only.  Errors: ZS_EINVAL_PSI/ND/RANK/LAYOUT(align < 1)/STAGE,
 * ZS_ENULL (out). */
int zs_layout(int64_t psi, int32_t n_d, int32_t rank, int64_t align, int32_t stage,
              int32_t out_mode, zs_shard* out);

/* Bytes of device workspace shard_grad_sqnorm needs for the squared norm of
 * "Data parallelism, ZeRO and FSDP", section 7 "Common mistakes" (global
 * clipping of sharded gradients): one fp64 partial sum
 * per block of its first pass (at most one block per 1024 parameters) plus
 * one per group of 4096 such partials, rounded up to 256 bytes -- 6.8 MB for
 * an 875M-parameter shard, at least 256 bytes (an empty shard).  Host only. */
size_t zs_workspace_bytes(const zs_shard* s);

/* Model-state bytes per GPU of the table of "Data parallelism, ZeRO and
 * FSDP", section 3, Theorem "ZeRO memory and communication" (the same
 * factors as state_bytes in "Distributed Training Basics -- DDP and FSDP",
 * "Memory accounting", whose argument checks this follows): weights and gradients
 * 2 bytes each, K optimizer bytes per parameter.  stage 0: (4+K)psi,
 * 1: 4psi + K psi/n_d, 2: 2psi + (2+K) psi/n_d, 3: (4+K) psi/n_d.
 * Returns -1 for psi <= 0, n_d < 1 or an unknown stage.  Host only. */
double zs_state_bytes(double psi, int32_t n_d, int32_t stage, double K);

/* Bytes each GPU sends per step, from the elements column of the same
 * Theorem ("Data parallelism, ZeRO and FSDP", section 3, proof items 5-7):
 * 2psi elements for stages 0-2, 3psi for
 * stage 3, times bytes_per_elem and (n_d-1)/n_d (ring collectives).
 * Returns -1 on invalid arguments.  Host only. */
double zs_comm_bytes(double psi, int32_t n_d, int32_t stage, double bytes_per_elem);

/* Clip pass: the reduce-scatter's local reduction plus this shard's squared
 * L2 norm.  "Data parallelism, ZeRO and FSDP": section 2 "The communication
 * is already there" (after the reduce-scatter GPU k holds slice k of the
 * gradients) with the averaging of section 2 "Two GPUs, one batch" and the
 * Proposition "DDP is exact" (the mean of the ranks' gradients; its order of
 * summation changes only the last bits, hence the fixed rank order here);
 * section 7 "Common mistakes" (a global clip over sharded gradients sums the
 * squared shard norms, which this call provides for this shard).
 *   grad_slices  host array of n_d device pointers; grad_slices[r] is rank
 *                r's bf16 gradient for this shard, valid_len elements.
 *   mean_out     device fp32[valid_len] or NULL.  If given, receives
 *                g_i = (sum over r = 0..n_d-1 in rank order of the widened
 *                bf16 values) / n_d.
 *   workspace    device, >= zs_workspace_bytes(s) bytes, 16-byte aligned;
 *                contents on entry are ignored.
 *   sqnorm_out   device, one double: sum of (double)g_i^2 over the shard.
 *                accumulate == 0 overwrites it; accumulate != 0 adds the
 *                shard's value to it (for a norm over several FSDP units,
 *                summed in call order).
 * The fp64 sum is taken in a fixed tree order (run-to-run deterministic for
 * one shape), not in ascending element order.  An empty shard (valid_len 0)
 * contributes 0.  Errors: ZS_ENULL, ZS_EINVAL_*, ZS_EALIGN, ZS_EUNSUPPORTED,
 * ZS_EWORKSPACE, ZS_ELAUNCH. */
int shard_grad_sqnorm(const zs_shard* s, const uint16_t* const* grad_slices, float* mean_out,
                      void* workspace, size_t workspace_bytes, double* sqnorm_out,
                      int32_t accumulate, void* stream);

/* Bytes of device workspace shard_grad_sqnorm_units needs for `units`
 * units of layout s: units x what one shard needs (6.8 MB per 875M
 * parameters of a unit).  Host only. */
size_t zs_workspace_bytes_units(const zs_shard* s, int32_t units);

/* The clip pass of `units` FSDP units that share one layout (e.g. identical
 * transformer blocks), as one call: the same result, bit for bit, as
 * shard_grad_sqnorm on unit 0 with `accumulate` followed by
 * shard_grad_sqnorm on units 1.. with accumulate = 1 -- the global squared
 * norm over the units ("Data parallelism, ZeRO and FSDP", section 7: the
 * norm of sharded gradients sums the squared shard norms), each unit's sum
 * taken in the fixed per-shard order and added in unit order -- but with
 * two partial-sum kernels in all instead of two per unit.
 *   grad_slices  host array of units x n_d device pointers, unit-major
 *                (unit u's rank r slice at [u*n_d + r]).
 *   mean_out     NULL, or a host array of `units` device pointers (each
 *                fp32[valid_len] or NULL) receiving each unit's mean.
 *   workspace    >= zs_workspace_bytes_units(s, units) bytes.
 * Errors: as shard_grad_sqnorm, plus ZS_EINVAL_UNITS; every unit's
 * pointers are checked before anything is enqueued. */
int shard_grad_sqnorm_units(const zs_shard* s, int32_t units, const uint16_t* const* grad_slices,
                            float* const* mean_out, void* workspace, size_t workspace_bytes,
                            double* sqnorm_out, int32_t accumulate, void* stream);

/* Element type of the gradient slices a reduction reads. */
#define ZS_GRAD_BF16 0   /* bf16, widened exactly to fp32 */
#define ZS_GRAD_F32  1   /* fp32 (the reduce_dtype=float32 policy) */

/* How shard_grad_reduce combines the ranks' slices and the micro-batches. */
typedef struct zs_reduce {
    int32_t grad_dtype;          /* ZS_GRAD_BF16 or ZS_GRAD_F32, every slice */
    int32_t micro;               /* j, this micro-batch: 0 <= j < micro_count */
    int32_t micro_count;         /* m >= 1 micro-batches per optimizer step
                                    (1: no gradient accumulation) */
    int32_t reserved;            /* must be 0 */
    const int64_t* rank_tokens;  /* NULL: the mean over ranks; else a host
                                    array of n_d valid-token counts, and the
                                    ranks are weighted by n_r / T */
} zs_reduce;

/* The general clip pass: reduces the ranks' slices of one micro-batch and
 * accumulates micro-batches into the shard's fp32 gradient.
 *   "Data parallelism, ZeRO and FSDP", section 3 "Gradient accumulation"
 *   (ZeRO-2 reduce-scatters after every micro-batch) and section 6 (Llama 3
 *   reduce-scattered gradients in fp32); "Distributed Training Basics --
 *   DDP and FSDP", "DDP: replicated state, partitioned examples" (weight
 *   ranks by valid tokens; a zero global count rejects the update) and
 *   "Accumulation, clipping and scaling measurements" (clip and step at the
 *   effective-update boundary).
 * Per element i < valid_len, in fp32:
 *   r_i = the mean over ranks, as shard_grad_sqnorm computes it, of bf16 or
 *         fp32 slices; or, with rank_tokens, ((w_0*G_0[i]) + (w_1*G_1[i]))
 *         + ... in rank order, w_r = f32(n_r / T) computed in double,
 *         T = sum of n_r, every product and sum rounded;
 *   micro == 0:                grad_out[i] = r_i
 *   0 < micro < m - 1:         grad_out[i] = grad_out[i] + r_i
 *   micro == m - 1 > 0:        grad_out[i] = (grad_out[i] + r_i) / m
 * so after the last micro-batch grad_out holds the step's gradient, the
 * mean over micro-batches, ready for zero_shard_step's mean_in.
 *   grad_slices  host array of n_d device pointers, each to valid_len
 *                elements of grad_dtype, 16-byte aligned.
 *   grad_out     device fp32[valid_len], 16-byte aligned; read and written
 *                in place for micro > 0.
 *   workspace, sqnorm_out, accumulate: as for shard_grad_sqnorm, applied to
 *                the values written.  sqnorm_out may be NULL (then no norm
 *                and no workspace are needed), e.g. before the last
 *                micro-batch.
 * Errors: ZS_ENULL, ZS_EINVAL_*, ZS_EINVAL_REDUCE, ZS_EZERO_TOKENS (nothing
 * enqueued), ZS_EALIGN, ZS_EUNSUPPORTED, ZS_EWORKSPACE, ZS_ELAUNCH. */
int shard_grad_reduce(const zs_shard* s, const zs_reduce* r, const void* const* grad_slices,
                      float* grad_out, void* workspace, size_t workspace_bytes,
                      double* sqnorm_out, int32_t accumulate, void* stream);

/* The fused optimizer step of this shard.  "Data parallelism, ZeRO and
 * FSDP": section 2 "What is redundant" (AdamW is elementwise, so GPU k
 * updates slice k from that slice's gradient, moments and fp32 master
 * weights alone) and the table of "The communication is already there" (the
 * update sits between the reduce-scatter and the all-gather of the new
 * weights); section 3 Theorem (K = 12 bytes of fp32 master weight, m and v
 * per parameter); section 5 "In code" (the AdamW expression order below);
 * section 7 "Common mistakes" (the clip uses the global norm).  Exactly one
 * gradient source:
 *   grad_slices  host array of n_d device pointers to bf16[valid_len]
 *                (reduced here, in rank order, as shard_grad_sqnorm does), or
 *   mean_in      device fp32[valid_len], the mean from shard_grad_sqnorm.
 * If h->max_grad_norm > 0: `sqnorm` (device, one double, this shard's or the
 * accumulated squared norm) is required and the global squared norm is
 * Q = *sqnorm + other_sqnorm (other_sqnorm stands for the scalar all-reduce
 * of the other ranks' squared shard norms; a negative value is rejected with
 * ZS_EINVAL_HPARAM, NaN and +Inf propagate as IEEE arithmetic does);
 * coef = f32(min(1, max_grad_norm / (sqrt(Q) + 1e-6))) in double, NaN kept,
 * and g = g * coef.  Otherwise `sqnorm` and other_sqnorm are ignored.
 * Then, for i < valid_len, in this order and in fp32 (b1 = f32(beta1),
 * c1 = f32(1 - beta1), bc1 = f32(1 - beta1^t), likewise b2, c2, bc2):
 *   m' = (b1*m) + (c1*g);  v' = (b2*v) + ((c2*g)*g)
 *   w' = w - lr*((m'/bc1) / (sqrt(v'/bc2) + eps) + wd*w)
 * master/exp_avg/exp_avg_sq (fp32[valid_len]) are updated in place, and
 * param_out receives bf16_rne(w') at its base (ZS_OUT_GATHER: param_out +
 * shard_offset; ZS_OUT_SHARD: param_out) followed by +0 in the
 * shard_len - valid_len pad positions.  Nothing beyond valid_len is read or
 * written in the state or gradient buffers, and nothing outside this
 * rank's slot of the gather buffer is written.  bf16_rne: round to nearest
 * even; any NaN becomes the canonical quiet NaN 0x7FC0.
 * Errors: ZS_ENULL, ZS_EINVAL_*, ZS_EALIGN, ZS_EUNSUPPORTED, ZS_ELAUNCH. */
int zero_shard_step(const zs_shard* s, const zs_adamw* h, const uint16_t* const* grad_slices,
                    const float* mean_in, const double* sqnorm, double other_sqnorm,
                    float* master, float* exp_avg, float* exp_avg_sq, uint16_t* param_out,
                    void* stream);

/* Cast and pack only: param_out (placed as in zero_shard_step) receives
 * bf16_rne(master[i]) for i < valid_len and +0 in the pads.  "Data
 * parallelism, ZeRO and FSDP", section 2 table (the all-gather of the new
 * weights after the update) and section 3 Theorem (bf16 weights of 2 bytes
 * next to the fp32 master copy); the slot layout of zs_layout.  The step of
 * the all-gather that needs no optimizer work (e.g. to publish weights after
 * loading a checkpoint).  Errors: ZS_ENULL, ZS_EINVAL_*, ZS_EALIGN,
 * ZS_ELAUNCH. */
int shard_pack_gather(const zs_shard* s, const float* master, uint16_t* param_out,
                      void* stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the clip
 * pass of shard_grad_sqnorm with the same arguments except the workspace,
 * computed by the same kernels into the same results bit for bit.  Its
 * block partials live in a static device array of ZS_SCRATCH_BYTES (16 MiB)
 * per device, held from the first use until the process ends; the call
 * itself allocates nothing and needs no zeroed memory.  Every call on one
 * device shares that device's array, so calls that overlap on one device
 * (several streams or host threads at once) race and give wrong results;
 * serialize them.  The array's device address is taken once per device by
 * zs_init or by the first call on that device (outside a capture, see the
 * HIP graph convention above).
 * Errors: as shard_grad_sqnorm without ZS_EWORKSPACE, plus ZS_ESCRATCH when
 * zs_workspace_bytes(s) > ZS_SCRATCH_BYTES (valid_len above
 * 2,146,959,360); nothing is enqueued then. */
int shard_grad_sqnorm_noalloc(const zs_shard* s, const uint16_t* const* grad_slices,
                              float* mean_out, double* sqnorm_out, int32_t accumulate,
                              void* stream);

/* ---- the vocabulary table: lookup and gradient, distillation ----------------------
 *
 * The operators at the two ends of a training step, whose parameter is the
 * (often tied) vocabulary table of a sharded unit: embed_lookup reads rows of
 * the vector the all-gather filled, embed_grad writes the gradient whose
 * slices shard_grad_reduce reads, and the distillation loss makes the gradient
 * both start from.  (It counts its rows on the device; zs_reduce.rank_tokens,
 * by which the ranks are weighed, is host memory that the program fills.)  All
 * conventions above hold, except: the table, its gradient, activations, logits
 * and their gradient need only the alignment of their element (rows of odd
 * length and tables inside a flat vector are allowed), and fp32 sums here may
 * use fused multiply-add. */

/* Element types of these calls, and the types of ids. */
#define ZS_BF16   0
#define ZS_F32    1
#define ZS_ID_I32 0
#define ZS_ID_I64 1

/* Tokens and table rows one embed_grad call takes at most, and the teacher
 * entries of a row. */
#define ZS_EMBED_MAX       ((int64_t)1 << 24)
#define ZS_DISTILL_MAX_K   1024

/* A call on a batch of token ids and `rows` consecutive rows of an embedding
 * table (the whole table, or the rows a rank holds).  A token is here when
 * first_row <= id < first_row + rows; any other id (padding, another rank's
 * rows) reads a row of zeros and has no gradient. */
typedef struct zs_embed {
    int64_t tokens;        /* T >= 0 ids, and rows of activations */
    int64_t rows;          /* R >= 1 table rows in the buffer */
    int64_t first_row;     /* id of the first of them, >= 0 */
    int64_t dim;           /* D >= 1 */
    int64_t table_pitch;   /* elements from one table row to the next, >= D */
    int64_t act_pitch;     /* elements from one activation row to the next, >= D */
    int32_t id_dtype;      /* ZS_ID_I32 or ZS_ID_I64 */
    int32_t table_dtype;   /* ZS_BF16 or ZS_F32: the table, or its gradient */
    int32_t act_dtype;     /* ZS_BF16 or ZS_F32: activations, or their gradient */
    int32_t reserved;      /* must be 0 */
    double scale;          /* rounded once to fp32; finite */
} zs_embed;

/* out[t, :] = scale * table[ids[t] - first_row, :], the product in fp32 and
 * rounded once to act_dtype; +0 for a token that is not here.
 *   ids    device, T ids.     table  device, R rows.     out  device, T rows.
 * Columns between D and the pitch are not read or written.
 * Errors: ZS_ENULL, ZS_EINVAL_EMBED, ZS_EALIGN, ZS_ELAUNCH. */
int embed_lookup(const zs_embed* e, const void* ids, const void* table, void* out, void* stream);

/* Bytes of device workspace embed_grad needs: the token positions sorted by
 * row (8 bytes a token), the row starts (4 bytes a row) and the partial sums
 * of rows with many tokens (2 D fp32 for every 8 to 64 tokens).  0 for a NULL
 * or invalid e and above ZS_EMBED_MAX.  Host only. */
size_t zs_embed_workspace_bytes(const zs_embed* e);

/* The gradient of embed_lookup with respect to the table, dense:
 *   G_r = scale * (sum of grad_out[t, :] over the tokens with row r)
 *   accumulate == 0: grad_table[r, :] = G_r for every row r (+0 without tokens)
 *   accumulate != 0: grad_table[r, :] += G_r for the rows that have tokens;
 *                    other rows are not read or written
 * (micro-batches after the first, or a tied table whose head's gradient is
 * there already).  Tokens are sorted by row, stably, and summed in fp32 in an
 * order that depends on the sizes and ids alone (run-to-run deterministic:
 * no floating-point atomics); the result is rounded once to table_dtype.  The
 * sort reads the ids once for every 512 rows of the table, at least 256 times:
 * its cost is tokens times rows / 512.  Where one row has most of the tokens,
 * a part of the sort reads them three times, and one block joins its sums.
 *   workspace  device, 16-byte aligned, >= zs_embed_workspace_bytes(e) bytes;
 *              contents on entry are ignored.
 * Errors: ZS_ENULL, ZS_EINVAL_EMBED, ZS_EALIGN, ZS_EUNSUPPORTED (more than
 * ZS_EMBED_MAX tokens or rows), ZS_EWORKSPACE, ZS_ELAUNCH. */
int embed_grad(const zs_embed* e, const void* ids, const void* grad_out, void* grad_table,
               int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream);

/* Distillation of student logits (T rows over a vocabulary of V) from the top
 * logits of a teacher, optionally mixed with the cross entropy of labels. */
typedef struct zs_distill {
    int64_t rows;          /* T >= 0 */
    int64_t vocab;         /* 1 <= V < 2^31 */
    int64_t logits_pitch;  /* elements from one row of logits to the next, >= V */
    int64_t grad_pitch;    /* the same of the logits' gradient */
    int32_t k;             /* teacher entries a row, 0..ZS_DISTILL_MAX_K */
    int32_t logits_dtype;  /* ZS_BF16 or ZS_F32: logits and their gradient */
    int32_t teacher_dtype; /* ZS_BF16 or ZS_F32: the teacher's logits */
    int32_t id_dtype;      /* ZS_ID_I32 or ZS_ID_I64: teacher ids and labels */
    double temperature;    /* tau > 0 */
    double alpha;          /* weight of the distillation, 0..1; the labels' cross
                              entropy has 1 - alpha */
    double scale;          /* of the gradient (not of the loss), finite */
} zs_distill;

/* What the student is held to.  Device pointers, rows contiguous. */
typedef struct zs_targets {
    const void* teacher_ids;     /* [T, k] columns; an id outside [0, V) is no entry */
    const void* teacher_logits;  /* [T, k] u, before the temperature; -Inf is no entry */
    const float* teacher_lse;    /* [T] or NULL: log(sum exp(u / tau)) over the teacher's
                                    whole vocabulary; NULL: the entries are all of it */
    const void* labels;          /* [T] or NULL: columns; a label outside [0, V) (-100)
                                    masks its row out of loss and gradient */
} zs_targets;

/* Bytes of device workspace distill_loss and distill_loss_grad need: a flag
 * per row, 16 bytes for each part a row may be cut into (2048 to 16384
 * logits), and for fewer than 128 rows of more than 1024 16-byte vectors of
 * logits 4 (k + 1) bytes a row.  0 for a NULL or invalid d.  Host only. */
size_t zs_distill_workspace_bytes(const zs_distill* d);

/* Row losses.  With s a row's logits, K its teacher entries, in fp32:
 *   lse_tau = log(sum over v of exp(s_v / tau)),  log q_v = s_v / tau - lse_tau
 *   log p_k = u_k / tau - (teacher_lse, or log(sum over K of exp(u / tau)))
 *   KD = sum over K of p_k (log p_k - log q_{id_k});   CE = lse_1 - s_label
 *   loss_out[t] = alpha tau^2 KD + (1 - alpha) CE
 * A row counts when its label (where labels are given) is in [0, V) and, if
 * alpha == 1, it has a teacher entry.  Any other row has loss 0, whatever its
 * logits hold.  An entry with p_k = 0 adds nothing; the same id twice
 * is two entries.  alpha < 1 needs labels; alpha == 0 reads no teacher.  NaN
 * and +Inf in a row that counts propagate; a logit of -Inf has probability 0.
 *   loss_out   fp32[T].
 *   lse_out    fp32[T, 2] or NULL (required by distill_loss): lse_tau and
 *              lse_1 (0 if alpha == 1); both 0 for a row that does not count.
 *              An lse_tau beyond fp32's range is its largest number.
 *   loss_sum   one fp32 or NULL: the sum of loss_out, taken in fp64 in a fixed
 *              order and rounded once.   counted  one int64 or NULL: how many
 *              rows count.  accumulate != 0 adds to what they hold.
 *   workspace  16-byte aligned, >= zs_distill_workspace_bytes(d) bytes.
 * Errors: ZS_ENULL, ZS_EINVAL_DISTILL, ZS_EALIGN, ZS_EWORKSPACE, ZS_ELAUNCH. */
int distill_loss(const zs_distill* d, const void* logits, const zs_targets* t, float* loss_out,
                 float* lse_out, float* loss_sum, int64_t* counted, int32_t accumulate,
                 void* workspace, size_t workspace_bytes, void* stream);

/* The gradient of the row losses, from the statistics distill_loss left:
 *   grad_out[t, v] = scale * row_grad[t] * (alpha tau (M q_v - sum of p_k with id_k = v)
 *                    + (1 - alpha) (exp(s_v - lse_1) - [v = label])),  M = sum of p_k
 * (M is 1 without teacher_lse), rounded once to logits_dtype; +0 in rows that
 * do not count.  q_v = exp(s_v / tau - lse_tau) is as exact as lse_in: fp32
 * holds it to |lse| 2^-24, and from |lse_tau| = 2^27 on q_v is held to 1 (a row
 * of equal values so far from zero is uniform in distill_loss_grad alone).
 *   row_grad  fp32[T] or NULL (1): the gradient each row's loss receives.
 *   grad_out  T rows; may be the logits themselves (then of the same pitch).
 * Errors: ZS_ENULL, ZS_EINVAL_DISTILL (also: in place with another pitch),
 * ZS_EALIGN, ZS_ELAUNCH. */
int distill_grad(const zs_distill* d, const void* logits, const zs_targets* t,
                 const float* lse_in, const float* row_grad, void* grad_out, void* stream);

/* Both in one call: the loss is usually the last operator of the forward
 * pass, so its gradient can be taken there.  From 128 rows on, and for rows of
 * at most 1024 16-byte vectors, the logits are read once (of a row, the first
 * 131072 in bf16, 65536 in fp32; where its largest logit times log2(e) / tau
 * is beyond 65536 in size, it is read again for the sums and for the
 * gradient).  Arguments and errors as above; lse_out may be NULL.  The loss
 * may differ from distill_loss's in its last bits, the gradient from
 * distill_grad's by what rounding lse to fp32 takes. */
int distill_loss_grad(const zs_distill* d, const void* logits, const zs_targets* t,
                      float* loss_out, float* lse_out, const float* row_grad, void* grad_out,
                      float* loss_sum, int64_t* counted, int32_t accumulate, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Per-device set-up for the current HIP device: queries its LDS size, raises
 * the kernels' dynamic-LDS limits and takes the address of the static
 * scratch array.  Optional; every entry point does what it needs itself on
 * its first call on a device.  Call it on each device before capturing
 * library calls into a HIP graph.  Returns ZS_OK or ZS_ELAUNCH. */
int zs_init(void);

/* Static description of an error code ("unknown error" otherwise). */
const char* zs_strerror(int code);

#ifdef __cplusplus
}
#endif
#endif
