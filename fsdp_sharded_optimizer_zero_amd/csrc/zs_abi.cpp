// zs_abi.cpp -- the C-ABI entry points that run the passes: argument
// validation (nothing is enqueued when a call is rejected), the scalars each
// pass needs, and the calls into the kernel part (enqueue_*, zs_kernels.hip).
// No HIP calls here.
//
// What each entry point computes is stated with its declaration in
// zero_shard.h, with the passage of "Data parallelism, ZeRO and FSDP" (and
// its companion pages) that defines it.
#include <cmath>
#include <cstdint>

#include "zs_internal.h"

namespace zs {
namespace {

bool is_pow2(int32_t n) { return n > 0 && (n & (n - 1)) == 0; }

// The n_d slice pointers of one unit into the kernel arguments; each must be
// non-null and 16-byte aligned unless the shard is empty.
int fill_slices(const zs_shard* s, const void* const* grad_slices, SlicePtrs* out)
{
    for (int r = 0; r < ZS_MAX_RANKS; ++r) out->p[r] = nullptr;
    if (!grad_slices) return ZS_ENULL;
    for (int r = 0; r < s->n_d; ++r) {
        const void* p = grad_slices[r];
        if (s->valid_len > 0) {
            if (!p) return ZS_ENULL;
            if (!aligned16(p)) return ZS_EALIGN;
        }
        out->p[r] = p;
    }
    return ZS_OK;
}

// Where the shard's bf16 values go: its slot of the gather buffer, or the
// rank's own shard buffer.
uint16_t* slot_base(const zs_shard* s, uint16_t* param_out)
{
    return s->out_mode == ZS_OUT_GATHER ? param_out + s->shard_offset : param_out;
}

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// The reduction's scalars for n_d ranks and m micro-batches (no weights).
SqArgs reduce_args(const zs_shard* s, float* grad_out, int32_t micro_count)
{
    SqArgs a{};
    a.mean_out = grad_out;
    a.valid_len = s->valid_len;
    a.n_d = s->n_d;
    a.nd = static_cast<float>(s->n_d);
    a.inv_nd = is_pow2(s->n_d) ? 1.0f / static_cast<float>(s->n_d) : 0.0f;
    a.micro_count = static_cast<float>(micro_count);
    a.inv_micro_count = is_pow2(micro_count) ? 1.0f / static_cast<float>(micro_count) : 0.0f;
    return a;
}

}  // namespace
}  // namespace zs

using namespace zs;

namespace zs {
namespace {

// The clip pass of one shard into the partials workspace `partials`; the
// shard, sqnorm_out and mean_out have been checked.
int sqnorm_pass(const zs_shard* s, const uint16_t* const* grad_slices, float* mean_out,
                double* partials, double* sqnorm_out, int32_t accumulate, void* stream)
{
    SqArgs a = reduce_args(s, mean_out, 1);
    int rc = fill_slices(s, reinterpret_cast<const void* const*>(grad_slices), &a.slices);
    if (rc != ZS_OK) return rc;
    rc = enqueue_reduce(a, false, false, kAccNone, mean_out != nullptr, partials, stream);
    if (rc != ZS_OK) return rc;
    return enqueue_sqnorm_sums(partials, reduce_blocks(s->valid_len, s->n_d, false, kAccNone), 1,
                               sqnorm_out, accumulate, stream);
}

}  // namespace
}  // namespace zs

extern "C" int zs_init(void)
{
    int rc = prepare_device();
    if (rc == ZS_OK) rc = prepare_vocab();
    if (rc == ZS_OK) rc = prepare_relpos();
    return rc != ZS_OK ? rc : prepare_tensors();
}

extern "C" int shard_grad_sqnorm(const zs_shard* s, const uint16_t* const* grad_slices,
                                 float* mean_out, void* workspace, size_t workspace_bytes,
                                 double* sqnorm_out, int32_t accumulate, void* stream)
{
    int rc = check_shard(s);
    if (rc != ZS_OK) return rc;
    if (!workspace || !sqnorm_out) return ZS_ENULL;
    if (!aligned16(workspace) || !aligned8(sqnorm_out)) return ZS_EALIGN;
    if (mean_out && !aligned16(mean_out)) return ZS_EALIGN;
    if (workspace_bytes < zs_workspace_bytes(s)) return ZS_EWORKSPACE;
    return sqnorm_pass(s, grad_slices, mean_out, static_cast<double*>(workspace), sqnorm_out,
                       accumulate, stream);
}

extern "C" int shard_grad_sqnorm_noalloc(const zs_shard* s, const uint16_t* const* grad_slices,
                                         float* mean_out, double* sqnorm_out,
                                         int32_t accumulate, void* stream)
{
    int rc = check_shard(s);
    if (rc != ZS_OK) return rc;
    if (!sqnorm_out) return ZS_ENULL;
    if (!aligned8(sqnorm_out)) return ZS_EALIGN;
    if (mean_out && !aligned16(mean_out)) return ZS_EALIGN;
    if (zs_workspace_bytes(s) > ZS_SCRATCH_BYTES) return ZS_ESCRATCH;
    SqArgs tmp;
    rc = fill_slices(s, reinterpret_cast<const void* const*>(grad_slices), &tmp.slices);
    if (rc != ZS_OK) return rc;
    void* ws = nullptr;
    if ((rc = static_scratch(&ws)) != ZS_OK) return rc;
    return sqnorm_pass(s, grad_slices, mean_out, static_cast<double*>(ws), sqnorm_out,
                       accumulate, stream);
}

extern "C" int shard_grad_sqnorm_units(const zs_shard* s, int32_t units,
                                       const uint16_t* const* grad_slices,
                                       float* const* mean_out, void* workspace,
                                       size_t workspace_bytes, double* sqnorm_out,
                                       int32_t accumulate, void* stream)
{
    int rc = check_shard(s);
    if (rc != ZS_OK) return rc;
    if (units < 1) return ZS_EINVAL_UNITS;
    if (!grad_slices || !workspace || !sqnorm_out) return ZS_ENULL;
    if (!aligned16(workspace) || !aligned8(sqnorm_out)) return ZS_EALIGN;
    if (workspace_bytes < zs_workspace_bytes_units(s, units)) return ZS_EWORKSPACE;
    // validate every unit before enqueueing anything
    for (int32_t u = 0; u < units; ++u) {
        SlicePtrs tmp;
        rc = fill_slices(s, reinterpret_cast<const void* const*>(grad_slices + u * s->n_d), &tmp);
        if (rc != ZS_OK) return rc;
        if (mean_out && mean_out[u] && !aligned16(mean_out[u])) return ZS_EALIGN;
    }
    const int64_t blocks = reduce_blocks(s->valid_len, s->n_d, false, kAccNone);
    double* partials = static_cast<double*>(workspace);
    for (int32_t u = 0; u < units; ++u) {
        SqArgs a = reduce_args(s, mean_out ? mean_out[u] : nullptr, 1);
        fill_slices(s, reinterpret_cast<const void* const*>(grad_slices + u * s->n_d), &a.slices);
        rc = enqueue_reduce(a, false, false, kAccNone, a.mean_out != nullptr,
                            partials + static_cast<int64_t>(u) * blocks, stream);
        if (rc != ZS_OK) return rc;
    }
    return enqueue_sqnorm_sums(partials, blocks, units, sqnorm_out, accumulate, stream);
}

extern "C" int shard_grad_reduce(const zs_shard* s, const zs_reduce* r,
                                 const void* const* grad_slices, float* grad_out,
                                 void* workspace, size_t workspace_bytes, double* sqnorm_out,
                                 int32_t accumulate, void* stream)
{
    int rc = check_shard(s);
    if (rc != ZS_OK) return rc;
    if (!r) return ZS_ENULL;
    if ((r->grad_dtype != ZS_GRAD_BF16 && r->grad_dtype != ZS_GRAD_F32) || r->reserved != 0 ||
        r->micro_count < 1 || r->micro < 0 || r->micro >= r->micro_count)
        return ZS_EINVAL_REDUCE;
    if (s->valid_len > 0 && !grad_out) return ZS_ENULL;
    if (grad_out && !aligned16(grad_out)) return ZS_EALIGN;
    if (sqnorm_out) {
        if (!workspace) return ZS_ENULL;
        if (!aligned16(workspace) || !aligned8(sqnorm_out)) return ZS_EALIGN;
        if (workspace_bytes < zs_workspace_bytes(s)) return ZS_EWORKSPACE;
    }
    SqArgs a = reduce_args(s, grad_out, r->micro_count);
    rc = fill_slices(s, grad_slices, &a.slices);
    if (rc != ZS_OK) return rc;
    const bool weighted = r->rank_tokens != nullptr;
    if (weighted) {
        // w_r = n_r / T in double, rounded once; T = 0 rejects the update.
        double T = 0.0;
        for (int k = 0; k < s->n_d; ++k) {
            if (r->rank_tokens[k] < 0) return ZS_EINVAL_REDUCE;
            T += static_cast<double>(r->rank_tokens[k]);
        }
        if (T == 0.0) return ZS_EZERO_TOKENS;
        for (int k = 0; k < s->n_d; ++k)
            a.wt[k] = static_cast<float>(static_cast<double>(r->rank_tokens[k]) / T);
    }
    const int acc = r->micro == 0 ? kAccNone
                  : (r->micro == r->micro_count - 1 ? kAccFinal : kAccAdd);
    double* partials = sqnorm_out ? static_cast<double*>(workspace) : nullptr;
    const bool f32 = r->grad_dtype == ZS_GRAD_F32;
    rc = enqueue_reduce(a, f32, weighted, acc, true, partials, stream);
    if (rc != ZS_OK || !sqnorm_out) return rc;
    return enqueue_sqnorm_sums(partials, reduce_blocks(s->valid_len, s->n_d, f32, acc), 1,
                               sqnorm_out, accumulate, stream);
}

extern "C" int zero_shard_step(const zs_shard* s, const zs_adamw* h,
                               const uint16_t* const* grad_slices, const float* mean_in,
                               const double* sqnorm, double other_sqnorm, float* master,
                               float* exp_avg, float* exp_avg_sq, uint16_t* param_out,
                               void* stream)
{
    int rc = check_shard(s);
    if (rc != ZS_OK) return rc;
    if ((rc = check_hparams(h)) != ZS_OK) return rc;
    if ((grad_slices == nullptr) == (mean_in == nullptr)) return ZS_ENULL;
    const bool clip = h->max_grad_norm > 0.0;
    if (clip) {
        // a sum of squares is never negative; NaN and +Inf propagate
        if (other_sqnorm < 0.0) return ZS_EINVAL_HPARAM;
        if (!sqnorm) return ZS_ENULL;
        if (!aligned8(sqnorm)) return ZS_EALIGN;
    }
    if (!param_out) return ZS_ENULL;
    if (!aligned16(param_out)) return ZS_EALIGN;
    if (s->valid_len > 0) {
        if (!master || !exp_avg || !exp_avg_sq) return ZS_ENULL;
        if (!aligned16(master) || !aligned16(exp_avg) || !aligned16(exp_avg_sq))
            return ZS_EALIGN;
        if (mean_in && !aligned16(mean_in)) return ZS_EALIGN;
    }
    StepArgs a{};
    if (grad_slices) {
        rc = fill_slices(s, reinterpret_cast<const void* const*>(grad_slices), &a.slices);
        if (rc != ZS_OK) return rc;
    }
    a.mean = mean_in;
    a.sqnorm = sqnorm;
    a.other_sqnorm = other_sqnorm;
    a.max_norm = h->max_grad_norm;
    a.w = master;
    a.m = exp_avg;
    a.v = exp_avg_sq;
    a.out = slot_base(s, param_out);
    a.valid_len = s->valid_len;
    a.shard_len = s->shard_len;
    a.n_d = s->n_d;
    a.nd = static_cast<float>(s->n_d);
    a.inv_nd = is_pow2(s->n_d) ? 1.0f / static_cast<float>(s->n_d) : 0.0f;
    a.c = make_consts(h);
    return enqueue_step(a, grad_slices != nullptr, clip, stream);
}

extern "C" int shard_pack_gather(const zs_shard* s, const float* master, uint16_t* param_out,
                                 void* stream)
{
    int rc = check_shard(s);
    if (rc != ZS_OK) return rc;
    if (!param_out) return ZS_ENULL;
    if (s->valid_len > 0 && !master) return ZS_ENULL;
    if (!aligned16(param_out) || (master && !aligned16(master))) return ZS_EALIGN;
    return enqueue_pack(master, slot_base(s, param_out), s->valid_len, s->shard_len, stream);
}

// ---- the vocabulary table --------------------------------------------------------

namespace zs {
namespace {

bool aligned_to(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
uintptr_t elem_bytes(int32_t dtype) { return dtype == ZS_F32 ? 4 : 2; }
uintptr_t id_bytes(int32_t dtype) { return dtype == ZS_ID_I64 ? 8 : 4; }

EmbedArgs embed_args(const zs_embed* e, const void* ids, const void* src, void* dst)
{
    EmbedArgs a{};
    a.ids = ids;
    a.src = src;
    a.dst = dst;
    a.tokens = e->tokens;
    a.rows = e->rows;
    a.first_row = e->first_row;
    a.dim = e->dim;
    a.table_pitch = e->table_pitch;
    a.act_pitch = e->act_pitch;
    a.scale = static_cast<float>(e->scale);
    a.id64 = e->id_dtype == ZS_ID_I64;
    a.table_f32 = e->table_dtype == ZS_F32;
    a.act_f32 = e->act_dtype == ZS_F32;
    return a;
}

// What the distillation calls share: the struct, the logits and the targets
// into the kernel arguments.
int distill_args(const zs_distill* d, const void* logits, const zs_targets* t, DistillArgs* a)
{
    int rc = check_distill(d);
    if (rc != ZS_OK) return rc;
    if (!t) return ZS_ENULL;
    const bool kd = d->alpha > 0.0, ce = d->alpha < 1.0;
    if (d->rows > 0) {
        if (!logits || (ce && !t->labels)) return ZS_ENULL;
        if (kd && d->k > 0 && (!t->teacher_ids || !t->teacher_logits)) return ZS_ENULL;
    }
    if (!aligned_to(logits, elem_bytes(d->logits_dtype)) ||
        !aligned_to(t->teacher_ids, id_bytes(d->id_dtype)) ||
        !aligned_to(t->teacher_logits, elem_bytes(d->teacher_dtype)) ||
        !aligned_to(t->teacher_lse, 4) || !aligned_to(t->labels, id_bytes(d->id_dtype)))
        return ZS_EALIGN;
    *a = DistillArgs{};
    a->logits = logits;
    a->teacher_ids = t->teacher_ids;
    a->teacher_logits = t->teacher_logits;
    a->teacher_lse = t->teacher_lse;
    a->labels = t->labels;
    a->rows = d->rows;
    a->vocab = d->vocab;
    a->logits_pitch = d->logits_pitch;
    a->grad_pitch = d->grad_pitch;
    a->k = kd ? d->k : 0;
    a->f32 = d->logits_dtype == ZS_F32;
    a->teacher_f32 = d->teacher_dtype == ZS_F32;
    a->id64 = d->id_dtype == ZS_ID_I64;
    a->kd = kd;
    a->ce = ce;
    a->inv_tau = static_cast<float>(1.0 / d->temperature);
    a->loss_kd = static_cast<float>(d->alpha * d->temperature * d->temperature);
    a->loss_ce = static_cast<float>(1.0 - d->alpha);
    a->grad_kd = static_cast<float>(d->alpha * d->temperature * d->scale);
    a->grad_ce = static_cast<float>((1.0 - d->alpha) * d->scale);
    return ZS_OK;
}

int set_grad(const zs_distill* d, const float* row_grad, void* grad_out, DistillArgs* a)
{
    if (d->rows > 0 && !grad_out) return ZS_ENULL;
    if (!aligned_to(grad_out, elem_bytes(d->logits_dtype)) || !aligned_to(row_grad, 4))
        return ZS_EALIGN;
    if (grad_out == a->logits && d->rows > 1 && d->grad_pitch != d->logits_pitch)
        return ZS_EINVAL_DISTILL;
    a->row_grad = row_grad;
    a->grad = grad_out;
    return ZS_OK;
}

int set_loss(const zs_distill* d, float* loss_out, float* lse_out, float* loss_sum,
             int64_t* counted, int32_t accumulate, void* workspace, size_t workspace_bytes,
             DistillArgs* a)
{
    if (!workspace || (d->rows > 0 && !loss_out)) return ZS_ENULL;
    if (!aligned16(workspace) || !aligned_to(loss_out, 4) || !aligned_to(lse_out, 4) ||
        !aligned_to(loss_sum, 4) || !aligned_to(counted, 8))
        return ZS_EALIGN;
    if (workspace_bytes < zs_distill_workspace_bytes(d)) return ZS_EWORKSPACE;
    const DistillSpace w = distill_space(d->rows, d->vocab, d->k, a->f32 != 0);
    char* base = static_cast<char*>(workspace);
    a->counts = reinterpret_cast<int32_t*>(base + w.counts);
    a->parts = reinterpret_cast<float*>(base + w.parts);
    a->picked = reinterpret_cast<float*>(base + w.picked);
    a->loss = loss_out;
    a->lse_out = lse_out;
    a->loss_sum = loss_sum;
    a->counted = counted;
    a->accumulate = accumulate ? 1 : 0;
    return ZS_OK;
}

}  // namespace
}  // namespace zs

extern "C" int embed_lookup(const zs_embed* e, const void* ids, const void* table, void* out,
                            void* stream)
{
    const int rc = check_embed(e);
    if (rc != ZS_OK) return rc;
    if (e->tokens == 0) return ZS_OK;
    if (!ids || !table || !out) return ZS_ENULL;
    if (!aligned_to(ids, id_bytes(e->id_dtype)) || !aligned_to(table, elem_bytes(e->table_dtype)) ||
        !aligned_to(out, elem_bytes(e->act_dtype)))
        return ZS_EALIGN;
    return enqueue_embed_lookup(embed_args(e, ids, table, out), stream);
}

extern "C" int embed_grad(const zs_embed* e, const void* ids, const void* grad_out,
                          void* grad_table, int32_t accumulate, void* workspace,
                          size_t workspace_bytes, void* stream)
{
    const int rc = check_embed(e);
    if (rc != ZS_OK) return rc;
    if (e->tokens > ZS_EMBED_MAX || e->rows > ZS_EMBED_MAX) return ZS_EUNSUPPORTED;
    if (!grad_table || !workspace) return ZS_ENULL;
    if (e->tokens > 0 && (!ids || !grad_out)) return ZS_ENULL;
    if (!aligned16(workspace) || !aligned_to(ids, id_bytes(e->id_dtype)) ||
        !aligned_to(grad_out, elem_bytes(e->act_dtype)) ||
        !aligned_to(grad_table, elem_bytes(e->table_dtype)))
        return ZS_EALIGN;
    if (workspace_bytes < zs_embed_workspace_bytes(e)) return ZS_EWORKSPACE;
    if (e->tokens == 0 && accumulate) return ZS_OK;
    return enqueue_embed_grad(embed_args(e, ids, grad_out, grad_table), accumulate != 0, workspace,
                              stream);
}

extern "C" int distill_loss(const zs_distill* d, const void* logits, const zs_targets* t,
                            float* loss_out, float* lse_out, float* loss_sum, int64_t* counted,
                            int32_t accumulate, void* workspace, size_t workspace_bytes,
                            void* stream)
{
    DistillArgs a;
    int rc = distill_args(d, logits, t, &a);
    if (rc != ZS_OK) return rc;
    if (d->rows > 0 && !lse_out) return ZS_ENULL;
    rc = set_loss(d, loss_out, lse_out, loss_sum, counted, accumulate, workspace, workspace_bytes,
                  &a);
    return rc != ZS_OK ? rc : enqueue_distill_loss(a, false, stream);
}

extern "C" int distill_grad(const zs_distill* d, const void* logits, const zs_targets* t,
                            const float* lse_in, const float* row_grad, void* grad_out,
                            void* stream)
{
    DistillArgs a;
    int rc = distill_args(d, logits, t, &a);
    if (rc != ZS_OK) return rc;
    if (d->rows > 0 && !lse_in) return ZS_ENULL;
    if (!aligned_to(lse_in, 4)) return ZS_EALIGN;
    if ((rc = set_grad(d, row_grad, grad_out, &a)) != ZS_OK) return rc;
    a.lse_in = lse_in;
    return enqueue_distill_grad(a, stream);
}

extern "C" int distill_loss_grad(const zs_distill* d, const void* logits, const zs_targets* t,
                                 float* loss_out, float* lse_out, const float* row_grad,
                                 void* grad_out, float* loss_sum, int64_t* counted,
                                 int32_t accumulate, void* workspace, size_t workspace_bytes,
                                 void* stream)
{
    DistillArgs a;
    int rc = distill_args(d, logits, t, &a);
    if (rc != ZS_OK) return rc;
    if ((rc = set_grad(d, row_grad, grad_out, &a)) != ZS_OK) return rc;
    rc = set_loss(d, loss_out, lse_out, loss_sum, counted, accumulate, workspace, workspace_bytes,
                  &a);
    return rc != ZS_OK ? rc : enqueue_distill_loss(a, true, stream);
}

// ---- the position-bias table ---------------------------------------------------------

namespace zs {
namespace {

// What both calls share: the struct into the kernel arguments, and the checks
// of what lies on the device.
int relpos_args(const zs_relpos* r, const void* in, void* out, const void* key_lengths,
                const void* query_starts, RelposArgs* a)
{
    const int rc = check_relpos(r);
    if (rc != ZS_OK) return rc;
    const uintptr_t size = elem_bytes(r->dtype);
    if (!aligned_to(in, size) || !aligned_to(out, size) ||
        !aligned_to(key_lengths, id_bytes(r->id_dtype)) ||
        !aligned_to(query_starts, id_bytes(r->id_dtype)))
        return ZS_EALIGN;
    const int64_t n[3] = {r->batch, r->heads, r->queries};
    *a = RelposArgs{};
    for (int k = 0; k < 3; ++k) {
        if (in && in == out && n[k] > 1 && r->in_pitch[k] != r->out_pitch[k])
            return ZS_EINVAL_RELPOS;
        a->in_pitch[k] = n[k] > 1 ? r->in_pitch[k] : 0;
        a->out_pitch[k] = n[k] > 1 ? r->out_pitch[k] : 0;
    }
    a->in = in;
    a->out = out;
    a->lengths = key_lengths;
    a->starts = query_starts;
    a->batch = r->batch;
    a->heads = r->heads;
    a->queries = r->queries;
    a->keys = r->keys;
    a->table_pitch = r->table_pitch;
    a->start = r->query_start;
    a->causal = r->causal;
    a->f32 = r->dtype == ZS_F32;
    a->table_f32 = r->table_dtype == ZS_F32;
    a->id64 = r->id_dtype == ZS_ID_I64;
    a->scale = static_cast<float>(r->scale);
    relpos_buckets(r, a);
    return ZS_OK;
}

bool relpos_empty(const zs_relpos* r) { return r->batch == 0 || r->queries == 0 || r->keys == 0; }

}  // namespace
}  // namespace zs

extern "C" int relpos_bias(const zs_relpos* r, const void* table, const void* scores,
                           const void* key_lengths, const void* query_starts, void* out,
                           void* stream)
{
    RelposArgs a;
    const int rc = relpos_args(r, scores, out, key_lengths, query_starts, &a);
    if (rc != ZS_OK) return rc;
    if (relpos_empty(r)) return ZS_OK;
    if (!table || !out) return ZS_ENULL;
    if (!aligned_to(table, elem_bytes(r->table_dtype))) return ZS_EALIGN;
    a.table = table;
    if (!relpos_bias_shape(&a)) return ZS_EUNSUPPORTED;
    return enqueue_relpos_bias(a, stream);
}

extern "C" int relpos_bias_grad(const zs_relpos* r, const void* grad, const void* key_lengths,
                                const void* query_starts, void* grad_table, void* grad_scores,
                                int32_t accumulate, void* workspace, size_t workspace_bytes,
                                void* stream)
{
    RelposArgs a;
    const int rc = relpos_args(r, grad, grad_scores, key_lengths, query_starts, &a);
    if (rc != ZS_OK) return rc;
    if (!grad_table || !workspace || (!grad && !relpos_empty(r))) return ZS_ENULL;
    if (!aligned16(workspace) || !aligned_to(grad_table, elem_bytes(r->table_dtype)))
        return ZS_EALIGN;
    if (!relpos_grad_shape(&a, grad_scores != nullptr)) return ZS_EUNSUPPORTED;
    // enough with and without grad_scores; 0: too many tiles in one of the two
    const size_t need = zs_relpos_workspace_bytes(r);
    if (need == 0) return ZS_EUNSUPPORTED;
    if (workspace_bytes < need) return ZS_EWORKSPACE;
    a.table_grad = grad_table;
    a.parts = static_cast<float*>(workspace);
    a.accumulate = accumulate ? 1 : 0;
    return enqueue_relpos_grad(a, stream);
}

// ---- many tensors -------------------------------------------------------------------

namespace zs {
namespace {

int tensors_args(const zs_tensors* t, void* plan, TensorsArgs* a)
{
    const int rc = check_tensors(t);
    if (rc != ZS_OK) return rc;
    if (!plan) return ZS_ENULL;
    if (!aligned16(plan)) return ZS_EALIGN;
    const TensorsSpace w = tensors_space(t->count, t->chunks);
    char* base = static_cast<char*>(plan);
    *a = TensorsArgs{};
    a->arrived = reinterpret_cast<uint32_t*>(base + w.arrived);
    a->table = reinterpret_cast<const TensorChunk*>(base + w.table);
    a->first = reinterpret_cast<const int64_t*>(base + w.first);
    a->partials = reinterpret_cast<double*>(base + w.partials);
    a->count = t->count;
    a->chunks = t->chunks;
    a->chunk_bytes = t->chunk_bytes;
    a->bytes = t->bytes;
    return ZS_OK;
}

int set_sqnorm(double* sqnorm_out, double* tensor_sqnorms, int32_t accumulate, TensorsArgs* a)
{
    if (!sqnorm_out) return ZS_ENULL;
    if (!aligned8(sqnorm_out) || !aligned8(tensor_sqnorms)) return ZS_EALIGN;
    a->sqnorm_out = sqnorm_out;
    a->each = tensor_sqnorms;
    a->accumulate = accumulate ? 1 : 0;
    return ZS_OK;
}

int set_clip(const zs_tensors* t, double max_norm, const double* sqnorm, double other_sqnorm,
             TensorsArgs* a)
{
    constexpr double kLargest = 1.7976931348623157e308;     // of the finite ones
    if (!(max_norm > 0.0 && max_norm <= kLargest) || other_sqnorm < 0.0)
        return ZS_EINVAL_HPARAM;
    if (!sqnorm || !t->has_out) return ZS_ENULL;
    if (!aligned8(sqnorm)) return ZS_EALIGN;
    a->sqnorm = sqnorm;
    a->other = other_sqnorm;
    a->max_norm = max_norm;
    // sqrt(Q) + 1e-6 <= max_norm, with room for the roundings on both sides; an
    // infinite Q, whose coefficient is 0, is above it whatever the limit
    const double most = max_norm - 1e-6;
    a->quiet = t->has_out == 2 && most > 0.0 ? std::fmin(most * most * (1.0 - 1e-9), kLargest)
                                             : -HUGE_VAL;
    return ZS_OK;
}

}  // namespace
}  // namespace zs

extern "C" int tensors_sqnorm(const zs_tensors* t, void* plan, double* sqnorm_out,
                              double* tensor_sqnorms, int32_t accumulate, void* stream)
{
    TensorsArgs a;
    int rc = tensors_args(t, plan, &a);
    if (rc != ZS_OK) return rc;
    if ((rc = set_sqnorm(sqnorm_out, tensor_sqnorms, accumulate, &a)) != ZS_OK) return rc;
    return enqueue_tensors_sqnorm(a, stream);
}

extern "C" int tensors_clip(const zs_tensors* t, void* plan, double max_norm, const double* sqnorm,
                            double other_sqnorm, void* stream)
{
    TensorsArgs a;
    int rc = tensors_args(t, plan, &a);
    if (rc != ZS_OK) return rc;
    if ((rc = set_clip(t, max_norm, sqnorm, other_sqnorm, &a)) != ZS_OK) return rc;
    return enqueue_tensors_clip(a, stream);
}

extern "C" int tensors_clip_norm(const zs_tensors* t, void* plan, double max_norm,
                                 double* sqnorm_out, double* tensor_sqnorms, int32_t accumulate,
                                 void* stream)
{
    TensorsArgs a;
    int rc = tensors_args(t, plan, &a);
    if (rc != ZS_OK) return rc;
    if ((rc = set_sqnorm(sqnorm_out, tensor_sqnorms, accumulate, &a)) != ZS_OK) return rc;
    if ((rc = set_clip(t, max_norm, sqnorm_out, 0.0, &a)) != ZS_OK) return rc;
    a.clip = 1;
    if ((rc = enqueue_tensors_sqnorm(a, stream)) != ZS_OK) return rc;
    return enqueue_tensors_clip(a, stream);
}
