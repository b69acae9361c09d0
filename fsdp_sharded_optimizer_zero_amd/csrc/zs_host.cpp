// zs_host.cpp -- host part of libzero_shard: shard layout, model-state and
// communication accounting, workspace layouts, argument checks, error
// strings.  No HIP calls.
//
// Layout: "Data parallelism, ZeRO and FSDP", section 2 "What is redundant"
// (rank k owns slice k) and "How FSDP implements ZeRO-3" step 1 (a unit's
// flat parameter cut into N_d equal chunks); padding sits at the tail of the
// flat vector so every slot has the same length S.
// Accounting: the same page's Theorem "ZeRO memory and communication" (table
// and proof); the error convention follows the state_bytes helper of
// "Distributed Training Basics -- DDP and FSDP" (Memory accounting).
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cstring>
#include <vector>

#include "zs_internal.h"

namespace zs {

static int64_t round_up(int64_t x, int64_t a) { return ((x + a - 1) / a) * a; }

int check_shard(const zs_shard* s)
{
    if (!s) return ZS_ENULL;
    zs_shard ref;
    int rc = zs_layout(s->psi, s->n_d, s->rank, s->align, s->stage, s->out_mode, &ref);
    if (rc != ZS_OK) return rc;
    if (s->shard_len != ref.shard_len || s->shard_offset != ref.shard_offset ||
        s->valid_len != ref.valid_len)
        return ZS_EINVAL_LAYOUT;
    if (s->n_d > ZS_MAX_RANKS) return ZS_EUNSUPPORTED;
    if (s->shard_len % 8 != 0) return ZS_EALIGN;
    return ZS_OK;
}

int check_hparams(const zs_adamw* h)
{
    if (!h) return ZS_ENULL;
    const double v[] = {h->lr, h->beta1, h->beta2, h->eps, h->weight_decay, h->max_grad_norm};
    for (double x : v)
        if (!std::isfinite(x)) return ZS_EINVAL_HPARAM;
    if (h->lr < 0.0) return ZS_EINVAL_HPARAM;
    if (!(h->beta1 >= 0.0 && h->beta1 < 1.0)) return ZS_EINVAL_HPARAM;
    if (!(h->beta2 >= 0.0 && h->beta2 < 1.0)) return ZS_EINVAL_HPARAM;
    if (!(h->eps > 0.0)) return ZS_EINVAL_HPARAM;
    if (h->weight_decay < 0.0) return ZS_EINVAL_HPARAM;
    if (h->step < 1) return ZS_EINVAL_HPARAM;
    return ZS_OK;
}

int check_embed(const zs_embed* e)
{
    if (!e) return ZS_ENULL;
    if (e->tokens < 0 || e->rows < 1 || e->first_row < 0 || e->dim < 1) return ZS_EINVAL_EMBED;
    // every buffer's size in bytes, and one past the last id, fit in 63 bits
    const int64_t most = int64_t(1) << 40;
    if (e->tokens > most || e->rows > most || e->first_row > INT64_MAX - e->rows)
        return ZS_EINVAL_EMBED;
    if (e->table_pitch < e->dim || e->act_pitch < e->dim) return ZS_EINVAL_EMBED;
    if (e->table_pitch > (int64_t(1) << 60) / e->rows ||
        e->act_pitch > (int64_t(1) << 60) / (e->tokens > 0 ? e->tokens : 1))
        return ZS_EINVAL_EMBED;
    if (e->id_dtype != ZS_ID_I32 && e->id_dtype != ZS_ID_I64) return ZS_EINVAL_EMBED;
    if (e->table_dtype != ZS_BF16 && e->table_dtype != ZS_F32) return ZS_EINVAL_EMBED;
    if (e->act_dtype != ZS_BF16 && e->act_dtype != ZS_F32) return ZS_EINVAL_EMBED;
    if (e->reserved != 0 || !std::isfinite(static_cast<float>(e->scale))) return ZS_EINVAL_EMBED;
    return ZS_OK;
}

int check_distill(const zs_distill* d)
{
    if (!d) return ZS_ENULL;
    if (d->rows < 0 || d->rows > INT32_MAX || d->vocab < 1 || d->vocab > INT32_MAX)
        return ZS_EINVAL_DISTILL;
    const int64_t pitch = (int64_t(1) << 60) / (d->rows > 0 ? d->rows : 1);
    if (d->logits_pitch < d->vocab || d->grad_pitch < d->vocab || d->logits_pitch > pitch ||
        d->grad_pitch > pitch)
        return ZS_EINVAL_DISTILL;
    if (d->k < 0 || d->k > ZS_DISTILL_MAX_K) return ZS_EINVAL_DISTILL;
    if (d->logits_dtype != ZS_BF16 && d->logits_dtype != ZS_F32) return ZS_EINVAL_DISTILL;
    if (d->teacher_dtype != ZS_BF16 && d->teacher_dtype != ZS_F32) return ZS_EINVAL_DISTILL;
    if (d->id_dtype != ZS_ID_I32 && d->id_dtype != ZS_ID_I64) return ZS_EINVAL_DISTILL;
    // tau, its reciprocal and its square are normal fp32 numbers
    if (!(d->temperature >= 1e-6 && d->temperature <= 1e6)) return ZS_EINVAL_DISTILL;
    if (!(d->alpha >= 0.0 && d->alpha <= 1.0)) return ZS_EINVAL_DISTILL;
    if (!std::isfinite(static_cast<float>(d->scale))) return ZS_EINVAL_DISTILL;
    return ZS_OK;
}

EmbedSpace embed_space(int64_t tokens, int64_t rows, int64_t dim)
{
    EmbedSpace w;
    w.order = 0;
    w.row_of = w.order + round_up(tokens * 4, 256);
    w.starts = w.row_of + round_up(tokens * 4, 256);
    w.partials = w.starts + round_up((embed_slots(rows) + 1) * 4, 256);
    // one chunk has no run that crosses into another
    const int64_t chunks = embed_chunks(tokens);
    w.bytes = w.partials + (chunks > 1 ? round_up(chunks * 2 * dim * 4, 256) : 0);
    return w;
}

DistillSpace distill_space(int64_t rows, int64_t vocab, int32_t k, bool f32)
{
    DistillSpace w;
    const DistillShape s = distill_shape(rows, vocab, f32);
    w.counts = 0;
    w.parts = round_up(rows > 0 ? rows * 4 : 4, 256);
    w.picked = w.parts +
               (s.rows_loss ? 0 : round_up(rows * s.splits * kDistillPart * int64_t(4), 256));
    w.bytes = w.picked + (s.rows_loss_grad ? 0 : round_up(rows * (k + 1) * int64_t(4), 256));
    return w;
}

TensorsSpace tensors_space(int64_t count, int64_t chunks)
{
    TensorsSpace w;
    w.arrived = 0;
    w.table = 256;
    w.first = w.table + round_up(chunks * static_cast<int64_t>(sizeof(TensorChunk)), 256);
    w.partials = w.first + round_up((count + 1) * 8, 256);
    w.bytes = w.partials + round_up(chunks > 0 ? chunks * 8 : 8, 256);
    return w;
}

// FNV-1a over the fields before the stamp.
static uint32_t tensors_stamp(const zs_tensors& t)
{
    unsigned char bytes[offsetof(zs_tensors, stamp)];
    std::memcpy(bytes, &t, sizeof bytes);
    uint32_t h = 2166136261u;
    for (unsigned char b : bytes) h = (h ^ b) * 16777619u;
    return h;
}

int check_tensors(const zs_tensors* t)
{
    if (!t) return ZS_ENULL;
    if (t->count < 0 || t->count > ZS_TENSORS_MAX || t->chunks < 0 || t->elements < t->chunks ||
        t->chunks > (int64_t(1) << 40) || t->stamp != tensors_stamp(*t) ||
        t->plan_bytes != tensors_space(t->count, t->chunks).bytes)
        return ZS_EINVAL_TENSORS;
    return ZS_OK;
}

namespace {

int64_t elem_size(int32_t dtype) { return dtype == ZS_F32 ? 4 : 2; }

int check_tensor(const zs_tensor& t)
{
    const int64_t most = int64_t(1) << 60;
    if (t.rows < 0 || t.cols < 0) return ZS_EINVAL_TENSORS;
    if ((t.in_dtype != ZS_BF16 && t.in_dtype != ZS_F32) ||
        (t.out_dtype != ZS_BF16 && t.out_dtype != ZS_F32))
        return ZS_EINVAL_TENSORS;
    if (t.rows == 0 || t.cols == 0) return ZS_OK;
    if (t.cols > most / t.rows) return ZS_EINVAL_TENSORS;
    if (t.rows > 1 && (t.in_pitch < t.cols || t.in_pitch > most / t.rows)) return ZS_EINVAL_TENSORS;
    if (!t.in) return ZS_ENULL;
    if (reinterpret_cast<uintptr_t>(t.in) % elem_size(t.in_dtype)) return ZS_EALIGN;
    if (!t.out) return ZS_OK;
    if (t.rows > 1 && (t.out_pitch < t.cols || t.out_pitch > most / t.rows))
        return ZS_EINVAL_TENSORS;
    if (reinterpret_cast<uintptr_t>(t.out) % elem_size(t.out_dtype)) return ZS_EALIGN;
    if (t.in == t.out &&
        (t.in_dtype != t.out_dtype || (t.rows > 1 && t.in_pitch != t.out_pitch)))
        return ZS_EINVAL_TENSORS;
    return ZS_OK;
}

// What one tensor reads or writes: `rows` runs of `width` bytes, `pitch` apart,
// from `begin` up to before `end`.
struct Extent {
    uint64_t begin, end, pitch, width;
    int64_t tensor;
    bool out;
};
Extent extent(const zs_tensor& t, int64_t i, bool out)
{
    const uint64_t size = static_cast<uint64_t>(elem_size(out ? t.out_dtype : t.in_dtype));
    const uint64_t rows = static_cast<uint64_t>(t.rows);
    const uint64_t pitch = rows > 1 ? (out ? t.out_pitch : t.in_pitch) * size : 0;
    Extent e;
    e.begin = reinterpret_cast<uint64_t>(out ? t.out : t.in);
    e.width = t.cols * size;
    e.pitch = pitch;
    e.end = e.begin + (rows - 1) * pitch + e.width;
    e.tensor = i;
    e.out = out;
    return e;
}

// Whether two extents that overlap have no byte in common all the same: columns
// of one matrix (a single row counts as one of the other's).
bool beside(const Extent& a, const Extent& b)
{
    const uint64_t pitch = a.pitch ? a.pitch : b.pitch;
    if (pitch == 0 || (a.pitch && b.pitch && a.pitch != b.pitch)) return false;
    if (a.width > pitch || b.width > pitch) return false;
    // b's columns as seen from a's first, in a row of `pitch`
    const uint64_t from = b.begin >= a.begin ? (b.begin - a.begin) % pitch
                                             : (pitch - (a.begin - b.begin) % pitch) % pitch;
    return from >= a.width && from + b.width <= pitch;
}

// No tensor is written where another one is read or written (the same tensor
// twice, in place, would be clipped twice, or once in places).
int check_overlap(const zs_tensor* list, int64_t count)
{
    std::vector<Extent> all;
    for (int64_t i = 0; i < count; ++i) {
        const zs_tensor& t = list[i];
        if (t.rows == 0 || t.cols == 0 || !t.out) continue;
        all.push_back(extent(t, i, true));
    }
    if (all.empty()) return ZS_OK;
    for (int64_t i = 0; i < count; ++i) {
        const zs_tensor& t = list[i];
        if (t.rows == 0 || t.cols == 0 || t.in == t.out) continue;
        all.push_back(extent(t, i, false));
    }
    std::sort(all.begin(), all.end(), [](const Extent& a, const Extent& b) {
        return a.begin != b.begin ? a.begin < b.begin : a.tensor < b.tensor;
    });
    // the extents that the next one may overlap
    std::vector<const Extent*> open;
    for (const Extent& e : all) {
        size_t kept = 0;
        for (const Extent* o : open) {
            if (o->end <= e.begin) continue;
            open[kept++] = o;
            if ((o->out || e.out) && !beside(*o, e)) return ZS_EINVAL_TENSORS;
        }
        open.resize(kept);
        open.push_back(&e);
    }
    return ZS_OK;
}

// Bytes an element has in the wider of a tensor's types, by which pieces are
// measured.
int64_t wide_size(const zs_tensor& t)
{
    return t.in_dtype == ZS_F32 || (t.out && t.out_dtype == ZS_F32) ? 4 : 2;
}

// A tensor as it is cut: its rows are one where nothing lies between them, and
// a piece has `take` elements of one row, or `take` whole rows.
struct Cut {
    int64_t rows, cols, take, pieces;
    bool whole_rows;
};
Cut cut_tensor(const zs_tensor& t, int64_t chunk_bytes)
{
    Cut c{t.rows, t.cols, 0, 0, false};
    if (c.rows == 0 || c.cols == 0) return Cut{0, 0, 1, 0, false};
    if (c.rows > 1 && t.in_pitch == c.cols && (!t.out || t.out_pitch == c.cols)) {
        c.cols *= c.rows;
        c.rows = 1;
    }
    const int64_t elems = chunk_bytes * (t.in == t.out ? kTensorPlace : 1) / wide_size(t);
    c.whole_rows = c.rows > 1 && c.cols <= elems;
    c.take = c.whole_rows ? elems / c.cols : elems;
    c.pieces = c.whole_rows ? (c.rows + c.take - 1) / c.take
                            : c.rows * ((c.cols + c.take - 1) / c.take);
    return c;
}

}  // namespace

// Whether an output has no two places in one: by size of their pitches, each
// dimension steps over all that the smaller ones take.
static bool places_apart(const int64_t pitch[3], const int64_t n[3], int64_t keys)
{
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return pitch[a] < pitch[b]; });
    int64_t span = keys;
    for (int k : order) {
        if (n[k] < 2) continue;
        if (pitch[k] < span) return false;
        span += (n[k] - 1) * pitch[k];      // (n pitch is at most 2^56)
    }
    return true;
}

int check_relpos(const zs_relpos* r)
{
    if (!r) return ZS_ENULL;
    const int64_t far = ZS_RELPOS_FAR;
    if (r->batch < 0 || r->batch > far || r->heads < 1 || r->heads > 65536 || r->queries < 0 ||
        r->queries > far || r->keys < 0 || r->keys > far)
        return ZS_EINVAL_RELPOS;
    // every place and every tile has a number of 62 bits
    const int64_t most = int64_t(1) << 56;
    const int64_t n[3] = {r->batch, r->heads, r->queries};
    int64_t places = r->keys > 0 ? r->keys : 1;
    const bool empty = r->batch == 0 || r->queries == 0 || r->keys == 0;
    for (int k = 0; k < 3; ++k) {
        const int64_t size = n[k] > 0 ? n[k] : 1;
        if (places > most / size) return ZS_EINVAL_RELPOS;
        places *= size;
        if (n[k] < 2 || empty) continue;
        if (r->in_pitch[k] < r->keys || r->out_pitch[k] < r->keys ||
            r->in_pitch[k] > most / n[k] || r->out_pitch[k] > most / n[k])
            return ZS_EINVAL_RELPOS;
    }
    if (!empty && !places_apart(r->out_pitch, n, r->keys)) return ZS_EINVAL_RELPOS;
    if (r->table_pitch < r->heads || r->table_pitch > most) return ZS_EINVAL_RELPOS;
    if (r->query_start < -far || r->query_start > far) return ZS_EINVAL_RELPOS;
    if ((r->bidirectional != 0 && r->bidirectional != 1) || (r->causal != 0 && r->causal != 1))
        return ZS_EINVAL_RELPOS;
    if (r->buckets < (r->bidirectional ? 4 : 2) || r->buckets > ZS_RELPOS_MAX_BUCKETS)
        return ZS_EINVAL_RELPOS;
    const int64_t exact = (r->bidirectional ? r->buckets / 2 : r->buckets) / 2;
    if (r->max_distance <= exact || r->max_distance > far) return ZS_EINVAL_RELPOS;
    if ((r->dtype != ZS_BF16 && r->dtype != ZS_F32) ||
        (r->table_dtype != ZS_BF16 && r->table_dtype != ZS_F32) ||
        (r->id_dtype != ZS_ID_I32 && r->id_dtype != ZS_ID_I64))
        return ZS_EINVAL_RELPOS;
    if (!std::isfinite(static_cast<float>(r->scale))) return ZS_EINVAL_RELPOS;
    return ZS_OK;
}

namespace {

// A whole number of up to 4096 bits, little end first.
struct Whole {
    uint32_t w[129];
    int n = 1;
    Whole() { w[0] = 1; }
    void times(uint32_t x)
    {
        uint64_t carry = 0;
        for (int i = 0; i < n; ++i) {
            carry += static_cast<uint64_t>(w[i]) * x;
            w[i] = static_cast<uint32_t>(carry);
            carry >>= 32;
        }
        if (carry) w[n++] = static_cast<uint32_t>(carry);
    }
    bool at_least(const Whole& o) const
    {
        if (n != o.n) return n > o.n;
        for (int i = n - 1; i >= 0; --i)
            if (w[i] != o.w[i]) return w[i] > o.w[i];
        return true;
    }
};

// Whether n^m >= exact^(m-k) far^k (each at most 2^29, m at most 128: 3712 bits).
bool reaches(uint32_t n, uint32_t exact, uint32_t far, int m, int k)
{
    Whole a, b;
    for (int i = 0; i < m; ++i) a.times(n);
    for (int i = 0; i < m; ++i) b.times(i < k ? far : exact);
    return a.at_least(b);
}

}  // namespace

void relpos_buckets(const zs_relpos* r, RelposArgs* a)
{
    a->buckets = r->buckets;
    a->two_sided = r->bidirectional;
    a->half = r->bidirectional ? r->buckets / 2 : r->buckets;
    a->exact = a->half / 2;
    const int m = a->half - a->exact;
    a->edge_count = m - 1;
    a->edge_span = 1;
    while (a->edge_span * 2 <= a->edge_count) a->edge_span *= 2;
    const double step = std::log(static_cast<double>(r->max_distance) / a->exact) / m;
    for (int k = 1; k < m; ++k) {
        // where the step is reached, in fp64 (off by at most some 1e-14 of it);
        // next to a whole number the whole numbers decide
        const double x = a->exact * std::exp(k * step), near = std::round(x);
        int64_t edge = static_cast<int64_t>(std::ceil(x));
        if (std::fabs(x - near) <= 1e-12 * x) {
            const int64_t c = static_cast<int64_t>(near);
            edge = reaches(static_cast<uint32_t>(c), static_cast<uint32_t>(a->exact),
                           static_cast<uint32_t>(r->max_distance), m, k)
                       ? c
                       : c + 1;
        }
        a->edges[k - 1] = static_cast<int32_t>(edge);
    }
    a->far = a->edge_count > 0 ? a->edges[a->edge_count - 1] : a->exact;
}

namespace {

constexpr int64_t kRelposWaves = kRelposThreads / 64;

bool past_caches(const RelposArgs& a)
{
    return a.batch * a.heads * a.queries * a.keys * (a.f32 ? 4 : 2) >= kRelposNt;
}

}  // namespace

bool relpos_bias_shape(RelposArgs* a)
{
    const int64_t n = a->f32 ? 4 : 8;
    a->lane_shift = 3;
    while (a->lane_shift < 6 && (n << a->lane_shift) < a->keys) ++a->lane_shift;
    // Of a bias alone: 32 lanes a row where that leaves out a sixth of the columns that
    // tiles of 64 cover (13 x 44 x 943 x 539 bf16: 122 us, with 64 132), or 16 for rows
    // of one tile (300 x 280: 27 us, with 64 36; longer ones lose, 300 x 1067 82 and
    // 75, and so does a bias onto scores, 300 x 380: 57 and 49).
    const auto covers = [&](int shift) { return round_up(a->keys, n << shift); };
    const int most = a->lane_shift;
    for (int shift = 5; !a->in && most == 6 && shift >= (a->keys <= n << 6 ? 4 : 5); --shift)
        if (a->queries >= (kRelposLaneRows * int64_t(64) >> shift) &&
            covers(shift) * 6 < covers(a->lane_shift) * 5)
            a->lane_shift = shift;
    const int64_t lanes = int64_t(1) << a->lane_shift, groups = 64 / lanes;
    const int64_t planes = a->batch * a->heads;
    a->col_tiles = (a->keys + lanes * n - 1) / (lanes * n);
    a->lane_vectors = 1;
    if (a->queries == 1 && planes * a->col_tiles >= kRelposManyTiles) {
        a->lane_vectors = kRelposLaneVectors;
        a->col_tiles = (a->col_tiles + kRelposLaneVectors - 1) / kRelposLaneVectors;
    }
    a->rows = static_cast<int32_t>(groups * (a->queries == 1 ? 1 : kRelposLaneRows));
    a->row_tiles = (a->queries + a->rows - 1) / a->rows;
    a->tiles = planes * a->row_tiles * a->col_tiles;
    a->blocks = (a->tiles + kRelposWaves - 1) / kRelposWaves;
    a->nt = past_caches(*a);
    return a->blocks <= INT32_MAX / kRelposWaves;
}

bool relpos_grad_shape(RelposArgs* a, bool scores)
{
    const int64_t n = a->f32 ? 4 : 8;
    a->lane_shift = 3;
    while (a->lane_shift < 6 && (n << a->lane_shift) < a->keys) ++a->lane_shift;
    const int64_t lanes = int64_t(1) << a->lane_shift, groups = 64 / lanes;
    a->col_tiles = (a->keys + lanes * n - 1) / (lanes * n);
    const int64_t planes = a->batch * a->heads;
    // a multiple of 8 rows: two batches of the kernel's
    int64_t rows = (scores ? kRelposScoreRows : kRelposRows) / groups;
    if (rows < 8) rows = 8;
    const auto row_tiles = [&] { return (a->queries + rows * groups - 1) / (rows * groups); };
    while (rows > 8 && planes * a->col_tiles * row_tiles() < kRelposGradTiles) rows /= 2;
    // so many tiles, of rows as near alike as multiples of 8 are (8 x 32 heads, 8 x
    // 4096 bf16: 8.7 us, with 64 rows 21.6; 65 x 4096 29 us and 35)
    const int64_t tall = groups * std::max<int64_t>(row_tiles(), 1);
    rows = std::max<int64_t>(round_up((a->queries + tall - 1) / tall, 8), 8);
    a->rows = static_cast<int32_t>(rows);
    a->row_tiles = row_tiles();
    a->plane_blocks = (a->row_tiles * a->col_tiles + kRelposWaves - 1) / kRelposWaves;
    a->blocks = planes * a->plane_blocks;
    a->tiles = kRelposWaves * a->blocks;
    a->nt = past_caches(*a);
    return a->blocks <= INT32_MAX / kRelposWaves;
}

int64_t relpos_parts_bytes(const RelposArgs& a)
{
    const int64_t bytes = a.blocks * a.buckets * 4;
    return round_up(bytes > 0 ? bytes : 1, 256);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The section 5 simulator's adamw evaluates 1 - beta and 1 - beta**t in
// double; each scalar is computed in double and rounded to fp32 once.
// A normal, positive power of two (its reciprocal is then exact).
static bool is_pow2f(float x)
{
    if (!(x >= 1.17549435e-38f) || !std::isfinite(x)) return false;
    int e = 0;
    return std::frexp(x, &e) == 0.5f;
}

StepConsts make_consts(const zs_adamw* h)
{
    const double t = static_cast<double>(h->step);
    StepConsts c;
    c.b1 = static_cast<float>(h->beta1);
    c.b2 = static_cast<float>(h->beta2);
    c.c1 = static_cast<float>(1.0 - h->beta1);
    c.c2 = static_cast<float>(1.0 - h->beta2);
    c.bc1 = static_cast<float>(1.0 - std::pow(h->beta1, t));
    c.bc2 = static_cast<float>(1.0 - std::pow(h->beta2, t));
    c.lr = static_cast<float>(h->lr);
    c.wd = static_cast<float>(h->weight_decay);
    c.eps = static_cast<float>(h->eps);
    c.bc1_pow2 = is_pow2f(c.bc1) ? 1 : 0;
    c.bc2_pow2 = is_pow2f(c.bc2) ? 1 : 0;
    c.inv_bc1 = c.bc1_pow2 ? 1.0f / c.bc1 : 0.0f;
    c.inv_bc2 = c.bc2_pow2 ? 1.0f / c.bc2 : 0.0f;
    return c;
}

}  // namespace zs

extern "C" {

int zs_layout(int64_t psi, int32_t n_d, int32_t rank, int64_t align, int32_t stage,
              int32_t out_mode, zs_shard* out)
{
    if (!out) return ZS_ENULL;
    if (psi <= 0) return ZS_EINVAL_PSI;
    if (n_d < 1) return ZS_EINVAL_ND;
    if (rank < 0 || rank >= n_d) return ZS_EINVAL_RANK;
    if (align < 1) return ZS_EINVAL_LAYOUT;
    if (stage < 0 || stage > 3) return ZS_EINVAL_STAGE;
    if (out_mode != ZS_OUT_GATHER && out_mode != ZS_OUT_SHARD) return ZS_EINVAL_STAGE;
    zs_shard s;
    s.psi = psi;
    s.n_d = n_d;
    s.rank = rank;
    s.align = align;
    s.stage = stage;
    s.out_mode = out_mode;
    if (stage == 0) {                    // DDP: the whole vector on every rank
        s.shard_len = zs::round_up(psi, align);
        s.shard_offset = 0;
        s.valid_len = psi;
    } else {
        const int64_t per_rank = psi / n_d + (psi % n_d != 0 ? 1 : 0);
        s.shard_len = zs::round_up(per_rank, align);
        s.shard_offset = static_cast<int64_t>(rank) * s.shard_len;
        const int64_t rest = psi - s.shard_offset;
        s.valid_len = rest <= 0 ? 0 : (rest < s.shard_len ? rest : s.shard_len);
    }
    *out = s;
    return ZS_OK;
}

size_t zs_workspace_bytes(const zs_shard* s)
{
    // One fp64 partial per clip-pass block and one per group of them,
    // rounded up to 256 bytes.
    const int64_t v = (s && s->valid_len > 0) ? s->valid_len : 0;
    const int64_t n = zs::sq_blocks(v);
    const int64_t bytes = (n + zs::sq_groups(n)) * static_cast<int64_t>(sizeof(double));
    return static_cast<size_t>(zs::round_up(bytes > 0 ? bytes : 1, 256));
}

size_t zs_workspace_bytes_units(const zs_shard* s, int32_t units)
{
    // units x (partials + group sums), rounded up to 256 bytes
    if (units < 1) units = 1;
    const int64_t v = (s && s->valid_len > 0) ? s->valid_len : 0;
    const int64_t n = zs::sq_blocks(v);
    const int64_t bytes =
        static_cast<int64_t>(units) * (n + zs::sq_groups(n)) * static_cast<int64_t>(sizeof(double));
    return static_cast<size_t>(zs::round_up(bytes > 0 ? bytes : 1, 256));
}

size_t zs_embed_workspace_bytes(const zs_embed* e)
{
    if (zs::check_embed(e) != ZS_OK || e->tokens > ZS_EMBED_MAX || e->rows > ZS_EMBED_MAX) return 0;
    return static_cast<size_t>(zs::embed_space(e->tokens, e->rows, e->dim).bytes);
}

size_t zs_relpos_workspace_bytes(const zs_relpos* r)
{
    if (zs::check_relpos(r) != ZS_OK) return 0;
    zs::RelposArgs a{};
    a.batch = r->batch;
    a.heads = r->heads;
    a.queries = r->queries;
    a.keys = r->keys;
    a.buckets = r->buckets;
    a.f32 = r->dtype == ZS_F32;
    // enough for either: with the scores' gradient and without
    if (!zs::relpos_grad_shape(&a, false)) return 0;
    const int64_t alone = zs::relpos_parts_bytes(a);
    if (!zs::relpos_grad_shape(&a, true)) return 0;
    const int64_t both = zs::relpos_parts_bytes(a);
    return static_cast<size_t>(alone > both ? alone : both);
}

size_t zs_distill_workspace_bytes(const zs_distill* d)
{
    if (zs::check_distill(d) != ZS_OK) return 0;
    return static_cast<size_t>(zs::distill_space(d->rows, d->vocab, d->k, d->logits_dtype == ZS_F32).bytes);
}

int zs_tensors_layout(const zs_tensor* list, int64_t count, zs_tensors* t)
{
    if (!t || (count > 0 && !list)) return ZS_ENULL;
    if (count < 0) return ZS_EINVAL_TENSORS;
    if (count > ZS_TENSORS_MAX) return ZS_EUNSUPPORTED;
    zs_tensors r{};
    r.count = count;
    bool place = true;
    r.has_out = 1;
    int64_t bytes = 0;
    for (int64_t i = 0; i < count; ++i) {
        const int rc = zs::check_tensor(list[i]);
        if (rc != ZS_OK) return rc;
        const int64_t n = list[i].rows * list[i].cols;
        if (n == 0) continue;
        r.elements += n;
        const bool here = list[i].in == list[i].out;
        bytes += n * zs::wide_size(list[i]) / (here ? zs::kTensorPlace : 1);
        r.bytes += n * zs::elem_size(list[i].in_dtype);
        place = place && here;
        // (each is at most 2^62: the sum is looked at before it can overflow)
        if (bytes > (int64_t(1) << 60)) return ZS_EINVAL_TENSORS;
        if (!list[i].out) r.has_out = 0;
    }
    if (r.has_out && place) r.has_out = 2;
    try {
        const int rc = zs::check_overlap(list, count);
        if (rc != ZS_OK) return rc;
    } catch (...) {
        return ZS_EUNSUPPORTED;         // host memory for the check
    }
    // as many pieces as fill the GPU, and no more than one block can join
    r.chunk_bytes = zs::kTensorChunkMin;
    while (r.chunk_bytes < 4 * zs::kTensorPart && bytes / r.chunk_bytes > zs::kTensorChunksMin)
        r.chunk_bytes *= 2;
    if (bytes / r.chunk_bytes > zs::kTensorChunks) {
        r.chunk_bytes = zs::round_up(bytes / zs::kTensorChunks, zs::kTensorPart);
        if (r.chunk_bytes > zs::kTensorChunkMax) r.chunk_bytes = zs::kTensorChunkMax;
    }
    for (int64_t i = 0; i < count; ++i)
        r.chunks += zs::cut_tensor(list[i], r.chunk_bytes).pieces;
    r.plan_bytes = zs::tensors_space(r.count, r.chunks).bytes;
    r.stamp = zs::tensors_stamp(r);
    *t = r;
    return ZS_OK;
}

int zs_tensors_plan(const zs_tensor* list, const zs_tensors* t, void* plan, size_t plan_bytes)
{
    if (!t || !plan) return ZS_ENULL;
    zs_tensors ref;
    const int rc = zs_tensors_layout(list, t->count, &ref);
    if (rc != ZS_OK) return rc;
    if (std::memcmp(&ref, t, sizeof ref) != 0) return ZS_EINVAL_TENSORS;
    if (plan_bytes < static_cast<size_t>(t->plan_bytes)) return ZS_EWORKSPACE;
    const zs::TensorsSpace w = zs::tensors_space(t->count, t->chunks);
    char* base = static_cast<char*>(plan);
    std::memset(base, 0, static_cast<size_t>(t->plan_bytes));
    char* at = base + w.table;
    int64_t pieces = 0;
    for (int64_t i = 0; i < t->count; ++i) {
        std::memcpy(base + w.first + i * 8, &pieces, 8);
        const zs_tensor& x = list[i];
        const zs::Cut c = zs::cut_tensor(x, t->chunk_bytes);
        const int64_t is = zs::elem_size(x.in_dtype), os = zs::elem_size(x.out_dtype);
        const auto put = [&](int64_t row, int64_t col, int64_t rows, int64_t cols) {
            zs::TensorChunk k{};
            k.in = reinterpret_cast<uint64_t>(x.in) + (row * x.in_pitch + col) * is;
            k.out = x.out ? reinterpret_cast<uint64_t>(x.out) + (row * x.out_pitch + col) * os : 0;
            k.in_pitch = x.in_pitch;
            k.out_pitch = x.out_pitch;
            k.rows = static_cast<int32_t>(rows);
            k.cols = static_cast<int32_t>(cols);
            k.kind = (x.in_dtype == ZS_F32 ? zs::kChunkInF32 : 0) |
                     (x.out_dtype == ZS_F32 ? zs::kChunkOutF32 : 0) |
                     (x.in == x.out ? zs::kChunkPlace : 0);
            k.tensor = static_cast<int32_t>(i);
            std::memcpy(at, &k, sizeof k);
            at += sizeof k;
            ++pieces;
        };
        if (c.whole_rows) {
            for (int64_t r = 0; r < c.rows; r += c.take)
                put(r, 0, c.rows - r < c.take ? c.rows - r : c.take, c.cols);
        } else {
            for (int64_t r = 0; r < c.rows; ++r)
                for (int64_t col = 0; col < c.cols; col += c.take)
                    put(r, col, 1, c.cols - col < c.take ? c.cols - col : c.take);
        }
    }
    std::memcpy(base + w.first + t->count * 8, &pieces, 8);
    return ZS_OK;
}

double zs_state_bytes(double psi, int32_t n_d, int32_t stage, double K)
{
    if (!(psi > 0.0) || n_d < 1) return -1.0;
    const double weights = 2.0 * psi, grads = 2.0 * psi, optim = K * psi;
    switch (stage) {
    case 0: return weights + grads + optim;
    case 1: return weights + grads + optim / n_d;
    case 2: return weights + (grads + optim) / n_d;
    case 3: return (weights + grads + optim) / n_d;
    default: return -1.0;
    }
}

double zs_comm_bytes(double psi, int32_t n_d, int32_t stage, double bytes_per_elem)
{
    if (!(psi > 0.0) || n_d < 1 || stage < 0 || stage > 3) return -1.0;
    // stages 0-2: one reduce-scatter and one all-gather of psi elements;
    // stage 3: a second all-gather for the backward pass.
    const double collectives = stage == 3 ? 3.0 : 2.0;
    return collectives * psi * bytes_per_elem * static_cast<double>(n_d - 1) / n_d;
}

const char* zs_strerror(int code)
{
    switch (code) {
    case ZS_OK: return "ok";
    case ZS_EINVAL_PSI: return "psi must be positive";
    case ZS_EINVAL_ND: return "n_d must be at least 1";
    case ZS_EINVAL_RANK: return "rank must be in [0, n_d)";
    case ZS_EINVAL_LAYOUT: return "align < 1 or shard fields inconsistent with zs_layout";
    case ZS_EALIGN: return "pointer not 16-byte aligned or shard_len not a multiple of 8";
    case ZS_EINVAL_HPARAM: return "invalid AdamW hyperparameter";
    case ZS_EINVAL_STAGE: return "invalid stage or out_mode";
    case ZS_ENULL: return "required pointer is NULL (or both/neither gradient source)";
    case ZS_EUNSUPPORTED: return "n_d exceeds ZS_MAX_RANKS";
    case ZS_EWORKSPACE: return "workspace smaller than zs_workspace_bytes";
    case ZS_ELAUNCH: return "the HIP runtime refused a kernel launch or a set-up call";
    case ZS_EINVAL_REDUCE: return "invalid zs_reduce (dtype, micro-batch index/count or token count)";
    case ZS_EZERO_TOKENS: return "global token count is zero: the update is rejected";
    case ZS_EINVAL_UNITS: return "units must be at least 1";
    case ZS_ESCRATCH: return "shard too large for the static scratch array (ZS_SCRATCH_BYTES)";
    case ZS_EINVAL_EMBED: return "invalid zs_embed (a size, pitch, type or scale out of range)";
    case ZS_EINVAL_DISTILL:
        return "invalid zs_distill (a size, pitch, type, temperature, alpha or scale out of range)";
    case ZS_EINVAL_TENSORS:
        return "invalid zs_tensor (a size, pitch or type out of range, in place with another, or "
               "written where another of the list is read or written), or zs_tensors not as "
               "zs_tensors_layout left it";
    case ZS_EINVAL_RELPOS:
        return "invalid zs_relpos (a size, pitch, type, position, bucket count, distance or scale "
               "out of range)";
    default: return "unknown error";
    }
}

}  // extern "C"
