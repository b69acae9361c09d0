// zs_internal.h -- declarations shared by the host parts (zs_host.cpp,
// zs_abi.cpp) and the kernel part (zs_kernels.hip) of libzero_shard.  Not
// part of the ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "zero_shard.h"

namespace zs {

// fp32 scalars of one AdamW step, each rounded once from double.
struct StepConsts {
    float b1, b2, c1, c2, bc1, bc2, lr, wd, eps;
    // When bc1 (bc2) is a power of two, x / bc equals x * (1 / bc) bit for
    // bit (both are the rounding of the same exact value), and the kernel
    // multiplies by the exact reciprocal instead of dividing.
    float inv_bc1, inv_bc2;
    int32_t bc1_pow2, bc2_pow2;
};

// The clip pass runs blocks of 128, 256 or 512 threads (one 8-parameter
// vector per thread, the size chosen per call by the kernel part) and writes
// one fp64 partial sum per block into the workspace; the workspace is sized
// for the smallest block.
constexpr int kSqThreadsMin = 128;

// Blocks of the clip pass over valid_len parameters at `threads` threads per
// block (the last vector may be partial).
inline int64_t sq_blocks(int64_t valid_len, int threads = kSqThreadsMin)
{
    const int64_t nvec = (valid_len + 7) / 8;
    return (nvec + threads - 1) / threads;
}

// The block partials are summed in two fixed-order stages: groups of
// kSqGroup partials, then the group sums.
constexpr int64_t kSqGroup = 4096;
inline int64_t sq_groups(int64_t partials) { return (partials + kSqGroup - 1) / kSqGroup; }

struct SlicePtrs {
    const void* p[ZS_MAX_RANKS];   // bf16 or fp32 rows, by the kernel's element type
};

struct StepArgs {
    SlicePtrs slices;
    const float* mean;
    const double* sqnorm;
    double other_sqnorm;
    double max_norm;
    float* w;
    float* m;
    float* v;
    uint16_t* out;          // slot base: shard element 0
    int64_t valid_len;
    int64_t shard_len;
    int64_t v0;             // first vector of this launch
    int32_t n_d;
    float nd;               // (float)n_d
    float inv_nd;           // 1/n_d, exact when n_d is a power of two
    StepConsts c;
};

struct SqArgs {
    SlicePtrs slices;
    float wt[ZS_MAX_RANKS]; // token weights (weighted reduction only)
    float* mean_out;        // the reduced gradient; also read in place when
                            // it is a micro-batch accumulator
    double* partials;       // one per block of this launch; null: no norm
    int64_t valid_len;
    int64_t v0;             // first vector of this launch
    int32_t n_d;
    float nd;
    float inv_nd;
    float micro_count;      // m, the divisor of the last micro-batch
    float inv_micro_count;  // 1/m when m is a power of two (exact), else 0
};

// What the clip pass does with the accumulator: write the reduced slice
// (no accumulation, or the first micro-batch), add it to the accumulator,
// or add it and divide by the micro-batch count (the last micro-batch).
enum AccMode { kAccNone = 0, kAccAdd = 1, kAccFinal = 2 };

// The passes (zs_kernels.hip).  Each enqueues its launches on `stream` (a
// hipStream_t), splitting a grid longer than one launch may hold, and
// returns ZS_OK or ZS_ELAUNCH; arguments are validated by the caller.
//   reduce_blocks: the number of blocks (fp64 partials) the clip pass runs
//     over valid_len parameters for this reduction (at most
//     sq_blocks(valid_len)).
//   enqueue_reduce: the clip pass / general reduction over a.valid_len
//     (a.v0 and a.partials are set per launch; partials: reduce_blocks(...)
//     fp64 slots, or null for no norm).  f32/weighted/acc select the general
//     reduction (always stored); otherwise bf16 rank-order mean, stored iff
//     `store`.
//   enqueue_sqnorm_sums: units x blocks partials (unit-major) -> *sqnorm_out
//     (added to it if accumulate), in a fixed order.
//   enqueue_step: the fused AdamW step over a.shard_len (a.v0 set per launch).
//   enqueue_pack: bf16 cast of master[0, valid_len) and +0 pads into out.
int64_t reduce_blocks(int64_t valid_len, int32_t n_d, bool f32, int acc);
int enqueue_reduce(SqArgs a, bool f32, bool weighted, int acc, bool store, double* partials,
                   void* stream);
int enqueue_sqnorm_sums(double* partials, int64_t blocks, int32_t units, double* sqnorm_out,
                        int accumulate, void* stream);
int enqueue_step(StepArgs a, bool from_slices, bool clip, void* stream);
int enqueue_pack(const float* master, uint16_t* out, int64_t valid_len, int64_t shard_len,
                 void* stream);

// Per-device set-up (zs_kernels.hip), for the current device; each returns
// ZS_OK or ZS_ELAUNCH.
//   prepare_device: the set-up calls every kernel launch needs (the LDS
//     query and the kernels' dynamic-LDS limits) and the address of the
//     static scratch array, so that later calls make none.
//   static_scratch: *ptr = this device's ZS_SCRATCH_BYTES scratch array.
int prepare_device();
int static_scratch(void** ptr);

// ---- the vocabulary table (zs_vocab.hip) -----------------------------------------

struct EmbedArgs {
    const void* ids;
    const void* src;        // lookup: table; gradient: activation gradients
    void* dst;              // lookup: activations; gradient: table gradient
    int64_t tokens, rows, first_row, dim;
    int64_t table_pitch, act_pitch;
    float scale;
    int32_t id64, table_f32, act_f32;
};

// embed_grad sorts the tokens by row, cuts the sorted order into chunks of
// embed_chunk positions and sums each chunk's runs; a run that crosses chunks
// leaves one partial row in each (at most two per chunk) for the join.
// Longer chunks mean fewer partials, shorter ones more parallel work: 8
// positions until the chunks number 1024, then twice as many, up to 64.
// Up to kEmbedFew tokens (one a lane) are not sorted at all.
constexpr int64_t kEmbedFew = 64;
inline int32_t embed_chunk(int64_t tokens)
{
    int32_t c = 8;
    while (c < 64 && tokens > 1024 * static_cast<int64_t>(c)) c *= 2;
    return c;
}
inline int64_t embed_chunks(int64_t tokens)
{
    const int64_t c = embed_chunk(tokens);
    return (tokens + c - 1) / c;
}

// The sort deals the rows to a power of two of buckets, at least kSortBuckets
// (rows permitting) and so many that none has more than kSortRows; the slots
// are the rows' places in the sorted order, a whole number per bucket.
constexpr int kSortRows = 512;
constexpr int kSortBuckets = 256;
struct SortShape {
    int32_t bucket_bits;    // log2 of the buckets
    int32_t rows;           // rows of a bucket
    int32_t row_bits;       // bits of a row's number in its bucket
};
inline SortShape sort_shape(int64_t rows)
{
    SortShape s{0, 0, 0};
    while ((int64_t(1) << s.bucket_bits) < kSortBuckets && (int64_t(1) << s.bucket_bits) < rows)
        ++s.bucket_bits;
    while ((rows - 1) >> s.bucket_bits >= kSortRows) ++s.bucket_bits;
    s.rows = static_cast<int32_t>(((rows - 1) >> s.bucket_bits) + 1);
    while ((1 << s.row_bits) < s.rows) ++s.row_bits;
    return s;
}
inline int64_t embed_slots(int64_t rows)
{
    const SortShape s = sort_shape(rows);
    return static_cast<int64_t>(s.rows) << s.bucket_bits;
}

// Workspace of embed_grad, in bytes from its start.
struct EmbedSpace {
    int64_t order;     // int32[tokens]: token positions sorted by row
    int64_t row_of;    // int32[tokens]: their rows
    int64_t starts;    // int32[slots + 1]: first sorted position of each slot
    int64_t partials;  // fp32[chunks][2][dim]
    int64_t bytes;
};
EmbedSpace embed_space(int64_t tokens, int64_t rows, int64_t dim);

int enqueue_embed_lookup(const EmbedArgs& a, void* stream);
int enqueue_embed_grad(const EmbedArgs& a, bool accumulate, void* workspace, void* stream);

struct DistillArgs {
    const void* logits;
    const void* teacher_ids;
    const void* teacher_logits;
    const float* teacher_lse;
    const void* labels;
    const float* lse_in;
    const float* row_grad;
    float* loss;
    float* lse_out;
    void* grad;
    int32_t* counts;        // workspace: 1 for a row that counts
    float* parts;           // workspace: fp32[rows][splits][kDistillPart]
    float* picked;          // workspace: fp32[rows][k + 1], logits at the entries and the label
    float* loss_sum;
    int64_t* counted;
    int64_t rows, vocab, logits_pitch, grad_pitch;
    int64_t part_cols;      // columns of one part (a multiple of 8)
    int32_t splits;         // parts a row is cut into
    int32_t k;              // 0 where alpha is 0
    int32_t entry_bits;     // log2 of the hash chains of the entries (set per launch)
    int32_t accumulate;
    int32_t f32, teacher_f32, id64, kd, ce;
    float inv_tau;          // 1/tau
    float loss_kd, loss_ce; // alpha tau^2, 1 - alpha
    float grad_kd, grad_ce; // alpha tau scale, (1 - alpha) scale
};

// A row cut into parts leaves per part: the maximum, and the sums of
// exp((s - max)/tau) and exp(s - max) (and a fourth number, unused: 16 bytes).
constexpr int kDistillPart = 4;

// How a call cuts its work.  A part is what a block of kDistillPartThreads
// holds in registers at `hold` 16-byte vectors a thread: 8, or 2 where 8 would
// make too few blocks to fill the GPU.
//  - The gradient from saved statistics always runs in parts.
//  - Loss and gradient in one call run a block a row (reading the logits
//    once) from kDistillRows rows on, or where a row is at most kDistillShort
//    vectors; fewer rows would leave CUs idle, and run in parts, twice (bf16,
//    a block a row against parts: 511 x 128256 56 us and 75, 128 x 128256 24
//    and 34, 64 x 128256 23 and 22, 8 x 128256 22 and 13, 8 x 8192 12 and 14;
//    the one size where parts win above the bound, 320 x 262144, 99 and 88).
//  - The loss runs a block a row where that does and a block of 256 threads
//    holds the row (then both calls' losses are the same bits; 511 x 32000 and
//    its gradient 33 us, in parts 37), otherwise in parts, then one wave a
//    row.
constexpr int kDistillPartThreads = 256;
constexpr int kDistillHold = 8;
constexpr int kDistillFewHold = 2;
constexpr int64_t kDistillBlocks = 2048;    // 8 blocks of 4 waves on each of 256 CUs
constexpr int64_t kDistillRows = 128;
constexpr int64_t kDistillShort = 1024;     // 8 vectors for each of 128 threads
struct DistillShape {
    int32_t splits;         // parts of a row
    int32_t hold;
    int64_t part_cols;      // columns of a part
    bool rows_loss;         // a block a row for the loss
    bool rows_loss_grad;    // the same for loss and gradient
};
inline DistillShape distill_shape(int64_t rows, int64_t vocab, bool f32)
{
    const int64_t vector = f32 ? 4 : 8;
    const auto parts = [&](int64_t hold) {
        const int64_t cols = hold * kDistillPartThreads * vector;
        return (vocab + cols - 1) / cols;
    };
    DistillShape s;
    s.hold = rows * parts(kDistillHold) >= kDistillBlocks ? kDistillHold : kDistillFewHold;
    s.splits = static_cast<int32_t>(parts(s.hold));
    s.part_cols = s.hold * kDistillPartThreads * vector;
    s.rows_loss_grad = rows >= kDistillRows || vocab / vector <= kDistillShort;
    s.rows_loss = s.rows_loss_grad && vocab / vector <= 16 * 256;
    return s;
}
struct DistillSpace {
    int64_t counts, parts, picked, bytes;
};
DistillSpace distill_space(int64_t rows, int64_t vocab, int32_t k, bool f32);

int enqueue_distill_loss(DistillArgs a, bool with_grad, void* stream);
int enqueue_distill_grad(DistillArgs a, void* stream);

// Loads the vocabulary kernels on the current device (so that a first call
// may be captured); ZS_OK or ZS_ELAUNCH.
int prepare_vocab();

int check_embed(const zs_embed* e);
int check_distill(const zs_distill* d);

// Host-side checks; each returns ZS_OK or the error code to report.
int check_shard(const zs_shard* s);
int check_hparams(const zs_adamw* h);
bool aligned16(const void* p);
StepConsts make_consts(const zs_adamw* h);

}  // namespace zs
