// zs_vocab.hip -- CDNA4 (gfx950) kernels of the vocabulary table: embedding
// lookup and gradient, distillation loss and gradient; their launch shapes,
// and the enqueue_* functions through which the C-ABI entry points
// (zs_abi.cpp) run them.
//
// What is computed is stated with the entry points in zero_shard.h.  All of
// it is bound by HBM: a lookup and an embedding gradient do one product or
// sum per element moved, a distillation about ten operations and one or two
// exponentials per logit (nothing here is a contraction, so no MFMA).
//
// Rows of odd length start anywhere: every 16-byte access is declared with
// the alignment of its element, which compiles to the same one instruction
// (global memory takes any byte address in the unaligned access mode the HSA
// ABI sets), and the elements behind a row's last full vector go one by one.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "zs_internal.h"

namespace zs {
namespace {

#ifndef ZS_MAX_LAUNCH_THREADS
#define ZS_MAX_LAUNCH_THREADS (int64_t(1) << 31)
#endif
constexpr int64_t max_blocks(int threads) { return ZS_MAX_LAUNCH_THREADS / threads; }

constexpr int kWave = 64;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLowest = -3.402823466e38f;

// ---- elements ------------------------------------------------------------------

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_u __attribute__((ext_vector_type(2), aligned(2)));

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// fp32 -> bf16 by the hardware's conversion: round to nearest even,
// subnormals kept, NaN stays NaN.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), b16x2));
}

__device__ __forceinline__ float widen(uint16_t x)
{
    return __uint_as_float(static_cast<uint32_t>(x) << 16);
}
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = static_cast<uint16_t>(pack_bf16x2(v, 0.0f)); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// N consecutive elements from any element address.
template <int N>
__device__ __forceinline__ void load_n(const uint16_t* p, float v[N])
{
    if constexpr (N == 8) {
        const u32x4_u b = *reinterpret_cast<const u32x4_u*>(p);
        v[0] = bf16_lo(b.x); v[1] = bf16_hi(b.x);
        v[2] = bf16_lo(b.y); v[3] = bf16_hi(b.y);
        v[4] = bf16_lo(b.z); v[5] = bf16_hi(b.z);
        v[6] = bf16_lo(b.w); v[7] = bf16_hi(b.w);
    } else {
        const u32x2_u b = *reinterpret_cast<const u32x2_u*>(p);
        v[0] = bf16_lo(b.x); v[1] = bf16_hi(b.x);
        v[2] = bf16_lo(b.y); v[3] = bf16_hi(b.y);
    }
}
template <int N>
__device__ __forceinline__ void load_n(const float* p, float v[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const f32x4_u b = *reinterpret_cast<const f32x4_u*>(p + i);
        v[i] = b.x; v[i + 1] = b.y; v[i + 2] = b.z; v[i + 3] = b.w;
    }
}
template <int N>
__device__ __forceinline__ void store_n(uint16_t* p, const float v[N])
{
    if constexpr (N == 8)
        *reinterpret_cast<u32x4_u*>(p) = u32x4_u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                 pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
    else
        *reinterpret_cast<u32x2_u*>(p) = u32x2_u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}
template <int N>
__device__ __forceinline__ void store_n(float* p, const float v[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 4)
        *reinterpret_cast<f32x4_u*>(p + i) = f32x4_u{v[i], v[i + 1], v[i + 2], v[i + 3]};
}

// The same past the caches' reuse: rows that are not read again soon.
template <int N>
__device__ __forceinline__ void store_nt(uint16_t* p, const float v[N])
{
    if constexpr (N == 8)
        __builtin_nontemporal_store(u32x4_u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])},
                                    reinterpret_cast<u32x4_u*>(p));
    else
        __builtin_nontemporal_store(u32x2_u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])},
                                    reinterpret_cast<u32x2_u*>(p));
}
template <int N>
__device__ __forceinline__ void store_nt(float* p, const float v[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 4)
        __builtin_nontemporal_store(f32x4_u{v[i], v[i + 1], v[i + 2], v[i + 3]},
                                    reinterpret_cast<f32x4_u*>(p + i));
}

// 16 bytes of elements as loaded: bf16 stays packed until it is used.
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
    static constexpr int N = 8;
    using M = u32x4_u;  // in memory
    using V = u32x4;    // in registers
    static __device__ __forceinline__ V lowest()    // -Inf in every place
    {
        constexpr uint32_t x = 0xFF80FF80u;
        return V{x, x, x, x};
    }
    static __device__ __forceinline__ V first(const uint16_t* p, int n)
    {
        const auto at = [&](int i) { return i < n ? static_cast<uint32_t>(p[i]) : 0u; };
        return V{at(0) | at(1) << 16, at(2) | at(3) << 16, at(4) | at(5) << 16,
                 at(6) | at(7) << 16};
    }
    static __device__ __forceinline__ void widen(V b, float v[8])
    {
        v[0] = bf16_lo(b.x); v[1] = bf16_hi(b.x);
        v[2] = bf16_lo(b.y); v[3] = bf16_hi(b.y);
        v[4] = bf16_lo(b.z); v[5] = bf16_hi(b.z);
        v[6] = bf16_lo(b.w); v[7] = bf16_hi(b.w);
    }
    static __device__ __forceinline__ V pack(const float v[8])
    {
        return V{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                 pack_bf16x2(v[6], v[7])};
    }
};
template <>
struct Raw<float> {
    static constexpr int N = 4;
    using M = f32x4_u;
    using V = f32x4;
    static __device__ __forceinline__ V lowest()
    {
        return V{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    }
    static __device__ __forceinline__ V first(const float* p, int n)
    {
        const auto at = [&](int i) { return i < n ? p[i] : 0.0f; };
        return V{at(0), at(1), at(2), at(3)};
    }
    static __device__ __forceinline__ void widen(V b, float v[4])
    {
        v[0] = b.x; v[1] = b.y; v[2] = b.z; v[3] = b.w;
    }
    static __device__ __forceinline__ V pack(const float v[4]) { return V{v[0], v[1], v[2], v[3]}; }
};
// All of a vector (past the caches' reuse), or its first n elements and 0.
template <typename T>
__device__ __forceinline__ typename Raw<T>::V load_raw(const T* p, int n)
{
    return n == Raw<T>::N
               ? __builtin_nontemporal_load(reinterpret_cast<const typename Raw<T>::M*>(p))
               : Raw<T>::first(p, n);
}

// Subtracting in 64 bits without a sign: an id below first gives a number
// above every row count.
__device__ __forceinline__ uint64_t row_of_id(int64_t id, int64_t first)
{
    return static_cast<uint64_t>(id) - static_cast<uint64_t>(first);
}

__device__ __forceinline__ int64_t read_id(const void* ids, int id64, int64_t i)
{
    return id64 ? static_cast<const int64_t*>(ids)[i]
                : static_cast<int64_t>(static_cast<const int32_t*>(ids)[i]);
}

// A value all lanes of the wave hold, in a scalar register.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ uint64_t uniform(uint64_t x)
{
    const uint64_t lo = static_cast<uint32_t>(uniform(static_cast<int>(x)));
    const uint64_t hi = static_cast<uint32_t>(uniform(static_cast<int>(x >> 32)));
    return hi << 32 | lo;
}

// ---- embedding lookup -------------------------------------------------------------

// Where the vector of N columns that would begin at c lies: the last one ends
// with the row and repeats columns of the one before it, where a vector's worth
// of the row's end element by element is a wave's slowest lane (16384 tokens of
// 771 bf16: the gradient 44 us, 60 with elements; 32768: the lookup 15, 18).
template <int N>
__device__ __forceinline__ int64_t in_row(int64_t c, int64_t dim)
{
    return c + N <= dim || dim < N ? c : dim - N;
}

constexpr int kEmbedThreads = 256;
constexpr int64_t kClearBytes = 16384;

// Lanes (a power of two, as a shift) that share one row of `dim` elements at
// n a lane, `most` at most.
int lane_shift(int64_t dim, int n, int most)
{
    int s = 0;
    while (s < most && (int64_t(n) << s) < dim) ++s;
    return s;
}

// 1 << shift lanes take one token; a block takes 256 >> shift.  A lane has
// TURNS loads under way (a row of 4096 bf16 is two turns of a block).  Bound
// by HBM: 16384 tokens of 4096 bf16 in 31.7 us, 5.9 TB/s (41 us with one load
// under way and plain stores).
template <typename TT, typename AT, int N, int TURNS>
__global__ void __launch_bounds__(kEmbedThreads)
    k_embed_lookup(EmbedArgs a, int shift, int64_t b0)
{
    const int64_t t = ((b0 + blockIdx.x) << (8 - shift)) + (threadIdx.x >> shift);
    if (t >= a.tokens) return;
    const int64_t step = static_cast<int64_t>(N) << shift;
    const uint64_t row = row_of_id(read_id(a.ids, a.id64, t), a.first_row);
    const bool here = row < static_cast<uint64_t>(a.rows);
    const TT* src = static_cast<const TT*>(a.src) + (here ? row * a.table_pitch : 0);
    AT* dst = static_cast<AT*>(a.dst) + t * a.act_pitch;
    for (int64_t c0 = static_cast<int64_t>(threadIdx.x & ((1 << shift) - 1)) * N; c0 < a.dim;
         c0 += step * TURNS) {
        float v[TURNS][N];
#pragma unroll
        for (int u = 0; u < TURNS; ++u) {
            const int64_t c = in_row<N>(c0 + u * step, a.dim);
            if (here && c0 + u * step < a.dim && c + N <= a.dim) {
                load_n<N>(src + c, v[u]);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) v[u][i] = 0.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < TURNS; ++u) {
            if (c0 + u * step >= a.dim) continue;
            const int64_t c = in_row<N>(c0 + u * step, a.dim);
            if (c + N <= a.dim) {
                if (here) {
#pragma unroll
                    for (int i = 0; i < N; ++i) v[u][i] *= a.scale;
                }
                store_nt<N>(dst + c, v[u]);
            } else {
                for (int64_t i = c; i < a.dim; ++i)
                    put(dst + i, here ? widen(src[i]) * a.scale : 0.0f);
            }
        }
    }
}

// ---- embedding gradient: sort -----------------------------------------------------

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kSortRowBits = 9;     // kSortRows rows
static_assert((1 << kSortRowBits) == kSortRows && ZS_EMBED_MAX / kSortWaves <= (1 << 20),
              "a token of a wave's part and a row of a bucket fit one entry");
// LDS of the sort: the 16 waves' counts, and what is left of 63 KB as their
// lists (at least 128 entries each, the queue of a second reading).
constexpr int kSortLds = 63 * 1024;
__host__ __device__ constexpr int sort_list(int rows)
{
    return (kSortLds / 4 - kSortWaves * rows) / kSortWaves;
}
static_assert(sort_list(kSortRows) >= 2 * kWave, "a queue of 64 and what comes on top");
constexpr int kSortLoads = 8;       // ids a lane has under way

// Rows are dealt to buckets in turn (bucket = row mod buckets), because the
// rows of small numbers tend to have most of the tokens.  The sorted order is
// by bucket, then by row; a row's slot is its place in it.
__device__ __forceinline__ int64_t sort_slot(const SortShape& s, int64_t row)
{
    return (row & ((int64_t(1) << s.bucket_bits) - 1)) * s.rows + (row >> s.bucket_bits);
}

// Lanes of the wave whose row equals this lane's, among those with `in`
// set (0 bits elsewhere): the intersection over the row's bits of the lanes
// that agree in that bit.
__device__ __forceinline__ uint64_t same_row(bool in, int row, int bits)
{
    uint64_t m = __ballot(in);
    for (int b = 0; b < bits; ++b) {
        const bool bit = (row >> b) & 1;
        const uint64_t set = __ballot(bit);
        m &= bit ? set : ~set;
    }
    return m;
}

// A stable counting sort of the tokens by slot, one block per bucket and no
// exchange between blocks: every block reads all ids (a batch of ids is small
// and comes from L2 after the first block), counts the tokens of earlier
// buckets (where its own part of the order begins) and of each of its rows,
// and then places its tokens.  Each wave takes one contiguous part of the
// tokens and lists those of the bucket, few of each 64, which are then
// handled 64 at a time.  A token's place is: its row's start, the tokens of
// that row in earlier waves, those handled earlier by its wave, and those in
// lower lanes (4096 tokens 7 us, 65536 23 us, 40 with a wait behind each
// load: every CU looks at every id, some 20 instructions for 64).  Where a
// wave's list is too short for its tokens (one id in most of them), all waves
// read the ids again and handle 64 whenever they have them, once to count and
// once to place.  Half of 65536 tokens with one id do that, as do 131072 with
// ids that fall as 1/v: the gradient of 128256 rows of 64 in bf16 takes 129 and
// 121 us then, 54 for 65536 such tokens without.
template <typename ID>
__global__ void __launch_bounds__(kSortThreads)
    k_embed_sort(EmbedArgs a, SortShape s, int32_t* order, int32_t* row_of, int32_t* starts)
{
    // per wave: its count of each row, then its list
    extern __shared__ __align__(16) int32_t sort_lds[];
    __shared__ int32_t wave_sum[kSortWaves];
    __shared__ int32_t wave_below[kSortWaves];
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    const uint32_t bucket = blockIdx.x, low = (1u << s.bucket_bits) - 1;
    const int tokens = static_cast<int>(a.tokens);
    constexpr int kSpan = kSortLoads * kWave;
    // tokens of one wave, a multiple of 64
    const int part = (tokens + kSortThreads - 1) / kSortThreads * kWave;
    const int t0 = wave * part, t1 = t0 + part < tokens ? t0 + part : tokens;
    const uint64_t lower = (uint64_t(1) << lane) - 1;
    const int room = sort_list(s.rows);
    int32_t* hist = sort_lds + wave * s.rows;
    const ID* ids = static_cast<const ID*>(a.ids);
    // entries (token - t0) << kSortRowBits | row in the bucket: 20 + 9 bits
    uint32_t* list =
        reinterpret_cast<uint32_t*>(sort_lds) + kSortWaves * s.rows + wave * room;
    for (int r = lane; r < s.rows; r += kWave) hist[r] = 0;

    // found(token, row, its bucket): 64 tokens; those without a row here are
    // of no bucket (UINT32_MAX)
    const auto read_ids = [&](auto found) {
        for (int base = t0; base < t1; base += kSpan) {
            // all loads first, without a branch between them
            ID id[kSortLoads];
#pragma unroll
            for (int u = 0; u < kSortLoads; ++u) {
                const int t = base + u * kWave + lane;
                id[u] = ids[t < t1 ? t : t1 - 1];
            }
#pragma unroll
            for (int u = 0; u < kSortLoads; ++u) {
                const int t = base + u * kWave + lane;
                const uint64_t r = row_of_id(id[u], a.first_row);
                const bool here = r < static_cast<uint64_t>(a.rows) && t < t1;
                const uint32_t row = static_cast<uint32_t>(r);
                found(t, row, here ? row & low : UINT32_MAX);
            }
        }
    };
    const auto entry = [&](int t, uint32_t row) {
        return static_cast<uint32_t>(t - t0) << kSortRowBits | row >> s.bucket_bits;
    };
    // count(e, in), place(e, in): one listed token a lane
    const auto count = [&](uint32_t e, bool in) {
        const int r = e & ((1 << kSortRowBits) - 1);
        const uint64_t same = same_row(in, r, s.row_bits);
        if (in && (same & lower) == 0) hist[r] += __popcll(same);
        __builtin_amdgcn_wave_barrier();
    };
    const auto place = [&](uint32_t e, bool in) {
        const int r = e & ((1 << kSortRowBits) - 1);
        const uint64_t same = same_row(in, r, s.row_bits);
        int first = 0;
        if (in) first = hist[r];
        // every lane has read before the first lane of each row adds
        __builtin_amdgcn_wave_barrier();
        if (in) {
            const int before = __popcll(same & lower);
            if (before == 0) hist[r] = first + __popcll(same);
            order[first + before] = t0 + static_cast<int>(e >> kSortRowBits);
            row_of[first + before] = r << s.bucket_bits | static_cast<int32_t>(bucket);
        }
        __builtin_amdgcn_wave_barrier();
    };
    // the listed tokens, or all of the bucket's by way of a queue of 64
    const auto from_list = [&](int n, auto handle) {
        for (int i = 0; i < n; i += kWave) {
            const bool in = i + lane < n;
            handle(in ? list[i + lane] : 0, in);
        }
    };
    const auto from_ids = [&](auto handle) {
        int queued = 0;
        read_ids([&](int t, uint32_t row, uint32_t of) {
            const bool in = of == bucket;
            const uint64_t mask = __ballot(in);
            if (mask == 0) return;
            if (in) list[queued + __popcll(mask & lower)] = entry(t, row);
            queued += __popcll(mask);
            __builtin_amdgcn_wave_barrier();
            if (queued < kWave) return;
            handle(list[lane], true);
            queued -= kWave;
            const uint32_t rest = list[kWave + lane];
            __builtin_amdgcn_wave_barrier();
            if (lane < queued) list[lane] = rest;
            __builtin_amdgcn_wave_barrier();
        });
        if (queued > 0) handle(list[lane], lane < queued);
    };

    int below = 0, n = 0;
    read_ids([&](int t, uint32_t row, uint32_t of) {
        const bool in = of == bucket;
        below += of < bucket;
        const uint64_t mask = __ballot(in);
        if (mask == 0) return;
        const int at = n + __popcll(mask & lower);
        if (in && at < room) list[at] = entry(t, row);
        n += __popcll(mask);
    });
    for (int o = kWave / 2; o > 0; o >>= 1) below += __shfl_xor(below, o);
    if (lane == 0) wave_below[wave] = below;
    const bool listed = __syncthreads_or(n > room) == 0;
    if (listed) from_list(n, count);
    else from_ids(count);
    __syncthreads();

    // per row: the tokens of earlier waves, and the row's start
    int total = 0;
    if (tid < s.rows) {
        int in_wave[kSortWaves];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) in_wave[w] = sort_lds[w * s.rows + tid];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            sort_lds[w * s.rows + tid] = total;
            total += in_wave[w];
        }
    }
    int incl = total;
    for (int o = 1; o < kWave; o <<= 1) {
        const int v = __shfl_up(incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == kWave - 1) wave_sum[wave] = incl;
    __syncthreads();
    int start = incl - total;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
        start += wave_below[w];
        if (w < wave) start += wave_sum[w];
    }
    if (tid < s.rows) {
        starts[bucket * s.rows + tid] = start;
        if (bucket == low && tid == s.rows - 1) starts[(low + 1) * s.rows] = start + total;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) sort_lds[w * s.rows + tid] += start;
    }
    __syncthreads();
    if (listed) from_list(n, place);
    else from_ids(place);
}

// ---- embedding gradient: sums -------------------------------------------------------

struct SumPlan {
    const int32_t* order;
    const int32_t* row_of;
    const int32_t* starts;  // first sorted position of each slot, and behind
                            // the last slot, at `count`, the tokens sorted
    const int32_t* count;
    SortShape sort;
    float* partials;        // [chunks][2][dim]: a run that began before the
                            // chunk, a run that goes on behind it
    int64_t chunks;
    int64_t splits;         // column parts of a row
    int64_t sum_blocks;     // blocks that sum; the rest clear empty rows
    int32_t chunk;          // sorted positions of a chunk
    int32_t zero_shift;     // log2 of the lanes that clear one row
    int32_t zero_rows;      // rows a block looks through, at most 64
};

// The gradient row's values at columns c.. but the first `skip`, for ADD.
template <typename GT, int N>
__device__ __forceinline__ void read_row(const EmbedArgs& a, int64_t row, int64_t c, float old[N],
                                         int skip = 0)
{
    const GT* g = static_cast<const GT*>(a.dst) + row * a.table_pitch + c;
    if (c + N <= a.dim && skip == 0) {
        load_n<N>(g, old);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            old[i] = i >= skip && c + i < a.dim ? widen(g[i]) : 0.0f;
    }
}

// scale * acc into the gradient row (with ADD: on top of what it held).
template <typename GT, int N, bool ADD>
__device__ __forceinline__ void put_row(const EmbedArgs& a, int64_t row, int64_t c,
                                        const float acc[N], const float old[N], int skip = 0)
{
    GT* g = static_cast<GT*>(a.dst) + row * a.table_pitch + c;
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = ADD ? old[i] + a.scale * acc[i] : a.scale * acc[i];
    if (c + N <= a.dim && skip == 0) {
        store_nt<N>(g, v);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i >= skip && c + i < a.dim) put(g + i, v[i]);
    }
}

template <int N>
__device__ __forceinline__ void put_partial(float* p, int64_t c, int64_t dim, const float acc[N])
{
    if (c + N <= dim) {
        store_n<N>(p + c, acc);
    } else {
        for (int i = 0; i < N; ++i)
            if (c + i < dim) p[c + i] = acc[i];
    }
}

// One block: +0 into those of zero_rows consecutive rows from r0 whose bit in
// `mask` is set (plain stores: 2.1 GB and its sums in 375 us, against 398 with
// nt ones).
template <typename GT>
__device__ __forceinline__ void clear_rows(const EmbedArgs& a, const SumPlan& p, int64_t r0,
                                           uint64_t mask)
{
    constexpr int N = 16 / sizeof(GT);
    const int lanes = 1 << p.zero_shift;
    const float z[N] = {};
    for (int i = threadIdx.x >> p.zero_shift; i < p.zero_rows; i += kEmbedThreads >> p.zero_shift) {
        if (!(mask >> i & 1)) continue;
        GT* g = static_cast<GT*>(a.dst) + (r0 + i) * a.table_pitch;
        for (int64_t c = static_cast<int64_t>(threadIdx.x & (lanes - 1)) * N; c < a.dim;
             c += static_cast<int64_t>(lanes) * N) {
            if (a.dim >= N) {
                store_n<N>(g + in_row<N>(c, a.dim), z);
            } else {
                for (int64_t j = c; j < a.dim; ++j) put(g + j, 0.0f);
            }
        }
    }
}

constexpr int kSumUnroll = 8;

// One wave sums one chunk of sorted positions over one part of the columns:
// equal work a wave whatever the ids, where a wave a row would leave the most
// frequent token to one wave.  What bounds it is HBM (65536 x 4096 bf16 into
// 128256 rows: 1.55 GB and 33 MB of partials in 269 us, 5.9 TB/s).
// Its lanes hold the chunk's tokens and rows, one position a lane, which the
// walk takes into scalar registers one by one: kSumUnroll loads in flight, and
// a run's sum handed on where the run ends or the chunk does.
template <typename AT, typename GT, int N, bool ADD>
__global__ void __launch_bounds__(kEmbedThreads)
    k_embed_sum(EmbedArgs a, SumPlan p, int64_t b0)
{
    const int64_t block = b0 + blockIdx.x;
    if (!ADD && block >= p.sum_blocks) {
        const int64_t r0 = (block - p.sum_blocks) * p.zero_rows;
        const int64_t r = r0 + threadIdx.x % kWave;
        bool empty = false;
        if (r < r0 + p.zero_rows && r < a.rows) {
            const int32_t* s = p.starts + sort_slot(p.sort, r);
            empty = s[0] == s[1];
        }
        clear_rows<GT>(a, p, r0, __ballot(empty));
        return;
    }
    constexpr int UNROLL = ADD ? kSumUnroll / 2 : kSumUnroll;
    const int wave = uniform(static_cast<int>(threadIdx.x / kWave)), lane = threadIdx.x % kWave;
    const int64_t worker = block * (kEmbedThreads / kWave) + wave;
    const int64_t chunk = worker / p.splits;
    const int64_t c = ((worker - chunk * p.splits) * kWave + lane) * N;
    const int64_t first = chunk * p.chunk;
    if (first >= a.tokens) return;
    // Position p0 + lane (the chunk has at most 64), the row behind it and the
    // one before the chunk, loaded beside the count of sorted positions: what
    // lies behind that count is not used.
    const int p0 = static_cast<int>(first), tokens = static_cast<int>(a.tokens);
    const int at0 = p0 + lane < tokens ? p0 + lane : tokens - 1;
    const int token = p.order[at0], row = p.row_of[at0];
    int row_next = p.row_of[at0 + 1 < tokens ? at0 + 1 : at0];
    const int row_before = p.row_of[p0 > 0 ? p0 - 1 : 0];
    const int n = *p.count;
    if (p0 >= n) return;
    const int len = p0 + p.chunk < n ? p.chunk : n - p0;
    if (at0 + 1 >= n) row_next = -1;
    // whether the run under way began in this chunk
    bool began = p0 == 0 || row_before != uniform(row);
    // Lanes behind the last column stay (the others read their token and row):
    // they load the first columns again and store nothing.
    const int64_t col = c < a.dim ? in_row<N>(c, a.dim) : 0;
    const AT* src = static_cast<const AT*>(a.src) + col;
    const int width = a.dim < N ? static_cast<int>(a.dim) : N;
    // A column that two lanes sum is stored by both, with the same bits, but
    // read and added to by one alone.
    const int skip = ADD && c < a.dim ? static_cast<int>(c - col) : 0;
    float* partial = p.partials + chunk * 2 * a.dim;
    float acc[N] = {};
    for (int q = 0; q < len; q += UNROLL) {
        typename Raw<AT>::V x[UNROLL];
        float old[ADD ? UNROLL : 1][N];
        const auto at = [&](int u) { return q + u < len ? q + u : len - 1; };
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            x[u] = load_raw(src + __builtin_amdgcn_readlane(token, at(u)) * a.act_pitch, width);
        }
        if constexpr (ADD) {
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int r = __builtin_amdgcn_readlane(row, at(u));
                if (q + u < len && __builtin_amdgcn_readlane(row_next, at(u)) != r)
                    read_row<GT, N>(a, r, col, old[u], skip);
            }
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if (q + u >= len) continue;
            float v[N];
            Raw<AT>::widen(x[u], v);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] += v[i];
            const int r = __builtin_amdgcn_readlane(row, at(u));
            const bool ends = __builtin_amdgcn_readlane(row_next, at(u)) != r;
            if (!ends && q + u + 1 < len) continue;
            if (c < a.dim) {
                if (!began) put_partial<N>(partial, col, a.dim, acc);
                else if (ends) put_row<GT, N, ADD>(a, r, col, acc, old[ADD ? u : 0], skip);
                else put_partial<N>(partial + a.dim, col, a.dim, acc);
            }
            began = true;
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = 0.0f;
        }
    }
}

// Up to 64 tokens: one launch, no sort (37 tokens of 768: 3.1 us, where sort,
// sums and join take 12).  Every wave has all of their rows, one a lane; a
// wave takes one token and one part of the columns, and if no earlier token
// has its row, sums the tokens that have it, in order.
template <typename AT, typename GT, int N, bool ADD>
__global__ void __launch_bounds__(kEmbedThreads)
    k_embed_few(EmbedArgs a, SumPlan p, int64_t b0)
{
    const int64_t block = b0 + blockIdx.x;
    const int wave = uniform(static_cast<int>(threadIdx.x / kWave)), lane = threadIdx.x % kWave;
    uint64_t id = UINT64_MAX;
    if (lane < a.tokens) id = row_of_id(read_id(a.ids, a.id64, lane), a.first_row);
    // rows are fewer than 2^24
    const int row = id < static_cast<uint64_t>(a.rows) ? static_cast<int>(id) : -1;
    if (!ADD && block >= p.sum_blocks) {
        const int64_t r0 = (block - p.sum_blocks) * p.zero_rows;
        const int64_t rest = a.rows - r0 < p.zero_rows ? a.rows - r0 : p.zero_rows;
        uint64_t mask = rest == 64 ? ~uint64_t(0) : (uint64_t(1) << rest) - 1;
        for (uint64_t m = __ballot(row >= r0 && row < r0 + rest); m; m &= m - 1)
            mask &= ~(uint64_t(1) << (__builtin_amdgcn_readlane(row, __builtin_ctzll(m)) - r0));
        clear_rows<GT>(a, p, r0, mask);
        return;
    }
    const int64_t worker = block * (kEmbedThreads / kWave) + wave;
    const int token = static_cast<int>(worker / p.splits);
    const int64_t c = ((worker - token * p.splits) * kWave + lane) * N;
    if (token >= a.tokens) return;
    const int r = __builtin_amdgcn_readlane(row, token);
    uint64_t same = __ballot(row == r);
    if (r < 0 || __builtin_ctzll(same) != token || c >= a.dim) return;
    const AT* src = static_cast<const AT*>(a.src) + c;
    const int width = c + N <= a.dim ? N : static_cast<int>(a.dim - c);
    float acc[N] = {}, old[N] = {};
    if constexpr (ADD) read_row<GT, N>(a, r, c, old);
    while (same) {
        typename Raw<AT>::V x[kSumUnroll] = {};
        uint64_t m = same;
#pragma unroll
        for (int u = 0; u < kSumUnroll; ++u) {
            if (m == 0) continue;
            x[u] = load_raw(src + __builtin_ctzll(m) * a.act_pitch, width);
            m &= m - 1;
        }
#pragma unroll
        for (int u = 0; u < kSumUnroll; ++u) {
            if (same == 0) continue;
            float v[N];
            Raw<AT>::widen(x[u], v);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] += v[i];
            same &= same - 1;
        }
    }
    put_row<GT, N, ADD>(a, r, c, acc, old);
}

// The runs that cross chunks (at 65536 tokens 11 us, most of it blocks that
// find none): the block of the chunk a run begins in adds its partials in
// order, each wave a contiguous part of them.  So the longest run is one
// block's work for its columns: with it, 65536 tokens of 4096 bf16 that all
// have one id take 459 us, 340 with ids that fall as 1/v.
template <typename GT, int N, bool ADD>
__global__ void __launch_bounds__(kEmbedThreads)
    k_embed_join(EmbedArgs a, SumPlan p, int64_t b0)
{
    __shared__ float sums[kEmbedThreads * N];
    const int64_t block = b0 + blockIdx.x;
    const int64_t chunk = block / p.splits;
    const int64_t p0 = chunk * p.chunk, p1 = p0 + p.chunk;
    if (p1 >= a.tokens) return;
    const int32_t row = p.row_of[p1], row_before = p.row_of[p1 - 1];
    if (p1 >= *p.count || row_before != row) return;        // no run crosses here
    const int32_t* span = p.starts + sort_slot(p.sort, row);
    if (span[0] < p0) return;                               // it begins in an earlier chunk
    const int64_t count = (span[1] - 1) / p.chunk - chunk + 1;
    constexpr int lanes = kWave, groups = kEmbedThreads / kWave;
    const int group = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int64_t c = ((block - chunk * p.splits) * lanes + lane) * N;
    float acc[N] = {}, old[N] = {};
    if (c < a.dim) {
        if (ADD && group == 0) read_row<GT, N>(a, row, c, old);
        const int64_t i0 = group * count / groups, i1 = (group + 1) * count / groups;
#pragma unroll 4
        for (int64_t i = i0; i < i1; ++i) {
            const float* s = p.partials + ((chunk + i) * 2 + (i == 0 ? 1 : 0)) * a.dim + c;
            float x[N];
            if (c + N <= a.dim) {
                load_n<N>(s, x);
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j) x[j] = c + j < a.dim ? s[j] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += x[j];
        }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) sums[threadIdx.x * N + j] = acc[j];
    __syncthreads();
    if (group != 0 || c >= a.dim) return;
    for (int g = 1; g < groups; ++g)
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] += sums[(g * lanes + lane) * N + j];
    put_row<GT, N, ADD>(a, row, c, acc, old);
}

// ---- distillation -------------------------------------------------------------------
//
// One row is one softmax (two with labels at another temperature) over the
// vocabulary plus K entries to look at.  The logits are what costs: HBM moves
// them, and each takes about six vector instructions and an exponential (four
// issue slots) in each of the two passes, together half the time the bytes
// take (8192 x 128256 bf16: without the exponentials 709 us, with them 726 to
// 740):
//  - exponentials are the hardware's base-2 one (1 ulp), their arguments one
//    fma each (see kFmaLimit), exact where the value is large;
//  - logits and gradients pass the caches (nt: the loss of 2048 x 50257 fp32
//    behind another kernel's stores took 75 us, with plain loads and stores
//    113), labels come through the scalar cache, and the teacher's entries
//    are a side job while a row's loads are under way.

constexpr int kWaves(int threads) { return threads / kWave; }

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ float wave_sum(float x)
{
    for (int o = kWave / 2; o > 0; o >>= 1) x += __shfl_xor(x, o);
    return x;
}
__device__ __forceinline__ float wave_max(float x)
{
    for (int o = kWave / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor(x, o));
    return x;
}

// Statistics of a softmax: the maximum and the sums of exp((s - m)/tau) and
// (CE) exp(s - m).  The maximum starts at the lowest finite value, so that
// -Inf logits have weight 0 and no Inf - Inf occurs.
struct Stat {
    float m, a, b;
};

// At tau = 1 both sums are one: SAME takes the exponentials once.
enum Terms { kKd = 0, kKdCe = 1, kSame = 2 };

template <Terms TM>
__device__ __forceinline__ void rescale(Stat& s, float m, float c)
{
    s.a *= exp2_hw((s.m - m) * c);
    if constexpr (TM == kKdCe) s.b *= exp2_hw((s.m - m) * kLog2e);
    s.m = m;
}

template <Terms TM>
__device__ __forceinline__ void join(Stat& s, Stat o, float c)
{
    const float m = fmaxf(s.m, o.m);
    rescale<TM>(s, m, c);
    rescale<TM>(o, m, c);
    s.a += o.a;
    if constexpr (TM == kKdCe) s.b += o.b;
}

// Over groups of `lanes` lanes (a power of two); all lanes get the result.
template <Terms TM>
__device__ __forceinline__ Stat lanes_join(Stat s, float c, int lanes)
{
    for (int o = lanes / 2; o > 0; o >>= 1) {
        Stat t;
        t.m = __shfl_xor(s.m, o);
        t.a = __shfl_xor(s.a, o);
        t.b = TM == kKdCe ? __shfl_xor(s.b, o) : 0.0f;
        join<TM>(s, t, c);
    }
    return s;
}

// Over the block, with its one barrier.
template <Terms TM, int THREADS>
__device__ __forceinline__ Stat block_join(Stat s, float c, float* red)
{
    s = lanes_join<TM>(s, c, kWave);
    const int lane = threadIdx.x % kWave;
    if (lane == 0) {
        float* r = red + threadIdx.x / kWave * 3;
        r[0] = s.m;
        r[1] = s.a;
        r[2] = s.b;
    }
    __syncthreads();
    const float* r = red + lane % kWaves(THREADS) * 3;
    s = lanes_join<TM>(Stat{r[0], r[1], r[2]}, c, kWaves(THREADS));
    if constexpr (TM == kSame) s.b = s.a;
    return s;
}

template <int N>
__device__ __forceinline__ float max_n(const float x[N], float m)
{
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, x[i]);
    return m;
}

// exp((x - m)/tau) of N elements, added to s.
template <Terms TM, int N>
__device__ __forceinline__ void add_exp(Stat& s, const float x[N], float c)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float d = x[i] - s.m;
        s.a += exp2_hw(d * c);
        if constexpr (TM == kKdCe) s.b += exp2_hw(d * kLog2e);
    }
}

// Vector v of the nv at a scalar address (held opaque, so that it stays one)
// and one 32-bit offset; beyond the last: the last, whose value is not used.
template <typename T>
__device__ __forceinline__ typename Raw<T>::V held_vector(uint64_t base, int v, int nv)
{
    v = v < nv ? v : nv - 1;
    using P = const __attribute__((address_space(1))) typename Raw<T>::M*;
    asm("" : "+s"(base));
    return __builtin_nontemporal_load((P)(base + static_cast<uint32_t>(v) * 16u));
}

template <typename T>
__device__ __forceinline__ void put_held(uint64_t base, int v, const float x[Raw<T>::N])
{
    using P = __attribute__((address_space(1))) typename Raw<T>::M*;
    asm("" : "+s"(base));
    const typename Raw<T>::M m = Raw<T>::pack(x);
    __builtin_nontemporal_store(m, (P)(base + static_cast<uint32_t>(v) * 16u));
}

// Keeps what was computed from v before out of what is computed after: the
// widened elements of a whole row would not fit the registers.
template <typename V>
__device__ __forceinline__ void forget(V& v)
{
    asm("" : "+v"(v));
}

// Below this |m c| an exponent may be taken as fma(x, c, -r), r = m c rounded:
// one instruction for two, and exact but for its own rounding and for what r
// was rounded by, at most 2^-8, which `rounded_by` gives back as a factor.
// Beyond it (and for a row of -Inf alone) the difference is taken first.
constexpr float kFmaLimit = 65536.0f;

__device__ __forceinline__ bool fma_range(float m, float c) { return fabsf(m * c) <= kFmaLimit; }
__device__ __forceinline__ float rounded_by(float m, float c)
{
    return exp2_hw(-__builtin_fmaf(m, c, -(m * c)));
}

// The statistics of the vectors raw[0..HOLD) of each thread, of which `own`
// are real: the maximum, and the sums where every |m c| allows the fma form
// (otherwise false is returned, for all lanes of the wave).
template <typename T, Terms TM, int HOLD, typename Own>
__device__ __forceinline__ bool held_stats(typename Raw<T>::V (&raw)[HOLD], Own own, float c,
                                           Stat& st)
{
    constexpr int N = Raw<T>::N;
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < HOLD; ++j) {
        if (!own(j)) raw[j] = Raw<T>::lowest();
        float x[N];
        Raw<T>::widen(raw[j], x);
        m = max_n<N>(x, m);
    }
    const bool none = m == -INFINITY;
    const float ref = none ? 0.0f : m;
    if (!__all(fma_range(ref, c) && (TM != kKdCe || fma_range(ref, kLog2e)))) return false;
    const float r = ref * c, r1 = ref * kLog2e;
    float a = 0.0f, b = 0.0f;
#pragma unroll
    for (int j = 0; j < HOLD; ++j) {
        float x[N];
        forget(raw[j]);
        Raw<T>::widen(raw[j], x);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            a += exp2_hw(__builtin_fmaf(x[i], c, -r));
            if constexpr (TM == kKdCe) b += exp2_hw(__builtin_fmaf(x[i], kLog2e, -r1));
        }
    }
    st.m = none ? kLowest : m;
    st.a = none ? a : a * rounded_by(ref, c);
    st.b = TM == kKdCe && !none ? b * rounded_by(ref, kLog2e) : b;
    return true;
}

// Elements of a row before its first 16-byte boundary, where its vectors
// begin: a bf16 row of odd length read from its start would take every vector
// across a boundary (5341 x 50257: 217 us, 248 from the start).
template <typename T>
__device__ __forceinline__ int row_head(const T* row, int64_t vocab)
{
    const int n = static_cast<int>((16 - (reinterpret_cast<uint64_t>(row) & 15)) & 15) /
                  static_cast<int>(sizeof(T));
    return static_cast<int>(n < vocab ? n : vocab);
}

// The statistics of a row's columns [0, head) and of its vectors from c0 to
// c1 and the elements behind them, over the block's threads, in one pass with
// the running maximum, BATCH loads under way.
template <typename T, Terms TM, int THREADS, int BATCH>
__device__ __forceinline__ Stat scan(Stat s, const T* row, int head, int64_t c0, int64_t c1,
                                     float c)
{
    constexpr int N = Raw<T>::N;
    const int nv = static_cast<int>((c1 - c0) / N);
    const typename Raw<T>::M* p = reinterpret_cast<const typename Raw<T>::M*>(row + c0);
    for (int v0 = threadIdx.x; v0 - static_cast<int>(threadIdx.x) < nv; v0 += BATCH * THREADS) {
        typename Raw<T>::V raw[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
            raw[j] = p[v0 + j * THREADS < nv ? v0 + j * THREADS : nv - 1];
        float m = s.m;
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            if (v0 + j * THREADS >= nv) raw[j] = Raw<T>::lowest();
            float x[N];
            Raw<T>::widen(raw[j], x);
            m = max_n<N>(x, m);
        }
        if (m > s.m) rescale<TM>(s, m, c);
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            float x[N];
            forget(raw[j]);
            Raw<T>::widen(raw[j], x);
            add_exp<TM, N>(s, x, c);
        }
    }
    const auto one = [&](int64_t col) {
        const float x = widen(row[col]);
        if (x > s.m) rescale<TM>(s, x, c);
        add_exp<TM, 1>(s, &x, c);
    };
    if (static_cast<int>(threadIdx.x) < head) one(threadIdx.x);
    const int64_t e = c0 + static_cast<int64_t>(nv) * N + threadIdx.x;
    if (e < c1) one(e);
    return s;
}

// A row's targets in LDS: entry k's column (-1: no entry), its log p and p,
// and the logit at it; with labels at alpha < 1 the label is entry K.
struct Entries {
    int32_t* col;
    float* logp;
    float* p;
    float* s;
    float* mass;    // sum of p, and behind it 1 if the row counts, else 0
    int32_t* heads; // more than 64 entries: the last entry of each hash of a
    int32_t* next;  // column, and the entry before each with its hash (-1: none)
    int n;          // K, or K + 1 with the label
    int hash_bits;
};

// Up to kWave entries, one wave reads them all and a column's others are
// found by looking through them; more are read by the whole block, and chained
// by a hash of their column.
__device__ __forceinline__ uint32_t entry_hash(const Entries& e, int col)
{
    return static_cast<uint32_t>(col) * 2654435769u >> (32 - e.hash_bits);
}

// Entries a row can hold, a multiple of 4.
__host__ __device__ constexpr int entry_slots(int k) { return (k + 1 + 3) / 4 * 4; }
// log2 of the chains of K > 64 entries: at least K.
__host__ __device__ constexpr int entry_hash_bits(int k)
{
    int b = 7;
    while ((1 << b) < k) ++b;
    return b;
}
size_t entry_bytes(int k)
{
    const size_t chains = k > kWave ? (size_t(1) << entry_hash_bits(k)) + entry_slots(k) : 0;
    return static_cast<size_t>(entry_slots(k)) * 16 + 16 + chains * 4;
}

__device__ __forceinline__ Entries entries_at(char* lds, const DistillArgs& a)
{
    const int slots = entry_slots(a.k);
    Entries e;
    e.col = reinterpret_cast<int32_t*>(lds);
    e.logp = reinterpret_cast<float*>(lds + slots * 4);
    e.p = e.logp + slots;
    e.s = e.p + slots;
    e.mass = e.s + slots;
    e.hash_bits = a.entry_bits;
    e.heads = reinterpret_cast<int32_t*>(e.mass + 4);
    e.next = e.heads + (1 << a.entry_bits);
    e.n = a.k + a.ce;
    return e;
}

__device__ __forceinline__ int read_column(const void* ids, int id64, int64_t i, int64_t vocab)
{
    const int64_t id = read_id(ids, id64, i);
    return id >= 0 && id < vocab ? static_cast<int>(id) : -1;
}

// Entry `at` of the teacher: its column and value.
__device__ __forceinline__ int read_entry(const DistillArgs& a, int64_t at, float* u)
{
    *u = a.teacher_f32 ? static_cast<const float*>(a.teacher_logits)[at]
                       : widen(static_cast<const uint16_t*>(a.teacher_logits)[at]);
    const int col = read_column(a.teacher_ids, a.id64, at, a.vocab);
    return *u == -INFINITY ? -1 : col;
}

// Whether the row's label lets it count (it may still have no entry), and the
// label (0 without labels).  `row` is uniform; the label comes through the
// scalar cache and does not wait for the vector loads under way.
__device__ __forceinline__ bool label_counts(const DistillArgs& a, int64_t row, int* label)
{
    *label = 0;
    if (!a.labels) return true;
    int64_t id;
    if (a.id64) {
        using P = const __attribute__((address_space(4))) int64_t*;
        id = ((P)reinterpret_cast<uint64_t>(a.labels))[row];
    } else {
        using P = const __attribute__((address_space(4))) int32_t*;
        id = ((P)reinterpret_cast<uint64_t>(a.labels))[row];
    }
    *label = static_cast<int>(id);
    return id >= 0 && id < a.vocab;
}

// The row's entries into LDS (u for log p), a part of them a thread (`thread`
// of `threads`), and the logits at those in columns [c0, c1).
template <typename T>
__device__ __forceinline__ void read_entries(const DistillArgs& a, const Entries& e, int64_t row,
                                             int label, const T* s, int64_t c0, int64_t c1,
                                             int thread, int threads)
{
    for (int k = thread; k < entry_slots(a.k); k += threads) {
        int col = -1;
        float u = 0.0f;
        if (k < a.k) {
            col = read_entry(a, row * a.k + k, &u);
        } else if (k == a.k && a.ce) {
            col = label;
        }
        e.col[k] = col;
        e.logp[k] = u;
        if (col >= c0 && col < c1) e.s[k] = widen(s[col]);
        if (a.k > kWave)
            e.next[k] = col < 0 ? -1 : atomicExch(e.heads + entry_hash(e, col), k);
    }
}

// Before read_entries, by the whole block, with a barrier behind it.
template <int THREADS>
__device__ __forceinline__ void clear_chains(const DistillArgs& a, const Entries& e)
{
    if (a.k <= kWave) return;
    for (int i = threadIdx.x; i < 1 << e.hash_bits; i += THREADS) e.heads[i] = -1;
    __syncthreads();
}

// One wave's work once they are there: log p, p and their sum.  The block's
// next barrier publishes them.
__device__ __forceinline__ void weigh_entries(const DistillArgs& a, const Entries& e, int64_t row)
{
    const int lane = threadIdx.x % kWave;
    float top = kLowest, mass = 0.0f;
    bool found = false;
    for (int k = lane; k < a.k; k += kWave) {
        if (e.col[k] < 0) continue;
        top = fmaxf(top, e.logp[k]);
        found = true;
    }
    const bool any = a.ce || __ballot(found) != 0;
    if (a.k > 0) {
        // log p = (u - from)/tau - norm: the difference first, so that no u/tau
        // overflows where the entries are all the whole distribution
        float from = 0.0f, norm;
        if (a.teacher_lse) {
            norm = a.teacher_lse[row];
        } else {
            from = wave_max(top);
            float sum = 0.0f;
            for (int k = lane; k < a.k; k += kWave)
                if (e.col[k] >= 0) sum += expf((e.logp[k] - from) * a.inv_tau);
            norm = logf(wave_sum(sum));
        }
        for (int k = lane; k < a.k; k += kWave) {
            const float logp = (e.logp[k] - from) * a.inv_tau - norm;
            const float p = e.col[k] >= 0 ? expf(logp) : 0.0f;
            e.logp[k] = logp;
            e.p[k] = p;
            mass += p;
        }
        mass = wave_sum(mass);
    }
    if (lane == 0) {
        e.mass[0] = mass;
        e.mass[1] = any ? 1.0f : 0.0f;
    }
}

// Both by one wave, beside the others' loads of the row.
template <typename T>
__device__ __forceinline__ void load_entries(const DistillArgs& a, const Entries& e, int64_t row,
                                             int label, const T* s)
{
    read_entries<T>(a, e, row, label, s, 0, a.vocab, threadIdx.x % kWave, kWave);
    // a lane reads in weigh_entries what it wrote here
    weigh_entries(a, e, row);
}

// Loss, statistics and flag of a row whose label lets it count, by one wave.
__device__ __forceinline__ void put_loss(const DistillArgs& a, const Entries& e, int64_t row,
                                         const Stat& st, const float* logit)
{
    const int lane = threadIdx.x % kWave;
    const float log_a = logf(st.a);
    float loss = 0.0f;
    if (a.kd) {
        for (int k = lane; k < a.k; k += kWave)
            if (e.col[k] >= 0 && e.p[k] != 0.0f)
                loss += e.p[k] * (e.logp[k] - ((logit[k] - st.m) * a.inv_tau - log_a));
        loss = a.loss_kd * wave_sum(loss);
    }
    const float log_b = a.ce ? logf(st.b) : 0.0f;
    if (a.ce) loss += a.loss_ce * (log_b - (logit[a.k] - st.m));
    if (lane != 0) return;
    const bool counts = e.mass[1] != 0.0f;
    a.loss[row] = counts ? loss : 0.0f;
    a.counts[row] = counts;
    if (a.lse_out) {
        // the quotient may pass the largest number; a row of -Inf alone (or
        // with NaN) keeps its -Inf (NaN)
        float lse = st.m * a.inv_tau + log_a;
        if (st.a > 0.0f) lse = fminf(fmaxf(lse, kLowest), -kLowest);
        a.lse_out[2 * row] = counts ? lse : 0.0f;
        a.lse_out[2 * row + 1] = a.ce ? st.m + log_b : 0.0f;
    }
}

// A row whose label masks it.
__device__ __forceinline__ void put_no_loss(const DistillArgs& a, int64_t row)
{
    if (threadIdx.x != 0) return;
    a.loss[row] = 0.0f;
    a.counts[row] = 0;
    if (a.lse_out) a.lse_out[2 * row] = a.lse_out[2 * row + 1] = 0.0f;
}

// A softmax's share of the gradient: g * exp2((s - m) * c), for both, the
// teacher's with an exponent e on top, and held to `top` at most.
struct Slope {
    float m_kd, g_kd, m_ce, g_ce, e_kd, top_kd;
};

template <Terms TM>
__device__ __forceinline__ float slope_at(const Slope& g, float x, float c)
{
    const float z = __builtin_fmaf(x - g.m_kd, c, g.e_kd);
    float v = g.g_kd * exp2_hw(z > g.top_kd ? g.top_kd : z);    // NaN stays
    if constexpr (TM == kKdCe) v += g.g_ce * exp2_hw((x - g.m_ce) * kLog2e);
    return v;
}

__device__ __forceinline__ Slope slope_of(const DistillArgs& a, float mass, const Stat& st,
                                          float row_grad, bool same)
{
    Slope g = {st.m, row_grad * a.grad_kd * mass / st.a, st.m,
               a.ce ? row_grad * a.grad_ce / st.b : 0.0f, 0.0f, INFINITY};
    if (same) g.g_kd += g.g_ce;
    return g;
}

// From this |lse| on its neighbours in fp32 are 16 apart, and it says which
// logits have a weight but not how much: their values are held to 1, where the
// rounding alone would take them to any size (rows of the type's lowest value).
constexpr float kVagueLse = 134217728.0f;

// The fma form of a slope, for the vectors a block holds.
struct FmaSlope {
    float r_kd, g_kd, r_ce, g_ce;
};
__device__ __forceinline__ FmaSlope fma_slope(const Slope& g, float c)
{
    return FmaSlope{g.m_kd * c, g.g_kd * (rounded_by(g.m_kd, c) * exp2_hw(g.e_kd)), g.m_ce * kLog2e,
                    g.g_ce * rounded_by(g.m_ce, kLog2e)};
}

template <Terms TM>
__device__ __forceinline__ bool slope_fma(const Slope& g, float c)
{
    return fma_range(g.m_kd, c) && (TM != kKdCe || fma_range(g.m_ce, kLog2e));
}

template <typename T, Terms TM, int HOLD, typename Vector>
__device__ __forceinline__ void put_held_slopes(T* out, typename Raw<T>::V (&raw)[HOLD],
                                                Vector vector, int nv, const FmaSlope& g, float c)
{
    constexpr int N = Raw<T>::N;
    const uint64_t to = reinterpret_cast<uint64_t>(out);
#pragma unroll
    for (int j = 0; j < HOLD; ++j) {
        const int v = vector(j);
        forget(raw[j]);
        if (v < nv) {
            float x[N];
            Raw<T>::widen(raw[j], x);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float y = g.g_kd * exp2_hw(__builtin_fmaf(x[i], c, -g.r_kd));
                if constexpr (TM == kKdCe)
                    y += g.g_ce * exp2_hw(__builtin_fmaf(x[i], kLog2e, -g.r_ce));
                x[i] = y;
            }
            put_held<T>(to, v, x);
        }
    }
}

// The gradient of a row's columns [0, head) and of its vectors from c0 to c1
// and the elements behind them.
template <typename T, Terms TM, int THREADS, int BATCH>
__device__ __forceinline__ void put_columns(const Slope& g, const T* row, T* out, int head,
                                            int64_t c0, int64_t c1, float c)
{
    constexpr int N = Raw<T>::N;
    const int nv = static_cast<int>((c1 - c0) / N);
    const typename Raw<T>::M* p = reinterpret_cast<const typename Raw<T>::M*>(row + c0);
    for (int v0 = threadIdx.x; v0 - static_cast<int>(threadIdx.x) < nv; v0 += BATCH * THREADS) {
        typename Raw<T>::V raw[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j)
            raw[j] = p[v0 + j * THREADS < nv ? v0 + j * THREADS : nv - 1];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            const int v = v0 + j * THREADS;
            if (v >= nv) continue;
            float x[N];
            Raw<T>::widen(raw[j], x);
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = slope_at<TM>(g, x[i], c);
            store_nt<N>(out + c0 + static_cast<int64_t>(v) * N, x);
        }
    }
    const auto one = [&](int64_t col) { put(out + col, slope_at<TM>(g, widen(row[col]), c)); };
    if (static_cast<int>(threadIdx.x) < head) one(threadIdx.x);
    const int64_t e = c0 + static_cast<int64_t>(nv) * N + threadIdx.x;
    if (e < c1) one(e);
}

// After a barrier behind the columns: the entries' columns once more, with
// their share taken off before the one rounding.  The first entry of a column
// takes off all of that column's, in their order.
template <typename T, Terms TM, int THREADS>
__device__ __forceinline__ void put_entries(const DistillArgs& a, const Entries& e, const Slope& g,
                                            float row_grad, T* out, int64_t c0, int64_t c1, float c)
{
    for (int k = threadIdx.x; k < e.n; k += THREADS) {
        const int col = e.col[k];
        if (col < c0 || col >= c1) continue;
        const auto share = [&](int j) {
            return row_grad * (j < a.k ? a.grad_kd * e.p[j] : a.grad_ce);
        };
        float take = 0.0f;
        bool first = true;
        int same = 3;
        if (a.k > kWave) {
            // one or two entries of the column: their sum has no order
            same = 0;
            for (int j = e.heads[entry_hash(e, col)]; j >= 0; j = e.next[j]) {
                if (e.col[j] != col) continue;
                first = first && j >= k;
                take += ++same <= 2 ? share(j) : 0.0f;
            }
        }
        if (same > 2) {
            take = 0.0f;
            first = true;
            for (int j = 0; j < e.n; j += 4) {
                const int4 o = *reinterpret_cast<const int4*>(e.col + j);
                if (!(o.x == col | o.y == col | o.z == col | o.w == col)) continue;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if ((i == 0 ? o.x : i == 1 ? o.y : i == 2 ? o.z : o.w) != col) continue;
                    first = first && j + i >= k;
                    take += share(j + i);
                }
            }
        }
        if (first) put(out + col, slope_at<TM>(g, e.s[k], c) - take);
    }
}

template <typename T, int THREADS>
__device__ __forceinline__ void put_zeros(T* out, int64_t c0, int64_t c1)
{
    constexpr int N = Raw<T>::N;
    const float z[N] = {};
    const int head = row_head(out + c0, c1 - c0);
    if (static_cast<int>(threadIdx.x) < head) put(out + c0 + threadIdx.x, 0.0f);
    c0 += head;
    const int nv = static_cast<int>((c1 - c0) / N);
    for (int v = threadIdx.x; v < nv; v += THREADS)
        store_nt<N>(out + c0 + static_cast<int64_t>(v) * N, z);
    const int64_t e = c0 + static_cast<int64_t>(nv) * N + threadIdx.x;
    if (e < c1) put(out + e, 0.0f);
}

// Vectors of a row each thread keeps in registers: 64 registers of the 128
// that 16 waves on a CU have each.  A block of 1024 threads so keeps 131072
// bf16 (65536 fp32) logits; what a longer row has beyond that is read again.
constexpr int kHold = 16;
// One block per row: the loss, and with GRAD the gradient, the row read once
// (8192 x 128256 bf16, an eighth of the rows masked: 3.94 GB in 726 us, 5.4
// TB/s; copying the rows in this pattern without arithmetic takes 660).
// Measured and not taken: two blocks of 512 threads on a CU, each holding half
// its row (865 us); loading the next row as this one's registers become free
// (840 us, one block a CU for all rows: a row's blocks in dispatch order suit
// the HBM better).
// (SHORT: a row may have no whole vector.)
template <typename T, Terms TM, bool GRAD, int THREADS, int HOLD, bool SHORT>
__global__ void __launch_bounds__(THREADS, 4) k_distill_row(DistillArgs a, int64_t b0)
{
    extern __shared__ __align__(16) char lds[];
    __shared__ float red[kWaves(THREADS) * 3];
    constexpr int N = Raw<T>::N;
    const int64_t row = b0 + blockIdx.x;
    const float c = a.inv_tau * kLog2e;
    const T* s = static_cast<const T*>(a.logits) + row * a.logits_pitch;
    T* out = static_cast<T*>(a.grad) + row * a.grad_pitch;
    int label;
    if (!label_counts(a, row, &label)) {
        put_no_loss(a, row);
        if constexpr (GRAD) put_zeros<T, THREADS>(out, 0, a.vocab);
        return;
    }
    const int head = row_head(s, a.vocab);
    const int64_t vectors = (a.vocab - head) / N;
    const int nv = static_cast<int>(vectors < HOLD * THREADS ? vectors : HOLD * THREADS);
    const int64_t behind = head + static_cast<int64_t>(nv) * N;     // the held vectors
    int tid = threadIdx.x;
    typename Raw<T>::V raw[HOLD];
    const auto vector = [&](int j) { return tid + j * THREADS; };
#pragma unroll
    for (int j = 0; j < HOLD; ++j)
        raw[j] = SHORT && nv == 0 ? Raw<T>::lowest()
                                  : held_vector<T>(reinterpret_cast<uint64_t>(s + head), vector(j), nv);
    const Entries e = entries_at(lds, a);
    if (a.k <= kWave) {
        if (threadIdx.x < kWave) load_entries<T>(a, e, row, label, s);
    } else {
        clear_chains<THREADS>(a, e);
        read_entries<T>(a, e, row, label, s, 0, a.vocab, threadIdx.x, THREADS);
        __syncthreads();
        if (threadIdx.x < kWave) weigh_entries(a, e, row);
    }
    Stat st = {kLowest, 0.0f, 0.0f};
    const bool sums = held_stats<T, TM>(raw, [&](int j) { return vector(j) < nv; }, c, st);
    st = scan<T, TM, THREADS, 4>(st, s, head, sums ? behind : head, a.vocab, c);
    st = block_join<TM, THREADS>(st, c, red);
    if (threadIdx.x / kWave == (THREADS > kWave ? 1 : 0)) put_loss(a, e, row, st, e.s);
    if constexpr (GRAD) {
        if (e.mass[1] == 0.0f) {
            put_zeros<T, THREADS>(out, 0, a.vocab);
            return;
        }
        const float rg = a.row_grad ? a.row_grad[row] : 1.0f;
        const Slope g = slope_of(a, *e.mass, st, rg, TM == kSame);
        const bool fma = slope_fma<TM>(g, c);
        forget(tid);
        if (fma) put_held_slopes<T, TM>(out + head, raw, vector, nv, fma_slope(g, c), c);
        put_columns<T, TM, THREADS, 4>(g, s, out, head, fma ? behind : head, a.vocab, c);
        __syncthreads();
        put_entries<T, TM, THREADS>(a, e, g, rg, out, 0, a.vocab, c);
    }
}

// A row cut into parts: a part is what one block of kPartThreads holds at HOLD
// vectors a thread, all of them loaded at once.  Parts are dispatched in the
// order of their addresses, so that the accesses under way are one window
// that moves through the logits, which suits the HBM best (2048 x 50257 fp32:
// the loss 60 + 7 us, its gradient 138; a block a row: 92 and 177).
constexpr int kPartThreads = kDistillPartThreads;

// A part of a row: its columns [c0, c1), of which `head` lie before the row's
// vectors (the first part's) and nv vectors from `from` on are held.
struct Part {
    int64_t c0, c1, from;
    int head, nv;
};
template <typename T, int HOLD>
__device__ __forceinline__ Part part_of(const DistillArgs& a, const T* row, int part)
{
    const int head = row_head(row, a.vocab);
    const auto bound = [&](int64_t i) {
        const int64_t c = head + i * a.part_cols;
        return i >= a.splits || c > a.vocab ? a.vocab : c;
    };
    Part p;
    p.from = bound(part);
    p.c0 = part == 0 ? 0 : p.from;
    p.c1 = bound(part + 1);
    p.head = part == 0 ? head : 0;
    const int64_t nv = (p.c1 - p.from) / Raw<T>::N;
    p.nv = static_cast<int>(nv < HOLD * kPartThreads ? nv : HOLD * kPartThreads);
    return p;
}

// The part's statistics, and, if a gradient follows (which may overwrite
// them), the logits at the entries in it.
template <typename T, Terms TM, int HOLD>
__global__ void __launch_bounds__(kPartThreads) k_distill_parts(DistillArgs a, int64_t b0)
{
    __shared__ float red[kWaves(kPartThreads) * 3];
    const int64_t block = b0 + blockIdx.x, row = block / a.splits;
    int label;
    if (!label_counts(a, row, &label)) return;
    const T* s = static_cast<const T*>(a.logits) + row * a.logits_pitch;
    const float c = a.inv_tau * kLog2e;
    const Part p = part_of<T, HOLD>(a, s, static_cast<int>(block - row * a.splits));
    const auto vector = [&](int j) { return static_cast<int>(threadIdx.x) + j * kPartThreads; };
    typename Raw<T>::V raw[HOLD];
#pragma unroll
    for (int j = 0; j < HOLD; ++j)
        raw[j] = p.nv == 0 ? Raw<T>::lowest()
                           : held_vector<T>(reinterpret_cast<uint64_t>(s + p.from), vector(j),
                                            p.nv);
    if (a.grad) {
        for (int k = threadIdx.x; k < a.k + a.ce; k += kPartThreads) {
            float u;
            const int col = k < a.k ? read_entry(a, row * a.k + k, &u) : label;
            if (col >= p.c0 && col < p.c1) a.picked[row * (a.k + 1) + k] = widen(s[col]);
        }
    }
    Stat st = {kLowest, 0.0f, 0.0f};
    const bool sums = held_stats<T, TM>(raw, [&](int j) { return vector(j) < p.nv; }, c, st);
    const int64_t rest = p.from + (sums ? static_cast<int64_t>(p.nv) * Raw<T>::N : 0);
    st = scan<T, TM, kPartThreads, 2>(st, s, p.head, rest, p.c1, c);
    st = block_join<TM, kPartThreads>(st, c, red);
    if (threadIdx.x == 0)
        *reinterpret_cast<float4*>(a.parts + block * kDistillPart) =
            float4{st.m, st.a, st.b, 0.0f};
}

// A row's statistics from its parts', by every wave for itself.
template <Terms TM>
__device__ __forceinline__ Stat join_parts(const DistillArgs& a, int64_t row, float c)
{
    Stat s = {kLowest, 0.0f, 0.0f};
    for (int i = threadIdx.x % kWave; i < a.splits; i += kWave) {
        const float4 o =
            *reinterpret_cast<const float4*>(a.parts + (row * a.splits + i) * kDistillPart);
        join<TM>(s, Stat{o.x, o.y, o.z}, c);
    }
    s = lanes_join<TM>(s, c, kWave);
    if constexpr (TM == kSame) s.b = s.a;
    return s;
}

// The loss of rows cut into parts, once the parts' statistics are there: one
// wave per row.
template <typename T, Terms TM>
__global__ void __launch_bounds__(kWave) k_distill_loss(DistillArgs a, int64_t b0)
{
    extern __shared__ __align__(16) char lds[];
    const int64_t row = b0 + blockIdx.x;
    int label;
    if (!label_counts(a, row, &label)) {
        put_no_loss(a, row);
        return;
    }
    const Entries e = entries_at(lds, a);
    clear_chains<kWave>(a, e);
    load_entries<T>(a, e, row, label, static_cast<const T*>(a.logits) + row * a.logits_pitch);
    put_loss(a, e, row, join_parts<TM>(a, row, a.inv_tau * kLog2e), e.s);
}

// The gradient of a part, from the parts' statistics (the first part's block
// writes the row's loss) or FROM_LSE, from saved ones.
template <typename T, Terms TM, int HOLD, bool FROM_LSE>
__global__ void __launch_bounds__(kPartThreads) k_distill_grad(DistillArgs a, int64_t b0)
{
    extern __shared__ __align__(16) char lds[];
    const int64_t block = b0 + blockIdx.x, row = block / a.splits;
    const int part = static_cast<int>(block - row * a.splits);
    const float c = a.inv_tau * kLog2e;
    const T* s = static_cast<const T*>(a.logits) + row * a.logits_pitch;
    T* out = static_cast<T*>(a.grad) + row * a.grad_pitch;
    const Part p = part_of<T, HOLD>(a, s, part);
    int label;
    if (!label_counts(a, row, &label)) {
        if (!FROM_LSE && part == 0) put_no_loss(a, row);
        put_zeros<T, kPartThreads>(out, p.c0, p.c1);
        return;
    }
    const auto vector = [&](int j) { return static_cast<int>(threadIdx.x) + j * kPartThreads; };
    typename Raw<T>::V raw[HOLD];
#pragma unroll
    for (int j = 0; j < HOLD; ++j)
        raw[j] = p.nv == 0 ? Raw<T>::lowest()
                           : held_vector<T>(reinterpret_cast<uint64_t>(s + p.from), vector(j),
                                            p.nv);
    const Entries e = entries_at(lds, a);
    clear_chains<kPartThreads>(a, e);
    read_entries<T>(a, e, row, label, s, p.c0, p.c1, threadIdx.x, kPartThreads);
    __syncthreads();
    if (threadIdx.x < kWave) weigh_entries(a, e, row);
    const float rg = a.row_grad ? a.row_grad[row] : 1.0f;
    Stat st = {};
    if constexpr (!FROM_LSE) st = join_parts<TM>(a, row, c);
    __syncthreads();
    if (e.mass[1] == 0.0f) {
        if (!FROM_LSE && part == 0) put_no_loss(a, row);
        put_zeros<T, kPartThreads>(out, p.c0, p.c1);
        return;
    }
    Slope g;
    if constexpr (FROM_LSE) {
        // exp(s/tau - lse) = exp((s - m)/tau + rest) with m = tau * lse
        // rounded and rest = m/tau - lse what the rounding leaves: near 0 for
        // an ordinary lse, above 1 past 2^24.  (The quotient of a finite lse
        // may pass the largest number by its rounding.)
        const float lse = a.lse_in[2 * row];
        const float m = fminf(fmaxf(lse / a.inv_tau, kLowest), -kLowest);
        const double rest = static_cast<double>(m) * a.inv_tau - lse;
        g.m_kd = m;
        g.g_kd = rg * a.grad_kd * *e.mass;
        g.e_kd = static_cast<float>(rest) * kLog2e;
        g.top_kd = fabsf(lse) >= kVagueLse ? 0.0f : INFINITY;
        g.m_ce = a.lse_in[2 * row + 1];
        g.g_ce = rg * a.grad_ce;
        if constexpr (TM == kSame) g.g_kd += g.g_ce;
    } else {
        g = slope_of(a, *e.mass, st, rg, TM == kSame);
    }
    const bool fma = slope_fma<TM>(g, c);
    if (fma) put_held_slopes<T, TM>(out + p.from, raw, vector, p.nv, fma_slope(g, c), c);
    const int64_t rest = p.from + (fma ? static_cast<int64_t>(p.nv) * Raw<T>::N : 0);
    put_columns<T, TM, kPartThreads, 2>(g, s, out, p.head, rest, p.c1, c);
    if (!FROM_LSE && part == 0 && threadIdx.x / kWave == 1)
        put_loss(a, e, row, st, a.picked + row * (a.k + 1));
    __syncthreads();
    put_entries<T, TM, kPartThreads>(a, e, g, rg, out, p.c0, p.c1, c);
}

constexpr int kTotalThreads = 1024;

// The sum of the row losses in fp64, in a fixed order, and the count.
__global__ void __launch_bounds__(kTotalThreads) k_distill_total(DistillArgs a)
{
    __shared__ double sums[kTotalThreads / kWave];
    __shared__ int64_t counts[kTotalThreads / kWave];
    double s = 0.0;
    int64_t n = 0;
    for (int64_t r = threadIdx.x; r < a.rows; r += kTotalThreads) {
        s += a.loss[r];
        n += a.counts[r];
    }
    for (int o = kWave / 2; o > 0; o >>= 1) {
        s += __shfl_xor(s, o);
        n += __shfl_xor(n, o);
    }
    if (threadIdx.x % kWave == 0) {
        sums[threadIdx.x / kWave] = s;
        counts[threadIdx.x / kWave] = n;
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < kTotalThreads / kWave; ++w) {
        s += sums[w];
        n += counts[w];
    }
    if (a.loss_sum) *a.loss_sum = static_cast<float>(a.accumulate ? *a.loss_sum + s : s);
    if (a.counted) *a.counted = a.accumulate ? *a.counted + n : n;
}

// ---- launch helpers -------------------------------------------------------------------

int launched() { return hipGetLastError() == hipSuccess ? ZS_OK : ZS_ELAUNCH; }

// blocks of `threads` threads of kernel(args..., first block), in as many
// launches as they need.
template <typename K, typename... Args>
int launch(K kernel, int64_t blocks, int threads, size_t lds, hipStream_t st, Args... args)
{
    const int64_t cap = max_blocks(threads);
    for (int64_t b0 = 0; b0 < blocks; b0 += cap) {
        const int64_t nb = blocks - b0 < cap ? blocks - b0 : cap;
        hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(nb)), dim3(threads), lds, st, args...,
                           b0);
        const int rc = launched();
        if (rc != ZS_OK) return rc;
    }
    return ZS_OK;
}

template <typename TT, typename AT, int N>
int lookup(const EmbedArgs& a, hipStream_t st)
{
    const int shift = lane_shift(a.dim, N, 8);
    const int64_t per = kEmbedThreads >> shift;
    const int64_t blocks = (a.tokens + per - 1) / per;
    // rows of one turn, or of several
    return a.dim <= N * kEmbedThreads
               ? launch(k_embed_lookup<TT, AT, N, 1>, blocks, kEmbedThreads, 0, st, a, shift)
               : launch(k_embed_lookup<TT, AT, N, 4>, blocks, kEmbedThreads, 0, st, a, shift);
}

template <typename AT, typename GT, bool ADD>
int embed_sums(const EmbedArgs& a, SumPlan p, hipStream_t st)
{
    constexpr int N = 16 / sizeof(AT);      // one 16-byte load of activations a lane
    p.zero_shift = lane_shift(a.dim, 16 / sizeof(GT), 8);
    // about 16 KB to clear a block (2.1 GB: 393 us, against 421 at 64 KB a block)
    const int64_t zr = kClearBytes / (a.dim * static_cast<int64_t>(sizeof(GT)));
    p.zero_rows = static_cast<int32_t>(zr < 1 ? 1 : (zr > kWave ? kWave : zr));
    constexpr int64_t cols = static_cast<int64_t>(N) * kWave;
    p.splits = (a.dim + cols - 1) / cols;
    constexpr int64_t per = kEmbedThreads / kWave;
    const int64_t zero_blocks = ADD ? 0 : (a.rows + p.zero_rows - 1) / p.zero_rows;
    if (a.tokens <= kEmbedFew) {
        p.sum_blocks = (a.tokens * p.splits + per - 1) / per;
        return launch(k_embed_few<AT, GT, N, ADD>, p.sum_blocks + zero_blocks, kEmbedThreads, 0,
                      st, a, p);
    }
    p.sum_blocks = (p.chunks * p.splits + per - 1) / per;
    const int rc = launch(k_embed_sum<AT, GT, N, ADD>, p.sum_blocks + zero_blocks, kEmbedThreads,
                          0, st, a, p);
    if (rc != ZS_OK || p.chunks <= 1) return rc;
    return launch(k_embed_join<GT, N, ADD>, p.chunks * p.splits, kEmbedThreads, 0, st, a, p);
}

template <typename AT, typename GT>
int embed_sums(const EmbedArgs& a, const SumPlan& p, bool add, hipStream_t st)
{
    return add ? embed_sums<AT, GT, true>(a, p, st) : embed_sums<AT, GT, false>(a, p, st);
}

// The smallest block that holds the row, so that 16 waves are on a CU at any
// length.  Short rows hold less and take one wave or two, so that more of them
// are under way (8192 rows of bf16, kernel: of 1000 logits 25 us and 44 with a
// block of 256 threads, of 4000 38 and 50, of 8000 53 and 58).
template <typename T, Terms TM, bool GRAD>
int distill_rows(const DistillArgs& a, hipStream_t st)
{
    const size_t lds = entry_bytes(a.k);
    const int64_t vectors = a.vocab / Raw<T>::N;
    if (vectors <= 4 * 64)
        return launch(k_distill_row<T, TM, GRAD, 64, 4, true>, a.rows, 64, lds, st, a);
    if (vectors <= 8 * 64)
        return launch(k_distill_row<T, TM, GRAD, 64, 8, false>, a.rows, 64, lds, st, a);
    if (vectors <= 8 * 128)
        return launch(k_distill_row<T, TM, GRAD, 128, 8, false>, a.rows, 128, lds, st, a);
    if (vectors <= kHold * 256)
        return launch(k_distill_row<T, TM, GRAD, 256, kHold, false>, a.rows, 256, lds, st, a);
    if (vectors <= kHold * 512)
        return launch(k_distill_row<T, TM, GRAD, 512, kHold, false>, a.rows, 512, lds, st, a);
    return launch(k_distill_row<T, TM, GRAD, 1024, kHold, false>, a.rows, 1024, lds, st, a);
}

template <typename T, Terms TM, int HOLD>
int distill_loss_parts(const DistillArgs& a, bool grad, hipStream_t st)
{
    const size_t lds = entry_bytes(a.k);
    const int64_t parts = a.rows * a.splits;
    const int rc = launch(k_distill_parts<T, TM, HOLD>, parts, kPartThreads, 0, st, a);
    if (rc != ZS_OK) return rc;
    return grad ? launch(k_distill_grad<T, TM, HOLD, false>, parts, kPartThreads, lds, st, a)
                : launch(k_distill_loss<T, TM>, a.rows, kWave, lds, st, a);
}

template <typename T, Terms TM>
int distill_loss_t(const DistillArgs& a, const DistillShape& s, bool grad, hipStream_t st)
{
    if (grad ? s.rows_loss_grad : s.rows_loss)
        return grad ? distill_rows<T, TM, true>(a, st) : distill_rows<T, TM, false>(a, st);
    return s.hold == kDistillHold ? distill_loss_parts<T, TM, kDistillHold>(a, grad, st)
                                  : distill_loss_parts<T, TM, kDistillFewHold>(a, grad, st);
}

template <typename T, Terms TM>
int distill_grad_t(const DistillArgs& a, const DistillShape& s, hipStream_t st)
{
    const int64_t parts = a.rows * a.splits;
    const size_t lds = entry_bytes(a.k);
    return s.hold == kDistillHold
               ? launch(k_distill_grad<T, TM, kDistillHold, true>, parts, kPartThreads, lds, st, a)
               : launch(k_distill_grad<T, TM, kDistillFewHold, true>, parts, kPartThreads, lds, st,
                        a);
}

// f(type tag, terms) for the call's element type and softmaxes.
template <typename F>
int by_type(const DistillArgs& a, F f)
{
    const Terms terms = !a.ce ? kKd : (a.inv_tau == 1.0f ? kSame : kKdCe);
    auto typed = [&](auto tag) {
        switch (terms) {
        case kKd: return f(tag, std::integral_constant<Terms, kKd>{});
        case kKdCe: return f(tag, std::integral_constant<Terms, kKdCe>{});
        default: return f(tag, std::integral_constant<Terms, kSame>{});
        }
    };
    return a.f32 ? typed(float{}) : typed(uint16_t{});
}

}  // namespace

int prepare_vocab()
{
    // one kernel's attributes load the code object that holds them all
    hipFuncAttributes f;
    return hipFuncGetAttributes(&f, reinterpret_cast<const void*>(k_distill_total)) == hipSuccess
               ? ZS_OK
               : ZS_ELAUNCH;
}

int enqueue_embed_lookup(const EmbedArgs& a, void* stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    if (a.table_f32)
        return a.act_f32 ? lookup<float, float, 4>(a, st) : lookup<float, uint16_t, 4>(a, st);
    return a.act_f32 ? lookup<uint16_t, float, 4>(a, st) : lookup<uint16_t, uint16_t, 8>(a, st);
}

int enqueue_embed_grad(const EmbedArgs& a, bool accumulate, void* workspace, void* stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    SumPlan p{};
    if (a.tokens > kEmbedFew) {
        const EmbedSpace w = embed_space(a.tokens, a.rows, a.dim);
        char* base = static_cast<char*>(workspace);
        int32_t* order = reinterpret_cast<int32_t*>(base + w.order);
        int32_t* row_of = reinterpret_cast<int32_t*>(base + w.row_of);
        int32_t* starts = reinterpret_cast<int32_t*>(base + w.starts);
        const SortShape s = sort_shape(a.rows);
        const int64_t buckets = int64_t(1) << s.bucket_bits;
        hipLaunchKernelGGL(a.id64 ? k_embed_sort<int64_t> : k_embed_sort<int32_t>,
                           dim3(static_cast<uint32_t>(buckets)), dim3(kSortThreads), kSortLds, st,
                           a, s, order, row_of, starts);
        const int rc = launched();
        if (rc != ZS_OK) return rc;
        p.order = order;
        p.row_of = row_of;
        p.starts = starts;
        p.count = starts + buckets * s.rows;
        p.sort = s;
        p.partials = reinterpret_cast<float*>(base + w.partials);
        p.chunk = embed_chunk(a.tokens);
        p.chunks = embed_chunks(a.tokens);
    }
    if (a.act_f32)
        return a.table_f32 ? embed_sums<float, float>(a, p, accumulate, st)
                           : embed_sums<float, uint16_t>(a, p, accumulate, st);
    return a.table_f32 ? embed_sums<uint16_t, float>(a, p, accumulate, st)
                       : embed_sums<uint16_t, uint16_t>(a, p, accumulate, st);
}

int enqueue_distill_loss(DistillArgs a, bool with_grad, void* stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    const DistillShape s = distill_shape(a.rows, a.vocab, a.f32);
    a.splits = s.splits;
    a.part_cols = s.part_cols;
    a.entry_bits = entry_hash_bits(a.k);
    int rc = ZS_OK;
    if (a.rows > 0)
        rc = by_type(a, [&](auto tag, auto terms) {
            return distill_loss_t<decltype(tag), decltype(terms)::value>(a, s, with_grad, st);
        });
    if (rc != ZS_OK || (!a.loss_sum && !a.counted)) return rc;
    hipLaunchKernelGGL(k_distill_total, dim3(1), dim3(kTotalThreads), 0, st, a);
    return launched();
}

int enqueue_distill_grad(DistillArgs a, void* stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    if (a.rows == 0) return ZS_OK;
    const DistillShape s = distill_shape(a.rows, a.vocab, a.f32);
    a.splits = s.splits;
    a.part_cols = s.part_cols;
    a.entry_bits = entry_hash_bits(a.k);
    return by_type(a, [&](auto tag, auto terms) {
        return distill_grad_t<decltype(tag), decltype(terms)::value>(a, s, st);
    });
}

}  // namespace zs
