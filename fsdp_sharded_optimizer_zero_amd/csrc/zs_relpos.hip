// zs_relpos.hip -- CDNA4 (gfx950) kernels of the position-bias table: the bias
// by buckets of relative position, alone or added to scores, and its gradient.
//
// What is computed is stated with the entry points in zero_shard.h.  Both are
// bound by HBM: the bias of a place depends on its diagonal (key minus query)
// alone, so a lane works out the bucket of a diagonal and not of a place, and the
// gradient sums diagonals in registers and turns them into buckets once at the
// end.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "zs_elements.h"
#include "zs_internal.h"

namespace zs {
namespace {

#ifndef ZS_MAX_LAUNCH_THREADS
#define ZS_MAX_LAUNCH_THREADS (int64_t(1) << 31)
#endif
constexpr int64_t max_blocks(int threads) { return ZS_MAX_LAUNCH_THREADS / threads; }

constexpr int kThreads = kRelposThreads;
constexpr int kWaves = kThreads / 64;
constexpr int kSumThreads = 1024;

// ---- buckets ----------------------------------------------------------------------

// The bucket of a distance n >= 0 on one side: itself below `exact`, then one
// more for each edge (the smallest distance of a bucket) it has reached.
__device__ __forceinline__ int side_bucket(const RelposArgs& a, const int32_t* edges, int n)
{
    if (n < a.exact) return n;
    if (n >= a.far) return a.half - 1;
    int at = 0;
    for (int half = a.edge_span; half > 0; half >>= 1)
        if (at + half <= a.edge_count && edges[at + half - 1] <= n) at += half;
    return a.exact + at;
}

__device__ __forceinline__ int bucket_of(const RelposArgs& a, const int32_t* edges, int d)
{
    const int n = d < 0 ? -d : (a.two_sided ? d : 0);
    const int u = side_bucket(a, edges, n);
    return a.two_sided && d > 0 ? a.half + u : u;
}

// The differences d from lo to hi that bucket u holds (none: lo > hi).
__device__ __forceinline__ void bucket_range(const RelposArgs& a, int u, int& lo, int& hi)
{
    const bool behind = u >= a.half;
    const int v = behind ? u - a.half : u;
    constexpr int kAll = INT32_MAX;
    // distances of one side, from begin up to before end
    const int begin = v <= a.exact ? v : a.edges[v - a.exact - 1];
    const int end = v == a.half - 1 ? kAll : v < a.exact ? v + 1 : a.edges[v - a.exact];
    if (behind) {
        lo = begin > 1 ? begin : 1;
        hi = end - 1;
    } else {
        lo = 1 - end;
        hi = v == 0 && !a.two_sided ? kAll : -begin;
    }
    if (u >= 2 * a.half) lo = 1, hi = 0;            // the odd bucket of a two-sided table
}

// ---- what a row sees ----------------------------------------------------------------

struct Sequence {
    int start;          // position of the first query
    int length;         // keys that are there
};
__device__ __forceinline__ int64_t read_int(const void* p, int id64, int64_t i)
{
    return id64 ? static_cast<const int64_t*>(p)[i]
                : static_cast<int64_t>(static_cast<const int32_t*>(p)[i]);
}
__device__ __forceinline__ Sequence sequence(const RelposArgs& a, int64_t b)
{
    constexpr int kFar = static_cast<int>(kRelposFar);
    Sequence s{static_cast<int>(a.start), static_cast<int>(a.keys)};
    if (a.starts) {
        // positions past the range a call may name are held to it
        const int64_t x = read_int(a.starts, a.id64, b);
        s.start = x < -kFar ? -kFar : x > kFar ? kFar : static_cast<int>(x);
    }
    if (a.lengths) {
        const int64_t x = read_int(a.lengths, a.id64, b);
        s.length = x < 0 ? 0 : x < s.length ? static_cast<int>(x) : s.length;
    }
    return s;
}
// Query i sees keys [0, limit).
__device__ __forceinline__ int row_limit(const RelposArgs& a, const Sequence& s, int i)
{
    if (!a.causal) return s.length;
    const int n = i + s.start + 1;
    return n < 0 ? 0 : n < s.length ? n : s.length;
}

// A value all lanes of the wave hold, in a scalar register.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// x = q d + r: returns q.
__device__ __forceinline__ uint32_t div_mod(uint32_t x, int64_t d, int& r)
{
    const uint32_t n = static_cast<uint32_t>(d), q = x / n;
    r = static_cast<int>(x - q * n);
    return q;
}

// ---- a row's vectors ----------------------------------------------------------------

// N elements as loaded, bf16 packed.
template <typename T>
struct Row;
template <>
struct Row<uint16_t> {
    static constexpr int N = 8;
    u32x4 b;
    __device__ __forceinline__ float at(int k) const
    {
        return k & 1 ? bf16_hi(b[k / 2]) : bf16_lo(b[k / 2]);
    }
    template <bool NT>
    __device__ __forceinline__ void load(const uint16_t* p)
    {
        const auto m = reinterpret_cast<const u32x4_u*>(p);
        b = NT ? __builtin_nontemporal_load(m) : *m;
    }
    // its first n elements
    __device__ __forceinline__ void part(const uint16_t* p, int n)
    {
        uint64_t lo = 0, hi = 0;
#pragma unroll 1
        for (int k = 0; k < n; ++k) {
            const uint64_t e = static_cast<uint64_t>(p[k]) << (16 * (k & 3));
            lo |= k < 4 ? e : 0;
            hi |= k < 4 ? 0 : e;
        }
        b = u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32),
                  static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)};
    }
    // keeps the first n elements, the others 0 whatever they were
    __device__ __forceinline__ void keep(int n)
    {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t mask = n >= 2 * k + 2 ? 0xFFFFFFFFu : n == 2 * k + 1 ? 0xFFFFu : 0u;
            b[k] &= mask;
        }
    }
    // without its first n elements
    __device__ __forceinline__ void drop(int n)
    {
        if (n & 1) b = u32x4{b[0] >> 16 | b[1] << 16, b[1] >> 16 | b[2] << 16,
                             b[2] >> 16 | b[3] << 16, b[3] >> 16};
        if (n & 2) b = u32x4{b[1], b[2], b[3], 0u};
        if (n & 4) b = u32x4{b[2], b[3], 0u, 0u};
    }
};
template <>
struct Row<float> {
    static constexpr int N = 4;
    f32x4 b;
    __device__ __forceinline__ float at(int k) const { return b[k]; }
    template <bool NT>
    __device__ __forceinline__ void load(const float* p)
    {
        const auto m = reinterpret_cast<const f32x4_u*>(p);
        b = NT ? __builtin_nontemporal_load(m) : *m;
    }
    __device__ __forceinline__ void part(const float* p, int n)
    {
        b = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int k = 0; k < n; ++k) {
            b[0] = k == 0 ? p[k] : b[0];
            b[1] = k == 1 ? p[k] : b[1];
            b[2] = k == 2 ? p[k] : b[2];
            b[3] = k == 3 ? p[k] : b[3];
        }
    }
    __device__ __forceinline__ void keep(int n)
    {
#pragma unroll
        for (int k = 0; k < 4; ++k) b[k] = k < n ? b[k] : 0.0f;
    }
    __device__ __forceinline__ void drop(int n)
    {
        if (n & 1) b = f32x4{b[1], b[2], b[3], 0.0f};
        if (n & 2) b = f32x4{b[2], b[3], 0.0f, 0.0f};
    }
};

// The first n of v, fewer than all, in at most three stores (both gradients, 48 x
// 1024 x 2047 bf16: 77 us, element by element 83).
__device__ __forceinline__ void store_part(uint16_t* p, const float (&v)[8], int n)
{
    typedef uint32_t u32_u __attribute__((aligned(2)));
    uint32_t a = pack_bf16x2(v[0], v[1]), b = pack_bf16x2(v[2], v[3]);
    if (n & 4) {
        *reinterpret_cast<u32x2_u*>(p) = u32x2_u{a, b};
        a = pack_bf16x2(v[4], v[5]);
        b = pack_bf16x2(v[6], v[7]);
        p += 4;
    }
    if (n & 2) {
        *reinterpret_cast<u32_u*>(p) = a;
        a = b;
        p += 2;
    }
    if (n & 1) *p = static_cast<uint16_t>(a);
}
__device__ __forceinline__ void store_part(float* p, const float (&v)[4], int n)
{
    typedef float f32x2_u __attribute__((ext_vector_type(2), aligned(4)));
    float a = v[0];
    if (n & 2) {
        *reinterpret_cast<f32x2_u*>(p) = f32x2_u{v[0], v[1]};
        a = v[2];
        p += 2;
    }
    if (n & 1) *p = a;
}

// A lane's N places of a row of `keys`, from column j on.  Those that reach
// past the row are loaded as the row's last N and moved down at use (element by
// element, a wave waits for each of its rows: 48 x 1024 x 2047 bf16, the gradient
// 79 us and 40); a row of fewer than N goes element by element.
template <typename T>
struct Span {
    static constexpr int N = Row<T>::N;
    int j, keys;
    int at;             // where the load begins
    int shift;          // elements of it before j
    __device__ __forceinline__ Span(int j, int keys)
        : j(j), keys(keys), at(j + N <= keys || keys < N ? j : keys - N), shift(j - at)
    {
    }
    // row: the row's first element
    template <bool NT>
    __device__ __forceinline__ Row<T> load(const T* row) const
    {
        Row<T> x;
        if (keys >= N) x.template load<NT>(row + at);
        else x.part(row + j, keys - j);
        return x;
    }
    __device__ __forceinline__ void align(Row<T>& x) const
    {
        if (shift > 0) x.drop(shift);
    }
    __device__ __forceinline__ void store(T* row, const float (&v)[N]) const
    {
        if (j + N <= keys) store_n<N>(row + j, v);
        else store_part(row + j, v, keys - j);
    }
};

// ---- bias -------------------------------------------------------------------------

constexpr int kFewEdges = 16;
// The buckets of W diagonals d0, d0 + 1, ...: for few edges by looking at all
// of them (scalars), else by search in LDS.
template <int W>
__device__ __forceinline__ void buckets_of(const RelposArgs& a, const int32_t* edges, int d0, int u[W])
{
    if (a.edge_count > kFewEdges) {
#pragma unroll
        for (int k = 0; k < W; ++k) u[k] = bucket_of(a, edges, d0 + k);
        return;
    }
    int n[W];
#pragma unroll
    for (int k = 0; k < W; ++k) {
        const int d = d0 + k;
        n[k] = d < 0 ? -d : (a.two_sided ? d : 0);
        u[k] = n[k] < a.exact ? n[k] : a.exact;
    }
    for (int e = 0; e < a.edge_count; ++e) {
        const int edge = a.edges[e];
#pragma unroll
        for (int k = 0; k < W; ++k) u[k] += n[k] >= edge ? 1 : 0;
    }
    if (a.two_sided) {
#pragma unroll
        for (int k = 0; k < W; ++k) u[k] += d0 + k > 0 ? a.half : 0;
    }
}

// One wave a tile: `lanes` lanes along the keys, N keys each, and 64 / lanes groups
// of R rows.  A lane holds N + R - 1 diagonals in registers for R rows, from one
// read of the table where they are all in a far bucket, which most are; it
// stores R times and ends.  Bound by HBM: 32 heads of 4096 x 4096 bf16 in 173 us,
// 6.2 TB/s (a bare fill in this pattern 166, in one row a block 153; two rows a
// lane 199, eight 184; diagonals built once in LDS for 16 rows and more 202-260).
// In the plain order of blocks 187 us, and rows that begin anywhere cost more (a
// fill 2 bytes off 211 us, in this order 153).  Waves and not blocks have tiles, so
// that a row's last few keys cost a wave (48 x 1024 x 2051: 35 us, with tiles of
// 256 lanes 53; 2048 keys 34).
// V > 1, for one query: vectors a tile's lanes apart (64 x 16 x 1 x 8192 onto
// scores: 12 us, one vector a lane 13; but 32 x 4099 alone 5.2 us and 4.4).
template <typename T, typename TT, bool SCORES, bool NT, int R, int V>
__global__ void __launch_bounds__(kThreads) k_relpos_bias(RelposArgs a, int64_t b0)
{
    constexpr int N = Row<T>::N;
    __shared__ int32_t edges[kRelposMaxEdges];
    if (a.edge_count > kFewEdges) {
        for (int e = threadIdx.x; e < a.edge_count; e += kThreads) edges[e] = a.edges[e];
        __syncthreads();
    }
    const uint32_t block = xcd_order<256>(static_cast<uint32_t>(b0) + blockIdx.x, a.blocks);
    const uint32_t tile = block * kWaves + uniform(threadIdx.x >> 6);
    if (tile >= a.tiles) return;
    int ct, rt, h;
    const int64_t b = div_mod(div_mod(div_mod(tile, a.col_tiles, ct), a.row_tiles, rt), a.heads, h);
    const TT* table = static_cast<const TT*>(a.table) + h;
    const Sequence s = sequence(a, b);
    const int lane = threadIdx.x & 63, l = lane & ((1 << a.lane_shift) - 1);
    const int step = N << a.lane_shift;             // keys of a tile's V-th part
    const int keys = static_cast<int>(a.keys);
    const int j0 = ct * (step * V) + l * N;
    const int i0 = rt * a.rows + (lane >> a.lane_shift) * R;
    const int rows = static_cast<int>(a.queries) - i0 < R ? static_cast<int>(a.queries) - i0 : R;
    if (j0 >= keys || rows <= 0) return;
    const T* in = static_cast<const T*>(a.in) + b * a.in_pitch[0] + h * a.in_pitch[1] + i0 * a.in_pitch[2];
    T* out = static_cast<T*>(a.out) + b * a.out_pitch[0] + h * a.out_pitch[1] + i0 * a.out_pitch[2];
    int limit[R];
#pragma unroll
    for (int r = 0; r < R; ++r) limit[r] = row_limit(a, s, i0 + r);
    // the row's last vector ends with the row, and repeats places of the one before:
    // both write the same bits (18 x 22 x 4044 x 22 fp32 onto scores 64 us; moved down
    // and stored element by element 78).  In place the other may have written them
    // already.
    const bool apart = a.in != a.out && keys >= N;
    const auto vector_at = [&](int v) {
        const int j = j0 + v * step;
        return apart && j < keys && j + N > keys ? keys - N : j;
    };
    Row<T> x[V][R];
    if constexpr (SCORES) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const Span<T> span(vector_at(v), keys);
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r < rows && span.j < limit[r]) x[v][r] = span.template load<NT>(in + r * a.in_pitch[2]);
        }
    }
    const int far = a.far;
    constexpr int W = N + R - 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (j0 + v * step >= keys) continue;
        const Span<T> span(vector_at(v), keys);
        const int j = span.j;
        // w[k - r + R - 1]: the bias of place (i0 + r, j + k)
        float w[W];
        const int d0 = j - i0 - s.start - (R - 1);
        // far away on one side, or all behind a one-sided query: one bucket
        if (d0 + W - 1 <= -far || (a.two_sided ? d0 >= far : d0 >= 0)) {
            const int u = d0 < 0 ? a.half - 1 : a.two_sided ? 2 * a.half - 1 : 0;
            const float q = widen(table[u * a.table_pitch]);
#pragma unroll
            for (int k = 0; k < W; ++k) w[k] = q;
        } else {
            int u[W];
            buckets_of<W>(a, edges, d0, u);
#pragma unroll
            for (int k = 0; k < W; ++k) w[k] = widen(table[u[k] * a.table_pitch]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r >= rows) continue;
            if constexpr (SCORES) span.align(x[v][r]);
            float q[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                q[k] = w[k - r + R - 1];
                if constexpr (SCORES) q[k] = __builtin_fmaf(a.scale, x[v][r].at(k), q[k]);
            }
            if (j + N > limit[r]) {
#pragma unroll
                for (int k = 0; k < N; ++k) q[k] = j + k < limit[r] ? q[k] : -INFINITY;
            }
            span.store(out + r * a.out_pitch[2], q);
        }
    }
}

// ---- gradient ---------------------------------------------------------------------

// x of another lane by DPP control.
template <int CTRL>
__device__ __forceinline__ float dpp(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float lane_of(float x, int lane)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}
// The sum over the wave, in every lane, in a fixed order: quad partners 1 and 2
// apart, rotations by 4 and 8 in a row of 16, the rows in order.
__device__ __forceinline__ float wave_sum(float q)
{
    q += dpp<0xB1>(q);
    q += dpp<0x4E>(q);
    q += dpp<0x124>(q);
    q += dpp<0x128>(q);
    return ((lane_of(q, 0) + lane_of(q, 16)) + lane_of(q, 32)) + lane_of(q, 48);
}

// The value of the lane below (0 in lane 0): a DPP move of the whole wave by one.
__device__ __forceinline__ float from_below(float x)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x138, 0xF, 0xF, true));
}

// One wave a tile: of a wave, `lanes` lanes take N columns each of one row, and
// 64 / lanes groups take a.rows rows each, one below the other.  N rows at a time,
// a lane's N x N places lie on 2N - 1 diagonals, summed in registers; N of them
// get nothing more from this lane and pass to the lane to the right, which meets
// them N rows later.  So each diagonal's sum leaves the wave once, at its right
// edge or below its last row, into LDS, where it is added to its bucket.  Bound
// by HBM: 8 x 16 x 2048 x 2048 bf16 in 165 us, 6.5 TB/s (over two buffers in turn
// 174-193), 606 MB of them seen in
// sequences of 0 to 2048 keys 112 (with the diagonals added to LDS every N rows
// 486 and 428; all of a bucket's diagonals by the whole wave, one bucket after the
// other, 20 us more a call).  The two loads of kBatch rows in turn keep one under way; 8
// rows loaded, then summed, 187 us; what is said of a row is worked out for all
// rows at once where they see the same (partly filled tiles are bound by that).
constexpr int kBatch = 4;
constexpr int kFewDiagonals = 16;   // of a bucket, up to which one lane sums them
// Of a tile of several groups, 64 at a time: 32 lanes' keys and its rows.  Joined
// before the buckets: 28 x 29 x 120 x 64 bf16 12.0 us, buckets by group 14.5 (the
// bytes' floor is 2).
template <int N>
constexpr int kGroupDiagonals = (32 * N + kRelposRows + 63) / 64;
template <typename T, bool SCORES, bool NT>
__global__ void __launch_bounds__(kThreads) k_relpos_grad(RelposArgs a, int64_t b0)
{
    constexpr int N = Row<T>::N;
    __shared__ float sums[kWaves][64 * N + kRelposRows];
    __shared__ float totals[kWaves][kRelposMaxBuckets];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float* mine = sums[wave];
    int in_plane, h, ct;
    const uint32_t plane = div_mod(static_cast<uint32_t>(b0) + blockIdx.x, a.plane_blocks, in_plane);
    const int64_t b = div_mod(plane, a.heads, h);
    const int rt = div_mod(uniform(in_plane * kWaves + wave), a.col_tiles, ct);
    const int lanes = 1 << a.lane_shift, groups = 64 >> a.lane_shift;
    const int group = lane >> a.lane_shift, l = lane & (lanes - 1);
    const int pitch = lanes * N + a.rows;           // of a group's diagonals
    const int keys = static_cast<int>(a.keys), queries = static_cast<int>(a.queries);
    const Sequence s = sequence(a, b);
    // a tile without a place that is seen leaves nothing (its last row sees most)
    const int rows_end = (rt + 1) * groups * a.rows;
    const bool here = rt < a.row_tiles && (SCORES || ct * lanes * N < row_limit(a, s, (rows_end < queries ? rows_end : queries) - 1));
    if (here) {
        const int i0 = (rt * groups + group) * a.rows, j = (ct * lanes + l) * N;
        const Span<T> span(j, keys);
        const T* in = static_cast<const T*>(a.in) + b * a.in_pitch[0] + h * a.in_pitch[1] +
                      i0 * a.in_pitch[2];
        T* out = static_cast<T*>(a.out) + b * a.out_pitch[0] + h * a.out_pitch[1] +
                 i0 * a.out_pitch[2];
        float* diag = mine + group * pitch;
        float acc[2 * N - 1], carry[N];
#pragma unroll
        for (int k = 0; k < 2 * N - 1; ++k) acc[k] = 0.0f;
#pragma unroll
        for (int k = 0; k < N; ++k) carry[k] = 0.0f;
        // elements of row i0 + r that this lane's vector has and sees
        const auto seen = [&](int r) {
            const int i = i0 + r;
            const int n = (i < queries ? row_limit(a, s, i) : 0) - j;
            return n < 0 ? 0 : n < N ? n : N;
        };
        const int fixed = seen(0);
        const T* next = in;
        // VARIES: rows see different numbers of keys, or are not there
        const auto load = [&](auto varies, Row<T>(&x)[kBatch], int r0) {
#pragma unroll
            for (int r = 0; r < kBatch; ++r) {
                x[r] = Row<T>{};
                if ((varies ? seen(r0 + r) : fixed) > 0) x[r] = span.template load<NT>(next);
                next += a.in_pitch[2];
            }
        };
        T* left = out;
        // PLACE: the batch's place among the N rows of the accumulators
        const auto work = [&](auto varies, auto place, Row<T>(&x)[kBatch], int r0) {
            constexpr int R = decltype(place)::value;
#pragma unroll
            for (int r = 0; r < kBatch; ++r) {
                const int n = varies ? seen(r0 + r) : fixed;
                // the places that this lane has and sees, the others 0
                span.align(x[r]);
                if (n < N) x[r].keep(n);
                if constexpr (SCORES) {
                    if ((!varies || i0 + r0 + r < queries) && j < keys) {
                        float v[N];
#pragma unroll
                        for (int k = 0; k < N; ++k) v[k] = a.scale * x[r].at(k);
                        if (n < N) {
#pragma unroll
                            for (int k = 0; k < N; ++k) v[k] = k < n ? v[k] : 0.0f;
                        }
                        span.store(left, v);
                    }
                    left += a.out_pitch[2];
                }
#pragma unroll
                for (int k = 0; k < N; ++k) acc[k - (R + r) + N - 1] += x[r].at(k);
            }
        };
        // the diagonals that get nothing more from this lane, with what the lane
        // to the left had of them N rows before
        const auto pass = [&](int r0, bool end) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float below = from_below(carry[k]);
                carry[k] = (l == 0 ? 0.0f : below) + acc[N - 1 + k];
            }
            if (end || l == lanes - 1) {
                float* f = diag + l * N - r0 + a.rows;
#pragma unroll
                for (int k = 0; k < N; ++k) f[k] = carry[k];
            }
#pragma unroll
            for (int k = 0; k < N - 1; ++k) acc[N + k] = acc[k];
#pragma unroll
            for (int k = 0; k < N; ++k) acc[k] = 0.0f;
        };
        // two batches of rows in turn, one under way while the other is summed
        using First = std::integral_constant<int, 0>;
        using Second = std::integral_constant<int, N == kBatch ? 0 : kBatch>;
        const auto walk = [&](auto varies) {
            Row<T> x[kBatch], y[kBatch];
            load(varies, x, 0);
            for (int r0 = 0; r0 < a.rows; r0 += 2 * kBatch) {
                load(varies, y, r0 + kBatch);
                work(varies, First{}, x, r0);
                if constexpr (N == kBatch) pass(r0, false);
                if (r0 + 2 * kBatch < a.rows) load(varies, x, r0 + 2 * kBatch);
                work(varies, Second{}, y, r0 + kBatch);
                pass(r0 + 2 * kBatch - N, false);
            }
        };
        if (__all(fixed == seen(a.rows - 1) && i0 + a.rows <= queries)) walk(std::false_type{});
        else walk(std::true_type{});
        pass(a.rows, true);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // the groups' diagonals to the tile's: group g's are (groups - 1 - g) * rows on
    const int last = pitch - 1 + (groups - 1) * a.rows;     // diagonals 1..last
    if (here && groups > 1) {
        float q[kGroupDiagonals<N>];
#pragma unroll
        for (int k = 0; k < kGroupDiagonals<N>; ++k) {
            q[k] = 0.0f;
            for (int g = 0; g < groups; ++g) {
                const int x = lane + 64 * k - (groups - 1 - g) * a.rows;
                if (x >= 1 && x < pitch) q[k] += mine[g * pitch + x];
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int k = 0; k < kGroupDiagonals<N>; ++k)
            if (lane + 64 * k <= last) mine[lane + 64 * k] = q[k];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    // the diagonals' sums to buckets, a bucket a lane; the last of each side, which
    // may have most of the diagonals, by all lanes.  mine[x] is of d = x + d0
    const int d0 = ct * lanes * N - ((rt + 1) * groups * a.rows + s.start);
    for (int u0 = 0; u0 < a.buckets; u0 += 64) {
        const int u = u0 + lane;
        float total = 0.0f;
        if (here) {
            // its distances, as places of diagonals: d from lo to hi
            int lo = 1, hi = 0;
            if (u < a.buckets) bucket_range(a, u, lo, hi);
            const bool wide = static_cast<int64_t>(hi) - lo >= kFewDiagonals;
            // (in 64 bits: distances may be 2^30, and a range all of them)
            const int64_t begin64 = static_cast<int64_t>(lo) - d0, end64 = static_cast<int64_t>(hi) - d0;
            const int x0 = begin64 < 1 ? 1 : begin64 > last ? last + 1 : static_cast<int>(begin64);
            const int x1 = end64 < 0 ? 0 : end64 > last ? last : static_cast<int>(end64);
            if (!wide) {
                for (int x = x0; x <= x1; x += 4) {
                    float q[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) q[k] = mine[x + k <= x1 ? x + k : x];
#pragma unroll
                    for (int k = 0; k < 4; ++k) total += x + k <= x1 ? q[k] : 0.0f;
                }
            }
            uint64_t many = __ballot(wide && x0 <= x1);
            while (many) {
                const int k = __builtin_ctzll(many);
                many &= many - 1;
                const int begin = __builtin_amdgcn_readlane(x0, k), end = __builtin_amdgcn_readlane(x1, k);
                float q = 0.0f;
                for (int x = begin + lane; x <= end; x += 64) q += mine[x];
                q = wave_sum(q);
                if (lane == k) total += q;
            }
        }
        if (u < a.buckets) totals[wave][u] = total;
    }
    __syncthreads();
    float* part = a.parts + ((static_cast<int64_t>(h) * a.batch + b) * a.plane_blocks + in_plane) * a.buckets;
    for (int u = threadIdx.x; u < a.buckets; u += kThreads) {
        float q = totals[0][u];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) q += totals[w][u];
        part[u] = q;
    }
}

// The table's gradient from the parts of the tiles' blocks (fp32), one block a head:
// buckets across the lanes, parts down; summed in fp64 in a fixed order.  Rounded to
// fp32, then to bf16: off by half a step of bf16 and at most half a step of fp32.
template <typename TT>
__global__ void __launch_bounds__(kSumThreads) k_relpos_sum(RelposArgs a)
{
    __shared__ double sums[kSumThreads];
    const int64_t h = blockIdx.x, n = a.batch * a.plane_blocks;
    const float* part = a.parts + h * n * a.buckets;
    // a power of two of lanes across the buckets
    int across = 1;
    while (across < a.buckets) across *= 2;
    const int u = threadIdx.x & (across - 1), down = kSumThreads / across;
    double q = 0.0;
    if (u < a.buckets) {
        constexpr int U = 8;
        for (int64_t t = threadIdx.x / across; t < n; t += int64_t(down) * U) {
            float x[U];
#pragma unroll
            for (int k = 0; k < U; ++k)
                x[k] = t + k * down < n ? part[(t + k * down) * a.buckets + u] : 0.0f;
#pragma unroll
            for (int k = 0; k < U; ++k) q += x[k];
        }
    }
    sums[threadIdx.x] = q;
    __syncthreads();
    for (int k = down / 2; k > 0; k /= 2) {
        if (static_cast<int>(threadIdx.x) < k * across) sums[threadIdx.x] += sums[threadIdx.x + k * across];
        __syncthreads();
    }
    if (static_cast<int>(threadIdx.x) < a.buckets) {
        TT* o = static_cast<TT*>(a.table_grad) + threadIdx.x * a.table_pitch + h;
        double v = sums[threadIdx.x];
        if (a.accumulate) v += widen(*o);
        put(o, static_cast<float>(v));
    }
}

template <typename T, typename TT, bool SCORES, bool NT>
void bias_launch(const RelposArgs& a, int64_t b0, uint32_t n, hipStream_t st)
{
    // one query past the caches is in tiles (of 64 lanes' vectors at most) enough for
    // kRelposLaneVectors
    static_assert(kRelposManyTiles * 64 * 16 <= kRelposNt, "NT with one vector a lane");
    if (a.lane_vectors > 1) {
        k_relpos_bias<T, TT, SCORES, NT, 1, kRelposLaneVectors><<<n, kThreads, 0, st>>>(a, b0);
        return;
    }
    if constexpr (!NT) {
        if (a.queries == 1) {
            k_relpos_bias<T, TT, SCORES, NT, 1, 1><<<n, kThreads, 0, st>>>(a, b0);
            return;
        }
    }
    k_relpos_bias<T, TT, SCORES, NT, kRelposLaneRows, 1><<<n, kThreads, 0, st>>>(a, b0);
}
template <typename T, typename TT>
void bias_launch(const RelposArgs& a, int64_t b0, uint32_t n, hipStream_t st)
{
    if (!a.in) bias_launch<T, TT, false, false>(a, b0, n, st);
    else if (a.nt) bias_launch<T, TT, true, true>(a, b0, n, st);
    else bias_launch<T, TT, true, false>(a, b0, n, st);
}
template <typename T>
void grad_launch(const RelposArgs& a, int64_t b0, uint32_t n, hipStream_t st)
{
    if (a.out)
        a.nt ? k_relpos_grad<T, true, true><<<n, kThreads, 0, st>>>(a, b0)
             : k_relpos_grad<T, true, false><<<n, kThreads, 0, st>>>(a, b0);
    else
        a.nt ? k_relpos_grad<T, false, true><<<n, kThreads, 0, st>>>(a, b0)
             : k_relpos_grad<T, false, false><<<n, kThreads, 0, st>>>(a, b0);
}

}  // namespace

int enqueue_relpos_bias(const RelposArgs& a, void* stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    for (int64_t b0 = 0; b0 < a.blocks; b0 += max_blocks(kThreads)) {
        const uint32_t n = static_cast<uint32_t>(
            a.blocks - b0 < max_blocks(kThreads) ? a.blocks - b0 : max_blocks(kThreads));
        if (a.f32)
            a.table_f32 ? bias_launch<float, float>(a, b0, n, st)
                        : bias_launch<float, uint16_t>(a, b0, n, st);
        else
            a.table_f32 ? bias_launch<uint16_t, float>(a, b0, n, st)
                        : bias_launch<uint16_t, uint16_t>(a, b0, n, st);
        if (hipGetLastError() != hipSuccess) return ZS_ELAUNCH;
    }
    return ZS_OK;
}

int enqueue_relpos_grad(const RelposArgs& a, void* stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    for (int64_t b0 = 0; b0 < a.blocks; b0 += max_blocks(kThreads)) {
        const uint32_t n = static_cast<uint32_t>(
            a.blocks - b0 < max_blocks(kThreads) ? a.blocks - b0 : max_blocks(kThreads));
        if (a.f32) grad_launch<float>(a, b0, n, st);
        else grad_launch<uint16_t>(a, b0, n, st);
        if (hipGetLastError() != hipSuccess) return ZS_ELAUNCH;
    }
    if (a.table_f32) k_relpos_sum<float><<<static_cast<uint32_t>(a.heads), kSumThreads, 0, st>>>(a);
    else k_relpos_sum<uint16_t><<<static_cast<uint32_t>(a.heads), kSumThreads, 0, st>>>(a);
    return hipGetLastError() == hipSuccess ? ZS_OK : ZS_ELAUNCH;
}

int prepare_relpos()
{
    hipFuncAttributes f;
    return hipFuncGetAttributes(&f, reinterpret_cast<const void*>(k_relpos_sum<float>)) == hipSuccess
               ? ZS_OK
               : ZS_ELAUNCH;
}

}  // namespace zs
