// zs_relpos.hip -- CDNA4 (gfx950) kernels of the position-bias table: the bias
// by buckets of relative position, alone or added to scores, and its gradient.
//
// What is computed is stated with the entry points in zero_shard.h.  Both are
// bound by HBM: the bias of a place depends on its diagonal (key minus query)
// alone, so a block works its buckets out once for a diagonal and not for a
// place, and the gradient sums diagonals in registers and turns them into
// buckets once at the end.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "zs_elements.h"
#include "zs_internal.h"

namespace zs {
namespace {

#ifndef ZS_MAX_LAUNCH_THREADS
#define ZS_MAX_LAUNCH_THREADS (int64_t(1) << 31)
#endif
constexpr int64_t max_blocks(int threads) { return ZS_MAX_LAUNCH_THREADS / threads; }

constexpr int kThreads = kRelposThreads;
constexpr int kSumThreads = 1024;

// ---- buckets ----------------------------------------------------------------------

// The bucket of a distance n >= 0 on one side: itself below `exact`, then one
// more for each edge (the smallest distance of a bucket) it has reached.
__device__ __forceinline__ int side_bucket(const RelposArgs& a, const int32_t* edges, int n)
{
    if (n < a.exact) return n;
    if (a.edge_count == 0 || n >= edges[a.edge_count - 1]) return a.exact + a.edge_count;
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

// Where bucket u of one side begins, as a distance.
__device__ __forceinline__ int side_begin(const RelposArgs& a, const int32_t* edges, int u)
{
    return u <= a.exact ? u : edges[u - a.exact - 1];
}

// ---- what a row sees ----------------------------------------------------------------

struct Sequence {
    int64_t start;      // position of the first query
    int64_t length;     // keys that are there
};
__device__ __forceinline__ int64_t read_int(const void* p, int id64, int64_t i)
{
    return id64 ? static_cast<const int64_t*>(p)[i]
                : static_cast<int64_t>(static_cast<const int32_t*>(p)[i]);
}
__device__ __forceinline__ Sequence sequence(const RelposArgs& a, int64_t b)
{
    Sequence s{a.start, a.keys};
    if (a.starts) {
        // positions past the range a call may name are held to it
        const int64_t x = read_int(a.starts, a.id64, b);
        s.start = x < -kRelposFar ? -kRelposFar : x > kRelposFar ? kRelposFar : x;
    }
    if (a.lengths) {
        const int64_t x = read_int(a.lengths, a.id64, b);
        s.length = x < 0 ? 0 : x < a.keys ? x : a.keys;
    }
    return s;
}
// Query i sees keys [0, limit).
__device__ __forceinline__ int64_t row_limit(const RelposArgs& a, const Sequence& s, int64_t i)
{
    if (!a.causal) return s.length;
    const int64_t n = i + s.start + 1;
    return n < 0 ? 0 : n < s.length ? n : s.length;
}

// ---- bias -------------------------------------------------------------------------

// Block b of n in an order in which each of the 8 XCDs, to which consecutive
// blocks are dealt in turn, has one stretch of the work: neighbours that share
// a cache line are then in one L2.
__device__ __forceinline__ int64_t xcd_order(int64_t b, int64_t n)
{
    const int64_t per = n / 8;
    return b < per * 8 ? (b & 7) * per + (b >> 3) : b;
}

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

// One block a tile of `lanes` lanes along the keys and kThreads / lanes groups of R
// rows.  A lane holds N + R - 1 diagonals in registers for R rows of N keys, from
// one read of the table where they are all in a far bucket, which most are; it
// stores R times and ends.  32 heads of 4096 x 4096 bf16 in 174 us, 6.2 TB/s (a
// bare fill in this pattern 166, in one row a block 153; two rows a lane 199, eight
// 184; diagonals built once in LDS for 16 rows and more 202-260).  Blocks in the
// order of xcd_order, by which also rows that begin anywhere cost nothing (a fill
// 2 bytes off 153 us, 211 in the plain order).
// V > 1, for one query: vectors a tile's lanes apart (64 x 16 x 1 x 8192 onto
// scores: 12 us, one vector a lane 13; but 32 x 4099 alone 5.2 us and 4.4).
template <typename T, typename TT, int N, bool SCORES, int R, int V>
__global__ void __launch_bounds__(kThreads) k_relpos_bias(RelposArgs a, int64_t b0)
{
    __shared__ int32_t edges[kRelposMaxEdges];
    int64_t ct, rt, h, b;
    const int64_t blk = xcd_order(b0 + blockIdx.x, a.tiles);
    if (a.tiles <= INT32_MAX) {
        const uint32_t x = static_cast<uint32_t>(blk), cts = static_cast<uint32_t>(a.col_tiles),
                       rts = static_cast<uint32_t>(a.row_tiles),
                       hs = static_cast<uint32_t>(a.heads);
        const uint32_t y = x / cts, z = y / rts, w = z / hs;
        ct = x - y * cts;
        rt = y - z * rts;
        h = z - w * hs;
        b = w;
    } else {
        const int64_t y = blk / a.col_tiles, z = y / a.row_tiles;
        ct = blk % a.col_tiles;
        rt = y % a.row_tiles;
        h = z % a.heads;
        b = z / a.heads;
    }
    const TT* table = static_cast<const TT*>(a.table) + h;
    if (a.edge_count > kFewEdges) {
        for (int e = threadIdx.x; e < a.edge_count; e += kThreads) edges[e] = a.edges[e];
        __syncthreads();
    }
    const Sequence s = sequence(a, b);
    const int lane = threadIdx.x & ((1 << a.lane_shift) - 1);
    const int step = N << a.lane_shift;             // keys of a tile's V-th part
    const int keys = static_cast<int>(a.keys);
    const int j0 = static_cast<int>(ct) * (step * V) + lane * N;
    const int64_t i0 = rt * a.rows + (threadIdx.x >> a.lane_shift) * R;
    const int rows = a.queries - i0 < R ? static_cast<int>(a.queries - i0) : R;
    if (j0 >= keys || rows <= 0) return;
    const T* in = static_cast<const T*>(a.in) + b * a.in_pitch[0] + h * a.in_pitch[1] + i0 * a.in_pitch[2];
    T* out = static_cast<T*>(a.out) + b * a.out_pitch[0] + h * a.out_pitch[1] + i0 * a.out_pitch[2];
    int limit[R];
#pragma unroll
    for (int r = 0; r < R; ++r) limit[r] = static_cast<int>(row_limit(a, s, i0 + r));
    float x[V][R][N];
    if constexpr (SCORES) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int j = j0 + v * step;
                if (r >= rows) continue;
                const T* p = in + r * a.in_pitch[2] + j;
                if (j + N <= limit[r]) {
                    load_n<N>(p, x[v][r]);
                } else {
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        x[v][r][k] = j + k < limit[r] ? widen(p[k]) : 0.0f;
                }
            }
    }
    const int far = a.edge_count > 0 ? a.edges[a.edge_count - 1] : a.exact;
    constexpr int W = N + R - 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int j = j0 + v * step;
        if (j >= keys) continue;
        // w[k - r + R - 1]: the bias of place (i0 + r, j + k)
        float w[W];
        const int d0 = static_cast<int>(j - i0 - s.start) - (R - 1);
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
            T* o = out + r * a.out_pitch[2] + j;
            float q[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                q[k] = w[k - r + R - 1];
                if constexpr (SCORES) q[k] = __builtin_fmaf(a.scale, x[v][r][k], q[k]);
            }
            if (j + N > limit[r]) {
#pragma unroll
                for (int k = 0; k < N; ++k) q[k] = j + k < limit[r] ? q[k] : -INFINITY;
            }
            if (j + N <= keys) {
                store_n<N>(o, q);
            } else {
#pragma unroll
                for (int k = 0; k < N; ++k)
                    if (j + k < keys) put(o + k, q[k]);
            }
        }
    }
}

// ---- gradient ---------------------------------------------------------------------

__device__ __forceinline__ float wave_sum(float q)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) q += __shfl_xor(q, d);
    return q;
}

// One wave a tile, kThreads / 64 tiles a block.  Of a wave, `lanes` lanes take
// N columns each of one row, and 64 / lanes groups take a.rows rows each, one
// below the other.  N rows at a time, a lane's N x N places lie on 2N - 1
// diagonals, summed in registers; N of them get nothing more from this lane and
// are added to the group's diagonals in LDS, where the lane to the left adds N
// rows later.  (A wave's LDS accesses are done in order, and in one access no
// two lanes have the same diagonal.)
template <typename T, int N, bool SCORES>
__global__ void __launch_bounds__(kThreads) k_relpos_grad(RelposArgs a, int64_t b0)
{
    __shared__ int32_t edges[kRelposMaxEdges];
    // per wave: 64 N columns and, for each group, its rows and N
    __shared__ float sums[kThreads / 64][64 * N + kRelposRows + 8 * N];
    for (int e = threadIdx.x; e < a.edge_count; e += kThreads) edges[e] = a.edges[e];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float* mine = sums[wave];
    for (int x = lane; x < 64 * N + kRelposRows + 8 * N; x += 64) mine[x] = 0.0f;
    __syncthreads();
    const int64_t tile = (b0 + blockIdx.x) * (kThreads / 64) + wave;
    if (tile >= a.tiles) return;
    int64_t rest = tile;
    const int64_t ct = rest % a.col_tiles;
    rest /= a.col_tiles;
    const int64_t rt = rest % a.row_tiles;
    rest /= a.row_tiles;
    const int64_t h = rest % a.heads, b = rest / a.heads;
    const Sequence s = sequence(a, b);
    const int lanes = 1 << a.lane_shift, groups = 64 >> a.lane_shift;
    const int group = lane >> a.lane_shift, l = lane & (lanes - 1);
    const int pitch = lanes * N + a.rows + N;       // of a group's diagonals
    const int64_t i0 = (rt * groups + group) * a.rows, c0 = ct * (static_cast<int64_t>(lanes) * N);
    const int64_t j = c0 + l * N;
    const T* in = static_cast<const T*>(a.in) + b * a.in_pitch[0] + h * a.in_pitch[1];
    T* out = static_cast<T*>(a.out) + b * a.out_pitch[0] + h * a.out_pitch[1];
    float* diag = mine + group * pitch;
    // diag[c - r + a.rows]: of column c0 + c and row i0 + r
    float acc[2 * N - 1];
#pragma unroll
    for (int k = 0; k < 2 * N - 1; ++k) acc[k] = 0.0f;
    for (int r0 = 0; r0 < a.rows; r0 += N) {
        float x[N][N];
#pragma unroll
        for (int r = 0; r < N; ++r) {
            const int64_t i = i0 + r0 + r;
            const int64_t limit = i < a.queries ? row_limit(a, s, i) : 0;
            const T* p = in + i * a.in_pitch[2] + j;
            if (j + N <= limit) {
                load_n<N>(p, x[r]);
            } else {
#pragma unroll
                for (int k = 0; k < N; ++k) x[r][k] = j + k < limit ? widen(p[k]) : 0.0f;
            }
        }
        if constexpr (SCORES) {
#pragma unroll
            for (int r = 0; r < N; ++r) {
                const int64_t i = i0 + r0 + r;
                if (i >= a.queries || j >= a.keys) continue;
                T* o = out + i * a.out_pitch[2] + j;
                float v[N];
#pragma unroll
                for (int k = 0; k < N; ++k) v[k] = a.scale * x[r][k];
                // (a place that is not seen is +0 whatever the scale's sign)
                const int64_t limit = row_limit(a, s, i);
                if (j + N > limit) {
#pragma unroll
                    for (int k = 0; k < N; ++k) v[k] = j + k < limit ? v[k] : 0.0f;
                }
                if (j + N <= a.keys) {
                    store_n<N>(o, v);
                } else {
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        if (j + k < a.keys) put(o + k, v[k]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < N; ++r)
#pragma unroll
            for (int k = 0; k < N; ++k) acc[k - r + N - 1] += x[r][k];
        float* f = diag + l * N - r0 + a.rows;
#pragma unroll
        for (int k = 0; k < N; ++k) f[k] += acc[N - 1 + k];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int k = 0; k < N - 1; ++k) acc[N + k] = acc[k];
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] = 0.0f;
    }
    // what the last rows left: the diagonals left of the lane's columns
    float* f = diag + l * N;
#pragma unroll
    for (int k = 0; k < N - 1; ++k) f[k + 1] += acc[N + k];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // the diagonals' sums to buckets: as d grows, the buckets follow one another
    float* part = a.parts + ((h * a.batch + b) * (a.row_tiles * a.col_tiles) + rt * a.col_tiles + ct) *
                                a.buckets;
    for (int u0 = 0; u0 < a.buckets; u0 += 64) {
        const int left = a.buckets - u0 < 64 ? a.buckets - u0 : 64;
        float total = 0.0f;                         // lane u's bucket u0 + u
        for (int g = 0; g < groups; ++g) {
            const float* from = mine + g * pitch;
            // d of from[x] is x + d0, 1 <= x < lanes N + a.rows
            const int64_t d0 = c0 - ((rt * groups + g) * static_cast<int64_t>(a.rows) + s.start) - a.rows;
            const int last = lanes * N + a.rows - 1;
            int x = 1;
            while (x <= last) {
                const int d = static_cast<int>(d0 + x);
                const int u = bucket_of(a, edges, d);
                // where this bucket ends
                int64_t end;
                if (d <= 0) {
                    const int side = u;
                    end = side == 0 ? (a.two_sided ? 0 : int64_t(1) << 40)
                                    : -static_cast<int64_t>(side_begin(a, edges, side));
                } else if (!a.two_sided || u == a.half * 2 - 1) {
                    end = int64_t(1) << 40;
                } else {
                    // the next bucket that begins later (edges may coincide)
                    int side = u - a.half + 1;
                    while (side < a.half - 1 && side_begin(a, edges, side) <= d) ++side;
                    end = static_cast<int64_t>(side_begin(a, edges, side)) - 1;
                    if (end < d) end = int64_t(1) << 40;
                }
                const int64_t stop = end - d0;
                const int to = stop < last ? static_cast<int>(stop) : last;
                if (u >= u0 && u < u0 + left) {
                    float q = 0.0f;
                    for (int y = x + lane; y <= to; y += 64) q += from[y];
                    q = wave_sum(q);
                    if (lane == u - u0) total += q;
                }
                x = to + 1;
            }
        }
        if (lane < left) part[u0 + lane] = total;
    }
}

// The table's gradient from the tiles' parts, one block a head: buckets across
// the lanes, tiles down; summed in fp64 in a fixed order.
template <typename TT>
__global__ void __launch_bounds__(kSumThreads) k_relpos_sum(RelposArgs a)
{
    __shared__ double sums[kSumThreads];
    const int64_t h = blockIdx.x, n = a.batch * a.row_tiles * a.col_tiles;
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

template <typename T, typename TT, int N, bool SCORES>
void bias_launch(const RelposArgs& a, int64_t b0, uint32_t n, hipStream_t st)
{
    if (a.lane_vectors > 1)
        k_relpos_bias<T, TT, N, SCORES, 1, kRelposLaneVectors><<<n, kThreads, 0, st>>>(a, b0);
    else if (a.queries == 1)
        k_relpos_bias<T, TT, N, SCORES, 1, 1><<<n, kThreads, 0, st>>>(a, b0);
    else
        k_relpos_bias<T, TT, N, SCORES, kRelposLaneRows, 1><<<n, kThreads, 0, st>>>(a, b0);
}
template <typename T, typename TT, int N>
void bias_launch(const RelposArgs& a, int64_t b0, uint32_t n, hipStream_t st)
{
    if (a.in) bias_launch<T, TT, N, true>(a, b0, n, st);
    else bias_launch<T, TT, N, false>(a, b0, n, st);
}

}  // namespace

int enqueue_relpos_bias(const RelposArgs& a, void* stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    for (int64_t b0 = 0; b0 < a.tiles; b0 += max_blocks(kThreads)) {
        const uint32_t n = static_cast<uint32_t>(
            a.tiles - b0 < max_blocks(kThreads) ? a.tiles - b0 : max_blocks(kThreads));
        if (a.f32)
            a.table_f32 ? bias_launch<float, float, 4>(a, b0, n, st)
                        : bias_launch<float, uint16_t, 4>(a, b0, n, st);
        else
            a.table_f32 ? bias_launch<uint16_t, float, 8>(a, b0, n, st)
                        : bias_launch<uint16_t, uint16_t, 8>(a, b0, n, st);
        if (hipGetLastError() != hipSuccess) return ZS_ELAUNCH;
    }
    return ZS_OK;
}

int enqueue_relpos_grad(const RelposArgs& a, void* stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    const int64_t blocks = (a.tiles + kThreads / 64 - 1) / (kThreads / 64);
    for (int64_t b0 = 0; b0 < blocks; b0 += max_blocks(kThreads)) {
        const uint32_t n = static_cast<uint32_t>(
            blocks - b0 < max_blocks(kThreads) ? blocks - b0 : max_blocks(kThreads));
        if (a.f32) {
            if (a.out) k_relpos_grad<float, 4, true><<<n, kThreads, 0, st>>>(a, b0);
            else k_relpos_grad<float, 4, false><<<n, kThreads, 0, st>>>(a, b0);
        } else {
            if (a.out) k_relpos_grad<uint16_t, 8, true><<<n, kThreads, 0, st>>>(a, b0);
            else k_relpos_grad<uint16_t, 8, false><<<n, kThreads, 0, st>>>(a, b0);
        }
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
