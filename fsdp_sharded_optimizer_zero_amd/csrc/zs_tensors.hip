// zs_tensors.hip -- CDNA4 (gfx950) kernels of the calls on many tensors: the
// squared norm over a list of tensors, and the list clipped to a global norm.
//
// What is computed is stated with the entry points in zero_shard.h.  Both are
// bound by HBM: one fp64 multiply-add, or one fp32 product, an element.  The
// list is cut on the host into pieces (zs_tensors_plan), so
// that a launch takes any number of tensors of any size; a piece is part of a
// tensor, or several rows of a tensor whose rows are apart.
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

constexpr int kThreads = kTensorThreads;
constexpr int kSumThreads = 1024;
constexpr int kUnroll = 4;      // 16-byte vectors a lane of the norm has under way

// N elements as loaded (bf16 stays packed until it is used: a lane's vectors
// take half the registers, and twice the waves fit), past the caches' reuse
// where NT.
template <typename T, int N>
struct Vec;
template <>
struct Vec<uint16_t, 8> {
    using M = u32x4_u;
    u32x4 b;
    __device__ __forceinline__ void widen(float v[8]) const
    {
        v[0] = bf16_lo(b.x); v[1] = bf16_hi(b.x);
        v[2] = bf16_lo(b.y); v[3] = bf16_hi(b.y);
        v[4] = bf16_lo(b.z); v[5] = bf16_hi(b.z);
        v[6] = bf16_lo(b.w); v[7] = bf16_hi(b.w);
    }
};
template <>
struct Vec<uint16_t, 4> {
    using M = u32x2_u;
    u32x2_u b;
    __device__ __forceinline__ void widen(float v[4]) const
    {
        v[0] = bf16_lo(b.x); v[1] = bf16_hi(b.x);
        v[2] = bf16_lo(b.y); v[3] = bf16_hi(b.y);
    }
};
template <>
struct Vec<float, 4> {
    using M = f32x4_u;
    f32x4 b;
    __device__ __forceinline__ void widen(float v[4]) const
    {
        v[0] = b.x; v[1] = b.y; v[2] = b.z; v[3] = b.w;
    }
};
template <bool NT, int N, typename T>
__device__ __forceinline__ Vec<T, N> load_vec(const T* p)
{
    using M = typename Vec<T, N>::M;
    const M* m = reinterpret_cast<const M*>(p);
    return Vec<T, N>{NT ? __builtin_nontemporal_load(m) : *m};
}

// ---- deterministic fp64 sums ------------------------------------------------------

// The sum over the 64 lanes of a wave, in a fixed order, in every lane.
__device__ __forceinline__ double wave_sum(double q)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) q += __shfl_xor(q, d);
    return q;
}

// The block's sum, the waves' sums in order; valid in thread 0.
template <int BS>
__device__ __forceinline__ double block_sum(double q)
{
    __shared__ double sums[BS / 64];
    q = wave_sum(q);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = q;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < BS / 64; ++w) t += sums[w];
    return t;
}

// ---- squared norm -----------------------------------------------------------------

// q + d*d: the square of a widened fp32 value is exact in fp64, the sum is
// rounded once.
__device__ __forceinline__ void add_squares(double& q, float x)
{
    const double d = x;
    q = __builtin_fma(d, d, q);
}

template <bool NT, typename T, int N>
__device__ double chunk_sqnorm(const TensorChunk& c)
{
    const T* in = reinterpret_cast<const T*>(c.in);
    double q = 0.0;
    if (c.rows == 1) {
        const int nvec = c.cols / N;
        for (int v0 = threadIdx.x; v0 < nvec; v0 += kThreads * kUnroll) {
            Vec<T, N> x[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                x[u] = v0 + u * kThreads < nvec
                           ? load_vec<NT, N>(in + static_cast<int64_t>(v0 + u * kThreads) * N)
                           : Vec<T, N>{};
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                float v[N];
                x[u].widen(v);
#pragma unroll
                for (int i = 0; i < N; ++i) add_squares(q, v[i]);
            }
        }
        const int e = nvec * N + threadIdx.x;
        if (e < c.cols) add_squares(q, widen(in[e]));
        return q;
    }
    // rows apart: the lanes take the rows' vectors in turn
    const uint32_t per_row = (c.cols + N - 1) / N;
    const uint32_t all = per_row * c.rows;
    for (uint32_t v = threadIdx.x; v < all; v += kThreads) {
        const uint32_t row = v / per_row, col = (v - row * per_row) * N;
        const T* p = in + row * c.in_pitch + col;
        if (col + N <= static_cast<uint32_t>(c.cols)) {
            float x[N];
            load_n<N>(p, x);
#pragma unroll
            for (int i = 0; i < N; ++i) add_squares(q, x[i]);
        } else {
            for (uint32_t i = col; i < static_cast<uint32_t>(c.cols); ++i)
                add_squares(q, widen(p[i - col]));
        }
    }
    return q;
}

// A piece's partial, as another block of the same launch wrote it (ONE), or an
// earlier launch.
template <bool ONE>
__device__ __forceinline__ double partial(const TensorsArgs& a, int64_t i)
{
    return ONE ? __hip_atomic_load(a.partials + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
               : a.partials[i];
}

// From the pieces' partials, by one block: the sum of each tensor's, and of
// all, both in an order that depends on the list's sizes alone.
template <int BS, bool ONE>
__device__ void finish(const TensorsArgs& a)
{
    double q = 0.0;
    constexpr int U = 8;
    for (int64_t i = threadIdx.x; i < a.chunks; i += int64_t(BS) * U) {
        double x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            x[u] = i + u * BS < a.chunks ? partial<ONE>(a, i + u * BS) : 0.0;
#pragma unroll
        for (int u = 0; u < U; ++u) q += x[u];
    }
    q = block_sum<BS>(q);
    if (threadIdx.x == 0) *a.sqnorm_out = a.accumulate ? *a.sqnorm_out + q : q;
    if (!a.each) return;
    // 64 tensors a wave: a lane sums a tensor of few pieces, the wave each of
    // many
    constexpr int kFew = 16;
    const int lane = threadIdx.x & 63;
    constexpr int kWaves = BS / 64;
    for (int64_t t0 = threadIdx.x >> 6; t0 < a.count; t0 += BS) {
        const int64_t t = t0 + lane * kWaves;
        const int64_t from = t < a.count ? a.first[t] : 0, to = t < a.count ? a.first[t + 1] : 0;
        if (t < a.count && to - from <= kFew) {
            double s = 0.0;
            for (int64_t i = from; i < to; ++i) s += partial<ONE>(a, i);
            a.each[t] = s;
        }
        uint64_t many = __ballot(to - from > kFew);
        while (many) {
            const int k = __builtin_ctzll(many);
            many &= many - 1;
            const int64_t begin = __shfl(from, k), end = __shfl(to, k);
            double s = 0.0;
            for (int64_t i = begin + lane; i < end; i += 64 * U) {
                double x[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    x[u] = i + u * 64 < end ? partial<ONE>(a, i + u * 64) : 0.0;
#pragma unroll
                for (int u = 0; u < U; ++u) s += x[u];
            }
            s = wave_sum(s);
            if (lane == 0) a.each[t0 + k * kWaves] = s;
        }
    }
}

// One block a piece, 4 vectors a lane under way in all 8 waves of a SIMD (8 as
// loaded, or 4 widened to fp32, leave room for 4 waves: 157 us, and 170, where
// this takes 133 with the join for 436 million bf16, 6.6 TB/s).  The fp64
// products and their conversions hide behind the loads.  ONE: the block that
// ends last joins the partials, in the fixed order of finish(); which block that
// is changes nothing.  A block's partial is visible to the whole GPU before its
// arrival is counted; the last block leaves the counter at 0 for the next call.
// An arrival takes 16 to 50 ns: 64 pieces 4.0 us, in two launches 4.0, 256
// pieces 8.0 and 4.1.
template <bool ONE, bool NT>
__global__ void __launch_bounds__(kThreads) k_tensors_sqnorm(TensorsArgs a, int64_t b0)
{
    const int64_t b = b0 + blockIdx.x;
    const TensorChunk c = a.table[b];
    double q = c.kind & kChunkInF32 ? chunk_sqnorm<NT, float, 4>(c)
                                   : chunk_sqnorm<NT, uint16_t, 8>(c);
    q = block_sum<kThreads>(q);
    if constexpr (!ONE) {
        if (threadIdx.x == 0) a.partials[b] = q;
    } else {
        __shared__ bool last;
        if (threadIdx.x == 0) {
            __hip_atomic_store(a.partials + b, q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const uint32_t before = __hip_atomic_fetch_add(a.arrived, 1u, __ATOMIC_ACQ_REL,
                                                           __HIP_MEMORY_SCOPE_AGENT);
            last = before + 1 == static_cast<uint32_t>(a.chunks);
            if (last)
                __hip_atomic_store(a.arrived, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (last) finish<kThreads, true>(a);
    }
}

__global__ void __launch_bounds__(kSumThreads) k_tensors_sum(TensorsArgs a)
{
    finish<kSumThreads, false>(a);
}

// ---- clipping ---------------------------------------------------------------------

// min(1, max_norm / (sqrt(Q) + 1e-6)) in double, rounded to fp32; a NaN
// quotient fails the comparison and stays NaN.  The step's coefficient.
__device__ __forceinline__ float clip_coef(double Q, double max_norm)
{
    double c = max_norm / (sqrt(Q) + 1e-6);
    c = (c > 1.0) ? 1.0 : c;
    return static_cast<float>(c);
}

// Part `part` of a piece's `parts`, UNROLL vectors a lane.
template <typename TI, typename TO, int N, int UNROLL>
__device__ void chunk_clip(const TensorsArgs& a, const TensorChunk& c, int part, int parts)
{
    const TI* in = reinterpret_cast<const TI*>(c.in);
    TO* out = reinterpret_cast<TO*>(c.out);
    const bool place = c.in == c.out;
    float coef = 0.0f;
    // in place, a coefficient of 1 leaves every value as it is
    if (place && (coef = clip_coef(*a.sqnorm + a.other, a.max_norm)) == 1.0f) return;
    if (c.rows == 1) {
        constexpr int kPart = kThreads * UNROLL;    // vectors
        if (static_cast<int64_t>(part) * kPart * N >= c.cols) return;
        const int nvec = c.cols / N, v0 = part * kPart + threadIdx.x;
        Vec<TI, N> x[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
            if (v0 + u * kThreads < nvec)
                x[u] = load_vec<true, N>(in + static_cast<int64_t>(v0 + u * kThreads) * N);
        // computed behind the loads
        if (!place) coef = clip_coef(*a.sqnorm + a.other, a.max_norm);
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            if (v0 + u * kThreads >= nvec) continue;
            float v[N];
            x[u].widen(v);
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] *= coef;
            store_nt<N>(out + static_cast<int64_t>(v0 + u * kThreads) * N, v);
        }
        // the elements behind the last vector, in the part they lie in
        const int e = nvec * N + threadIdx.x;
        if (nvec / kPart == part && e < c.cols) put(out + e, widen(in[e]) * coef);
        return;
    }
    if (!place) coef = clip_coef(*a.sqnorm + a.other, a.max_norm);
    const uint32_t per_row = (c.cols + N - 1) / N;
    const uint32_t all = per_row * c.rows;
    for (uint32_t v = part * kThreads + threadIdx.x; v < all; v += kThreads * parts) {
        const uint32_t row = v / per_row, col = (v - row * per_row) * N;
        const TI* p = in + row * c.in_pitch + col;
        TO* o = out + row * c.out_pitch + col;
        if (col + N <= static_cast<uint32_t>(c.cols)) {
            float x[N];
            load_n<N>(p, x);
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] *= coef;
            store_n<N>(o, x);
        } else {
            for (uint32_t i = 0; col + i < static_cast<uint32_t>(c.cols); ++i)
                put(o + i, widen(p[i]) * coef);
        }
    }
}

// A block takes one part of a piece and ends: 32 bytes a lane of the wider of
// the two types, nt loads and stores, all loads first, in stretches by XCD.  436
// million elements: fp32 to fp32 554 us (6.3 TB/s), bf16 to fp32 411 (6.4), bf16
// to bf16 275, one element off 574, 447 and 302 (in the plain order 576, 417 and
// 291; 611, 447 and 308); blocks that walk through their piece 635-680 us for the
// first, with the next loads under way or not; plain stores 5% slower.  In place
// a lane has 64 bytes (583 us; 32: 575): what is then within the limit costs half
// as many waves that only look.
__global__ void __launch_bounds__(kThreads) k_tensors_clip(TensorsArgs a, int parts, int64_t b0)
{
    // a list in place and well within the limit: no wave looks at its piece
    // (436 million fp32: 24 us, with the division in every wave 55)
    if (*a.sqnorm + a.other <= a.quiet) return;
    const int64_t b = xcd_order<64>(b0 + blockIdx.x, a.chunks * parts), k = b / parts;
    const int part = static_cast<int>(b - k * parts);
    const TensorChunk c = a.table[k];
    constexpr int P = kTensorPlace;
    switch (c.kind) {
    case 0: return chunk_clip<uint16_t, uint16_t, 8, 2>(a, c, part, parts);
    case kChunkInF32: return chunk_clip<float, uint16_t, 4, 2>(a, c, part, parts);
    case kChunkOutF32: return chunk_clip<uint16_t, float, 4, 2>(a, c, part, parts);
    case kChunkInF32 | kChunkOutF32: return chunk_clip<float, float, 4, 2>(a, c, part, parts);
    case kChunkPlace: return chunk_clip<uint16_t, uint16_t, 8, 2 * P>(a, c, part, parts);
    default: return chunk_clip<float, float, 4, 2 * P>(a, c, part, parts);
    }
}

// Runs launch(first block, blocks) for `blocks` blocks of kThreads.
template <typename F>
int launches(int64_t blocks, F launch)
{
    for (int64_t b0 = 0; b0 < blocks; b0 += max_blocks(kThreads)) {
        const int64_t n = blocks - b0 < max_blocks(kThreads) ? blocks - b0 : max_blocks(kThreads);
        launch(b0, static_cast<uint32_t>(n));
        if (hipGetLastError() != hipSuccess) return ZS_ELAUNCH;
    }
    return ZS_OK;
}

}  // namespace

int enqueue_tensors_sqnorm(const TensorsArgs& a, void* stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    const bool nt = a.bytes >= (a.clip ? kTensorNtClip : kTensorNt);
    const int rc = launches(a.chunks, [&](int64_t b0, uint32_t n) {
        if (a.chunks <= kTensorOneLaunch) k_tensors_sqnorm<true, false><<<n, kThreads, 0, st>>>(a, b0);
        else if (nt) k_tensors_sqnorm<false, true><<<n, kThreads, 0, st>>>(a, b0);
        else k_tensors_sqnorm<false, false><<<n, kThreads, 0, st>>>(a, b0);
    });
    if (rc != ZS_OK || (a.chunks > 0 && a.chunks <= kTensorOneLaunch)) return rc;
    k_tensors_sum<<<1, kSumThreads, 0, st>>>(a);
    return hipGetLastError() == hipSuccess ? ZS_OK : ZS_ELAUNCH;
}

int enqueue_tensors_clip(const TensorsArgs& a, void* stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    const int parts = static_cast<int>((a.chunk_bytes + kTensorPart - 1) / kTensorPart);
    return launches(a.chunks * parts, [&](int64_t b0, uint32_t n) {
        k_tensors_clip<<<n, kThreads, 0, st>>>(a, parts, b0);
    });
}

int prepare_tensors()
{
    hipFuncAttributes f;
    return hipFuncGetAttributes(&f, reinterpret_cast<const void*>(k_tensors_sum)) == hipSuccess
               ? ZS_OK
               : ZS_ELAUNCH;
}

}  // namespace zs
