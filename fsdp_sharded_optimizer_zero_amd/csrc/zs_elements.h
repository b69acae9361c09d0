// zs_elements.h -- device helpers on elements of both types (bf16 bit patterns
// and fp32) shared by the kernel parts that read rows from any element address
// (zs_vocab.hip, zs_tensors.hip, zs_relpos.hip).  Not part of the ABI.
//
// Every 16-byte access is declared with the alignment of its element, which
// compiles to the same one instruction (global memory takes any byte address
// in the unaligned access mode the HSA ABI sets).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace zs {
namespace {

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

// Block b of n in an order in which each of the 8 XCDs, to which consecutive
// blocks are dealt in turn, has stretches of STRETCH blocks (a power of two):
// neighbours that share a cache line or a page of HBM are then mostly on one XCD,
// and work that is uneven over n still falls to all.
template <int STRETCH, typename I>
__device__ __forceinline__ I xcd_order(I b, int64_t n)
{
    const I in = b & (8 * STRETCH - 1), first = b - in;
    return first + 8 * STRETCH <= n ? first + (in & 7) * STRETCH + (in >> 3) : b;
}

}  // namespace
}  // namespace zs
