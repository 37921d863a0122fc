// ops_common.hpp -- types and small device helpers of the operators beside
// the compressed weights (ops_logprobs.hpp, ops_adapters.hpp, ops_moe.hpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wc.h"

namespace wc {
namespace ops {

constexpr uint32_t kCus = 256;  // compute units of an MI355X: what the launch shapes are planned for

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// The same vectors at any element's address: gfx950 loads and stores up to
// 16 bytes at any address, so rows that start anywhere take the wide
// accesses too.
template <int kAlign>
struct Unaligned;
template <>
struct Unaligned<2> {
    typedef uint32_t x2 __attribute__((ext_vector_type(2), aligned(2)));
    typedef uint32_t x4 __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct Unaligned<4> {
    typedef uint32_t x2 __attribute__((ext_vector_type(2), aligned(4)));
    typedef uint32_t x4 __attribute__((ext_vector_type(4), aligned(4)));
};

template <int T>
struct Type;

template <>
struct Type<WC_T_FP32> {
    using elem = float;
    static constexpr int kBytes = 4, kPer16 = 4;  // elements in 16 bytes
    __device__ static float to_f32(elem v) { return v; }
    __device__ static elem from_f32(float v) { return v; }
    __device__ static void unpack(u32x4 v, float *f)
    {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t w = v[i];  // a bit cast of the vector's element itself reads element 0
            f[i] = __builtin_bit_cast(float, w);
        }
    }
    __device__ static u32x4 pack(const float *f)
    {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = __builtin_bit_cast(uint32_t, f[i]);
        return v;
    }
};

template <>
struct Type<WC_T_BF16> {
    using elem = uint16_t;
    using x8 = bf16x8;
    static constexpr int kBytes = 2, kPer16 = 8;
    __device__ static float to_f32(elem v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
    __device__ static elem from_f32(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }  // nearest even
    __device__ static void unpack(u32x4 v, float *f)
    {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            f[2 * i] = __builtin_bit_cast(float, v[i] << 16);
            f[2 * i + 1] = __builtin_bit_cast(float, v[i] & 0xFFFF0000u);
        }
    }
    __device__ static u32x4 pack(const float *f)
    {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = (uint32_t)from_f32(f[2 * i]) | ((uint32_t)from_f32(f[2 * i + 1]) << 16);
        return v;
    }
    __device__ static f32x4 mfma(x8 a, x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
};

template <>
struct Type<WC_T_FP16> {
    using elem = uint16_t;
    using x8 = f16x8;
    static constexpr int kBytes = 2, kPer16 = 8;
    __device__ static float to_f32(elem v) { return (float)__builtin_bit_cast(_Float16, v); }
    __device__ static elem from_f32(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }  // nearest even
    __device__ static void unpack(u32x4 v, float *f)
    {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            f[2 * i] = to_f32((uint16_t)(v[i] & 0xFFFFu));
            f[2 * i + 1] = to_f32((uint16_t)(v[i] >> 16));
        }
    }
    __device__ static u32x4 pack(const float *f)
    {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = (uint32_t)from_f32(f[2 * i]) | ((uint32_t)from_f32(f[2 * i + 1]) << 16);
        return v;
    }
    __device__ static f32x4 mfma(x8 a, x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
};

// 16 bytes at an address that is a multiple of kAlign
template <int kAlign>
__device__ __forceinline__ u32x4 load16(const void *p)
{
    if constexpr (kAlign >= 16) return *static_cast<const u32x4 *>(p);
    else return (u32x4)(*static_cast<const typename Unaligned<kAlign>::x4 *>(p));
}
template <int kAlign>
__device__ __forceinline__ void store16(void *p, u32x4 v)
{
    if constexpr (kAlign >= 16) *static_cast<u32x4 *>(p) = v;
    else *static_cast<typename Unaligned<kAlign>::x4 *>(p) = (typename Unaligned<kAlign>::x4)v;
}

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float nan32() { return __builtin_bit_cast(float, 0x7FC00000u); }
constexpr float kInf = __builtin_inff();

// Whole numbers in the order of floats (-0 = 0), 1 for NaN, 0 for nothing.
__device__ __forceinline__ uint32_t key_of(float f)
{
    if (f != f) return 1u;
    const uint32_t b = __builtin_bit_cast(uint32_t, f + 0.0f);  // -0 + 0 = 0
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    if (k <= 1u) return nan32();
    return __builtin_bit_cast(float, (k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// A word of LDS that is the same for the whole block, read to the end: a
// plain read may still be under way when its wave reaches the next barrier,
// after which another wave may write the word again.
__device__ __forceinline__ uint32_t lds_uniform(const uint32_t &v)
{
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)*(const volatile uint32_t *)&v);
}

__device__ __forceinline__ void report(uint32_t *err, uint32_t bits)
{
    if (err) atomicOr(err, bits);
}

}  // namespace ops
}  // namespace wc
