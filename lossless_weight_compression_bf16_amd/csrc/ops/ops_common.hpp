// ops_common.hpp -- types and small device helpers of the operators beside
// the compressed weights (ops_logprobs.hpp, ops_adapters.hpp, ops_moe.hpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wc.h"

namespace wc {
namespace ops {

constexpr uint32_t kCus = 256;  // compute units of an MI355X: what the launch shapes are planned for

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
    typedef uint32_t x4 __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct Unaligned<4> {
    typedef uint32_t x4 __attribute__((ext_vector_type(4), aligned(4)));
};
template <>
struct Unaligned<16> {
    typedef u32x4 x4;
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
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{f[2 * i], f[2 * i + 1]}), bf16x2));
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

// The same, with kStream past the caches: for memory that is read, or
// written, once, in whole 128-byte lines, and more of it than the last cache
// holds (a gradient over 502 MiB of logits: 192 -> 180 us; over 19: 11.6 ->
// 12.4 us).  Where a
// line's halves are taken by different instructions it costs more than it
// gives, the line being gone before its second half is asked for.
template <int kAlign, bool kStream>
__device__ __forceinline__ u32x4 read16(const void *p)
{
    if constexpr (kStream) return (u32x4)__builtin_nontemporal_load(static_cast<const typename Unaligned<kAlign>::x4 *>(p));
    else return load16<kAlign>(p);
}
template <int kAlign, bool kStream>
__device__ __forceinline__ void write16(void *p, u32x4 v)
{
    if constexpr (kStream)
        __builtin_nontemporal_store((typename Unaligned<kAlign>::x4)v, static_cast<typename Unaligned<kAlign>::x4 *>(p));
    else store16<kAlign>(p, v);
}

__device__ __forceinline__ u32x4 only(bool in, u32x4 v)  // all lanes load, some drop what they got
{
#pragma unroll
    for (int e = 0; e < 4; e++) v[e] = in ? v[e] : 0u;
    return v;
}

// Sixteen rows of a 16-bit matrix through LDS, 256 columns at a time.
// Read in operand order, an instruction takes 64 bytes of each of 16 rows,
// halves of lines; read along the rows, 512 bytes of each of two, whole
// lines, past the caches: 7.1 against 5.8 TB/s over a large buffer, and 6.3
// against 3.6 TB/s where every compute unit has 256 KiB to read.  LDS turns
// one order into the other; rows lie 576 bytes apart, so that the 16 rows of
// an operand spread over all banks.
constexpr uint32_t kStripCols = 256, kStripPitch = 36;  // pitch in 16 bytes
struct Strip {
    u32x4 q[16 * kStripPitch];
};

// The j-th step of 32 columns (64 bytes of a row) of wave `wave` of W: two
// steps in a row, so that one wave's loads take a 128-byte line together.
// The L1 cache holds 256 lines, and a kernel that only streams is bound by how
// many of them it can have on their way: half used lines halve its rate.
template <uint32_t W>
__device__ __forceinline__ uint32_t wave_step(uint32_t wave, uint32_t j)
{
    return (j >> 1) * (2 * W) + 2 * wave + (j & 1);
}

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float nan32() { return __builtin_bit_cast(float, 0x7FC00000u); }
constexpr float kInf = __builtin_inff();

// Eight fp32 numbers as sums of 16-bit ones, for the matrix cores.  BF16: three
// terms, the number itself (each is truncated, so that what two of 8 bits leave
// is the third).  FP16: two, of numbers scaled as below, 22 bits and a sign.
// An infinity is its own first term.
template <int T>
struct Terms;
template <>
struct Terms<WC_T_BF16> {
    static constexpr int kCount = 3;
    __device__ __forceinline__ static void split(const float *f, bf16x8 *out)
    {
        u32x4 v[kCount];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            float lo = f[2 * e], hi = f[2 * e + 1];
#pragma unroll
            for (int c = 0; c < kCount; c++) {
                const uint32_t l = __builtin_bit_cast(uint32_t, lo), h = __builtin_bit_cast(uint32_t, hi);
                v[c][e] = __builtin_amdgcn_perm(h, l, 0x07060302u);  // the upper halves of both
                const float tl = __builtin_bit_cast(float, l & 0xFFFF0000u), th = __builtin_bit_cast(float, h & 0xFFFF0000u);
                lo = c || fabsf(lo) < kInf ? lo - tl : 0.f;
                hi = c || fabsf(hi) < kInf ? hi - th : 0.f;
            }
        }
#pragma unroll
        for (int c = 0; c < kCount; c++) out[c] = __builtin_bit_cast(bf16x8, v[c]);
    }
};
template <>
struct Terms<WC_T_FP16> {
    static constexpr int kCount = 2;
    __device__ __forceinline__ static void split(const float *f, f16x8 *out)
    {
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const _Float16 a = (_Float16)f[e];
            out[0][e] = a;
            out[1][e] = (_Float16)(fabsf((float)a) < kInf ? f[e] - (float)a : 0.f);
        }
    }
};

// What FP16 values are multiplied by before they are split: the power of two
// that brings `most`, the largest of them, to 2^14..2^15; its inverse in
// `unscale`.  1 for BF16, whose range is that of FP32.
template <int T>
__device__ __forceinline__ float term_scale(float most, float &unscale)
{
    unscale = 1.f;
    if (T != WC_T_FP16 || !(most > 0.f && most < kInf)) return 1.f;
    const int ex = min(100, 15 - __builtin_amdgcn_frexp_expf(most));  // -113 at least; 2^-100 for the smallest values
    unscale = __builtin_ldexpf(1.f, -ex);
    return __builtin_ldexpf(1.f, ex);
}

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

// Reductions over a wave by lane moves within the vector registers (a
// shuffle through LDS costs several times as much), the result in every
// lane: sums of 1, 2, 4, 8 lanes of a row of 16, then of rows, end in lane 63.
template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t lanes_moved(uint32_t v, uint32_t none)
{
    return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, kCtrl, kRows, 0xF, false);
}
template <class Op>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, uint32_t none, Op op)
{
    v = op(v, lanes_moved<0x111, 0xF>(v, none));  // from 1, 2, 4, 8 lanes below in the row
    v = op(v, lanes_moved<0x112, 0xF>(v, none));
    v = op(v, lanes_moved<0x114, 0xF>(v, none));
    v = op(v, lanes_moved<0x118, 0xF>(v, none));
    v = op(v, lanes_moved<0x142, 0xA>(v, none));  // lane 15 of the row below into rows 1 and 3
    v = op(v, lanes_moved<0x143, 0xC>(v, none));  // lane 31 into rows 2 and 3
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_sum(float v)
{
    return __builtin_bit_cast(float, wave_reduce(__builtin_bit_cast(uint32_t, v), 0u, [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
    }));
}
__device__ __forceinline__ float wave_max(float v)
{
    return __builtin_bit_cast(float, wave_reduce(__builtin_bit_cast(uint32_t, v), 0xFF800000u, [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
    }));
}
__device__ __forceinline__ uint32_t wave_min(uint32_t v)
{
    return wave_reduce(v, ~0u, [](uint32_t a, uint32_t b) { return min(a, b); });
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
