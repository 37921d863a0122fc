// ops_host.hpp -- what the C entries of the operators share: argument checks and launch limits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wc.h"

namespace {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }
constexpr uint64_t kMaxRows = 0x7FFFFFFFull;
// Blocks of a launch: HIP counts a grid's threads along x in 32 bits.
constexpr uint64_t max_blocks(uint64_t threads) { return 0xFFFFFFFFull / threads; }

inline bool valid_type(uint32_t t) { return t <= WC_T_FP32; }
inline uintptr_t type_bytes(uint32_t t) { return t == WC_T_FP32 ? 4 : 2; }

// Whether two sets of m rows have no byte in common, rows and pitches in
// bytes: apart as a whole, or side by side in rows of one pitch.
inline bool rows_apart(const void *a, uint64_t a_pitch, uint64_t a_row, const void *b, uint64_t b_pitch, uint64_t b_row, uint64_t m)
{
    const uint64_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    if (p + (m - 1) * a_pitch + a_row <= q || q + (m - 1) * b_pitch + b_row <= p) return true;
    if (m == 1 || a_pitch != b_pitch) return false;
    const uint64_t off = q >= p ? (q - p) % a_pitch : (a_pitch - (p - q) % a_pitch) % a_pitch;  // of b's rows in a's
    return off >= a_row && off + b_row <= a_pitch;
}

inline wc_status launched() { return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP; }

}  // namespace
