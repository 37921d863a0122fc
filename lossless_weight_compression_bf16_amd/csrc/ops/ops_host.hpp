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

// Rows of memory: `n` of `width` bytes, `pitch` bytes from one to the next.
struct Rows {
    const void *at;
    uint64_t pitch, width, n;

    uint64_t bytes() const { return n ? (n - 1) * pitch + width : 0; }
};
inline Rows line(const void *at, uint64_t bytes) { return {at, bytes, bytes, bytes ? 1u : 0u}; }
// Rows of 16-bit numbers, `stride` of them from one to the next.
inline Rows rows_of(const void *at, uint64_t stride, uint64_t cols, uint64_t n) { return {at, 2 * stride, 2 * cols, n}; }
// Weights of experts: rows of one pitch where they are that, else all that lies between the first and the last of them.
inline Rows experts_of(const void *at, uint64_t expert, uint64_t row, uint64_t cols, uint64_t rows, uint64_t experts)
{
    if (expert % row == 0) return rows_of(at, row, cols, (experts - 1) * (expert / row) + rows);
    return line(at, 2 * ((experts - 1) * expert + (rows - 1) * row + cols));
}
// Whether two such have no byte in common: apart as a whole, or side by side in rows of one pitch.  Nothing is apart from all.
inline bool apart(const Rows &a, const Rows &b)
{
    if (!a.at || !b.at || !a.n || !b.n) return true;
    const uint64_t p = reinterpret_cast<uintptr_t>(a.at), q = reinterpret_cast<uintptr_t>(b.at);
    if (p + a.bytes() <= q || q + b.bytes() <= p) return true;
    if ((a.n == 1 && b.n == 1) || (a.n > 1 && b.n > 1 && a.pitch != b.pitch)) return false;
    const uint64_t pitch = a.n > 1 ? a.pitch : b.pitch;
    const uint64_t off = q >= p ? (q - p) % pitch : (pitch - (p - q) % pitch) % pitch;  // of b's rows in a's
    return off >= a.width && off + b.width <= pitch;
}
template <class... More>
bool apart(const Rows &a, const Rows &b, const More &...more)
{
    return apart(a, b) && apart(a, more...);
}

inline wc_status launched() { return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP; }

}  // namespace
