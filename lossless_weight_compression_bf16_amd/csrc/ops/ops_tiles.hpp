// ops_tiles.hpp -- one tile of a matrix product on the matrix cores, for the
// products of ops_grouped.hpp and ops_loss.hpp:  D[m][n] = sum_k Q[m][k] P[n][k]
// with fp32 sums of exact products, Q and P each stored with k along the rows of
// memory or across them.
//
// A block of four waves has BM x BN of D, a wave (BM / 2) x (BN / 2).  k goes by
// stages of 64: while one is multiplied the next one is on its way from memory
// straight into LDS (no registers), and within a stage the operands of one half
// are read while the other half is multiplied, a read or a load between every
// few products, so that a wave alone on its SIMD keeps its matrix core fed; one
// barrier per stage.  256 x 256 takes 256 accumulators and 147 KB of LDS, one
// block on a compute unit.  What bounds it: the clock under the matrix cores'
// load.  8192^3, BF16, dense: k along both 1455 TFLOP/s, along and across 1399,
// across both 1411, where a library's product reaches 1396.  (The same with eight waves
// of 128 x 64, whose reads of LDS take half as long again: 1106 and, in two
// groups that take turns at reading and multiplying, 1145.)  128 x 128 takes 64
// accumulators and 64 KB, two blocks on a compute unit, for few rows.
//
// MFMA 16x16x32 (lane l = 16 g + i): A operand row i, k = 8 g .. 8 g + 7;
// B operand column i, the same k; D column i, rows 4 g .. 4 g + 3.  Here A is
// P and B is Q, so that a lane has four neighbours along a row of D.
#pragma once

#include "ops_common.hpp"

namespace wc {
namespace ops {

typedef __attribute__((address_space(3))) void lds_void;
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kTileK = 64;         // k of one stage
constexpr uint32_t kNowhere = 1u << 31;  // an offset past the end of every window

// What is the same in every lane, said so: a window in vector registers would be
// taken apart lane by lane at every load.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }
template <class P>
__device__ __forceinline__ const P *uniform(const P *p)
{
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    return reinterpret_cast<const P *>((uint64_t)uniform((uint32_t)(v >> 32)) << 32 | uniform((uint32_t)v));
}

// One operand of a tile: R rows (of D, or columns of it) by kTileK values of k,
// loaded 1024 bytes at a time, and every load in a place of its own in LDS.
// kAlong: k runs along the rows of memory, a load takes 8 rows of 128 bytes; 16-byte
// chunk c of row r lies where c ^ (r >> 1 & 7) would.  Otherwise k counts the rows
// of memory, and a load takes 512 / R rows of 2 R bytes.
template <int R, bool kAlong, int kWaves>
struct Operand {
    static_assert(R == 64 || R == 128 || R == 256, "and 64 only along");
    static constexpr uint32_t kLoads = R / 8 / kWaves;  // of each wave and stage
    static_assert(R / 8 % kWaves == 0, "whole loads");
    static constexpr uint32_t kRowsOfLoad = kAlong ? 8 : 512 / R;

    __device__ __forceinline__ static constexpr uint32_t place(uint32_t load)
    {
        if (kAlong) return load * 1024;
        if (R == 256) return load * 1088 + (load >> 2) * 128;
        return load * 1024 + (load >> 1) * 128;
    }
    static constexpr uint32_t kBytes = place(R / 8 - 1) + 1024;
    __device__ __forceinline__ static uint32_t swap(uint32_t k) { return R == 256 ? 2 * (k & 1) : 2 * (k & 3); }

    const char *base;
    uint32_t pitch;        // bytes, below 2^23
    uint32_t rows;         // of memory that exist
    uint32_t width;        // bytes of a row that exist
    uint32_t off[kLoads];  // the lane's in each load

    // kAlong: `from` is the tile's first row, `n` rows exist, each of `k` values.
    // Otherwise `from` is the tile's first column in row 0 of `n` rows of k;
    // `k` columns exist from there on.
    __device__ __forceinline__ void init(const void *from, uint64_t row_elems, uint32_t n, uint32_t k)
    {
        const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
        base = uniform(static_cast<const char *>(from));
        pitch = uniform(2 * (uint32_t)row_elems);
        rows = uniform(n);
        width = uniform(2 * k);
#pragma unroll
        for (uint32_t j = 0; j < kLoads; j++) {
            constexpr uint32_t kPerRow = 64 / kRowsOfLoad;  // lanes of a row
            const uint32_t r = (wave * kLoads + j) * kRowsOfLoad + lane / kPerRow;
            off[j] = r * pitch + 16 * ((lane % kPerRow) ^ (kAlong ? (r >> 1) & 7 : swap(r)));
        }
    }

    struct Stage {
        __amdgpu_buffer_rsrc_t window;  // what lies past it reads as zero
        uint32_t none[2];               // of every second load: past the window for lanes whose k do not exist
    };
    // The stage of k0 .. k0 + 63, of `k` values of k in all.
    __device__ __forceinline__ Stage stage(uint32_t k0, uint32_t k) const
    {
        Stage s;
        if constexpr (kAlong) {
            const uint32_t n = rows && k0 < k ? (rows - 1) * pitch + width - 2 * k0 : 0;
            s.window = __builtin_amdgcn_make_buffer_rsrc((void *)(base + 2ull * k0), 0, n, 0x00020000);
#pragma unroll
            for (uint32_t j = 0; j < 2; j++) {
                const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = (wave * kLoads + j) * 8 + (lane >> 3);
                s.none[j] = k0 + 8 * ((lane & 7) ^ ((r >> 1) & 7)) < k ? 0u : kNowhere;
            }
        } else {
            const uint32_t left = k0 < rows ? rows - k0 : 0, n = left ? (min(left, kTileK) - 1) * pitch + width : 0;
            s.window = __builtin_amdgcn_make_buffer_rsrc((void *)(base + (uint64_t)k0 * pitch), 0, n, 0x00020000);
        }
        return s;
    }
    __device__ __forceinline__ void load(const Stage &s, char *to, uint32_t wave, uint32_t j) const
    {
        const uint32_t at = kAlong ? off[j] | s.none[j & 1] : off[j];
        __builtin_amdgcn_raw_ptr_buffer_load_lds(s.window, (lds_void *)(to + place(wave * kLoads + j)), 16, at, 0, 0, 0);
    }

    // Sixteen rows from r0 on (a multiple of 16) and 32 values of k, half `sub` of the stage, in operand order.
    __device__ __forceinline__ static u32x4 operand(const char *from, uint32_t r0, uint32_t sub)
    {
        const uint32_t lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
        if constexpr (kAlong) {
            const uint32_t at = place(r0 / 8) + 128 * i + 16 * ((4 * sub + gr) ^ (i >> 1));
            return *reinterpret_cast<const u32x4 *>(from + at);
        } else {
            const uint32_t k = 32 * sub + 8 * gr + (i >> 2);
            const uint32_t at = place(k / kRowsOfLoad) + (k % kRowsOfLoad) * (2 * R) + 16 * ((r0 / 8 + ((i & 3) >> 1)) ^ swap(k)) +
                                8 * (i & 1);
            const uint32_t next = place((k + 4) / kRowsOfLoad) - place(k / kRowsOfLoad);
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(from + at));
            const s16x4 hi =
                __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(from + at + next));
            return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

// Blocks of a tile's kernel on a compute unit.
constexpr int tile_blocks(int BM, int BN) { return BM + BN > 384 ? 1 : 2; }

// A wave has every kWavesM-th 16 rows of Q and every kWavesN-th of P.
template <int T, int BM, int BN, bool kQAlong, bool kPAlong, int kStages = 2>
struct Tile {
    static constexpr int kWavesM = BM == 64 ? 1 : 2, kWavesN = 4 / kWavesM;
    static constexpr int kWaves = 4;
    static constexpr int kM = BM / kWavesM / 16, kN = BN / kWavesN / 16;
    using Q = Operand<BM, kQAlong, kWaves>;
    using P = Operand<BN, kPAlong, kWaves>;
    using X8 = typename Type<T>::x8;

    Q q;
    P p;
    f32x4 acc[kN][kM];

    // 256 accumulators of a lane are more than the compiler keeps in place by
    // itself: they are named as accumulation registers.
    static constexpr bool kNamed = kM * kN * 4 > 128;
    __device__ __forceinline__ static void mfma(X8 a, X8 b, f32x4 &c)
    {
        if constexpr (!kNamed) c = Type<T>::mfma(a, b, c);
        else if constexpr (T == WC_T_BF16) asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
        else asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
    }
    // The wait between the last of these and the first use of a result, which
    // the compiler puts in for its own products only (16 cycles each: the last one's passes and more).
    __device__ __forceinline__ void settle()
    {
        if constexpr (kNamed) {
#pragma unroll
            for (int a = 0; a < kN; a++)
#pragma unroll
                for (int b = 0; b < kM; b += 4)
                    asm volatile("s_nop 15" : "+a"(acc[a][b]), "+a"(acc[a][b + 1]), "+a"(acc[a][b + 2]), "+a"(acc[a][b + 3]));
        }
    }

    // Branches of the whole wave around products of rows that do not exist.  Not
    // where the accumulators are named: around branches the compiler moves
    // them, without the waits that it does not know of.  Not for 64 rows, where
    // reading P is the bound and the branches cost (61 rows of 128256 x 4096
    // against all of them: 207 us, 178 without).
    static constexpr bool kSkip = BM == 128;

    struct Half {  // operands of 32 values of k
        X8 p[kN], q[kM];
    };

    __device__ __forceinline__ static void read(Half &h, const char *qs, const char *ps, uint32_t wave, uint32_t sub, int n)
    {
        if (n < kN) h.p[n] = __builtin_bit_cast(X8, P::operand(ps, 16 * (wave % kWavesN) + 16 * kWavesN * n, sub));
        else h.q[n - kN] = __builtin_bit_cast(X8, Q::operand(qs, 16 * (wave / kWavesN) + 16 * kWavesM * (n - kN), sub));
    }
    static constexpr int kLoads = Q::kLoads + P::kLoads;
    struct Stage {
        typename Q::Stage q;
        typename P::Stage p;
    };
    __device__ __forceinline__ Stage begin(uint32_t k0, uint32_t k) const { return {q.stage(k0, k), p.stage(k0, k)}; }
    __device__ __forceinline__ void load(const Stage &s, char *qs, char *ps, uint32_t wave, int j) const
    {
        if (j < (int)Q::kLoads) q.load(s.q, qs, wave, j);
        else p.load(s.p, ps, wave, j - Q::kLoads);
    }

    // The products of h, with the reading of `into` spread among them, and
    // kEach loads of a later stage with each of the first ones.  Sixteens of
    // Q's rows from `live` on do not exist: tiles of 128 leave them out (kSkip).
    template <int kEach>
    __device__ __forceinline__ void multiply(const Half &h, Half &into, const char *qs, const char *ps, uint32_t sub,
                                             const Stage &s, char *ql, char *pl, uint32_t wave, int live)
    {
        constexpr int kReads = kM + kN, kProducts = kM * kN, kPer = kProducts / kReads;
        static_assert(!kEach || kEach * kReads >= kLoads, "all loads");
#pragma unroll
        for (int n = 0; n < kReads; n++) {
            if (!kSkip || n < kN || n - kN < live) read(into, qs, ps, wave, sub, n);
            if constexpr (kEach > 0) {
#pragma unroll
                for (int j = kEach * n; j < kEach * (n + 1); j++)
                    if (j < kLoads) load(s, ql, pl, wave, j);
            }
            if (!kSkip || n * kPer / kN < live) {
#pragma unroll
                for (int e = 0; e < kPer; e++) {
                    const int at = n * kPer + e;
                    mfma(h.p[at % kN], h.q[at / kN], acc[at % kN][at / kN]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int at = kReads * kPer; at < kProducts; at++) mfma(h.p[at % kN], h.q[at / kN], acc[at % kN][at / kN]);
    }

    static constexpr int kEach = (kLoads + kM + kN - 1) / (kM + kN);

    // The wait for reads of LDS, and for all loads but the last n.
    template <int n>
    __device__ __forceinline__ static void wait_all_but()
    {
        __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | 0x0070);
    }

    // One stage, whose first half is in h[0]; the next one has come at the end of
    // the first half, and the one kStages after it comes into its place.
    __device__ __forceinline__ void stage(Half *h, char *here, const char *next, uint32_t wave, int live, uint32_t k0, uint32_t k)
    {
        const Stage s = begin(k0 + kStages * kTileK, k);
        multiply<0>(h[0], h[1], here, here + Q::kBytes, 1, s, nullptr, nullptr, wave, live);
        wait_all_but<(kStages - 2) * kLoads>();
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        multiply<kEach>(h[1], h[0], next, next + Q::kBytes, 0, s, here, here + Q::kBytes, wave, live);
    }

    static constexpr uint32_t kBytes = Q::kBytes + P::kBytes;  // of a stage in LDS
    static constexpr uint32_t kThird = kStages == 3 ? kBytes : 16;

    // The product over k values of k, of `rows` of Q's rows.  s2: where kStages is 3.
    __device__ __forceinline__ void product(char *s0, char *s1, char *s2, uint32_t k, uint32_t rows = BM)
    {
        k = uniform(k);
        const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        // this wave's sixteens: wave / kWavesN, and every kWavesM-th after it
        const int sixteens = (int)((uniform(rows) + 15) / 16) - (int)(wave / kWavesN);
        const int live = sixteens <= 0 ? 0 : (sixteens + kWavesM - 1) / kWavesM;
#pragma unroll
        for (int a = 0; a < kN; a++)
#pragma unroll
            for (int b = 0; b < kM; b++) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = 0; n < kStages; n++) {
            const Stage s = begin(n * kTileK, k);
            char *to = n == 0 ? s0 : n == 1 ? s1 : s2;
#pragma unroll
            for (int j = 0; j < kLoads; j++) load(s, to, to + Q::kBytes, wave, j);
        }
        wait_all_but<(kStages - 1) * kLoads>();
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        Half h[2];
#pragma unroll
        for (int n = 0; n < kM + kN; n++) read(h[0], s0, s0 + Q::kBytes, wave, 0, n);
        uint32_t k0 = 0;
        if constexpr (kStages == 2) {
            for (; k0 + kTileK < k; k0 += 2 * kTileK) {
                stage(h, s0, s1, wave, live, k0, k);
                stage(h, s1, s0, wave, live, k0 + kTileK, k);
            }
            if (k0 < k) stage(h, s0, s1, wave, live, k0, k);
        } else {
            for (; k0 + 2 * kTileK < k; k0 += 3 * kTileK) {
                stage(h, s0, s1, wave, live, k0, k);
                stage(h, s1, s2, wave, live, k0 + kTileK, k);
                stage(h, s2, s0, wave, live, k0 + 2 * kTileK, k);
            }
            if (k0 < k) stage(h, s0, s1, wave, live, k0, k);
            if (k0 + kTileK < k) stage(h, s1, s2, wave, live, k0 + kTileK, k);
        }
        settle();
        wait_all_but<0>();  // loads past the last k have not landed before
        __syncthreads();
    }
};

// Block b of a grid of at least 8 ceil(n / 8) to one of n pieces of work, each
// of the 8 XCDs (every eighth block) with a contiguous range of them; n or more: none.
__device__ __forceinline__ uint32_t xcd_piece(uint32_t b, uint32_t n)
{
    const uint32_t per = (n + 7) / 8;
    return b / 8 < per ? (b % 8) * per + b / 8 : n;
}

// Piece t of rows x cols tiles, eight rows of tiles at a time, column by
// column, so that blocks that run together share their operands.
__device__ __forceinline__ void tile_of(uint32_t t, uint32_t rows, uint32_t cols, uint32_t &r, uint32_t &c)
{
    const uint32_t band = t / (8 * cols), at = t % (8 * cols), high = min(8u, rows - 8 * band);
    r = 8 * band + at % high;
    c = at / high;
}

// f(row of the tile, column, the four values of D from there on) for every four of this lane.
template <class Tile, class F>
__device__ __forceinline__ void each_four(const Tile &t, F f)
{
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, gr = lane >> 4;
#pragma unroll
    for (int b = 0; b < Tile::kM; b++)
#pragma unroll
        for (int a = 0; a < Tile::kN; a++)
            f(16 * (wave / Tile::kWavesN + Tile::kWavesM * b) + i,
              16 * (wave % Tile::kWavesN + Tile::kWavesN * a) + 4 * gr, t.acc[a][b]);
}

template <int T>
__device__ __forceinline__ void store_four(uint16_t *to, f32x4 v)
{
    uint64_t q = 0;
#pragma unroll
    for (int e = 0; e < 4; e++) q |= (uint64_t)Type<T>::from_f32(v[e]) << (16 * e);
    *reinterpret_cast<uint64_t *>(to) = q;
}

}  // namespace ops
}  // namespace wc
