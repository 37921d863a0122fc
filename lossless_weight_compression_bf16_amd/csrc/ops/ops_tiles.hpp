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

    // Where an operand lies.  kAlong: `base` is the tile's first row, `rows` exist, each
    // of width / 2 values of k.  Otherwise `base` is the tile's first column in
    // row 0 of `rows` rows of k, of which `width` bytes exist from there on.
    struct Where {
        const char *base;
        uint32_t rows, width;

        __device__ __forceinline__ Where said_uniform() const { return {uniform(base), uniform(rows), uniform(width)}; }
        __device__ __forceinline__ static Where at(const void *from, uint32_t n, uint32_t values)
        {
            return {static_cast<const char *>(from), n, 2 * values};
        }
    };

    uint32_t pitch;        // bytes, below 2^23
    uint32_t off[kLoads];  // the lane's in each load

    __device__ __forceinline__ void init(uint64_t row_elems)
    {
        const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
        pitch = uniform(2 * (uint32_t)row_elems);
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
    __device__ __forceinline__ Stage stage(const Where &w, uint32_t k0, uint32_t k) const
    {
        Stage s;
        if constexpr (kAlong) {
            const uint32_t n = w.rows && k0 < k ? (w.rows - 1) * pitch + w.width - 2 * k0 : 0;
            s.window = __builtin_amdgcn_make_buffer_rsrc((void *)uniform(w.base + 2ull * k0), 0, uniform(n), 0x00020000);
#pragma unroll
            for (uint32_t j = 0; j < 2; j++) {
                const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = (wave * kLoads + j) * 8 + (lane >> 3);
                s.none[j] = k0 + 8 * ((lane & 7) ^ ((r >> 1) & 7)) < k ? 0u : kNowhere;
            }
        } else {
            const uint32_t left = k0 < w.rows ? w.rows - k0 : 0, n = left ? (min(left, kTileK) - 1) * pitch + w.width : 0;
            s.window = __builtin_amdgcn_make_buffer_rsrc((void *)uniform(w.base + (uint64_t)k0 * pitch), 0, uniform(n), 0x00020000);
        }
        return s;
    }
    __device__ __forceinline__ void load(const Stage &s, char *to, uint32_t wave, uint32_t j, bool stream) const
    {
        const uint32_t at = kAlong ? off[j] | s.none[j & 1] : off[j];
        lds_void *const there = (lds_void *)(to + place(wave * kLoads + j));
        if (stream) __builtin_amdgcn_raw_ptr_buffer_load_lds(s.window, there, 16, at, 0, 0, 2);  // not to be kept in the caches
        else __builtin_amdgcn_raw_ptr_buffer_load_lds(s.window, there, 16, at, 0, 0, 0);
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

// A compute unit's blocks of a kernel of tiles.
constexpr int tile_blocks(int BM, int BN) { return BM + BN > 384 ? 1 : 2; }

// A wave has every kWavesM-th 16 rows of Q and every kWavesN-th 32 rows of P.
template <int T, int BM, int BN, bool kQAlong, bool kPAlong>
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
    struct Place {  // of a tile's operands, with k values of k
        typename Q::Where q;
        typename P::Where p;
        uint32_t k;

        __device__ __forceinline__ Place said_uniform() const { return {q.said_uniform(), p.said_uniform(), uniform(k)}; }
    };

    __device__ __forceinline__ Tile(uint64_t q_pitch, uint64_t p_pitch)
    {
        q.init(q_pitch);
        p.init(p_pitch);
    }

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

    // Tiles of 64 rows are bound by reading P, once and past the caches.  us of 61
    // rows on a vocabulary of 128256 x 4096 and of 122 rows of 8 experts of 14336 x
    // 4096: through the caches 208 and 167, past them 188 and 148, and with every
    // two blocks beginning at another stage 161 and 149.
    static constexpr bool kStreamP = BM == 64;

    // Branches of the whole wave around products of rows that do not exist.  Not
    // where the accumulators are named: around branches the compiler moves
    // them, without the waits that it does not know of.  Not for 64 rows, where
    // reading P is the bound and the branches cost (61 rows of 128256 x 4096
    // against all of them: 207 us, 178 without).
    static constexpr bool kSkip = BM == 128;

    // A result where it is used: until there it stays in its accumulation register.
    __device__ __forceinline__ f32x4 result(int a, int b) const
    {
        f32x4 v = acc[a][b];
        if constexpr (kNamed) asm volatile("" : "+a"(v));
        return v;
    }

    // The first row within the tile of the wave's b-th sixteen of Q, and of its a-th of P.
    __device__ __forceinline__ static constexpr uint32_t q_row(uint32_t wave, int b) { return 16 * (wave / kWavesN + kWavesM * b); }
    __device__ __forceinline__ static constexpr uint32_t p_row(uint32_t wave, int a)
    {
        return 32 * (wave % kWavesN + kWavesN * (a / 2)) + 16 * (a % 2);
    }

    struct Half {  // operands of 32 values of k
        X8 p[kN], q[kM];
    };

    __device__ __forceinline__ static void read(Half &h, const char *qs, const char *ps, uint32_t wave, uint32_t sub, int n)
    {
        if (n < kN) h.p[n] = __builtin_bit_cast(X8, P::operand(ps, p_row(wave, n), sub));
        else h.q[n - kN] = __builtin_bit_cast(X8, Q::operand(qs, q_row(wave, n - kN), sub));
    }
    static constexpr int kLoads = Q::kLoads + P::kLoads;
    struct Stage {
        typename Q::Stage q;
        typename P::Stage p;
    };
    __device__ __forceinline__ Stage begin(const Place &w, uint32_t k0) const { return {q.stage(w.q, k0, w.k), p.stage(w.p, k0, w.k)}; }
    __device__ __forceinline__ void load(const Stage &s, char *qs, char *ps, uint32_t wave, int j) const
    {
        if (j < (int)Q::kLoads) q.load(s.q, qs, wave, j, false);
        else p.load(s.p, ps, wave, j - Q::kLoads, kStreamP);
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

    // Every wave's reads of LDS, and its loads, are done.
    __device__ __forceinline__ static void all_done()
    {
        __builtin_amdgcn_s_waitcnt(0x0070);
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }

    static constexpr uint32_t kBytes = Q::kBytes + P::kBytes;  // of a stage in LDS

    // One stage, whose first half is in h[0]; the next one, in `next`, has come at
    // the end of the first half, and stage `s`, the one after it, comes into this one's place.
    __device__ __forceinline__ void stage(Half *h, char *here, const char *next, const Stage &s, uint32_t wave, int live)
    {
        multiply<0>(h[0], h[1], here, here + Q::kBytes, 1, s, nullptr, nullptr, wave, live);
        all_done();
        multiply<kEach>(h[1], h[0], next, next + Q::kBytes, 0, s, here, here + Q::kBytes, wave, live);
    }

    // The first two stages on their way, and the first half read.
    __device__ __forceinline__ void first(Stage s, const Stage &second, Half *h, char *s0, char *s1) const
    {
        const uint32_t wave = uniform(threadIdx.x >> 6);
#pragma unroll
        for (int j = 0; j < kLoads; j++) load(s, s0, s0 + Q::kBytes, wave, j);
        s = second;
#pragma unroll
        for (int j = 0; j < kLoads; j++) load(s, s1, s1 + Q::kBytes, wave, j);
        __builtin_amdgcn_s_waitcnt((kLoads & 15) | ((kLoads >> 4) << 14) | 0x0070);  // all but the second stage's
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < kM + kN; n++) read(h[0], s0, s0 + Q::kBytes, wave, 0, n);
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int a = 0; a < kN; a++)
#pragma unroll
            for (int b = 0; b < kM; b++) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
        settle();
    }

    // Where Q is a sum of kTerms matrices, `again` bytes apart: the sum of their products
    // with P, one after the other over all of k.

    // The product of a tile of which `rows` of Q's rows exist.  Where P is streamed,
    // blocks begin at different stages (pairs of an XCD's at the same one), so
    // that not all of them ask for the same columns of all rows at the same time.
    template <int kTerms>
    __device__ __forceinline__ void product(const Place &of, char *s0, char *s1, uint32_t rows, uint64_t again)
    {
        static_assert(kTerms == 1 || !kStreamP, "every term from its first stage on");
        const Place w = of.said_uniform();
        const uint32_t wave = uniform(threadIdx.x >> 6);
        // this wave's sixteens: wave / kWavesN, and every kWavesM-th after it
        const int sixteens = (int)((uniform(rows) + 15) / 16) - (int)(wave / kWavesN);
        const int live = sixteens <= 0 ? 0 : (sixteens + kWavesM - 1) / kWavesM;
        const uint32_t k = w.k, of_term = (k + kTileK - 1) / kTileK, stages = kTerms * of_term;
        uint32_t next = kStreamP && stages ? kTileK * (blockIdx.x / 16 % stages) : 0;
        uint32_t left = stages;  // whose loads have not been asked for
        auto turn = [&]() {      // the next stage; past the last k when there is none
            Place to = w;
            if (kTerms > 1) to.q.base += left > of_term ? 0 : again;
            const uint32_t at = left ? next : k;
            left -= left ? 1 : 0;
            next = next + kTileK < k ? next + kTileK : 0;
            return begin(to, at);
        };
        Half h[2];
        clear();
        const Stage a = turn(), b = turn();
        first(a, b, h, s0, s1);
        uint32_t n = 0;
        for (; n + 1 < stages; n += 2) {
            stage(h, s0, s1, turn(), wave, live);
            stage(h, s1, s0, turn(), wave, live);
        }
        if (n < stages) stage(h, s0, s1, turn(), wave, live);
        settle();
    }

    // The same within a row of tiles: the first half is in h[0] and the first two
    // stages are in s0 and s1, or on their way, and so are those of `next` when
    // this one is done.  Stages are taken by twos, at least two.
    template <int kTerms>
    __device__ __forceinline__ void product(const Place &of, const Place &after, Half *h, char *s0, char *s1, uint64_t again)
    {
        static_assert(kTerms <= 2, "one and another");
        const Place w = of.said_uniform(), next = after.said_uniform();
        const uint32_t wave = uniform(threadIdx.x >> 6), of_term = w.k > 2 * kTileK ? (w.k + 2 * kTileK - 1) / (2 * kTileK) : 1;
        const uint32_t most = kTerms * of_term;
        clear();
        for (uint32_t n = 1; n <= most; n++) {
            const bool last = n == most, second = kTerms > 1 && n >= of_term;
            Place to{last ? next.q : w.q, last ? next.p : w.p, last ? next.k : w.k};
            if (kTerms > 1) to.q.base += second && !last ? again : 0;
            const uint32_t k0 = last ? 0 : 2 * (second ? n - of_term : n) * kTileK;
            stage(h, s0, s1, begin(to, k0), wave, kM);
            stage(h, s1, s0, begin(to, k0 + kTileK), wave, kM);
        }
        settle();
    }
};

// The tiles of a block: job(n, j) gives its n-th, or none, and done(t, j) has its
// product.  Where a tile fills the compute unit (256 x 256) the block takes
// one after the other, a grid of kCus blocks, with the next one's first stages on their
// way before this one is stored; otherwise a block has one, and those beside it fill such gaps.
// again: between Q's two terms, where it has as many.
template <class Tile, class Job, int kTerms = 1, class Get, class Done>
__device__ __forceinline__ void each_tile(Tile &t, char *s0, char *s1, Get get, Done done, uint64_t again = 0)
{
    Job j;
    if (!get(0, j)) return;
    if constexpr (Tile::kNamed) {
        typename Tile::Half h[2];
        t.first(t.begin(j.place, 0), t.begin(j.place, kTileK), h, s0, s1);
        for (uint32_t n = 1;; n++) {
            Job next;
            const bool more = uniform((uint32_t)get(n, next)) != 0;
            if (!more) next.place = {{j.place.q.base, 0, 0}, {j.place.p.base, 0, 0}, 0};
            t.template product<kTerms>(j.place, next.place, h, s0, s1, again);
            done(t, j);
            if (!more) break;
            j = next;
        }
        __builtin_amdgcn_s_waitcnt(0x0070);
    } else {
        t.template product<kTerms>(j.place, s0, s1, j.rows, again);
        done(t, j);
    }
}

// A barrier for what the waves have written to LDS, which does not wait for loads.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("s_barrier" ::: "memory");
}


// The n-th piece of this block is that of block b of a grid of one piece a block.
__device__ __forceinline__ uint32_t block_of(uint32_t n) { return blockIdx.x + n * gridDim.x; }

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

// The lane's number, which the compiler does not know to be that of the last
// tile: it would compute all places of all results before the first tile, and
// have no registers for them.
__device__ __forceinline__ uint32_t lane_here()
{
    uint32_t lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    return lane;
}

// f(row of the tile, column, the four values of D from there on) for every four of this lane.
template <class Tile, class F>
__device__ __forceinline__ void each_four(const Tile &t, F f)
{
    const uint32_t wave = uniform(threadIdx.x >> 6), lane = lane_here(), i = lane & 15, gr = lane >> 4;
#pragma unroll
    for (int b = 0; b < Tile::kM; b++) {
#pragma unroll
        for (int a = 0; a < Tile::kN; a++) f(Tile::q_row(wave, b) + i, Tile::p_row(wave, a) + 4 * gr, t.result(a, b));
        __builtin_amdgcn_sched_barrier(0);  // or all accumulators are copied at once, for which there are no registers
    }
}

// Four numbers as 16-bit ones.
template <int T>
__device__ __forceinline__ uint64_t pack_four(f32x4 v)
{
    const float f[8] = {v[0], v[1], v[2], v[3], 0.f, 0.f, 0.f, 0.f};
    const u32x4 p = Type<T>::pack(f);
    return (uint64_t)p[1] << 32 | p[0];
}
template <int T>
__device__ __forceinline__ void store_four(uint16_t *to, f32x4 v)
{
    *reinterpret_cast<uint64_t *>(to) = pack_four<T>(v);
}

// f(row of the tile, column, eight 16-bit values of D from there on) for every eight of this lane, of
// what g(row, column, four of D) makes of D.  Lanes of neighbouring groups trade their
// halves of two sixteens, so that a lane stores 16 bytes and four of them
// 64 bytes of a row: half as many stores, of twice the length, as fours would take (dW of
// 100 rows on a vocabulary of 50257 x 768, 77 MB: 39.6 us, 31.0 so).
template <int T, class Tile, class G, class F>
__device__ __forceinline__ void each_eight(const Tile &t, G g, F f)
{
    const uint32_t wave = uniform(threadIdx.x >> 6), lane = lane_here(), i = lane & 15, gr = lane >> 4;
#pragma unroll
    for (int b = 0; b < Tile::kM; b++) {
        const uint32_t row = Tile::q_row(wave, b) + i;
#pragma unroll
        for (int a = 0; a < Tile::kN; a += 2) {
            const uint32_t col = Tile::p_row(wave, a);
            const uint64_t one = pack_four<T>(g(row, col + 4 * gr, t.result(a, b)));
            const uint64_t two = pack_four<T>(g(row, col + 16 + 4 * gr, t.result(a + 1, b)));
            // odd groups' `one` against even groups' `two`
            const auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)one, (uint32_t)two, false, false);
            const auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(one >> 32), (uint32_t)(two >> 32), false, false);
            f(row, col + 16 * (gr & 1) + 8 * (gr >> 1), u32x4{lo[0], hi[0], lo[1], hi[1]});
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}
// What the type leaves of four numbers, themselves packed in `of`; 0 where that is an infinity.
template <int T>
__device__ __forceinline__ f32x4 rest_of(f32x4 v, uint64_t of)
{
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const float had = Type<T>::to_f32((uint16_t)(of >> (16 * e)));
        v[e] = fabsf(had) < kInf ? v[e] - had : 0.f;
    }
    return v;
}
// The same as each_eight in two terms: f(row, column, eight values, eight of what they leave of D).
template <int T, class Tile, class G, class F>
__device__ __forceinline__ void each_eight_whole(const Tile &t, G g, F f)
{
    const uint32_t wave = uniform(threadIdx.x >> 6), lane = lane_here(), i = lane & 15, gr = lane >> 4;
    const auto swapped = [](uint64_t one, uint64_t two) {
        const auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)one, (uint32_t)two, false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(one >> 32), (uint32_t)(two >> 32), false, false);
        return u32x4{lo[0], hi[0], lo[1], hi[1]};
    };
#pragma unroll
    for (int b = 0; b < Tile::kM; b++) {
        const uint32_t row = Tile::q_row(wave, b) + i;
#pragma unroll
        for (int a = 0; a < Tile::kN; a += 2) {
            const uint32_t col = Tile::p_row(wave, a);
            const f32x4 u = g(row, col + 4 * gr, t.result(a, b)), v = g(row, col + 16 + 4 * gr, t.result(a + 1, b));
            const uint64_t one = pack_four<T>(u), two = pack_four<T>(v);
            const uint64_t rest = pack_four<T>(rest_of<T>(u, one)), rest2 = pack_four<T>(rest_of<T>(v, two));
            f(row, col + 16 * (gr & 1) + 8 * (gr >> 1), swapped(one, two), swapped(rest, rest2));
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}
struct AsIs {
    __device__ __forceinline__ f32x4 operator()(uint32_t, uint32_t, f32x4 v) const { return v; }
};

}  // namespace ops
}  // namespace wc
