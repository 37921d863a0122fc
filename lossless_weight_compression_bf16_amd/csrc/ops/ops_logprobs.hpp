// ops_logprobs.hpp -- log probabilities of given tokens, with the entropy and
// the most likely alternatives of every row, and their gradient.
//
//   lse = log sum_j exp z_j,  logprob = z_t - lse,  p_j = exp(z_j - lse)
//   H = -sum_j p_j log p_j = lse - sum_j p_j z_j
//   d logprob / d z_j = [j = t] - p_j,   d H / d z_j = -p_j (log p_j + H)
//
// One pass over the logits.  Every thread keeps the largest logit m it has
// seen, S = sum 2^d and W = sum 2^d d with d = (z - m) log2 e, and corrects S
// and W when a batch of 32 logits raises m:
//   S' = c S,  W' = c (W + delta S),  delta = (m - m') log2 e,  c = 2^delta.
// With the row's M, S, W: lse = M + ln S, H = ln S - ln 2 W / S.  The maximum
// is subtracted first: that is exact for the logits near it and 0 for itself,
// whatever their size.  (z log2 e - m log2 e in one fused operation leaves the
// rounding of m log2 e in every d: past 2^127 at m = 3e9.)
//
// The alternatives need no sort of the row.  Let T be the n-th largest of
// the maxima of 256 classes of threads: at least n logits are >= T, so every
// logit among the n largest is >= T (so a T a little lower does as well).
// The largest logit of every batch is kept in LDS, so
// the logits >= T are found by looking again at the batches whose maximum is
// >= T only (about n of V / 32), and ranked by counting.  Rows with so many
// equal logits that the lists overflow take the scan of top_slow.
//
// Order of the alternatives: larger logits first, equal ones (-0 = 0) by
// their index, NaN after everything else.
#pragma once

#include "ops_common.hpp"

namespace wc {
namespace ops {

constexpr uint32_t kJoinThreads = 256;
constexpr uint32_t kBatch = 32;                          // logits a thread takes per round
constexpr uint32_t kMaxSlice = 131072;                   // logits of one block
constexpr uint32_t kMaxSlices = 64;                      // blocks of one row
constexpr uint32_t kClasses = 256;                       // groups of threads whose maxima give the threshold
constexpr uint32_t kMaxTop = 64;
constexpr uint32_t kMaxVocab = kMaxSlice * kMaxSlices / 2;
constexpr uint32_t kListCap = 1024;                      // candidates ranked by counting
constexpr float kFloor = -1e30f;                         // a thread's maximum before its first logit

// Softmax statistics in base 2: see the file's comment.
struct Stat {
    float m, s, w;
};
__device__ __forceinline__ void raise(Stat &a, float m)  // m >= a.m
{
    const float delta = fmaxf((a.m - m) * kLog2e, kFloor);  // finite, so that a zero S stays zero
    const float c = exp2_fast(delta);
    a.w = c * (a.w + delta * a.s);
    a.s = c * a.s;
    a.m = m;
}
__device__ __forceinline__ Stat merge(Stat a, Stat b)
{
    const float m = fmaxf(a.m, b.m);
    raise(a, m);
    raise(b, m);
    return Stat{m, a.s + b.s, a.w + b.w};
}

template <bool kTop, bool kSlice, int NT_>
struct RowShared {
    static constexpr uint32_t NT = NT_;  // threads of the block
    uint64_t list[kTop ? kListCap : 1];                               // candidates: key << 32 | ~index
    uint32_t batch_max[kTop && kSlice ? kMaxSlice / kBatch : 1];      // bits of the largest logit of batch NT i + thread
    uint32_t hits[kTop && kSlice ? kListCap : 1];                     // batches to look at again
    uint32_t keys[kTop && kSlice ? kClasses : 4];
    float part[3 * (NT / 64)];
    uint64_t thresh64;
    uint32_t thresh, n_list, n_hits, wave_count[NT / 64];
};

__device__ __forceinline__ uint64_t entry(uint32_t key, uint32_t index) { return ((uint64_t)key << 32) | (uint32_t)~index; }

// The wave's statistics, in every lane.
__device__ __forceinline__ Stat wave_stat(Stat a)
{
    raise(a, wave_max(a.m));
    return Stat{a.m, wave_sum(a.s), wave_sum(a.w)};
}

// The block's statistics, in every thread.
template <class Sh>
__device__ inline Stat block_stat(Stat a, Sh &sh)
{
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    a = wave_stat(a);
    if (lane == 0) {
        sh.part[3 * wave] = a.m;
        sh.part[3 * wave + 1] = a.s;
        sh.part[3 * wave + 2] = a.w;
    }
    __syncthreads();
    a = Stat{-kInf, 0.f, 0.f};
    if (lane < Sh::NT / 64) a = Stat{sh.part[3 * lane], sh.part[3 * lane + 1], sh.part[3 * lane + 2]};
    return wave_stat(a);
}

// A key that at least n of the 256 classes of threads reach (0 if fewer than
// n have one), and hardly more: the n-th largest, or a lower one if at most
// 64 and n + 8 classes reach it.  A class is a thread, or four threads side by
// side, and its key the largest of theirs.  Found by bisection between the
// smallest and the largest, every wave counting all classes by itself.
template <class Sh>
__device__ inline uint32_t nth_key(uint32_t key, uint32_t n, Sh &sh)
{
    constexpr uint32_t kPer = Sh::NT / kClasses;
    if constexpr (kPer == 4) {
        key = max(key, lanes_moved<0xB1, 0xF>(key, 0u));  // lanes 1 0 3 2 of each four
        key = max(key, lanes_moved<0x4E, 0xF>(key, 0u));  // lanes 2 3 0 1
    }
    static_assert(kPer == 1 || kPer == 4, "classes");
    if (threadIdx.x % kPer == 0) sh.keys[threadIdx.x / kPer] = key;
    __syncthreads();
    const u32x4 k = *reinterpret_cast<const u32x4 *>(&sh.keys[4 * (threadIdx.x & 63)]);
    auto reach = [&](uint32_t c) {
        return (uint32_t)(__popcll(__ballot(k[0] >= c)) + __popcll(__ballot(k[1] >= c)) +
                          __popcll(__ballot(k[2] >= c)) + __popcll(__ballot(k[3] >= c)));
    };
    const uint32_t few = min(n + 8, 64u);
    uint32_t count = reach(1u);
    if (count < n) return 0;
    // none of the keys is below lo but 0; count classes reach lo, fewer than n reach hi + 1
    uint32_t lo = wave_min(min(min(k[0] - 1, k[1] - 1), min(k[2] - 1, k[3] - 1))) + 1;
    uint32_t hi = ~wave_min(min(min(~k[0], ~k[1]), min(~k[2], ~k[3])));
    while (count > few && lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2, c = reach(mid);
        if (c >= n) {
            lo = mid;
            count = c;
        } else {
            hi = mid - 1;
        }
    }
    return lo;
}

// Writes the n largest entries of the list, in order; fewer entries than n
// leave zeros.
template <class Sh, class Put>
__device__ inline void rank_list(uint32_t count, uint32_t n, const Sh &sh, Put put)
{
    for (uint32_t i = threadIdx.x; i < count; i += Sh::NT) {
        const uint64_t mine = sh.list[i];
        uint32_t above = 0;
#pragma unroll 4
        for (uint32_t j = 0; j < count; j++) above += sh.list[j] > mine;
        if (above < n) put(above, mine);
    }
    for (uint32_t i = count + threadIdx.x; i < n; i += Sh::NT) put(i, 0ull);
}

// Adds to the list, in the order of the index, the first elements of
// [lo, hi) whose key is `key` until it holds n entries; the new count.
template <int T, class Sh>
__device__ inline uint32_t fill_equal(const typename Type<T>::elem *row, uint32_t lo, uint32_t hi, uint32_t n,
                                      uint32_t count, uint32_t key, Sh &sh)
{
    const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    for (uint32_t j0 = lo; count < n && j0 < hi; j0 += Sh::NT) {
        const uint32_t j = j0 + threadIdx.x;
        const bool eq = j < hi && key_of(Type<T>::to_f32(row[j])) == key;
        const uint64_t votes = __ballot(eq);
        if (lane == 0) sh.wave_count[wave] = (uint32_t)__popcll(votes);
        __syncthreads();
        uint32_t at = count + (uint32_t)__popcll(votes & ((1ull << lane) - 1)), total = 0;
        for (uint32_t i = 0; i < Sh::NT / 64; i++) {
            if (i < wave) at += sh.wave_count[i];
            total += sh.wave_count[i];
        }
        if (eq && at < n) sh.list[at] = entry(key, j);
        count = min(count + total, n);
        __syncthreads();
    }
    return count;
}

// The candidates where more elements than the list holds are above `thresh`,
// a key that at least n elements reach: the n-th largest of those in the
// list is a higher key that n elements reach, and the scan starts again from
// there.  The key grows every time, so this ends; it takes rows in which few
// threads hold more than a thousand of the largest logits.
template <int T, class Sh>
__device__ __noinline__ uint32_t top_slow(const typename Type<T>::elem *row, uint32_t lo, uint32_t hi, uint32_t n,
                                          uint32_t thresh, Sh &sh)
{
    for (;;) {
        __syncthreads();
        if (threadIdx.x == 0) {
            sh.n_list = 0;
            sh.thresh = ~0u;
        }
        __syncthreads();
        for (uint32_t j = lo + threadIdx.x; j < hi; j += Sh::NT) {
            const uint32_t key = key_of(Type<T>::to_f32(row[j]));
            if (key > thresh) {
                const uint32_t at = atomicAdd(&sh.n_list, 1u);
                if (at < kListCap) sh.list[at] = entry(key, j);
            }
        }
        __syncthreads();
        const uint32_t count = lds_uniform(sh.n_list);
        if (count <= kListCap) return fill_equal<T>(row, lo, hi, n, count, thresh, sh);
        for (uint32_t i = threadIdx.x; i < kListCap; i += Sh::NT) {
            const uint32_t key = (uint32_t)(sh.list[i] >> 32);
            uint32_t above = 0;
            for (uint32_t j = 0; j < kListCap; j++) above += (uint32_t)(sh.list[j] >> 32) > key;
            if (above < n) atomicMin(&sh.thresh, key);
        }
        __syncthreads();
        thresh = lds_uniform(sh.thresh);
    }
}

// Collects the elements of [lo, hi) whose key is at least `limit` from the
// batches that have one.  False if they are too many for the lists.
template <int T, class Sh>
__device__ inline bool collect(const typename Type<T>::elem *row, uint32_t lo, uint32_t hi, uint32_t rounds,
                               uint32_t limit, Sh &sh)
{
    using Ty = Type<T>;
    constexpr uint32_t kPer = Ty::kPer16, kVecs = kBatch / kPer, kSweep = Sh::NT * kBatch;
    const uint32_t tid = threadIdx.x;
    __syncthreads();
    if (tid == 0) sh.n_list = sh.n_hits = 0;
    __syncthreads();
#pragma unroll 4
    for (uint32_t i = 0; i < rounds; i++) {
        if (key_of(__builtin_bit_cast(float, sh.batch_max[Sh::NT * i + tid])) >= limit) {
            const uint32_t at = atomicAdd(&sh.n_hits, 1u);
            if (at < kListCap) sh.hits[at] = Sh::NT * i + tid;
        }
    }
    __syncthreads();
    const uint32_t hits = lds_uniform(sh.n_hits);
    if (hits > kListCap) return false;
    for (uint32_t i = tid; i < hits * kVecs; i += Sh::NT) {
        const uint32_t b = sh.hits[i / kVecs];
        const uint32_t j = lo + (b / Sh::NT) * kSweep + (Sh::NT * (i % kVecs) + b % Sh::NT) * kPer;
        float f[kPer];
        if (j + kPer <= hi) {
            Ty::unpack(load16<Ty::kBytes>(row + j), f);
        } else {
#pragma unroll
            for (uint32_t q = 0; q < kPer; q++) f[q] = j + q < hi ? Ty::to_f32(row[j + q]) : 0.f;
        }
        uint32_t has = 0;
#pragma unroll
        for (uint32_t q = 0; q < kPer; q++) has |= (j + q < hi && key_of(f[q]) >= limit) ? 1u << q : 0u;
        if (has) {
            uint32_t at = atomicAdd(&sh.n_list, (uint32_t)__popc(has));
#pragma unroll
            for (uint32_t q = 0; q < kPer; q++)
                if ((has >> q) & 1) {
                    if (at < kListCap) sh.list[at] = entry(key_of(f[q]), j + q);
                    at++;
                }
        }
    }
    __syncthreads();
    return lds_uniform(sh.n_list) <= kListCap;
}

// The candidates of a slice where many logits equal the threshold (a masked
// row), or fewer than n are above -inf: those above it (in the batches of at
// most 64 classes, 16 of each), then the first that equal it, then NaN.
template <int T, class Sh>
__device__ __noinline__ uint32_t candidates_many(const typename Type<T>::elem *row, uint32_t lo, uint32_t hi,
                                                 uint32_t rounds, uint32_t thresh, uint32_t n, Sh &sh)
{
    if (!collect<T>(row, lo, hi, rounds, thresh + 1, sh)) return top_slow<T>(row, lo, hi, n, thresh, sh);
    uint32_t count = lds_uniform(sh.n_list);
    for (uint32_t key = thresh;; key = 1u) {
        count = fill_equal<T>(row, lo, hi, n, count, key, sh);
        if (key != key_of(-kInf)) return count;
    }
}

// The candidates of a slice in sh.list: their number.  best: the key of the
// thread's largest logit (0: it had none).
template <int T, class Sh>
__device__ inline uint32_t candidates(const typename Type<T>::elem *row, uint32_t lo, uint32_t hi, uint32_t rounds,
                                      uint32_t best, uint32_t n, Sh &sh)
{
    const uint32_t none = key_of(-kInf);
    const uint32_t thresh = max(nth_key(best, n, sh), none);
    if (thresh > none && collect<T>(row, lo, hi, rounds, thresh, sh)) return lds_uniform(sh.n_list);
    return candidates_many<T>(row, lo, hi, rounds, thresh, n, sh);
}

// Statistics of elements [lo, hi) of a row, in every thread, and with kTop
// the number of candidates in sh.list.  All rounds run the same code (a
// second copy for the last, partial one costs a short row more in fetching
// instructions than it saves): a vector that crosses the end is read ending
// there, and what is not its own counts as -inf.
template <int T, bool kTop, class Sh>
__device__ inline Stat slice_pass(const typename Type<T>::elem *row, uint32_t lo, uint32_t hi, uint32_t n, Sh &sh,
                                  uint32_t *count)
{
    using Ty = Type<T>;
    constexpr uint32_t kPer = Ty::kPer16, kVecs = kBatch / kPer;
    constexpr uint32_t kSweep = Sh::NT * kBatch;  // logits of a round of the block
    const uint32_t tid = threadIdx.x;
    Stat a{kFloor, 0.f, 0.f};
    float best = -kInf;   // the largest of the thread's batches
    uint32_t round = 0;
    u32x4 cur[kVecs], nxt[kVecs];
    // a round's vector u of a thread: elements base + (NT u + tid) kPer ..
    // Past the caches with 256 threads, that is, where rows are many: us past
    // them and through them, BF16, 2048 rows of 128256 93 and 104, 512 rows 32
    // and 33, 1024 rows of 32000 21.4 and 21.1, 1000 of 8192 13.6 both.
    auto fetch = [&](u32x4 *v, uint32_t base) {
#pragma unroll
        for (uint32_t u = 0; u < kVecs; u++)
            v[u] = read16<Ty::kBytes, Sh::NT == 256>(row + min(base + (Sh::NT * u + tid) * kPer, hi - kPer));
    };
    const bool tiny = hi < kPer;  // a row shorter than a vector
    if (!tiny) fetch(cur, lo);
    for (uint32_t base = lo; base < hi; base += kSweep, round++) {
        if (hi - base > kSweep) fetch(nxt, base + kSweep);
        float f[kBatch];
        if (!tiny) {
#pragma unroll
            for (uint32_t u = 0; u < kVecs; u++) Ty::unpack(cur[u], f + kPer * u);
            if (hi - base < kSweep) {
#pragma unroll
                for (uint32_t u = 0; u < kVecs; u++) {
                    const uint32_t j = base + (Sh::NT * u + tid) * kPer, at = min(j, hi - kPer);
#pragma unroll
                    for (uint32_t i = 0; i < kPer; i++) f[kPer * u + i] = at + i >= j ? f[kPer * u + i] : -kInf;
                }
            }
        } else {
#pragma unroll
            for (uint32_t i = 0; i < kBatch; i++) f[i] = i < kPer && tid == 0 && i < hi ? Ty::to_f32(row[i]) : -kInf;
        }
        float bmax = f[0];
#pragma unroll
        for (uint32_t i = 1; i < kBatch; i++) bmax = fmaxf(bmax, f[i]);
        if (bmax > a.m) raise(a, bmax);
#pragma unroll
        for (uint32_t i = 0; i < kBatch; i++) {
            const float d = (f[i] - a.m) * kLog2e;
            const float e = exp2_fast(d);
            a.s += e;
            a.w = __builtin_fmaf(e, fmaxf(d, -1000.f), a.w);  // a masked logit adds 0 * -1000, not 0 * -inf
        }
        if constexpr (kTop) {
            // a batch of nothing but NaN counts as -inf: its elements are looked at if the threshold is that low
            bmax = fmaxf(bmax, -kInf);
            sh.batch_max[Sh::NT * round + tid] = __builtin_bit_cast(uint32_t, bmax);
            best = fmaxf(best, bmax);
        }
#pragma unroll
        for (uint32_t u = 0; u < kVecs; u++) cur[u] = nxt[u];
    }
    if constexpr (kTop) *count = candidates<T>(row, lo, hi, round, lo + tid * kPer < hi ? key_of(best) : 0u, n, sh);
    return block_stat(a, sh);
}

// A row's statistics with its true maximum, by the whole block: for rows
// whose logits are all below kFloor, and for the gradient.
template <int T, class Sh>
__device__ __noinline__ Stat exact_stat(const typename Type<T>::elem *row, uint32_t vocab, Sh &sh)
{
    __syncthreads();
    float m = -kInf;
    for (uint32_t j = threadIdx.x; j < vocab; j += Sh::NT) m = fmaxf(m, Type<T>::to_f32(row[j]));
    m = block_stat(Stat{m, 0.f, 0.f}, sh).m;
    Stat b{0.f, 0.f, 0.f};
    for (uint32_t j = threadIdx.x; j < vocab; j += Sh::NT) {
        const float d = (Type<T>::to_f32(row[j]) - m) * kLog2e;
        const float e = m == -kInf ? 0.f : exp2_fast(d);
        b.s += e;
        b.w += e > 0.f ? e * d : 0.f;
    }
    __syncthreads();
    b = block_stat(b, sh);
    return Stat{m, b.s, b.w};
}

struct LogprobArgs {
    const void *logits;
    uint64_t stride;
    const int64_t *tokens;
    uint32_t vocab, top, slices, slice;  // slice: logits per block, a multiple of 8
    float *logprob, *entropy, *lse, *top_logprobs;
    int64_t *top_ids;
    float *part;        // (row, slice): M, S, W and a spare, when slices > 1
    uint64_t *part_top; // (row, slice): the slice's top entries in order
    uint32_t *err;
};

// Writes a row's statistics; returns its lse for the alternatives.  Called
// by the whole block; z is the logit of the row's token t.  S is 0 where every
// logit is below kFloor (masks of the type's lowest value in a whole row, -inf
// in a whole row): such a row is computed again with its true maximum.
template <int T, class Sh>
__device__ inline float write_row(const LogprobArgs &g, uint64_t r, Stat a, int64_t t, float z, Sh &sh)
{
    using Ty = Type<T>;
    const typename Ty::elem *row = static_cast<const typename Ty::elem *>(g.logits) + r * g.stride;
    float lse, entropy;
    if (a.s == 0.f) a = exact_stat<T>(row, g.vocab, sh);
    if (a.s == 0.f) {  // nothing but -inf: no token is possible
        lse = -kInf;
        entropy = 0.f;
    } else if (!(a.s < kInf)) {  // a NaN or +inf among the logits
        lse = entropy = nan32();
    } else {
        const float ln_s = __logf(a.s);
        lse = a.m + ln_s;
        entropy = fmaxf(ln_s - kLn2 * (a.w / a.s), 0.f);
    }
    if (threadIdx.x == 0) {
        float lp = 0.f;
        if (t >= 0 && t < (int64_t)g.vocab) {
            lp = z == -kInf && lse == lse ? -kInf : z - lse;
        } else if (t != -1) {
            lp = nan32();
            report(g.err, WC_EF_BAD_INDEX);
        }
        g.logprob[r] = lp;
        g.entropy[r] = entropy;
        g.lse[r] = lse;
    }
    return lse;
}

__device__ __forceinline__ void put_top(const LogprobArgs &g, uint64_t r, uint32_t at, uint64_t e, float lse)
{
    const float z = key_value((uint32_t)(e >> 32));
    g.top_logprobs[r * g.top + at] = z == -kInf && lse == lse ? -kInf : z - lse;
    g.top_ids[r * g.top + at] = (int64_t)(uint32_t)~(uint32_t)e;
}

// A row's token and its logit (0 for none), read before anything else.
template <int T>
__device__ __forceinline__ float given_logit(const LogprobArgs &g, uint64_t r, int64_t &t)
{
    t = g.tokens[r];
    if (t < 0 || t >= (int64_t)g.vocab) return 0.f;
    return Type<T>::to_f32(static_cast<const typename Type<T>::elem *>(g.logits)[r * g.stride + t]);
}

// One block per slice of a row; with one slice it writes the row.  Many rows:
// reading them is the bound (2048 rows of 128256 in BF16, 5 best: 94 us a call
// in a row of calls, 5.6 TB/s, 101 under a kernel trace; 7.1 is what reading
// alone reaches), and 256 threads a row leave room for the blocks that hide
// one another's choice of the best.  Few rows: the passes over a row by its one
// block, for which 1024 threads are there (64 rows, 20 best: 17 us; one row of
// 50257, FP32: 9.8 us).
template <int T, bool kTop, int NT>
__global__ __launch_bounds__(NT) void k_logprobs(LogprobArgs g)
{
    __shared__ RowShared<kTop, true, NT> sh;
    const uint64_t r = blockIdx.x / g.slices;
    const uint32_t s = blockIdx.x % g.slices;
    const typename Type<T>::elem *row = static_cast<const typename Type<T>::elem *>(g.logits) + r * g.stride;
    const uint32_t lo = s * g.slice, hi = min(g.vocab, lo + g.slice);
    uint32_t count = 0;
    int64_t token;
    const float z = given_logit<T>(g, r, token);
    const Stat a = slice_pass<T, kTop>(row, lo, hi, g.top, sh, &count);
    if (g.slices == 1) {
        const float lse = write_row<T>(g, r, a, token, z, sh);
        if constexpr (kTop) rank_list(count, g.top, sh, [&](uint32_t at, uint64_t e) { put_top(g, r, at, e, lse); });
        return;
    }
    if (threadIdx.x == 0) *reinterpret_cast<f32x4 *>(g.part + 4 * (uint64_t)blockIdx.x) = f32x4{a.m, a.s, a.w, 0.f};
    if constexpr (kTop)
        rank_list(count, g.top, sh, [&](uint32_t at, uint64_t e) { g.part_top[(uint64_t)blockIdx.x * g.top + at] = e; });
}

// Joins the slices of a row: one block per row.  The n largest of the
// slices' lists are found as in a slice, T being the n-th largest of the
// threads' largest entries.  No two entries are equal, so exactly n threads
// hold entries >= T, and a thread holds at most 16 (64 slices x 64 / 256).
template <int T, bool kTop>
__global__ __launch_bounds__(kJoinThreads) void k_logprobs_join(LogprobArgs g)
{
    __shared__ RowShared<kTop, false, kJoinThreads> sh;
    static_assert(kMaxSlices * kMaxTop / kJoinThreads * kMaxTop <= kListCap, "the join's list");
    const uint32_t tid = threadIdx.x;
    const uint64_t r = blockIdx.x;
    Stat a{kFloor, 0.f, 0.f};
    if (tid < g.slices) {
        const f32x4 p = *reinterpret_cast<const f32x4 *>(g.part + 4 * (r * g.slices + tid));
        a = Stat{p[0], p[1], p[2]};
    }
    int64_t token;
    const float z = given_logit<T>(g, r, token);
    a = block_stat(a, sh);
    const float lse = write_row<T>(g, r, a, token, z, sh);
    if constexpr (kTop) {
        const uint64_t *tops = g.part_top + r * g.slices * g.top;
        const uint32_t total = g.slices * g.top;
        uint64_t best = 0;
        for (uint32_t i = tid; i < total; i += kJoinThreads) best = max(best, tops[i]);
        sh.list[tid] = best;
        if (tid == 0) {
            sh.thresh64 = ~0ull;
            sh.n_list = 0;
        }
        __syncthreads();
        uint32_t above = 0;
        for (uint32_t i = 0; i < kJoinThreads; i++) above += sh.list[i] > best;
        if (above < g.top) atomicMin(reinterpret_cast<unsigned long long *>(&sh.thresh64), (unsigned long long)best);
        __syncthreads();
        const uint64_t thresh = sh.thresh64;
        for (uint32_t i = tid; i < total; i += kJoinThreads) {
            const uint64_t e = tops[i];
            if (e && e >= thresh) sh.list[atomicAdd(&sh.n_list, 1u)] = e;
        }
        __syncthreads();
        rank_list(lds_uniform(sh.n_list), g.top, sh, [&](uint32_t at, uint64_t e) { put_top(g, r, at, e, lse); });
    }
}

// The gradient: with g and h the gradients of a row's log probability and
// entropy, dz_j = g [j = t] - p_j (g + h (log p_j + H)), one pass that reads
// and writes every logit once; a thread takes 32 of them per round.  Every
// element is read and written by one thread, the read first, so dz may be
// the logits' own memory.  Reading and writing is the bound: 2048 rows of
// 128256 in BF16, masked, 180 us, 5.8 TB/s of both, where a copy of as much
// reaches 6.5; 100 rows of 50257 in FP32 10.4 us.
//
// log p_j = z_j - lse; an lse of 2^16 or more (a row of nothing but the
// type's lowest value, say) has no bits left for the probabilities in 32
// bits, so such a row's maximum and log of the sum are computed again.  That
// reads the whole row: in the logits' own memory a row has only one block.
constexpr uint32_t kGradThreads = 256;

struct LogprobGradArgs {
    const void *logits;
    void *out;
    uint64_t stride, out_stride;
    const int64_t *tokens;
    const float *lse, *entropy, *grad_logprob, *grad_entropy;  // the gradients may be null: zero
    uint32_t vocab, blocks;                                    // blocks per row
    uint32_t *err;
};

template <int T, bool kStream>
__global__ __launch_bounds__(kGradThreads) void k_logprobs_grad(LogprobGradArgs a)
{
    using Ty = Type<T>;
    using E = typename Ty::elem;
    constexpr int kPer = Ty::kPer16, kVecs = kBatch / kPer;
    constexpr uint32_t kSweep = kGradThreads * kBatch;
    const uint64_t r = blockIdx.x / a.blocks;
    const uint32_t first = (blockIdx.x % a.blocks) * kSweep, tid = threadIdx.x;
    const E *row = static_cast<const E *>(a.logits) + r * a.stride;
    __shared__ RowShared<false, true, kGradThreads> sh;
    E *out = static_cast<E *>(a.out) + r * a.out_stride;
    const int64_t t64 = a.tokens[r];
    const bool given = t64 >= 0 && t64 < (int64_t)a.vocab;
    if (!given && t64 != -1 && first == 0 && tid == 0) report(a.err, WC_EF_BAD_INDEX);
    const uint32_t t = given ? (uint32_t)t64 : ~0u;
    float g = given && a.grad_logprob ? a.grad_logprob[r] : 0.f;
    float h = a.grad_entropy ? a.grad_entropy[r] : 0.f;
    float lse = a.lse[r];
    if (lse == -kInf) {  // nothing but -inf: constant outputs, no gradient
        g = h = 0.f;
        lse = kInf;  // every p becomes exp(-inf) = 0
    }
    float shift = 0.f;
    if (fabsf(lse) >= 65536.f && fabsf(lse) < kInf) {
        const Stat st = exact_stat<T>(row, a.vocab, sh);
        lse = st.m;
        shift = __logf(st.s);
    }
    const float gh = __builtin_fmaf(h, h != 0.f ? a.entropy[r] : 0.f, g);
    auto grad = [&](float z, uint32_t j) {
        const float lp = (z - lse) - shift;
        const float p = exp2_fast(lp * kLog2e);
        const float d = -p * __builtin_fmaf(h, fmaxf(lp, -200.f), gh);  // p is 0 below -104: 0 times a finite number
        return j == t ? d + g : d;
    };
    for (uint32_t base = first; base < a.vocab; base += a.blocks * kSweep) {
        uint32_t at[kVecs];
        u32x4 v[kVecs];
#pragma unroll
        for (int u = 0; u < kVecs; u++) {
            at[u] = base + (kGradThreads * u + tid) * kPer;
            if (at[u] + kPer <= a.vocab) v[u] = read16<Ty::kBytes, kStream>(row + at[u]);
        }
#pragma unroll
        for (int u = 0; u < kVecs; u++) {
            if (at[u] + kPer <= a.vocab) {
                float f[kPer];
                Ty::unpack(v[u], f);
#pragma unroll
                for (int i = 0; i < kPer; i++) f[i] = grad(f[i], at[u] + i);
                write16<Ty::kBytes, kStream>(out + at[u], Ty::pack(f));
            } else {
                for (int i = 0; i < kPer; i++)
                    if (at[u] + i < a.vocab) out[at[u] + i] = Ty::from_f32(grad(Ty::to_f32(row[at[u] + i]), at[u] + i));
            }
        }
    }
}

}  // namespace ops
}  // namespace wc
