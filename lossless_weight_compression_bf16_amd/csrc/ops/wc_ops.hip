// wc_ops.hip -- C ABI of the operators beside the compressed weights (see
// include/wc.h): argument checks, launch shapes and scratch layout.  Like
// the codec's calls these only enqueue on the caller's stream; no
// allocation, no synchronisation, no global state.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wc.h"
#include "ops_common.hpp"
#include "ops_logprobs.hpp"

using namespace wc::ops;

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }
constexpr uint64_t kMaxGrid = 0x7FFFFFFFull;

bool valid_type(uint32_t t) { return t <= WC_T_FP32; }
uintptr_t type_bytes(uint32_t t) { return t == WC_T_FP32 ? 4 : 2; }

wc_status launched() { return hipGetLastError() == hipSuccess ? WC_OK : WC_ERR_HIP; }

// Blocks of a row of the log probabilities.  A block's first round is 8,192
// logits, but with few rows more, smaller blocks fill the GPU better: 4 per
// compute unit, at least 2,048 logits each.
void logprob_slices(uint64_t m, uint32_t vocab, uint32_t *slices, uint32_t *slice)
{
    uint64_t s = ceil_div(4 * kCus, m);
    const uint64_t most = ceil_div(vocab, kMinSlice);
    if (s > most) s = most;
    if (s > kMaxSlices) s = kMaxSlices;
    const uint64_t least = ceil_div(vocab, kMaxSlice);
    if (s < least) s = least;
    *slice = (uint32_t)((ceil_div(vocab, s) + 7) / 8 * 8);
    *slices = (uint32_t)ceil_div(vocab, *slice);
}

uint64_t logprob_scratch(uint64_t m, uint32_t vocab, uint32_t top)
{
    uint32_t slices, slice;
    logprob_slices(m, vocab, &slices, &slice);
    return slices == 1 ? 0 : m * slices * (16 + 8ull * top);
}

template <int T>
wc_status launch_logprobs(const LogprobArgs &g, uint64_t m, hipStream_t stream)
{
    const dim3 grid((uint32_t)(m * g.slices)), block(kRowThreads);
    if (g.top) hipLaunchKernelGGL((k_logprobs<T, true>), grid, block, 0, stream, g);
    else hipLaunchKernelGGL((k_logprobs<T, false>), grid, block, 0, stream, g);
    if (g.slices > 1) {
        if (g.top) hipLaunchKernelGGL((k_logprobs_join<T, true>), dim3((uint32_t)m), block, 0, stream, g);
        else hipLaunchKernelGGL((k_logprobs_join<T, false>), dim3((uint32_t)m), block, 0, stream, g);
    }
    return launched();
}

}  // namespace

extern "C" {

uint64_t wc_token_logprobs_scratch(uint64_t m, uint32_t vocab, uint32_t top)
{
    if (m == 0 || vocab == 0 || vocab > kMaxVocab || top > kMaxTop) return 0;
    return logprob_scratch(m, vocab, top);
}

wc_status wc_token_logprobs(const wc_logprobs *a, void *d_scratch, uint64_t scratch_bytes, uint32_t *d_err,
                            hipStream_t stream)
{
    if (!a || !valid_type(a->type) || a->vocab == 0 || a->vocab > kMaxVocab || a->top > kMaxTop || a->top > a->vocab)
        return WC_ERR_ARG;
    if (d_err && !aligned(d_err, 4)) return WC_ERR_ARG;
    if (a->m == 0) return WC_OK;
    if (a->m > kMaxGrid || (a->m > 1 && a->stride < a->vocab)) return WC_ERR_ARG;
    if (!a->logits || !aligned(a->logits, type_bytes(a->type)) || !a->tokens || !aligned(a->tokens, 8))
        return WC_ERR_ARG;
    if (!a->logprob || !a->entropy || !a->lse || !aligned(a->logprob, 4) || !aligned(a->entropy, 4) ||
        !aligned(a->lse, 4))
        return WC_ERR_ARG;
    if (a->top && (!a->top_logprobs || !a->top_ids || !aligned(a->top_logprobs, 4) || !aligned(a->top_ids, 8)))
        return WC_ERR_ARG;
    LogprobArgs g{};
    logprob_slices(a->m, a->vocab, &g.slices, &g.slice);
    if (a->m * g.slices > kMaxGrid) return WC_ERR_ARG;
    const uint64_t need = logprob_scratch(a->m, a->vocab, a->top);
    if (scratch_bytes < need) return WC_ERR_CAPACITY;
    if (need && (!d_scratch || !aligned(d_scratch, 16))) return WC_ERR_ARG;
    g.logits = a->logits;
    g.stride = a->stride;
    g.tokens = a->tokens;
    g.vocab = a->vocab;
    g.top = a->top;
    g.logprob = a->logprob;
    g.entropy = a->entropy;
    g.lse = a->lse;
    g.top_logprobs = a->top_logprobs;
    g.top_ids = a->top_ids;
    g.part = static_cast<float *>(d_scratch);
    g.part_top = need ? reinterpret_cast<uint64_t *>(static_cast<char *>(d_scratch) + 16 * a->m * g.slices) : nullptr;
    g.err = d_err;
    switch (a->type) {
    case WC_T_BF16: return launch_logprobs<WC_T_BF16>(g, a->m, stream);
    case WC_T_FP16: return launch_logprobs<WC_T_FP16>(g, a->m, stream);
    default: return launch_logprobs<WC_T_FP32>(g, a->m, stream);
    }
}

wc_status wc_token_logprobs_backward(const wc_logprobs_grad *a, uint32_t *d_err, hipStream_t stream)
{
    if (!a || !valid_type(a->type) || a->vocab == 0 || a->vocab > kMaxVocab) return WC_ERR_ARG;
    if (d_err && !aligned(d_err, 4)) return WC_ERR_ARG;
    if (a->m == 0) return WC_OK;
    if (a->m > 1 && (a->stride < a->vocab || a->out_stride < a->vocab)) return WC_ERR_ARG;
    const uintptr_t es = type_bytes(a->type);
    if (!a->logits || !a->out || !aligned(a->logits, es) || !aligned(a->out, es)) return WC_ERR_ARG;
    if (a->out == a->logits && a->m > 1 && a->out_stride != a->stride) return WC_ERR_ARG;
    if (!a->tokens || !aligned(a->tokens, 8) || !a->lse || !aligned(a->lse, 4)) return WC_ERR_ARG;
    if (!aligned(a->grad_logprob, 4) || !aligned(a->grad_entropy, 4)) return WC_ERR_ARG;
    if (a->grad_entropy && (!a->entropy || !aligned(a->entropy, 4))) return WC_ERR_ARG;
    LogprobGradArgs g{};
    g.logits = a->logits;
    g.out = a->out;
    g.stride = a->stride;
    g.out_stride = a->out_stride;
    g.tokens = a->tokens;
    g.lse = a->lse;
    g.entropy = a->entropy;
    g.grad_logprob = a->grad_logprob;
    g.grad_entropy = a->grad_entropy;
    g.vocab = a->vocab;
    g.blocks = a->out == a->logits ? 1 : (uint32_t)ceil_div(a->vocab, kSweep);
    g.err = d_err;
    if (a->m > kMaxGrid / g.blocks) return WC_ERR_ARG;
    const dim3 grid((uint32_t)(a->m * g.blocks)), block(kRowThreads);
    switch (a->type) {
    case WC_T_BF16: hipLaunchKernelGGL(k_logprobs_grad<WC_T_BF16>, grid, block, 0, stream, g); break;
    case WC_T_FP16: hipLaunchKernelGGL(k_logprobs_grad<WC_T_FP16>, grid, block, 0, stream, g); break;
    default: hipLaunchKernelGGL(k_logprobs_grad<WC_T_FP32>, grid, block, 0, stream, g); break;
    }
    return launched();
}

}  // extern "C"
