"""The products of one serving step, from weights that are kept compressed.

A batch of tokens goes through a shared projection with an adapter per
request, a mixture-of-experts layer and the output layer, and its next tokens
are scored:

  y = X W^T straight from the compressed W (decode fused with the product),
      plus each request's low-rank adapter, added into the same y;
  h = x + experts(y), the experts decoded into buffers that the layer reads;
  logits = h V^T straight from the compressed output layer;
  log probability and entropy of the given tokens, the best alternatives, and
      the gradient that a fine-tuning step would send back into the logits.

Run it on an MI355X:  python examples/serve_step.py
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from lossless_weight_compression_bf16_amd import adapters, codec, gemm, logprobs, moe  # noqa: E402


@dataclass
class Model:
    """Weights of a layer and an output layer: compressed ones, and small ones that are kept as they are."""
    projection: gemm.EncodedWeights   # cols x cols
    output: gemm.EncodedWeights       # vocabulary x cols
    experts: codec.EncodedBatch       # w1, w3 (inner x cols) and w2 (cols x inner) of every expert
    buffers: list                     # w1, w3, w2: experts x ..., what the experts are decoded into
    router: torch.Tensor              # experts x cols
    a: torch.Tensor                   # adapters x rank x cols
    b: torch.Tensor                   # adapters x cols x rank
    scales: torch.Tensor


def random_weights(cols=512, inner=256, experts=8, vocab=1024, n_adapters=4, rank=16, seed=0, device="cuda"):
    """Random weights of the shapes above (there are no checkpoints here)."""
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, std):
        return torch.empty(shape, dtype=torch.bfloat16, device=device).normal_(0.0, std, generator=g)
    return {"projection": normal(cols, cols, std=cols ** -0.5), "output": normal(vocab, cols, std=3 * cols ** -0.5),
            "w1": normal(experts, inner, cols, std=cols ** -0.5), "w3": normal(experts, inner, cols, std=cols ** -0.5),
            "w2": normal(experts, cols, inner, std=inner ** -0.5), "router": normal(experts, cols, std=cols ** -0.5),
            "a": normal(n_adapters, rank, cols, std=cols ** -0.5), "b": normal(n_adapters, cols, rank, std=0.1),
            "scales": 0.5 + torch.rand(n_adapters, generator=g, device=device)}


def compress(w) -> Model:
    experts = codec.encode_batch([*w["w1"], *w["w3"], *w["w2"]])
    return Model(gemm.encode_weights([w["projection"]]), gemm.encode_weights([w["output"]]), experts,
                 [torch.empty_like(w[k]) for k in ("w1", "w3", "w2")], w["router"], w["a"], w["b"], w["scales"])


def step(model: Model, x, ids, tokens, top_k=2, top=5):
    """x: m x cols BF16, m at most 64, ids: an adapter per token or -1,
    tokens: the next tokens to score.  Scores, logits and their gradient."""
    y, = gemm.decode_gemm(model.projection, [x])
    adapters.add_adapters(x, y, model.a, model.b, ids, model.scales)
    codec.decode_batch(model.experts, outs=[e for w in model.buffers for e in w])
    h = x + moe.moe_layer(y.to(torch.bfloat16), model.router, *model.buffers, top_k)
    logits, = gemm.decode_gemm(model.output, [h])
    scores = logprobs.token_logprobs(logits, tokens, top=top)
    # minus the mean log probability, a tenth of the mean entropy kept high
    m = x.shape[0]
    gradient = logprobs.token_logprobs_backward(
        logits, tokens, scores.lse, scores.entropy, torch.full((m,), -1.0 / m, device=x.device),
        torch.full((m,), -0.1 / m, device=x.device))
    return scores, logits, gradient


def main():
    w = random_weights()
    model = compress(w)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((8, 512), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    ids = torch.tensor([0, 1, -1, 2, 3, 1, 1, -1], device="cuda")
    tokens = torch.randint(0, 1024, (8,), generator=g, device="cuda")
    scores, _, gradient = step(model, x, ids, tokens)
    print(f"compressed: projection {model.projection.ratio:.3f}, output {model.output.ratio:.3f}, "
          f"experts {model.experts.ratio:.3f} of their size")
    for r in range(8):
        best = ", ".join(f"{int(i)} ({float(p):.2f})" for i, p in zip(scores.top_ids[r], scores.top_logprobs[r]))
        print(f"token {int(tokens[r]):4d}: log probability {float(scores.logprob[r]):7.3f}, entropy "
              f"{float(scores.entropy[r]):.3f}, best {best}")
    print(f"gradient of the logits: {tuple(gradient.shape)}, norm {float(gradient.norm()):.4f}")


if __name__ == "__main__":
    main()
