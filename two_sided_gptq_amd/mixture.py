"""A rounded mixture layer in use: routed, adapted by request, and drafting for its original.

    python -m two_sided_gptq_amd.mixture [--experts 8 --choices 2 --tokens 512 --width 512 --requests 16]

Tokens come in the order of their requests.  `forward` takes them through the library's
calls as a server would:

  1. a gate's largest log probabilities choose each token's experts (token_logprobs);
  2. the choices are sorted by expert (group_sort), the tokens rounded to fp8 once and copied
     to their places (group_gather_fp8), multiplied with the experts' rounded weights
     (fp8_matmul) and brought back with the gate's weights (group_combine);
  3. each request's low-rank adapter is added in place (group_sort, adapter_matmul).

`backward` is the way back through the layer in 16 bits, for training the adapters and the
gate's weights; `verify` lets the original layer keep or refuse what the rounded one drafted
(verify_drafts).
"""
from __future__ import annotations

import argparse

import torch

from two_sided_gptq_amd import bakron


def route(X, gate, choices):
    """(experts (tokens, choices) int64, weights that sum to 1) of a gate (experts, width)."""
    logits = bakron.grouped_matmul(X, gate, out_dtype=torch.float32)
    none = torch.full((X.shape[0],), -1, dtype=torch.int64, device=X.device)
    top = bakron.token_logprobs(logits, none, top=choices)
    return top["top_ids"], top["top_logprob"].softmax(1)


def forward(X, experts, weights, W8, scales, adapters=None):
    """The layer's outputs (tokens, N).  W8 (experts, N, K) in fp8 with the rows' scales;
    adapters: None or (request's adapter of each token, A, B, scale)."""
    offsets, _, slots = bakron.group_sort(experts, W8.shape[0])
    X8, sx = bakron.group_gather_fp8(X, slots, offsets)
    Y = bakron.fp8_matmul(X8, sx, W8, scales, offsets=offsets)
    out = bakron.group_combine(Y, slots, offsets, weights)
    return out if adapters is None else adapted(X, out, adapters)


def forward_original(X, experts, weights, W, adapters=None):
    """(outputs, what `backward` needs) of the layer in 16 bits."""
    offsets, _, slots = bakron.group_sort(experts, W.shape[0])
    Xs = bakron.group_gather(X, slots, offsets)
    Y = bakron.grouped_matmul(Xs, W, offsets)
    out = bakron.group_combine(Y, slots, offsets, weights)
    return out if adapters is None else adapted(X, out, adapters), (Xs, Y, slots, offsets)


def adapted(X, out, adapters):
    of, A, B, scale = adapters
    places, order, _ = bakron.group_sort(of, A.shape[0])
    return bakron.adapter_matmul(X, A, B, places, order, scale, base=out, out=out)


def backward(dout, X, weights, W, kept, adapters=None):
    """Gradients of X, of the gate's weights and of the experts' (and of A and B)."""
    Xs, Y, slots, offsets = kept
    dY, dweights = bakron.group_combine_grad(dout, Y, slots, offsets, weights)
    dXs, dW = bakron.grouped_matmul_grad(dY, Xs, W, offsets)
    dX = bakron.group_combine(dXs, slots, offsets)
    if adapters is None:
        return dX, dweights, dW
    of, A, B, scale = adapters
    places, order, _ = bakron.group_sort(of, A.shape[0])
    dX, dA, dB = bakron.adapter_matmul_grad(dout, X, A, B, places, order, scale, base=dX, out=dX)
    return dX, dweights, dW, dA, dB


def verify(p, q, generator=None):
    """Drafts drawn from q (requests, n, vocab) and what p (requests, n + 1, vocab) keeps."""
    requests, n, vocab = q.shape
    drafts = torch.multinomial(q.view(-1, vocab), 1, generator=generator).view(requests, n)
    u = torch.rand(requests, n, device=q.device, generator=generator)
    v = torch.rand(requests, device=q.device, generator=generator)
    return drafts, *bakron.verify_drafts(p, q, drafts, u, v)


def example(experts=8, choices=2, tokens=512, width=512, requests=16, rank=16, bits=4, seed=1):
    """Random inputs of a layer: (X, gate, W, W8, scales, adapters).  One request in four has no
    adapter; the rounded weights are those of a solve with factors that are the identity."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, size=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * size).bfloat16()
    X = normal(tokens, width)
    gate, W = normal(experts, width, size=width ** -0.5), normal(experts, width, width, size=width ** -0.5)
    A, B = normal(requests, rank, width, size=width ** -0.5), normal(requests, width, rank, size=0.1)
    of = torch.arange(requests, device="cuda").repeat_interleave(-(-tokens // requests))[:tokens]
    of = torch.where(of % 4 == 3, -1, of)
    W8 = torch.empty((experts, width, width), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((experts, width), device="cuda")
    eye = torch.eye(width, device="cuda")
    for e in range(experts):
        out = bakron.quantize(W[e].float(), eye, eye, bits=bits)
        bakron.fp8_from_codes(out["codes"], bits=bits, out=W8[e])
        scales[e] = out["scales"]
    return X, gate, W, W8, scales, (of, A, B, torch.ones(requests, device="cuda"))


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--experts", type=int, default=8)
    p.add_argument("--choices", type=int, default=2)
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--width", type=int, default=512)
    p.add_argument("--requests", type=int, default=16)
    p.add_argument("--bits", type=int, default=4, choices=(2, 3, 4))
    a = p.parse_args()
    if not 1 <= a.choices <= a.experts:
        p.error(f"a token cannot choose {a.choices} of {a.experts} experts")
    if a.requests < 1 or a.tokens % a.requests or a.tokens < 2 * a.requests:
        p.error(f"{a.tokens} tokens are not two or more for each of {a.requests} requests, of the same number")
    X, gate, W, W8, scales, adapters = example(a.experts, a.choices, a.tokens, a.width, a.requests, bits=a.bits)
    experts, weights = route(X, gate, a.choices)
    rounded = forward(X, experts, weights, W8, scales, adapters)
    original, kept = forward_original(X, experts, weights, W, adapters)
    grads = backward(original, X, weights, W, kept, adapters)
    off = ((rounded.float() - original.float()).norm() / original.float().norm()).item()
    # each request's last tokens as drafts; a head of the width's columns
    n = min(4, a.tokens // a.requests - 1)
    logits = [y.float().view(a.requests, -1, a.width)[:, -(n + 1):] for y in (original, rounded)]
    drafts, accepted, tokens = verify(logits[0].softmax(2), logits[1][:, :n].softmax(2).contiguous())
    print(f"{a.experts} experts of {a.width} x {a.width}, {a.choices} a token, {a.tokens} tokens of {a.requests} requests, "
          f"{a.bits} bits")
    print(f"rounded layer off by {off:.4f}, gradients' norms "
          + ", ".join(f"{g.float().norm().item():.3g}" for g in grads)
          + f", drafts kept {accepted.float().mean().item():.2f} of {n}")


if __name__ == "__main__":
    main()
