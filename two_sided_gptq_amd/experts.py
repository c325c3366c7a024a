"""Rounding the experts of a layer, multiplying with them and scoring what it cost.

    python -m two_sided_gptq_amd.experts [--experts 8 --tokens 2048 --width 512 --bits 4]

A small mixture layer with random weights: tokens sorted by expert, one weight
matrix an expert, a common output head.  `round_experts` takes it through the
library's calls as a post-training quantiser would:

  1. forward in bf16 (grouped_matmul), log probabilities of the targets
     (token_logprobs) and their gradient back to the experts' outputs
     (token_logprobs_grad, grouped_matmul_grad);
  2. for each expert that saw tokens, the factors of its inputs and of its outputs'
     gradients (hessian, factor) and the two-sided rounding (quantize);
  3. the codes as fp8 weights, exactly (fp8_from_codes), the activations in fp8 with
     a scale for each 128 (fp8_quantize), and the layer's product (fp8_matmul);
  4. log probabilities again, from the rounded layer.
"""
from __future__ import annotations

import argparse

import torch

from two_sided_gptq_amd import bakron, synth


def forward(X, W, head, offsets, targets, top=1):
    """(experts' outputs, logits, scores) of the layer in bf16."""
    Y = bakron.grouped_matmul(X, W, offsets)
    logits = bakron.grouped_matmul(Y, head, out_dtype=torch.float32)
    return Y, logits, bakron.token_logprobs(logits, targets, top=top)


def output_gradients(Y, logits, scores, head, targets):
    """Gradient of the targets' log probabilities with respect to the experts' outputs:
    the samples of the output-side factors."""
    ones = torch.ones(logits.shape[0], device=logits.device)
    d = bakron.token_logprobs_grad(logits, targets, scores["lse"], None, ones)
    dY, _ = bakron.grouped_matmul_grad(d.to(torch.bfloat16), Y, head, want_w=False)
    return dY


def round_experts(X, W, head, offsets, targets, kind=bakron.Q_SYM, bits=4):
    """X (tokens, K) sorted by expert, W (experts, N, K) and head (vocab, N) in bf16,
    offsets (int32, experts + 1) and targets (int64) on the GPU.  Returns a dict with
    the rounded weights and the scores before and after."""
    experts, N, K = W.shape
    Y, logits, before = forward(X, W, head, offsets, targets)
    dY = output_gradients(Y, logits, before, head, targets)
    at = offsets.tolist()
    W8 = torch.empty((experts, N, K), dtype=torch.float8_e4m3fn, device=X.device)
    scales = torch.ones((experts, N), device=X.device)
    V = W.float()
    status = torch.zeros(1, dtype=torch.int32, device=X.device)
    eye = {}
    for e in range(experts):
        a, b = at[e], at[e + 1]
        if a == b:  # no tokens: rounded to nearest, by factors that are the identity
            for n in (K, N):
                eye.setdefault(n, torch.eye(n, device=X.device))
            LA, LB = eye[K], eye[N]
        else:
            LA = bakron.factor(bakron.hessian(X[a:b].float(), synth.DAMP), dev_status=status)
            LB = bakron.factor(bakron.hessian(dY[a:b].float(), synth.DAMP), dev_status=status)
        out = bakron.quantize(W[e].float(), LA, LB, kind=kind, bits=bits, dev_status=status)
        bakron.fp8_from_codes(out["codes"], out["zeros"], kind=kind, bits=bits, out=W8[e])
        scales[e], V[e] = out["scales"], out["V"]
    X8, sx = bakron.fp8_quantize(X, dev_status=status)
    Y8 = bakron.fp8_matmul(X8, sx, W8, scales, offsets=offsets, dev_status=status)
    logits8 = bakron.grouped_matmul(Y8, head, out_dtype=torch.float32, dev_status=status)
    after = bakron.token_logprobs(logits8, targets, top=1, dev_status=status)
    return dict(W8=W8, scales=scales, V=V, X8=X8, sx=sx, Y=Y, Y8=Y8, before=before, after=after, status=status)


def example(experts=8, tokens=2048, width=512, vocab=4096, seed=1):
    """Random inputs of round_experts: uneven experts, one of them without tokens."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    share = 1.0 / torch.arange(1, experts + 1, device="cuda")
    share[-1] = 0.0 if experts > 1 else 1.0
    to = torch.multinomial(share, tokens, replacement=True, generator=g)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(to, minlength=experts).cumsum(0)
    X = torch.randn(tokens, width, device="cuda", generator=g)
    X[:, ::97] *= 20.0
    W = torch.randn(experts, width, width, device="cuda", generator=g) * 0.02
    head = torch.randn(vocab, width, device="cuda", generator=g) * width ** -0.5
    X, W, head = X.bfloat16(), W.bfloat16(), head.bfloat16()
    # targets as the layer itself would draw them
    logits = bakron.grouped_matmul(bakron.grouped_matmul(X, W, offsets), head, out_dtype=torch.float32)
    targets = torch.multinomial(logits.softmax(1), 1, generator=g).squeeze(1)
    return X, W, head, offsets, targets


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--experts", type=int, default=8)
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--width", type=int, default=512)
    p.add_argument("--bits", type=int, default=4, choices=(2, 3, 4))
    a = p.parse_args()
    X, W, head, offsets, targets = example(a.experts, a.tokens, a.width)
    r = round_experts(X, W, head, offsets, targets, bits=a.bits)
    before, after = r["before"], r["after"]
    same = (before["top_ids"] == after["top_ids"]).float().mean().item()
    print(f"{a.experts} experts of {a.width} x {a.width}, {a.tokens} tokens, {a.bits} bits")
    print(f"mean log probability {before['logprob'].mean().item():.4f} -> {after['logprob'].mean().item():.4f}, "
          f"entropy {before['entropy'].mean().item():.4f} -> {after['entropy'].mean().item():.4f}, "
          f"same first token {same:.3f}, status {int(r['status'])}")


if __name__ == "__main__":
    main()
