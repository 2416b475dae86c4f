"""The output end of a language model, trained and then served.

Training step: the residual stream goes through the norm and into the loss over
the vocabulary, which keeps no logits; the gradients of the stream, the norm's
weight and the vocabulary's matrix come back and are clipped together. Serving:
the matrix is rounded once, to 8-bit integers and to 4-bit floating point; each
token's norm leaves its kernel in 8 bits, or is rounded to 4, and the products run
on those.

    python examples/output_head.py [tokens] [words] [width]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dense_fp32_gemm_gb300 import binding  # noqa: E402
from dense_fp32_gemm_gb300.layers import linear_cross_entropy, rms_norm  # noqa: E402


def loss_of(x, residual, gain, words, target):
    y, _ = rms_norm(x, gain, residual=residual)
    return linear_cross_entropy(y, words, target)


def run(tokens=512, vocabulary=2000, width=256, steps=10, seed=0, lr=0.5):
    """Trains gain and words on random tokens; returns (losses, norms, relative errors of the logits in 8 and in 4
    bits)."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    x, residual = normal(tokens, width).bfloat16(), normal(tokens, width).bfloat16()
    target = torch.randint(0, vocabulary, (tokens,), generator=g, device="cuda")
    target[::7] = -100                                   # not counted, as a prompt's words are not
    gain = torch.ones(width, device="cuda", requires_grad=True)
    words = normal(vocabulary, width, scale=width ** -0.5).bfloat16().requires_grad_()

    losses, norms = [], []
    for _ in range(steps):
        loss = loss_of(x, residual, gain, words, target)
        grads = torch.autograd.grad(loss, [gain, words])
        norms.append(binding.clip_grad_norm(grads, 1.0))
        with torch.no_grad():
            for w, d in zip((gain, words), grads):
                w -= lr * d
        losses.append(loss.detach())

    with torch.no_grad():
        y, h, _ = binding.rms_norm(x, gain, residual=residual)
        logits = y.float() @ words.float().mT
        q8, s8, _ = binding.rms_norm_i8(x, gain, residual=residual)
        logits8 = binding.i8_gemm(q8, s8, *binding.i8_quantize(words), out_dtype=torch.float32)
        q4, s4 = binding.mx4_quantize(y)
        logits4 = binding.mx4_gemm(q4, s4, *binding.mx4_quantize(words), out_dtype=torch.float32)
        errors = [(v - logits).norm() / logits.norm() for v in (logits8, logits4)]
    return [float(v) for v in losses], [float(v) for v in norms], [float(v) for v in errors]


if __name__ == "__main__":
    losses, norms, errors = run(*(int(v) for v in sys.argv[1:4]))
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}, gradient norm {norms[0]:.4f} -> {norms[-1]:.4f}, "
          f"logits off by {100 * errors[0]:.2f} % in 8 bits and {100 * errors[1]:.2f} % in 4")
