"""One block of routed experts, trained and then served.

Training step: tokens are sorted by expert, go through the experts' grouped
product and a dense projection (a single group), the gradients of inputs and
weights come back through the same kernels, and all gradients are clipped
together. Serving: the projection's weights are quantised to 8 bits once, the
activations token by token, and the product runs on 8-bit integers.

    python examples/expert_layer.py [tokens] [experts] [width]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dense_fp32_gemm_gb300 import binding  # noqa: E402
from dense_fp32_gemm_gb300.layers import expert_linear  # noqa: E402


def route(scores):
    """Each token's best expert: the order that sorts tokens by expert and the
    experts' row bounds, all on the device."""
    expert = scores.argmax(dim=1)
    order = torch.argsort(expert, stable=True)
    counts = torch.bincount(expert, minlength=scores.shape[1])
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return order, offsets


def run(tokens=1024, experts=8, width=512, steps=20, seed=0, lr=0.2):
    """Fits the block to a random teacher; returns (losses, norms, error of the
    8-bit projection relative to the bf16 one)."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda") * scale

    x = normal(tokens, width).bfloat16()
    order, offsets = route(normal(tokens, experts))
    x = x[order]
    target = torch.tanh(normal(tokens, width))
    up = normal(experts, 2 * width, width, scale=width ** -0.5).bfloat16().requires_grad_()
    down = normal(1, width, 2 * width, scale=(2 * width) ** -0.5).bfloat16().requires_grad_()
    one = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")

    def block(x):
        hidden = torch.relu(expert_linear(x, up, offsets))
        return hidden, expert_linear(hidden, down, one)

    losses, norms = [], []
    for _ in range(steps):
        _, y = block(x)
        loss = (y.float() - target).square().mean()
        grads = torch.autograd.grad(loss, [up, down])
        norms.append(binding.clip_grad_norm(grads, 1.0))
        with torch.no_grad():
            for w, d in zip((up, down), grads):
                w -= lr * tokens ** 0.5 * d
        losses.append(loss.detach())

    with torch.no_grad():
        hidden, y = block(x)
        qw, sw = binding.i8_quantize(down[0])      # a scale for each output channel
        qh, sh = binding.i8_quantize(hidden)       # a scale for each token
        y8 = binding.i8_gemm(qh, sh, qw, sw, out_dtype=torch.bfloat16)
        error = (y8.float() - y.float()).norm() / y.float().norm()
    return [float(v) for v in losses], [float(v) for v in norms], float(error)


if __name__ == "__main__":
    sizes = [int(v) for v in sys.argv[1:4]]
    losses, norms, error = run(*sizes)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}, gradient norm {norms[0]:.4f} -> {norms[-1]:.4f}, "
          f"8-bit projection off by {100 * error:.2f} %")
