"""What is measured of the operators around a linear layer of experts.

Four operators, each in its plain form (elementary torch operations in 32
bits, rounded once at the end) and as the calls a user makes of the library:

  rows   Y[r] = X[r] op(W_e) for the rows r of expert e, the rows of one expert
         adjacent and their bounds in `offsets` (forward product with op "T",
         W_e stored N x K; gradient of the input with op "N", W_e stored K x N)
  wgrad  C_e = A_e^T B_e, the gradient of the experts' weights
  i8     activations quantised to 8 bits token by token, then the product with
         8-bit weights, scaled by token and channel
  clip   the 2-norm of many gradients taken together, and their clipping
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # 16 token rows spread over 32 experts: one decode step of a small batch
        dict(name="rows_decode_bf16", kind="rows", op="T", type="bf16", e=32, rows=16, n=1024, k=2048),
        # a prompt's tokens through eight experts: the throughput case
        dict(name="rows_prompt_bf16", kind="rows", op="T", type="bf16", e=8, rows=8192, n=4096, k=4096),
        # gradient of the input with odd sizes, tight rows (no 16-byte alignment)
        dict(name="rows_dx_odd_f16", kind="rows", op="N", type="f16", e=16, rows=2049, n=777, k=1000),
        # full-precision experts, as a user of the FP32 products has them
        dict(name="rows_f32", kind="rows", op="T", type="f32", e=8, rows=2048, n=1024, k=2048),
        # weight gradient of a training step, kept in 32 bits
        dict(name="wgrad_bf16_f32", kind="wgrad", type="bf16", out="f32", e=8, rows=8192, m=4096, n=1024),
        # short ragged groups, gradients in the weights' own type
        dict(name="wgrad_f16", kind="wgrad", type="f16", out="f16", e=16, rows=1000, m=520, n=264),
        # one token of one sequence
        dict(name="i8_token_bf16", kind="i8", type="bf16", m=1, n=4096, k=4096),
        # a decode batch, odd in every size
        dict(name="i8_batch_odd_f16", kind="i8", type="f16", m=133, n=8191, k=1000),
        # a prompt
        dict(name="i8_prompt_bf16", kind="i8", type="bf16", m=4096, n=4096, k=4096),
        # the gradients of a small model: latency
        dict(name="clip_small_f32", kind="clip", type="f32", tensors=48, numel=1 << 20, clipped=True),
        # bf16 gradients of odd sizes, packed one behind the other in one buffer
        dict(name="clip_large_bf16", kind="clip", type="bf16", tensors=300, numel=400_000_003, clipped=True),
        # a step whose norm stays below the bound, in place
        dict(name="clip_unclipped_f32", kind="clip", type="f32", tensors=150, numel=60_000_001, clipped=False),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["rows", "rows", "wgrad", "i8", "i8", "clip"])
    if kind == "clip":
        return dict(kind=kind, type=rng.choice(["f32", "bf16", "f16"]), tensors=_spread(rng, 1, 300),
                    numel=_spread(rng, 1 << 16, 200_000_000), clipped=rng.random() < 0.7)
    if kind == "i8":
        return dict(kind=kind, type=rng.choice(["f32", "bf16", "f16"]), m=_spread(rng, 1, 4096),
                    n=_spread(rng, 256, 4096), k=_spread(rng, 256, 4096))
    e = _spread(rng, 1, 64)
    a = _spread(rng, 64, 4096)
    b = _spread(rng, 64, min(4096, (1 << 27) // (e * a)))
    if rng.random() < 0.5:
        a, b = -(-a // 8) * 8, -(-b // 8) * 8
    if kind == "rows":
        return dict(kind=kind, op=rng.choice(["T", "N"]), type=rng.choice(["f32", "bf16", "f16"]), e=e,
                    rows=_spread(rng, 1, 8192), n=a, k=b)
    t = rng.choice(["f32", "bf16", "f16"])
    return dict(kind=kind, type=t, out=rng.choice(["f32", t]), e=e, rows=_spread(rng, 1, 8192), m=a, n=b)


def _counts(case):
    """Rows of each expert, largest first: a skewed routing, the same for every seed (the seed says which
    expert has which share). About one expert in eight of a longer list has none."""
    e, rows = case["e"], case["rows"]
    r = np.random.RandomState((e * 7919 + rows) % (1 << 31))
    p = r.exponential(size=e) + 0.05
    if e >= 8:
        p[r.permutation(e)[: e // 8]] = 0.0
    return sorted(r.multinomial(rows, p / p.sum()).tolist(), reverse=True)


def _bounds(case, seed):
    c = np.array(_counts(case))[np.random.RandomState(seed % (1 << 31)).permutation(case["e"])]
    return [0] + np.cumsum(c).tolist()


def _sizes(case):
    """Sizes of the tensors of a "clip" case: vectors and matrices of all sizes, odd ones among them."""
    n, total = case["tensors"], case["numel"]
    w = np.random.RandomState(n + 17).lognormal(0.0, 1.5, size=n)
    cut = np.concatenate([[0], np.round(np.cumsum(w) / w.sum() * total)]).astype(np.int64)
    cut[-1] = total
    return np.diff(cut).tolist()


def _normal(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return torch.randn(shape, generator=g, device="cuda").mul_(scale)


def _activations(rows, cols, seed):
    """Normal, with a few channels that are much larger, as activations are."""
    x = _normal((rows, cols), seed)
    x[:, seed % 61:: 61] *= 8.0
    return x


def prepare(case, seed):
    kind = case["kind"]
    t = TYPES[case["type"]]
    if kind == "rows":
        n, k = case["n"], case["k"]
        b = _bounds(case, seed)
        shape = (case["e"], n, k) if case["op"] == "T" else (case["e"], k, n)
        return dict(case=case, x=_activations(case["rows"], k, seed).to(t),
                    w=_normal(shape, seed + 1, k ** -0.5).to(t), bounds=b,
                    offsets=torch.tensor(b, dtype=torch.int32, device="cuda"))
    if kind == "wgrad":
        b = _bounds(case, seed)
        return dict(case=case, a=_normal((case["rows"], case["m"]), seed, 0.05).to(t),
                    b=_activations(case["rows"], case["n"], seed + 1).to(t), bounds=b,
                    offsets=torch.tensor(b, dtype=torch.int32, device="cuda"))
    if kind == "i8":
        w = _normal((case["n"], case["k"]), seed + 1, 40.0).round_().clamp_(-127, 127).to(torch.int8)
        return dict(case=case, x=_activations(case["m"], case["k"], seed).to(t), w=w,
                    sw=_normal((case["n"],), seed + 2).abs_().add_(0.5).mul_(1e-3),
                    most=torch.full((), 127.0, device="cuda"))
    sizes = _sizes(case)
    flat = _normal((case["numel"],), seed, 1e-3).to(t)
    norm = 1e-3 * math.sqrt(case["numel"])
    out = torch.empty_like(flat) if case["clipped"] else flat
    return dict(case=case, flat=flat, grads=list(flat.split(sizes)), out_flat=out, out=list(out.split(sizes)),
                max_norm=norm * (0.3 if case["clipped"] else 3.0))


def run(state):
    return _calls(state) if own else _plain(state)


def _calls(s):
    from dense_fp32_gemm_gb300 import binding

    case = s["case"]
    if case["kind"] == "rows":
        return binding.grouped_gemm(s["x"], s["w"], s["offsets"], op=case["op"])
    if case["kind"] == "wgrad":
        return binding.grouped_wgrad(s["a"], s["b"], s["offsets"], out_dtype=TYPES[case["out"]])
    if case["kind"] == "i8":
        q, sx = binding.i8_quantize(s["x"])
        return {"y": binding.i8_gemm(q, sx, s["w"], s["sw"], out_dtype=s["x"].dtype), "q": q, "scale": sx}
    norm = binding.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"])
    return {"norm": norm, "grads": s["out_flat"]}


def _plain(s):
    case = s["case"]
    if case["kind"] == "rows":
        w = s["w"].mT if case["op"] == "T" else s["w"]
        return torch.cat([s["x"][a:b].float() @ w[e].float()
                          for e, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:])) if b > a]).to(s["x"].dtype)
    if case["kind"] == "wgrad":
        return torch.stack([s["a"][a:b].float().mT @ s["b"][a:b].float()
                            for a, b in zip(s["bounds"], s["bounds"][1:])]).to(TYPES[case["out"]])
    if case["kind"] == "i8":
        x = s["x"].float()
        scale = x.abs().amax(dim=1) / s["most"]
        # (a row of zeros has scale 0 and is all zeros)
        q = torch.where(scale[:, None] > 0, x / scale[:, None], torch.zeros_like(x)).round().clamp(-127, 127)
        y = (q @ s["w"].float().mT) * scale[:, None] * s["sw"]
        return {"y": y.to(s["x"].dtype), "q": q.to(torch.int8), "scale": scale}
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    s["out_flat"].copy_(s["flat"].float() * coef)
    return {"norm": norm, "grads": s["out_flat"]}


def work(case):
    kind = case["kind"]
    size = TYPES[case["type"]].itemsize
    if kind == "rows":
        active = sum(c > 0 for c in _counts(case))
        rows, n, k = case["rows"], case["n"], case["k"]
        return {"bytes": size * (rows * k + active * n * k + rows * n) + 4 * (case["e"] + 1),
                "flops": 2 * rows * n * k}
    if kind == "wgrad":
        rows, m, n = case["rows"], case["m"], case["n"]
        return {"bytes": size * rows * (m + n) + TYPES[case["out"]].itemsize * case["e"] * m * n + 4 * (case["e"] + 1),
                "flops": 2 * rows * m * n}
    if kind == "i8":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": size * m * k + m * k + 4 * m + n * k + 4 * n + size * m * n, "flops": 2 * m * n * k}
    return {"bytes": case["numel"] * size * (2 if case["clipped"] else 1), "flops": 3 * case["numel"]}


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("rows", "wgrad"):
        ends = s["bounds"]
        if kind == "rows":
            y = torch.zeros((case["rows"], case["n"]), dtype=torch.float64, device="cuda")
            for e in range(case["e"]):
                rows = slice(ends[e], ends[e + 1])
                y[rows] = torch.einsum("rk,nk->rn" if case["op"] == "T" else "rk,kn->rn",
                                       s["x"][rows].double(), s["w"][e].double())
            return y
        c = torch.zeros((case["e"], case["m"], case["n"]), dtype=torch.float64, device="cuda")
        for e in range(case["e"]):
            rows = slice(ends[e], ends[e + 1])
            c[e] = torch.einsum("rm,rn->mn", s["a"][rows].double(), s["b"][rows].double())
        return c
    if kind == "i8":
        x = s["x"].double()
        # the scale and the quotient are FP32 values by definition, rounded to nearest
        scale = (x.abs().max(dim=1).values / 127.0).float().double()
        safe = torch.where(scale == 0, torch.ones_like(scale), scale)
        q = torch.clamp(torch.round((x / safe[:, None]).float().double()), -127, 127)
        y = torch.einsum("mk,nk->mn", q, s["w"].double()) * torch.outer(scale, s["sw"].double())
        return {"y": y, "q": q.to(torch.int8), "scale": scale}
    total = sum(float(c.double().pow(2).sum()) for c in s["flat"].split(1 << 26))
    norm = math.sqrt(total)
    coef = min(1.0, s["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": s["flat"].double() * coef}
