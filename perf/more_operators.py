"""What is measured of the operators at a model's output end.

Three operators, each in its plain form (elementary torch operations in 32
bits, rounded once at the end) and as the calls a user makes of the library:

  norm   h = x + residual in the type of x, y = h / rms(h) * weight; y as 8-bit
         integers with a scale a row; and a training step's forward and
         backward pass
  ce     softmax cross entropy of x @ w.T over a vocabulary, row by row, and
         its gradients
  mx4    activations to 4-bit floating point in blocks of 32 with a power of
         two each, then the product with 4-bit weights; and the values that a
         matrix is rounded to
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
IGNORE = -100


def listed():
    return [
        # one token of one sequence, on its way into an 8-bit layer: latency
        dict(name="norm_token_i8_bf16", kind="norm", form="i8", type="bf16", weight="bf16", m=1, n=4096, residual=True),
        # a decode batch of odd sizes
        dict(name="norm_batch_odd_f16", kind="norm", form="y", type="f16", weight="f32", m=133, n=1001, residual=True),
        # a prompt, on its way into an 8-bit layer
        dict(name="norm_prompt_i8_bf16", kind="norm", form="i8", type="bf16", weight="bf16", m=8192, n=4096, residual=True),
        # a training step
        dict(name="norm_train_bf16", kind="norm", form="train", type="bf16", weight="f32", m=8192, n=4096, residual=True),
        # a training step of a small model: latency
        dict(name="ce_train_small_f16", kind="ce", form="train", type="f16", t=65, v=1000, h=256),
        # the loss of an evaluation
        dict(name="ce_eval_bf16", kind="ce", form="loss", type="bf16", t=2048, v=65536, h=2048),
        # a training step over a large vocabulary
        dict(name="ce_train_large_bf16", kind="ce", form="train", type="bf16", t=4096, v=100003, h=4096),
        # full precision, odd sizes, tight rows
        dict(name="ce_train_odd_f32", kind="ce", form="train", type="f32", t=1000, v=8191, h=777),
        # one token through a layer of 4-bit weights
        dict(name="mx4_token_bf16", kind="mx4", form="layer", type="bf16", m=1, n=4096, k=4096),
        # a decode batch, odd in every size
        dict(name="mx4_batch_odd_f16", kind="mx4", form="layer", type="f16", m=133, n=8191, k=1000),
        # a prompt
        dict(name="mx4_prompt_bf16", kind="mx4", form="layer", type="bf16", m=8192, n=8192, k=4096),
        # the rounding of a weight matrix, to see what it costs in quality
        dict(name="mx4_round_f32", kind="mx4", form="round", type="f32", m=8192, k=4096),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["norm", "ce", "mx4"])
    t = rng.choice(["f32", "bf16", "f16"])
    even = rng.random() < 0.5      # sizes as models have them, or any

    def size(low, high):
        v = _spread(rng, low, high)
        return -(-v // 64) * 64 if even else v

    if kind == "norm":
        n = size(64, 16384)
        return dict(kind=kind, form=rng.choice(["y", "i8", "train"]), type=t, weight=rng.choice([t, "f32"]),
                    m=_spread(rng, 1, min(8192, (1 << 25) // n)), n=n, residual=rng.random() < 0.7)
    if kind == "ce":
        h = size(64, 4096)
        return dict(kind=kind, form=rng.choice(["loss", "train", "train"]), type=t, t=_spread(rng, 1, 4096),
                    v=size(64, 65536), h=h)
    if rng.random() < 0.3:
        return dict(kind=kind, form="round", type=t, m=_spread(rng, 1, 4096), k=size(32, 8192))
    return dict(kind=kind, form="layer", type=t, m=_spread(rng, 1, 8192), n=size(64, 8192), k=size(64, 4096))


def _normal(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    return torch.randn(shape, generator=g, device="cuda").mul_(scale)


def _activations(rows, cols, seed):
    """Normal, with a few channels that are much larger, as activations are."""
    x = _normal((rows, cols), seed)
    x[:, seed % 61:: 61] *= 8.0
    return x


def prepare(case, seed):
    kind, t = case["kind"], TYPES[case["type"]]
    if kind == "norm":
        m, n = case["m"], case["n"]
        s = dict(case=case, x=_activations(m, n, seed).to(t),
                 residual=_normal((m, n), seed + 1, 3.0).to(t) if case["residual"] else None,
                 weight=_normal((n,), seed + 2, 0.2).add_(1.0).to(TYPES[case["weight"]]),
                 most=torch.full((), 127.0, device="cuda"))
        if case["form"] == "train":
            s["dy"] = _normal((m, n), seed + 3).to(t)
            s["dh"] = _normal((m, n), seed + 4).to(t)
        return s
    if kind == "ce":
        rows, v, h = case["t"], case["v"], case["h"]
        g = torch.Generator(device="cuda").manual_seed(int(seed) + 2)
        # frequent words and rare ones; about one row in 16 is not counted
        u = torch.rand((rows,), generator=g, device="cuda")
        target = (v ** u.double()).long().clamp(max=v) - 1
        target[torch.rand((rows,), generator=g, device="cuda") < 1 / 16] = IGNORE
        # (a training step in 16-bit floating point scales its loss)
        scale = 1024.0 if t == torch.float16 else 1.0
        d = torch.full((rows,), scale, device="cuda") / (target != IGNORE).sum().clamp(min=1)
        return dict(case=case, x=_activations(rows, h, seed).to(t), w=_normal((v, h), seed + 1, 2 * h ** -0.5).to(t),
                    target=target, dloss=d)
    m, k = case["m"], case["k"]
    s = dict(case=case, x=_activations(m, k, seed).to(t))
    if case["form"] == "layer":
        codes, power = _to_mx4(_normal((case["n"], k), seed + 1, k ** -0.5))
        # two codes a byte, the first in the low half
        s["w"] = codes[:, 0::2] | (codes[:, 1::2] << 4)
        s["w_scale"] = _tiled(power)
    return s


def _to_mx4(x):
    """The codes (0 to 15, rows filled up to whole blocks of 32) and the biased powers of two of the blocks."""
    x = x.float()
    rows, k = x.shape
    blocks = -(-k // 32)
    x = torch.nn.functional.pad(x, (0, 32 * blocks - k)).view(rows, blocks, 32)
    most = x.abs().amax(dim=2)
    # floor(log2(most)) - 2, so that the largest lies in 4 .. 8 units; blocks of zeros and those below 2^-125 get
    # the least power, -127
    power = torch.where(most > 0, torch.frexp(most).exponent.int() - 3, -127).clamp(min=-127)
    v = x * ((127 - power) << 23).view(torch.float32)[:, :, None]
    a = v.abs()
    # 0, 0.5, 1, 1.5, 2, 3, 4, 6: steps of a half, of one and of two; ties to the even code
    code = torch.where(a < 2, (2 * a).round(), torch.where(a < 4, a.round() + 2, ((a / 2).round() + 4).clamp(max=7)))
    code = code.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    return code.view(rows, 32 * blocks), (power + 127).to(torch.uint8)


def _tile_places(rows, blocks, device):
    """Where the scales stand: tiles of 128 rows x 4 blocks of 512 bytes, in a tile 32 lines of 4 rows (r, r + 32,
    r + 64, r + 96) of 4 blocks."""
    r = torch.arange(rows, device=device)[:, None]
    b = torch.arange(blocks, device=device)[None, :]
    return ((r // 128) * (-(-blocks // 4)) + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4


def _tiled(power):
    rows, blocks = power.shape
    s = torch.zeros(-(-rows // 128) * -(-blocks // 4) * 512, dtype=torch.uint8, device=power.device)
    s[_tile_places(rows, blocks, power.device)] = power
    return s


def _from_mx4(codes, power):
    """The values in 32 bits."""
    c = codes.int()
    e, half = (c >> 1) & 3, (c & 1).float() / 2
    v = torch.where(e == 0, half, (half + 1) * (1 << (e - 1).clamp(min=0)).float())
    v = torch.where(c >= 8, -v, v).view(codes.shape[0], -1, 32)
    p = power.int()
    # 2^-127 is below the normal numbers: half of 2^-126
    scale = torch.where(p > 0, (p << 23).view(torch.float32), torch.full_like(v[:, :, 0], 2.0 ** -127))
    return (v * scale[:, :, None]).view(codes.shape[0], -1)


def run(state):
    return _calls(state) if own else _plain(state)


def _calls(s):
    from dense_fp32_gemm_gb300 import binding

    case = s["case"]
    form = case["form"]
    if case["kind"] == "norm":
        if form == "i8":
            q, scale, h = binding.rms_norm_i8(s["x"], s["weight"], residual=s["residual"], eps=EPS)
            return {"q": q, "scale": scale, "h": h}
        y, h, rstd = binding.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        if form == "y":
            return {"y": y, "h": h}
        dx, dweight = binding.rms_norm_grad(s["dy"], h, s["weight"], rstd, dH=s["dh"])
        return {"y": y, "h": h, "dx": dx, "dweight": dweight}
    if case["kind"] == "ce":
        loss, lse = binding.linear_cross_entropy(s["x"], s["w"], s["target"], ignore_index=IGNORE)
        if form == "loss":
            return {"loss": loss, "lse": lse}
        dx, dw = binding.linear_cross_entropy_grad(s["x"], s["w"], s["target"], lse, s["dloss"], ignore_index=IGNORE)
        return {"loss": loss, "dx": dx, "dw": dw}
    q, scale = binding.mx4_quantize(s["x"])
    if form == "round":
        return binding.mx4_dequantize(q, scale, case["k"], out_dtype=s["x"].dtype)
    return binding.mx4_gemm(q, scale, s["w"], s["w_scale"], out_dtype=s["x"].dtype)


def _plain(s):
    case = s["case"]
    form, t = case["form"], s["x"].dtype
    if case["kind"] == "norm":
        h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(t)
        v, w = h.float(), s["weight"].float()
        rstd = (v.square().mean(dim=1, keepdim=True) + EPS).rsqrt()
        if form == "i8":
            # the scale's factor rstd is common to a row: its integers do not depend on it
            u = v * w
            step = u.abs().amax(dim=1) / s["most"]
            q = torch.where(step[:, None] > 0, u / step[:, None], torch.zeros_like(u)).round().clamp(-127, 127)
            return {"q": q.to(torch.int8), "scale": step * rstd[:, 0], "h": h}
        n = v * rstd
        out = {"y": (n * w).to(t), "h": h}
        if form == "train":
            dy = s["dy"].float()
            dn = dy * w
            dx = (dn - n * (dn * n).mean(dim=1, keepdim=True)) * rstd + s["dh"].float()
            out["dx"] = dx.to(t)
            out["dweight"] = (dy * n).sum(dim=0).to(s["weight"].dtype)
        return out
    if case["kind"] == "ce":
        logits = s["x"].float() @ s["w"].float().mT
        counted = s["target"] != IGNORE
        target = torch.where(counted, s["target"], 0)[:, None]
        most = logits.amax(dim=1, keepdim=True)
        lse = most + (logits - most).exp().sum(dim=1, keepdim=True).log()
        loss = torch.where(counted, (lse - logits.gather(1, target))[:, 0], 0.0)
        if form == "loss":
            return {"loss": loss, "lse": lse[:, 0]}
        d = torch.where(counted, s["dloss"], 0.0)[:, None]
        p = (logits - lse).exp_()
        p = p.scatter_add_(1, target, torch.full_like(lse, -1.0)).mul_(d)
        return {"loss": loss, "dx": (p @ s["w"].float()).to(t), "dw": (p.mT @ s["x"].float()).to(t)}
    codes, power = _to_mx4(s["x"])
    if form == "round":
        return _from_mx4(codes, power)[:, : case["k"]].to(t)
    w = torch.stack([s["w"] & 15, s["w"] >> 4], dim=2).view(case["n"], -1)
    w_power = s["w_scale"][_tile_places(case["n"], w.shape[1] // 32, w.device)]
    return (_from_mx4(codes, power) @ _from_mx4(w, w_power).mT).to(t)


def work(case):
    size = TYPES[case["type"]].itemsize
    form = case["form"]
    if case["kind"] == "norm":
        m, n = case["m"], case["n"]
        weight = TYPES[case["weight"]].itemsize * n
        there = size * m * n * (3 if case["residual"] else 1)            # x, residual, h
        if form == "i8":
            return {"bytes": there + m * n + 4 * m + weight, "flops": 6 * m * n}
        if form == "y":
            return {"bytes": there + size * m * n + weight, "flops": 5 * m * n}
        return {"bytes": there + size * m * n * 5 + 3 * weight, "flops": 15 * m * n}   # y; dy, dh, h, dx
    if case["kind"] == "ce":
        t, v, h = case["t"], case["v"], case["h"]
        there = size * h * (t + v) + 16 * t
        if form == "loss":
            return {"bytes": there, "flops": 2 * t * v * h}
        return {"bytes": 2 * there, "flops": 6 * t * v * h}
    m, k = case["m"], case["k"]
    if form == "round":
        return {"bytes": 2 * size * m * k, "flops": 4 * m * k}
    n = case["n"]
    return {"bytes": size * m * k + n * -(-k // 32) * 17 + size * m * n, "flops": 2 * m * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    kind, form = case["kind"], case["form"]
    x = s["x"].double()
    if kind == "norm":
        h = x
        if s["residual"] is not None:
            h = torch.add(x, s["residual"].double()).to(s["x"].dtype)
        w = s["weight"].double()
        f = h.double()
        r = 1.0 / torch.sqrt(torch.einsum("ij,ij->i", f, f) / f.shape[1] + EPS)
        if form == "i8":
            # product and quotients are FP32 values by definition, rounded to nearest
            u = (f * w).float().double()
            step = (u.abs().max(dim=1).values / 127.0).float().double()
            safe = torch.where(step == 0, torch.ones_like(step), step)
            q = torch.clamp(torch.round((u / safe[:, None]).float().double()), -127, 127)
            return {"q": q.to(torch.int8), "scale": step * r, "h": h}
        z = f * r[:, None]
        out = {"y": z * w, "h": h}
        if form == "train":
            g = s["dy"].double()
            gw = g * w
            share = torch.einsum("ij,ij->i", gw, z) / f.shape[1]
            out["dx"] = r[:, None] * (gw - share[:, None] * z) + s["dh"].double()
            out["dweight"] = torch.einsum("ij,ij->j", g, z)
        return out
    if kind == "ce":
        w = s["w"].double()
        z = torch.einsum("th,vh->tv", x, w)
        lse = torch.logsumexp(z, dim=1)
        rows = torch.nonzero(s["target"] != IGNORE)[:, 0]
        at = s["target"][rows]
        loss = torch.zeros_like(lse)
        loss[rows] = lse[rows] - z[rows, at]
        if form == "loss":
            return {"loss": loss, "lse": lse}
        z.sub_(lse[:, None]).exp_()
        z[rows, at] -= 1.0
        d = torch.zeros_like(lse)
        d[rows] = s["dloss"].double()[rows]
        z.mul_(d[:, None])
        return {"loss": loss, "dx": torch.einsum("tv,vh->th", z, w), "dw": torch.einsum("tv,th->vh", z, x)}

    powers = torch.tensor([2.0 ** p for p in range(-127, 129)], dtype=torch.float64, device=x.device)

    def rounded(v):
        """The nearest of the 4-bit values, block by block, found by the borders between them."""
        rows, k = v.shape
        b = torch.zeros((rows, -(-k // 32) * 32), dtype=torch.float64, device=v.device)
        b[:, :k] = v
        b = b.view(rows, -1, 32)
        top = b.abs().max(dim=2).values
        # the last power of two that is at most the block's largest, two steps down
        at = torch.searchsorted(powers, top.contiguous(), right=True) - 1
        unit = powers[(at - 2).clamp(min=0)][:, :, None]
        a, out = (b / unit).abs(), torch.zeros_like(b)
        for border, step, up in ((0.25, 0.5, False), (0.75, 0.5, True), (1.25, 0.5, False), (1.75, 0.5, True),
                                 (2.5, 1.0, False), (3.5, 1.0, True), (5.0, 2.0, False)):
            out += step * ((a >= border) if up else (a > border))
        return (out * torch.sign(b) * unit).view(rows, -1)

    q = rounded(x)
    if form == "round":
        return q[:, : case["k"]]
    low, high = s["w"].long() % 16, s["w"].long() // 16
    codes = torch.stack([low, high], dim=-1).flatten(1)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=codes.device)
    table = torch.cat([table, -table])
    n, k = codes.shape
    # from the tiles of 128 rows x 4 blocks: (row tile, block tile, r % 32, r // 32, b % 4)
    tiles = s["w_scale"].view(-(-n // 128), -1, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-(-n // 128) * 128, -1)
    w = table[codes].view(n, -1, 32) * powers[tiles[:n, : k // 32].long()][:, :, None]
    return torch.einsum("mk,nk->mn", q, w.view(n, k))
