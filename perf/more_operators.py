"""What is measured of the training step around a gated feed-forward block: both
projections, the activation and the product in one call, its backward pass, the
global norm over a list of gradient tensors, and their clipping.

Sizes are those of the benchmark and the tests: hidden 4096 with FFN 14336 at
8192 tokens, hidden 5120 with FFN 20480, the MLP's 512 and 2048, and ragged ones
between them; the gradient lists are those of such blocks' weights.

``run`` computes the operators in elementary torch operations in 32 bits (sums
of squares in 64), or, where ``own`` is set, calls the framework.
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
# the largest listed case's products (tokens x hidden x FFN) and gradient elements
MOST_MACS = 8192 * 4096 * 14336
MOST_GRADS = 900_000_000


def listed():
    return [
        # one token of a decode step: the weights stream past it
        dict(name="ffn 1x4096x14336", op="ffn", M=1, K=4096, F=14336, type="bf16", keep=False),
        # a small batch of sequences, one token each
        dict(name="ffn 33x5120x20480", op="ffn", M=33, K=5120, F=20480, type="bf16", keep=False),
        # a training step's block, with the projections kept for the backward pass
        dict(name="ffn 8192x4096x14336 keep", op="ffn", M=8192, K=4096, F=14336, type="bf16", keep=True),
        # a prompt of ragged length
        dict(name="ffn 1000x4096x14336", op="ffn", M=1000, K=4096, F=14336, type="bf16", keep=False),
        # the MLP's widths in FP16 at an odd token count
        dict(name="ffn-bwd 777x512x2048 f16", op="ffn_backward", M=777, K=512, F=2048, type="f16", saved="stored"),
        # the training step's backward pass from the kept projections
        dict(name="ffn-bwd 8192x4096x14336 stored", op="ffn_backward", M=8192, K=4096, F=14336, type="bf16", saved="stored"),
        # the same block under activation checkpointing: the projections are formed again, y comes with them
        dict(name="ffn-bwd 4000x5120x10240 again", op="ffn_backward", M=4000, K=5120, F=10240, type="bf16", saved="again"),
        # odd widths, rows that are not 16-byte aligned
        dict(name="ffn-bwd 300x1001x2047 odd", op="ffn_backward", M=300, K=1001, F=2047, type="bf16", saved="stored"),
        # the two-layer MLP's four gradients in FP16 under loss scaling: the launch and its latency
        dict(name="norm mlp f16", op="norm", list="mlp", layers=1, hidden=512, ffn=2048, type="f16", overflow=False),
        # four blocks' weight gradients, the norm that a step clips by
        dict(name="norm 4 blocks bf16", op="norm", list="blocks", layers=4, hidden=4096, ffn=14336, type="bf16", overflow=False),
        # many small tensors of odd lengths that start anywhere, clipped in place of their FP32 accumulators
        dict(name="clip 700 ragged f32", op="clip", list="ragged", layers=700, hidden=64, ffn=2048, type="f32", out="f32"),
        # BF16 gradients unscaled and clipped into FP32 for the optimizer
        dict(name="clip 4 blocks bf16 to f32", op="clip", list="blocks", layers=4, hidden=4096, ffn=14336, type="bf16", out="f32"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["ffn", "ffn", "ffn_backward", "ffn_backward", "norm", "clip"])
    if op in ("ffn", "ffn_backward"):
        K, F = spread(64, 5120), spread(128, 20480)
        how = rng.random()
        if how < 0.45:                 # whole tiles, as models have them
            K, F = max(64, K // 128 * 128), max(128, F // 256 * 256)
        elif how < 0.8:                # whole 16-byte vectors
            K, F = max(8, K // 8 * 8), max(8, F // 8 * 8)
        most = MOST_MACS // (1 if op == "ffn" else 2) // (K * F)
        case = dict(op=op, M=spread(1, max(1, min(8192, most))), K=K, F=F, type=rng.choice(["bf16", "bf16", "f16"]))
        if op == "ffn":
            case["keep"] = rng.random() < 0.4
        else:
            case["saved"] = rng.choice(["stored", "again"])
        return case
    which = rng.choice(["mlp", "blocks", "ragged"])
    hidden, ffn = spread(64, 4096), spread(256, 14336)
    each = {"mlp": 12 * hidden * ffn, "blocks": 2 * hidden * (hidden + hidden // 4) + 3 * hidden * ffn, "ragged": ffn}[which]
    layers = spread(1, max(1, min(1500 if which == "ragged" else 48, MOST_GRADS // 2 // each)))
    case = dict(op=op, list=which, layers=layers, hidden=hidden, ffn=ffn, type=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if op == "norm":
        case["overflow"] = rng.random() < 0.2
    else:
        case["out"] = rng.choice([case["type"], "f32", "bf16"])
    return case


def _lengths(case):
    """Elements of each gradient tensor of the case."""
    h, f = case["hidden"], case["ffn"]
    if case["list"] == "mlp":          # two linear layers with biases, ten classes
        return [h * f, f, f * 10, 10] * case["layers"]
    if case["list"] == "blocks":       # QKV with grouped heads, output, gate and up, down, two norms
        return [h * (h + h // 4 * 2), h * h, 2 * f * h, h * f, h, h] * case["layers"]
    # lengths from 1 to twice the mean, in an order without pattern
    return [1 + (i * 7919 + 13 * h) % (2 * f) for i in range(case["layers"])]


# ------------------------------------------------------------------ inputs ---

def prepare(case, seed):
    d = "cuda"
    gen = torch.Generator(device=d).manual_seed(seed)
    t = TYPES[case["type"]]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=d, dtype=dtype)

    def out(*shape, dtype=t):
        return torch.empty(*shape, device=d, dtype=dtype)

    s = {"case": case}
    op = case["op"]
    if op in ("ffn", "ffn_backward"):
        M, K, F = case["M"], case["K"], case["F"]
        # normalised token rows with a few loud channels; projections of unit variance
        s["x"] = normal(M, K).mul_(normal(K).mul_(0.25).exp_()).to(t)
        s["w"] = normal(2 * F, K).mul_(K ** -0.5).to(t)
        if op == "ffn":
            s["y"] = out(M, F)
            if case["keep"]:
                s["gu"] = out(M, 2 * F)
        else:
            # a gradient whose size differs from token to token, under a loss scale in FP16
            s["dy"] = normal(M, F).mul_(normal(M, 1).mul_(0.5).exp_() * (0.16 if t is torch.float16 else 0.01)).to(t)
            if case["saved"] == "stored":
                s["gu"] = normal(M, 2 * F).to(t)
            else:
                s["y"] = out(M, F)
            s["dgu"], s["dx"], s["dw"] = out(M, 2 * F), out(M, K), out(2 * F, K)
            if own:                    # the work area that a training program keeps for its products
                import mixed_precision_numerics_amd as amp
                s["work"] = out(amp.GEMM_SWIGLU_WORK, dtype=torch.float32)
        return s
    # gradients under a loss scale (FP16), each tensor of its own size, one after another in memory as they were made
    lengths = _lengths(case)
    S = 1024.0 if t is torch.float16 else 1.0
    room = [n + 1 if case["list"] == "ragged" else -(-n // 8) * 8 for n in lengths]
    flat = torch.empty(sum(room), device=d, dtype=t)
    at, grads = 0, []
    size = normal(len(lengths)).exp_().mul_(1e-3 * S).cpu().tolist()
    for n, r, k in zip(lengths, room, size):
        grads.append(flat[at:at + n].copy_(normal(n, dtype=t).mul_(k)))
        at += r
    if case.get("overflow"):
        g = grads[len(grads) // 2]
        g[g.numel() // 3] = float("inf")
    s["grads"], s["scale"], s["max_norm"] = grads, S, 1.0
    # what the framework's step holds: the scaler's state and, for the norm, its accumulator
    s["state"] = torch.zeros(10, device=d, dtype=torch.int32)
    s["state"].view(torch.float32)[0] = S
    if op == "norm":
        s["norm"] = torch.zeros(1025, device=d, dtype=torch.float64)
        s["result"] = torch.empty(2, device=d)
    else:
        s["coef"] = torch.full((1,), 0.37, device=d) * (1.0 + 0.1 * torch.rand(1, generator=gen, device=d))
        # the clipped gradients lie end to end
        s["out"] = torch.empty(sum(lengths), device=d, dtype=TYPES[case["out"]])
        s["outs"] = list(s["out"].split(lengths))
    if own:
        # the lists that a training program makes once, beside its parameters
        import mixed_precision_numerics_amd as amp
        kind = {"bf16": amp.BF16, "f16": amp.F16, "f32": amp.F32}
        s["list"] = amp.TensorList([(g, g.numel(), kind[case["type"]]) for g in grads])
        if op == "clip":
            s["list_out"] = amp.TensorList([(o, o.numel(), kind[case["out"]]) for o in s["outs"]])
    return s


# ------------------------------------------------------------- plain forms ---

def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "ffn":
        F, t = case["F"], s["x"].dtype
        gu = s["x"].float() @ s["w"].float().t()
        g, u = gu[:, :F], gu[:, F:]
        out = {"y": (g / (1.0 + torch.exp(-g)) * u).to(t)}
        if case["keep"]:
            out["gu"] = gu.to(t)
        return out
    if op == "ffn_backward":
        F, t = case["F"], s["x"].dtype
        x, w = s["x"].float(), s["w"].float()
        gu = s["gu"].float() if "gu" in s else x @ w.t()
        g, u = gu[:, :F], gu[:, F:]
        dy = s["dy"].float()
        sig = 1.0 / (1.0 + torch.exp(-g))
        silu = g * sig
        out = {}
        if "gu" not in s:
            out["y"] = (silu * u).to(t)
        dgu = torch.cat([dy * u * sig * (1.0 + g * (1.0 - sig)), dy * silu], 1)
        out["dgu"], out["dx"], out["dw"] = dgu.to(t), (dgu @ w).to(t), (dgu.t() @ x).to(t)
        return out
    inv = 1.0 / s["scale"]
    if op == "norm":
        total = torch.zeros((), device="cuda", dtype=torch.float64)
        bad = torch.zeros((), device="cuda", dtype=torch.bool)
        for g in s["grads"]:
            v = g.float() * inv
            total = total + v.double().square().sum()
            bad = bad | ~torch.isfinite(v).all()
        norm = torch.where(bad, torch.full_like(total, math.inf), total.sqrt()).float()
        coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
        return {"coef": torch.where(bad, torch.ones_like(coef), coef).reshape(1), "norm": norm.reshape(1), "found_inf": bad.int().reshape(1)}
    for g, o in zip(s["grads"], s["outs"]):
        o.copy_((g.float() * inv) * s["coef"])
    return {"grads": s["out"]}


# ------------------------------------------------------ the framework's own ---

def _own(s):
    import mixed_precision_numerics_amd as amp
    case = s["case"]
    op = case["op"]
    t = {"bf16": amp.BF16, "f16": amp.F16, "f32": amp.F32}[case["type"]]
    if op == "ffn":
        M, K, F = case["M"], case["K"], case["F"]
        amp.amp_gemm_swiglu(M, F, K, s["x"], t, K, s["w"], K, s["y"], F, s.get("gu"), 2 * F)
        return {k: s[k] for k in ("y", "gu") if k in s}
    if op == "ffn_backward":
        M, K, F = case["M"], case["K"], case["F"]
        amp.amp_gemm_swiglu_backward(M, F, K, s["dy"], t, F, s["x"], K, s["w"], K, s.get("gu"), 2 * F, s["dgu"], 2 * F,
                                     s.get("y"), F, s["dx"], K, s["dw"], t, K, s["work"])
        return {k: s[k] for k in ("y", "dgu", "dx", "dw") if k in s}
    if op == "norm":
        amp.amp_grad_norm_list(s["list"], True, s["state"], s["norm"], s["max_norm"], s["result"])
        return {"coef": s["result"][:1], "norm": s["result"][1:], "found_inf": s["state"][2:3]}
    amp.amp_grad_clip_list(s["list"], s["list_out"], s["state"], s["coef"])
    return {"grads": s["out"]}


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work ---

def work(case):
    e = BYTES[case["type"]]
    op = case["op"]
    if op == "ffn":
        M, K, F = case["M"], case["K"], case["F"]
        return {"bytes": e * (M * K + 2 * F * K + M * F * (3 if case["keep"] else 1)), "flops": 4 * M * K * F + 10 * M * F}
    if op == "ffn_backward":
        M, K, F = case["M"], case["K"], case["F"]
        # in: dy, x, w and the kept projections; out: dgu, dx, dw, or y where the projections are formed again
        b = M * F + M * K + 2 * F * K + 2 * M * F + M * K + 2 * F * K + (2 * M * F if case["saved"] == "stored" else M * F)
        return {"bytes": e * b, "flops": (8 if case["saved"] == "stored" else 12) * M * K * F + 20 * M * F}
    n = sum(_lengths(case))
    if op == "norm":
        return {"bytes": e * n + 8, "flops": 3 * n}
    return {"bytes": (e + BYTES[case["out"]]) * n + 4, "flops": 2 * n}


# ----------------------------------------------------------- 64-bit values ---

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("ffn", "ffn_backward"):
        F = case["F"]
        x, wg, wu = s["x"].double(), s["w"][:F].double(), s["w"][F:].double()
        g, u = (s["gu"][:, :F].double(), s["gu"][:, F:].double()) if "gu" in s and op == "ffn_backward" else (
            torch.mm(x, wg.t()), torch.mm(x, wu.t()))
        p = torch.sigmoid(g)
        out = {}
        if op == "ffn":
            out["y"] = g * p * u
            if case["keep"]:
                out["gu"] = torch.cat([g, u], 1)
            return out
        if "gu" not in s:
            out["y"] = g * p * u
        # d(g p)/dg = p + g p (1 - p), and 1 - p(g) = p(-g)
        dy = s["dy"].double()
        dg = dy * u * (p + g * p * torch.sigmoid(-g))
        du = dy * g * p
        out["dgu"] = torch.cat([dg, du], 1)
        out["dx"] = torch.mm(dg, wg) + torch.mm(du, wu)
        out["dw"] = torch.cat([torch.mm(dg.t(), x), torch.mm(du.t(), x)], 0)
        return out
    S = s["scale"]
    if op == "norm":
        bad = any(bool(torch.isinf(g).any() | torch.isnan(g).any()) for g in s["grads"])
        found = torch.tensor([bad], device="cuda").int()
        if bad:
            one = torch.ones(1, device="cuda", dtype=torch.float64)
            return {"coef": one, "norm": one * math.inf, "found_inf": found}
        parts = [torch.linalg.vector_norm(c.double()) / S for g in s["grads"] for c in g.split(1 << 26)]
        norm = torch.linalg.vector_norm(torch.stack(parts)).reshape(1)
        return {"coef": (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0), "norm": norm, "found_inf": found}
    return {"grads": torch.cat([g.double() * (s["coef"].double() / S) for g in s["grads"]])}
