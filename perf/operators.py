"""What is measured of the fused block operators: RMS norm and gated activation
with FP8 outputs, their backward passes from FP8 activation checkpoints, and
the transposed requantization of a checkpoint.

Sizes are those of the benchmark and the tests: hidden 4096 with FFN 14336 at
8192 tokens, hidden 5120 with FFN 20480 at 16384 tokens, the MLP's 512 and
2048, and ragged ones between them.

``run`` computes the operators in elementary torch operations in 32 bits, or,
where ``own`` is set, calls the framework.  FP8 tensors are returned as torch's
FP8 types, so that codes are compared as the values they stand for.
"""
from __future__ import annotations

import math

import torch

own = False

TILE = 128
FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
# the largest listed case's elements of the wide side (rows x FFN)
MOST = 8192 * 14336


def listed():
    return [
        # one token of a decode step: the launch and one row's latency
        dict(name="norm 1x4096 tiles", op="norm", rows=1, cols=4096, type="bf16", out="tiles", residual=True, checkpoint=False),
        # the norm before a block's FFN at a training step: FP8 operand, FP8 checkpoint of the residual stream
        dict(name="norm 8192x4096 tiles+ckpt", op="norm", rows=8192, cols=4096, type="bf16", out="tiles", residual=True, checkpoint=True),
        # a ragged token count under delayed scaling (one known scale, the amax recorded)
        dict(name="norm 16381x5120 delayed", op="norm", rows=16381, cols=5120, type="bf16", out="delayed", residual=True, checkpoint=False),
        # its backward from the 8-bit checkpoint, joining the residual branch's gradient
        dict(name="norm-bwd 8192x4096 ckpt", op="norm_backward", rows=8192, cols=4096, type="bf16", saved="checkpoint", residual=True),
        # odd row length (rows not 16-byte aligned) with the stored 16-bit input
        dict(name="norm-bwd 1000x2047 stored", op="norm_backward", rows=1000, cols=2047, type="f16", saved="stored", residual=False),
        # one token through the gated activation
        dict(name="swiglu 1x14336 tiles", op="swiglu", rows=1, cols=14336, type="bf16", out="tiles", checkpoint=False),
        # the FFN's activation at a training step: FP8 operand, FP8 checkpoint of the up projection
        dict(name="swiglu 8192x14336 tiles+ckpt", op="swiglu", rows=8192, cols=14336, type="bf16", out="tiles", checkpoint=True),
        # its backward from the checkpoint, with every FP8 operand that dgrad and wgrad read
        dict(name="swiglu-bwd 8192x14336 ckpt", op="swiglu_backward", rows=8192, cols=14336, type="bf16", saved="checkpoint", out="tiles"),
        # FP16 training with stored activations at an odd width
        dict(name="swiglu-bwd 777x2049 stored", op="swiglu_backward", rows=777, cols=2049, type="f16", saved="stored", out="same"),
        # the normalised tensor as the weight gradient's operand, recomputed from the checkpoint
        dict(name="requant 8192x4096 norm", op="requantize", rows=8192, cols=4096, type="bf16", factors=True),
        # a plain transposition at ragged sizes
        dict(name="requant 4099x1111", op="requantize", rows=4099, cols=1111, type="bf16", factors=False),
        # a wide hidden state in FP32 with a 16-bit output
        dict(name="norm 2048x20480 f32", op="norm", rows=2048, cols=20480, type="f32", out="half", residual=False, checkpoint=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm_backward", "swiglu", "swiglu_backward", "requantize"])
    cols = spread(64, 20480)
    how = rng.random()
    if how < 0.4:                      # whole tiles
        cols = max(128, cols // 128 * 128)
    elif how < 0.7:                    # whole 16-byte vectors
        cols = max(8, cols // 8 * 8)
    t = rng.choice(["bf16", "bf16", "f16", "f32"])
    rows = spread(1, max(1, min(16384, MOST // 2 // cols)))
    case = dict(op=op, rows=rows, cols=cols, type=t)
    if op in ("norm", "swiglu"):
        case["out"] = rng.choice(["tiles", "delayed", "half"])
        case["checkpoint"] = rng.random() < 0.5
    if op in ("norm", "norm_backward"):
        case["residual"] = rng.random() < 0.5
    if op in ("norm_backward", "swiglu_backward"):
        case["saved"] = rng.choice(["checkpoint", "stored"])
    if op == "swiglu_backward":
        case["out"] = rng.choice(["tiles", "same"])
        if case["out"] == "tiles":     # a GEMM operand's tiles must not straddle the two halves
            case["cols"] = max(128, cols // 128 * 128)
    if op == "requantize":
        case["type"] = rng.choice(["bf16", "f16"])
        case["factors"] = rng.random() < 0.5
    return case


def _blocks(n):
    return -(-n // TILE)


# ------------------------------------------------------------------ inputs ---

def prepare(case, seed):
    d = "cuda"
    gen = torch.Generator(device=d).manual_seed(seed)
    rows, cols, t = case["rows"], case["cols"], TYPES[case["type"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=d)

    def heavy(r, c):                   # token rows with a few loud channels
        return normal(r, c).mul_(normal(c).mul_(0.5).exp_()).to(t)

    def bytes_(*shape):
        return torch.empty(*shape, dtype=torch.uint8, device=d)

    def f32(*shape):
        return torch.empty(*shape, dtype=torch.float32, device=d)

    s = {"case": case}
    op = case["op"]
    if op in ("norm", "norm_backward") or case.get("factors"):
        s["gamma"] = (1.0 + 0.1 * normal(cols)).to(t)
    if op == "norm":
        s["x"] = heavy(rows, cols)
        if case["residual"]:
            s["res"] = heavy(rows, cols)
            s["h"] = torch.empty_like(s["x"])
    elif op == "swiglu":
        s["x"] = heavy(rows, 2 * cols)
    if op in ("norm", "swiglu"):
        wide = cols if op == "norm" else 2 * cols
        if case["out"] == "half":
            s["y"] = torch.empty(rows, cols, dtype=torch.float16 if t is torch.float16 else torch.bfloat16, device=d)
        else:
            s["q"] = bytes_(rows, cols)
        if case["out"] == "tiles":
            s["s"] = f32(_blocks(cols), rows)
        if case["out"] == "delayed":
            s["scale"] = torch.full((1,), FP8_MAX / 64.0, device=d)
            s["amax"] = torch.zeros(1, device=d)
        if case["checkpoint"]:
            s["cq"] = bytes_(rows, wide)
            s["cs"] = f32(_blocks(cols) * (wide // cols), rows)
        if op == "norm":
            s["rstd"] = f32(rows)
    if op in ("norm_backward", "swiglu_backward"):
        wide = cols if op == "norm_backward" else 2 * cols
        x = heavy(rows, wide)
        s["dy"] = normal(rows, cols).mul_(normal(rows, 1).mul_(0.5).exp_() * 1e-2).to(t)
        if op == "norm_backward":
            s["rstd"] = (x.float().square().mean(1) + EPS).rsqrt()
            s["work"] = f32(min(rows, 512), cols)
            s["dgamma"] = f32(cols)
            if case["residual"]:
                s["dres"] = normal(rows, cols).mul_(1e-2).to(t)
        if case["saved"] == "stored":
            s["x"] = x
        else:
            halves = [_encode_tiles(p.float()) for p in x.split(cols, 1)]
            s["cq"] = torch.cat([q for q, _ in halves], 1).view(torch.uint8)
            s["cs"] = torch.cat([c for _, c in halves], 0)
        if case.get("out", "same") == "same":
            s["dx"] = torch.empty(rows, wide, dtype=t, device=d)
        else:
            s["q"], s["s"] = bytes_(rows, 2 * cols), f32(2 * _blocks(cols), rows)
            s["qt"], s["st"] = bytes_(2 * cols, rows), f32(_blocks(rows), 2 * cols)
            s["yt"], s["yst"] = bytes_(cols, rows), f32(_blocks(rows), cols)
    if op == "requantize":
        x = heavy(rows, cols)
        q, s["cs"] = _encode_tiles(x.float())
        s["cq"] = q.view(torch.uint8)
        if case["factors"]:
            s["rstd"] = (x.float().square().mean(1) + EPS).rsqrt()
        s["qt"], s["st"] = bytes_(cols, rows), f32(_blocks(rows), cols)
    return s


# ------------------------------------------------------------- plain forms ---

def _encode_tiles(v):
    """FP8 codes of 32-bit values [rows, cols] in 1x128 tiles, and scale_inv [blocks, rows]."""
    rows, cols = v.shape
    nb = _blocks(cols)
    p = torch.nn.functional.pad(v, (0, nb * TILE - cols)).view(rows, nb, TILE)
    amax = p.abs().amax(2)
    scale = torch.where(amax > 0, FP8_MAX / amax, torch.ones_like(amax))
    q = (p * scale[:, :, None]).clamp(-FP8_MAX, FP8_MAX).to(FP8)
    return q.view(rows, nb * TILE)[:, :cols].contiguous(), (1.0 / scale).t().contiguous()


def _decode_tiles(q, s, cols):
    """32-bit values of FP8 codes [rows, cols * parts], tiles starting again at each part."""
    rows = q.shape[0]
    out = []
    for part, sp in zip(q.view(FP8).split(cols, 1), s.split(_blocks(cols), 0)):
        each = sp.t().repeat_interleave(TILE, 1)[:, :cols]
        out.append(part.float() * each)
    return out


def _outputs(s, y, out):
    case = s["case"]
    if case["out"] == "half":
        out["y"] = y.to(s["y"].dtype)
    elif case["out"] == "delayed":
        out["q"] = (y * s["scale"]).clamp(-FP8_MAX, FP8_MAX).to(FP8)
        out["amax"] = torch.maximum(s["amax"], y.abs().amax())
    else:
        out["q"], out["s"] = _encode_tiles(y)


def _plain(s):
    case = s["case"]
    op, cols = case["op"], case["cols"]
    out = {}
    if op == "norm":
        h = s["x"]
        if case["residual"]:
            h = (h.float() + s["res"].float()).to(h.dtype)
            out["h"] = h
        h = h.float()
        r = 1.0 / torch.sqrt(h.square().mean(1) + EPS)
        out["rstd"] = r
        _outputs(s, h * r[:, None] * s["gamma"].float(), out)
        if case["checkpoint"]:
            out["cq"], out["cs"] = _encode_tiles(h)
    elif op == "norm_backward":
        h = s["x"].float() if "x" in s else _decode_tiles(s["cq"], s["cs"], cols)[0]
        dy, r = s["dy"].float(), s["rstd"][:, None]
        n = h * r
        g = dy * s["gamma"].float()
        dx = r * (g - n * (g * n).mean(1, keepdim=True))
        if case["residual"]:
            dx = dx + s["dres"].float()
        out["dx"] = dx.to(s["dy"].dtype)
        out["dgamma"] = (dy * n).sum(0)
    elif op == "swiglu":
        g, u = s["x"].float().split(cols, 1)
        _outputs(s, g / (1.0 + torch.exp(-g)) * u, out)
        if case["checkpoint"]:
            a, b = _encode_tiles(g), _encode_tiles(u)
            out["cq"], out["cs"] = torch.cat([a[0].view(torch.uint8), b[0].view(torch.uint8)], 1).view(FP8), torch.cat([a[1], b[1]], 0)
    elif op == "swiglu_backward":
        g, u = s["x"].float().split(cols, 1) if "x" in s else _decode_tiles(s["cq"], s["cs"], cols)
        dy = s["dy"].float()
        sig = 1.0 / (1.0 + torch.exp(-g))
        silu = g * sig
        dx = torch.cat([dy * u * sig * (1.0 + g * (1.0 - sig)), dy * silu], 1)
        if case["out"] == "same":
            out["dx"] = dx.to(s["dy"].dtype)
        else:
            out["q"], out["s"] = _encode_tiles(dx)
            out["qt"], out["st"] = _encode_tiles(dx.t())
            out["yt"], out["yst"] = _encode_tiles((silu * u).t())
    else:
        v = _decode_tiles(s["cq"], s["cs"], cols)[0]
        if case["factors"]:
            v = v * s["rstd"][:, None] * s["gamma"].float()
        out["qt"], out["st"] = _encode_tiles(v.t())
    return out


# ------------------------------------------------------ the framework's own ---

def _own(s):
    import mixed_precision_numerics_amd as amp
    case = s["case"]
    op, rows, cols = case["op"], case["rows"], case["cols"]
    t = {"bf16": amp.BF16, "f16": amp.F16, "f32": amp.F32}[case["type"]]

    def tiles(q, scales):
        return amp.Fp8Tiles(s[q], s[scales], s[q].shape[1], s[scales].shape[1], amp.E4M3) if q in s and scales in s else None

    out = {}
    if op in ("norm", "swiglu"):
        half = case["out"] == "half"
        yt = (amp.F16 if t == amp.F16 else amp.BF16) if half else amp.E4M3
        y = s["y"] if half else s["q"] if case["out"] == "delayed" else None
        yq, ckpt = tiles("q", "s"), tiles("cq", "cs")
        if op == "norm":
            amp.amp_rmsnorm(s["x"], t, rows, cols, cols, s.get("res"), cols, s["gamma"], t, EPS, s.get("h"), cols,
                            y, yt, cols, s.get("scale"), s.get("amax"), yq, ckpt, s["rstd"])
        else:
            amp.amp_swiglu(s["x"], t, rows, cols, 2 * cols, y, yt, cols, s.get("scale"), s.get("amax"), yq, ckpt)
        names = ("h", "rstd", "y", "q", "s", "amax", "cq", "cs")
    elif op == "norm_backward":
        amp.amp_rmsnorm_backward(s["dy"], t, rows, cols, cols, s.get("x"), cols, tiles("cq", "cs"), s["gamma"], t, s["rstd"],
                                 s.get("dres"), cols, s["dx"], cols, s["dgamma"], s["work"])
        names = ("dx", "dgamma")
    elif op == "swiglu_backward":
        amp.amp_swiglu_backward(s["dy"], t, rows, cols, cols, s.get("x"), 2 * cols, tiles("cq", "cs"), s.get("dx"), 2 * cols,
                                tiles("q", "s"), tiles("qt", "st"), tiles("yt", "yst"))
        names = ("dx", "q", "s", "qt", "st", "yt", "yst")
    else:
        amp.amp_requantize_blockwise(tiles("cq", "cs"), rows, cols, s.get("rstd"), s.get("gamma"), t, tiles("qt", "st"))
        names = ("qt", "st")
    for n in names:
        if n in s:
            out[n] = s[n].view(FP8) if s[n].dtype == torch.uint8 else s[n]
    return out


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work ---

def work(case):
    rows, cols, op = case["rows"], case["cols"], case["op"]
    n, e = rows * cols, BYTES[case["type"]]
    scales = 4 * rows * _blocks(cols)
    scales_t = 4 * cols * _blocks(rows)
    y = {"half": 2 * n, "delayed": n, "tiles": n + scales}
    if op == "norm":
        b = n * e + cols * e + 4 * rows + y[case["out"]]
        b += 2 * n * e if case["residual"] else 0
        b += n + scales if case["checkpoint"] else 0
        f = 8 * n
    elif op == "norm_backward":
        b = 2 * n * e + cols * (e + 4) + 4 * rows
        b += n * e if case["residual"] else 0
        b += n * e if case["saved"] == "stored" else n + scales
        f = 12 * n
    elif op == "swiglu":
        b = 2 * n * e + y[case["out"]]
        b += 2 * (n + scales) if case["checkpoint"] else 0
        f = 10 * n
    elif op == "swiglu_backward":
        b = n * e + (2 * n * e if case["saved"] == "stored" else 2 * (n + scales))
        b += 2 * n * e if case["out"] == "same" else 2 * (n + scales) + 3 * (n + scales_t)
        f = 20 * n
    else:
        b = 2 * n + scales + scales_t + (4 * rows + cols * e if case["factors"] else 0)
        f = 4 * n
    return {"bytes": b, "flops": f}


# ----------------------------------------------------------- 64-bit values ---

def _wide(q, s, first, cols):
    """Values in 64 bits of the part of a checkpoint whose columns start at `first`."""
    at = torch.arange(cols, device=q.device)
    return q[:, first:first + cols].view(FP8).double() * s.double()[first // cols * _blocks(cols) + at // TILE].t()


def _scaled(v):
    """What tile codes stand for before their rounding, and scale_inv: a loop over the K blocks in 64 bits."""
    q, inv = torch.empty_like(v), []
    for c in range(0, v.shape[1], TILE):
        top = v[:, c:c + TILE].abs().max(1).values
        k = torch.where(top == 0, torch.ones_like(top), top / FP8_MAX)
        q[:, c:c + TILE] = v[:, c:c + TILE] / k[:, None]
        inv.append(k)
    return q, torch.stack(inv)


def exact(case, seed):
    s = prepare(case, seed)
    op, cols = case["op"], case["cols"]
    out = {}
    y = None
    if op == "norm":
        h = s["x"].double()
        if case["residual"]:
            h = (h + s["res"].double()).to(s["x"].dtype).double()   # the stored stream is what is normalised
            out["h"] = h
        ms = torch.linalg.vector_norm(h, dim=1) ** 2 / cols
        out["rstd"] = (ms + EPS) ** -0.5
        y = h * s["gamma"].double() * out["rstd"].unsqueeze(1)
        if case["checkpoint"]:
            out["cq"], out["cs"] = _scaled(h)
    elif op == "swiglu":
        g, u = s["x"][:, :cols].double(), s["x"][:, cols:].double()
        y = u * g * torch.sigmoid(g)
        if case["checkpoint"]:
            (a, i), (b, j) = _scaled(g), _scaled(u)
            out["cq"], out["cs"] = torch.cat([a, b], 1), torch.cat([i, j])
    elif op == "norm_backward":
        # y_i = gamma_i h_i r and r^-2 = mean(h^2) + eps give dr/dh_i = -h_i r^3 / N
        h = s["x"].double() if "x" in s else _wide(s["cq"], s["cs"], 0, cols)
        r, dy, gamma = s["rstd"].double(), s["dy"].double(), s["gamma"].double()
        dr = (dy * h * gamma).sum(1)
        dx = (dy * gamma) * r.unsqueeze(1) - h * (dr * r ** 3 / cols).unsqueeze(1)
        out["dx"] = dx + s["dres"].double() if case["residual"] else dx
        out["dgamma"] = (dy * h * r.unsqueeze(1)).sum(0)
    elif op == "swiglu_backward":
        g, u = (s["x"][:, :cols].double(), s["x"][:, cols:].double()) if "x" in s else (
            _wide(s["cq"], s["cs"], 0, cols), _wide(s["cq"], s["cs"], cols, cols))
        dy = s["dy"].double()
        p, m = torch.sigmoid(g), torch.sigmoid(-g)
        du = dy * g * p
        dg = dy * u * (p + g * p * m)
        if case["out"] == "same":
            out["dx"] = torch.cat([dg, du], 1)
        else:
            (a, i), (b, j) = _scaled(dg), _scaled(du)
            out["q"], out["s"] = torch.cat([a, b], 1), torch.cat([i, j])
            (a, i), (b, j) = _scaled(dg.t()), _scaled(du.t())
            out["qt"], out["st"] = torch.cat([a, b], 0), torch.cat([i, j], 1)
            out["yt"], out["yst"] = _scaled((g * p * u).t())
    else:
        v = _wide(s["cq"], s["cs"], 0, cols)
        if case["factors"]:
            v = v * s["gamma"].double() * s["rstd"].double().unsqueeze(1)
        out["qt"], out["st"] = _scaled(v.t())
    if y is not None:
        if case["out"] == "half":
            out["y"] = y
        elif case["out"] == "delayed":
            out["q"] = (y * s["scale"].double()).clamp(-FP8_MAX, FP8_MAX)
            out["amax"] = y.abs().max().reshape(1)
        else:
            out["q"], out["s"] = _scaled(y)
    return out
