"""Norm and gated activation between fine-grained FP8 GEMMs, and their
gradients (oracle).

Test infrastructure only (see ``oracle/__init__``).

Plain float64 formulas over decoded values; the only roundings are those that
the definition makes before further use (the residual stream's).  Scaling
tiles are those of ``blockwise`` (1x128 along K, ``s[kb, r]``), with a scale of
1 where ``fmax / amax`` is not a positive finite FP32 number.
"""
from __future__ import annotations

import numpy as np

from . import formats as F
from .blockwise import FMAX, TILE, _ceil


def residual_add(x, res, fmt: F.Fmt):
    """The stream after the addition, rounded once to its type."""
    return F.round_to(np.asarray(x, np.float64) + np.asarray(res, np.float64), fmt)


def rmsnorm(h, gamma, eps):
    """(y, r): y = h r gamma, r = 1 / sqrt(mean(h^2) + eps), row by row."""
    h = np.asarray(h, np.float64)
    with np.errstate(all="ignore"):
        r = 1.0 / np.sqrt((h * h).mean(axis=1) + float(np.float32(eps)))
        return h * r[:, None] * np.asarray(gamma, np.float64), r


def rmsnorm_backward(dy, h, gamma, r, dres=None):
    """(dx, dgamma) for given r: dx = r (g - n mean(g n)) + dres, n = h r, g = dy gamma."""
    n = h * r[:, None]
    g = dy * gamma
    dx = r[:, None] * (g - n * (g * n).mean(axis=1, keepdims=True))
    return (dx if dres is None else dx + dres), (dy * n).sum(axis=0)


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(g, np.float64)))


def swiglu(g, u):
    with np.errstate(invalid="ignore"):
        return g * sigmoid(g) * u


def swiglu_backward(dy, g, u):
    """(dg, du)."""
    s = sigmoid(g)
    return dy * u * s * (1.0 + g * sigmoid(-np.asarray(g, np.float64))), dy * g * s


def tile_amax(v):
    """Largest |v| of each 1x128 tile, [K blocks, rows]; NaN if a tile holds one."""
    R, K = v.shape
    out = np.zeros((_ceil(K, TILE), R))
    for kb in range(out.shape[0]):
        out[kb] = np.abs(v[:, kb * TILE:(kb + 1) * TILE]).max(axis=1)
    return out


def tile_scale(amax, fmt: F.Fmt):
    """FP32 scale of tiles with these maxima (FP32 values)."""
    with np.errstate(all="ignore"):
        sc = F.f32(FMAX[fmt.name] / F.f32(amax))
    return np.where(np.isfinite(sc) & (sc > 0), sc, 1.0)


def quantize(v, fmt: F.Fmt):
    """(codes [R, K], scale_inv [K blocks, R]) of FP32 values in 1x128 tiles."""
    v = np.asarray(v, np.float64)
    sc = tile_scale(tile_amax(v), fmt)
    each = np.repeat(sc, TILE, axis=0)[:v.shape[1]].T
    return F.encode(F.f32(v * each), fmt), F.f32(1.0 / sc)


def dequantize(codes, s, fmt: F.Fmt, parts: int = 1):
    """Values of codes [R, K]; the tiles start again at each of `parts` equal parts."""
    v = F.decode(codes, fmt)
    K = v.shape[1] // parts
    nb = _ceil(K, TILE)
    k = np.arange(v.shape[1])
    return v * np.asarray(s, np.float64)[k // K * nb + k % K // TILE].T
