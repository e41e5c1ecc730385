"""Checks of rounded outputs by intervals: a kernel's FP32 value lies within a
derived error of the float64 value, rounding is monotone, so the stored value
lies between the roundings of the interval's ends.  No other tolerance."""
import numpy as np

from oracle import block as B
from oracle import formats as F
from oracle.blockwise import FMAX, TILE

U = 2.0 ** -24            # an FP32 rounding, relative


def report(ok, got, lo, hi, what):
    bad = np.argwhere(~ok)
    assert bad.size == 0, (what, len(bad), bad[0], got[tuple(bad[0])], lo[tuple(bad[0])], hi[tuple(bad[0])])


def check_values(got, fmt, v, err, what=""):
    """got: values stored in fmt; v: float64 values; err: their FP32 counterparts' error."""
    got, v = np.asarray(got, np.float64), np.asarray(v, np.float64)
    nan = np.isnan(v)
    with np.errstate(invalid="ignore"):
        lo, hi = F.round_to(F.f32(v - err), fmt), F.round_to(F.f32(v + err), fmt)
        ok = (got >= lo) & (got <= hi)
    report(np.where(nan, np.isnan(got), ok), got, lo, hi, what)


def check_scaled(codes, fmt, v, err, sc_lo, sc_hi, what=""):
    """codes: FP8 codes of v times a scale between sc_lo and sc_hi."""
    got = F.decode(codes, fmt)
    nan = np.isnan(v)
    a = np.abs(np.where(nan, 0.0, v))
    err = np.where(nan, 0.0, np.broadcast_to(err, v.shape))
    with np.errstate(over="ignore"):
        lo = F.round_to(F.f32(F.f32(np.maximum(a - err, 0.0)) * sc_lo), fmt)
        hi = F.round_to(F.f32(F.f32(a + err) * sc_hi), fmt)
    ok = (np.abs(got) >= lo) & (np.abs(got) <= hi) & ((np.sign(got) * np.sign(v) >= 0) | (a <= err))
    report(np.where(nan, codes == 0x7F, ok), got, lo, hi, what)


def check_tiles(codes, s, fmt, v, err, what=""):
    """codes [R, K], s [K blocks, R]: v in 1x128 tiles."""
    v = np.asarray(v, np.float64)
    err = np.broadcast_to(np.asarray(err, np.float64), v.shape)
    nan = np.isnan(v)
    top = B.tile_amax(v)
    a = np.where(nan, 0.0, np.abs(v))
    e = np.where(nan | np.isinf(v), 0.0, err)
    special = ~np.isfinite(top)
    lo = np.where(special, np.nan, B.tile_amax(np.maximum(a - e, 0.0)))
    hi = np.where(special, np.nan, B.tile_amax(a + e))
    sc_lo, sc_hi = B.tile_scale(F.f32(hi), fmt), B.tile_scale(F.f32(lo), fmt)
    s = np.asarray(s, np.float64)
    # the scale is not monotone where fmax / amax overflows: below, it is 1.  A
    # tile whose interval reaches across that border may lie on either side of
    # it: at a scale of 1, or at one between fmax / hi and FLT_MAX.
    across = (sc_hi == 1.0) & (sc_lo != 1.0) & (hi < 1.0)
    sc_lo, sc_hi = np.where(across & (s == 1.0), 1.0, sc_lo), np.where(across & (s != 1.0), F.F32.max_finite, sc_hi)
    inv_lo, inv_hi = F.f32(1.0 / sc_hi), F.f32(1.0 / sc_lo)
    report((s >= inv_lo) & (s <= inv_hi), s, inv_lo, inv_hi, what + " scale_inv")

    def each(sc):
        return np.repeat(sc, TILE, axis=0)[:v.shape[1]].T
    check_scaled(codes, fmt, v, e, each(sc_lo), each(sc_hi), what)


# ---- FP32 errors of the operators, from their sequences of roundings --------

def norm_err(cols):
    """Relative error of r: a thread sums at most cols / 64 + 8 squares, a row's
    threads join in 6 + 16 additions; each is a rounding of a sum of positive
    terms, and the square root halves their total; then /N, +eps, sqrt, 1/x."""
    return ((cols / 64 + 8 + 22 + 1 + 2) / 2 + 2) * U


def dx_err(dy, h, gamma, r, dres, dx):
    """dx = r (g - n m) (+ dres): n carries 2 roundings (3 from a checkpoint),
    g one, the mean of g n its terms' 5 and the sum's cols / 64 + 31."""
    cols = h.shape[1]
    n, g = np.abs(h * r[:, None]), np.abs(dy * gamma)
    mean = (g * n).mean(axis=1, keepdims=True)
    e = np.abs(r)[:, None] * (3 * U * g + n * mean * (cols / 64 + 31 + 5 + 2 + 7) * U)
    return e + 2 * U * np.abs(dx) + (0 if dres is None else U * np.abs(dres))


def gate_err(g):
    """Relative errors of s and 1 - s: exp(-g) carries |g| (3 roundings of its
    argument, one more from a checkpoint) and 2 for the instruction's ulp, the
    reciprocal 2; weakened by 1 - s in s."""
    s, om = B.sigmoid(g), B.sigmoid(-g)
    es = (om * (4 * np.abs(g) + 2) + 4) * U
    return s, om, es, (4 * np.abs(g) + 2 + 1) * U + es


TINY = 2.0 ** -120        # results below the normal range may be flushed


def swiglu_err(g, u):
    s, _, es, _ = gate_err(g)
    return np.abs(g * u) * (s * (es + 5 * U) + TINY)


def swiglu_back_err(dy, g, u):
    s, om, es, eo = gate_err(g)
    f = np.abs(1 + g * om)
    dg = np.abs(dy * u) * (s * (f * (es + 6 * U) + np.abs(g) * om * (eo + 3 * U)) + TINY * (1 + np.abs(g)))
    return dg, np.abs(dy * g) * (s * (es + 5 * U) + TINY)
