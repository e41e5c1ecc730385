"""Gated feed-forward block (both projections, activation and product in one
call) and its backward pass on the GPU, against oracle/ffn.py in float64.

Bounds: products of 16-bit values are exact in FP32; a sum of n of them is off
by at most 2 n U sum |a||b| (each addition rounds, to nearest or not, a partial
sum of at most sum |a||b|).  |silu'| <= 1.1 and |silu''| <= 0.5 carry the
projections' errors on; the activation's own are those of block_util."""
import numpy as np
import pytest
import torch

import mixed_precision_numerics_amd as amp
from oracle import ffn as O
from oracle import formats as F
from block_util import U, check_values, swiglu_back_err, swiglu_err
from gpu_util import dev, host
from test_gpu_block import FMT, NPT, Mat, rand
from test_gpu_block_edges import Hollow

pytestmark = pytest.mark.gpu

TYPES = [amp.BF16, amp.F16]


def sum_err(n, a, b):
    return 2 * n * U * (np.abs(a) @ np.abs(b))


def projections(x, w):
    """(y, g, u) and the errors of the FP32 g and u."""
    y, g, u = O.forward(x, w)
    e = sum_err(x.shape[1], x, w.T)
    f = w.shape[0] // 2
    return y, g, u, e[:, :f], e[:, f:]


def y_err(g, u, eg, eu):
    return 1.1 * (np.abs(u) + eu) * eg + (np.abs(g) + eg) * eu + swiglu_err(np.abs(g) + eg, np.abs(u) + eu) + swiglu_err(g, u)


def dgu_err(dy, g, u, eg, eu):
    a, b = swiglu_back_err(dy, g, u)
    more = np.abs(dy) * (0.5 * (np.abs(u) + eu) * eg + 1.1 * eu)
    # the formula's own roundings at the FP32 g and u instead of the exact ones: their bounds move by a share of eg, eu
    return np.concatenate([1.01 * a + more * (1 + 64 * U), 1.01 * b + 1.1 * np.abs(dy) * eg * (1 + 64 * U)], axis=1)


def operands(M, Fn, K, t, pad, mat=Mat, seed=0):
    x = mat(M, K, t, pad, rand(seed + 1, M, K))
    w = mat(2 * Fn, K, t, pad, rand(seed + 2, 2 * Fn, K, scale=K ** -0.5))
    return x, w


def run_forward(M, Fn, K, t, pad, mat=Mat, keep=True):
    x, w = operands(M, Fn, K, t, pad, mat)
    y, gu = Mat(M, Fn, t, pad), Mat(M, 2 * Fn, t, pad)
    amp.amp_gemm_swiglu(M, Fn, K, x.d, t, x.ld, w.d, w.ld, y.d, y.ld, gu.d if keep else None, gu.ld)
    wy, g, u, eg, eu = projections(x.v, w.v)
    check_values(y.values(), FMT[t], wy, y_err(g, u, eg, eu), "y")
    if keep:
        check_values(gu.values(), FMT[t], np.concatenate([g, u], 1), np.concatenate([eg, eu], 1), "gu")
    else:
        gu.codes()


# one token to two tiles of tokens; features and summed lengths that end inside
# a 16- or 64-wide tile, a 16-byte piece, a step; pads with and without 16-byte rows
SHAPES = [(1, 1, 1), (1, 16, 128), (2, 40, 200), (16, 17, 1000), (17, 64, 72), (33, 130, 1096), (64, 24, 264), (65, 1, 7), (70, 200, 64),
          (128, 64, 128), (129, 65, 129), (200, 136, 520), (300, 33, 8)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("M,Fn,K", SHAPES)
def test_forward(M, Fn, K, pad, t):
    run_forward(M, Fn, K, t, pad, keep=pad != 0)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("pad", [8, 3])
@pytest.mark.parametrize("M,Fn,K", SHAPES)
def test_forward_reads_its_rows_alone(M, Fn, K, pad, t):
    run_forward(M, Fn, K, t, pad, Hollow)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,Fn,K", [(5, 40, 200), (100, 72, 136)])
def test_forward_that_only_keeps_the_projections(M, Fn, K, t):
    x, w = operands(M, Fn, K, t, 0)
    gu = Mat(M, 2 * Fn, t)
    amp.amp_gemm_swiglu(M, Fn, K, x.d, t, x.ld, w.d, w.ld, None, 0, gu.d, gu.ld)
    _, g, u, eg, eu = projections(x.v, w.v)
    check_values(gu.values(), FMT[t], np.concatenate([g, u], 1), np.concatenate([eg, eu], 1), "gu")


@pytest.mark.parametrize("M", [3, 100])
def test_forward_of_no_length_writes_zeros(M):
    y, gu = Mat(M, 40, amp.BF16), Mat(M, 80, amp.BF16)
    amp.amp_gemm_swiglu(M, 40, 0, None, amp.BF16, 0, None, 0, y.d, y.ld, gu.d, gu.ld)
    assert not y.codes().any() and not gu.codes().any()


def run_backward(M, Fn, K, t, pad, saved, dwt, mat=Mat, work=True, in_place=False):
    x, w = operands(M, Fn, K, t, pad, mat, 10)
    dy = mat(M, Fn, t, pad, rand(13, M, Fn))
    gu = mat(M, 2 * Fn, t, pad, rand(14, M, 2 * Fn, scale=2.0)) if saved else None
    dgu, y = (gu if in_place else Mat(M, 2 * Fn, t, pad)), Mat(M, Fn, t, pad)
    dx, dw = Mat(M, K, t, pad), Mat(2 * Fn, K, dwt, pad)
    area = torch.full((amp.GEMM_SWIGLU_WORK,), float("nan"), device="cuda") if work else None
    amp.amp_gemm_swiglu_backward(M, Fn, K, dy.d, t, dy.ld, x.d, x.ld, w.d, w.ld, gu.d if gu else None, gu.ld if gu else 0, dgu.d, dgu.ld,
                                 None if gu else y.d, y.ld, dx.d, dx.ld, dw.d, dwt, dw.ld, area)
    if gu:
        g, u = gu.v[:, :Fn], gu.v[:, Fn:]
        err = np.concatenate(swiglu_back_err(dy.v, g, u), 1)
        y.codes()
    else:
        wy, g, u, eg, eu = projections(x.v, w.v)
        check_values(y.values(), FMT[t], wy, y_err(g, u, eg, eu), "y")
        err = dgu_err(dy.v, g, u, eg, eu)
    got = dgu.values() if not (in_place and mat is Hollow) else F.decode(host(dgu.d, NPT[t])[:M * dgu.ld].reshape(M, dgu.ld)[:, :2 * Fn], FMT[t])
    check_values(got, FMT[t], O.activation_backward(dy.v, g, u), err, "dgu")
    wx, ww = O.gradients(got, x.v, w.v)
    check_values(dx.values(), FMT[t], wx, sum_err(2 * Fn, got, w.v), "dx")
    check_values(dw.values(), FMT[dwt], ww, sum_err(M, got.T, x.v), "dw")


# the summed dimensions are F and M here; the third and fourth are split into parts
BACK_SHAPES = [(1, 1, 1), (1, 16, 128), (3, 40, 200), (17, 520, 72), (40, 1024, 256), (64, 24, 264), (65, 4, 7), (129, 65, 129), (200, 136, 520),
               (2100, 64, 72), (1300, 33, 40)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("saved", [True, False])
@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("M,Fn,K", BACK_SHAPES)
def test_backward(M, Fn, K, pad, saved, t):
    run_backward(M, Fn, K, t, pad, saved, amp.F32 if pad else t)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("saved", [True, False])
@pytest.mark.parametrize("pad", [8, 3])
@pytest.mark.parametrize("M,Fn,K", BACK_SHAPES)
def test_backward_reads_its_rows_alone(M, Fn, K, pad, saved, t):
    run_backward(M, Fn, K, t, pad, saved, t, Hollow)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,Fn,K", [(3, 40, 200), (40, 1024, 256), (130, 72, 136)])
def test_backward_without_work_area_and_in_place(M, Fn, K, t):
    run_backward(M, Fn, K, t, 0, True, t, work=False)
    run_backward(M, Fn, K, t, 8, True, t, in_place=True)


@pytest.mark.parametrize("t", TYPES)
def test_backward_of_no_tokens_or_features(t):
    area = torch.empty(amp.GEMM_SWIGLU_WORK, device="cuda")
    dx, dw = Mat(5, 40, t), Mat(48, 40, amp.F32)
    w = Mat(48, 40, t, 0, rand(1, 48, 40))
    amp.amp_gemm_swiglu_backward(0, 24, 40, None, t, 24, None, 40, w.d, 40, None, 0, None, 48, None, 0, None, 0, dw.d, amp.F32, dw.ld, area)
    assert not dw.codes().any()
    amp.amp_gemm_swiglu_backward(5, 0, 40, None, t, 0, None, 40, None, 40, None, 0, None, 0, None, 0, dx.d, dx.ld, None, t, 0, area)
    assert not dx.codes().any()


# more tokens than the kernel for few of them takes, in tiles that hold little
TILE_SHAPES = [(129, 1, 1), (130, 17, 1000), (144, 130, 72), (257, 40, 7), (161, 64, 192), (400, 9, 65)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("M,Fn,K", TILE_SHAPES)
def test_small_tiles(M, Fn, K, pad, t):
    run_forward(M, Fn, K, t, pad, Hollow)
    run_backward(M, Fn, K, t, pad, False, t, Hollow)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("M,Fn,K", [(1, 300, 2050), (18, 130, 4161), (128, 33, 1025), (100, 100, 63)])
def test_few_tokens_recomputed(M, Fn, K, t):
    """The last waves' turns past the end of the summed dimension, groups of 16 tokens that are not full."""
    for pad in (0, 3):
        run_forward(M, Fn, K, t, pad, Hollow)
        run_backward(M, Fn, K, t, pad, False, amp.F32, Hollow)


def test_one_token_of_the_most_features():
    """F = 2^26 with K = 1: y of every feature is that of its own two weights."""
    Fn = 1 << 26
    w = torch.randint(-300, 300, (2 * Fn, 1), device="cuda").float().div_(64).to(torch.bfloat16)
    x, y = torch.ones(1, 1, dtype=torch.bfloat16, device="cuda"), torch.full((1, Fn), float("nan"), dtype=torch.bfloat16, device="cuda")
    amp.amp_gemm_swiglu(1, Fn, 1, x, amp.BF16, 1, w, 1, y, Fn)
    at = torch.cat([torch.randint(0, Fn, (4000,), device="cuda"), torch.tensor([0, Fn // 2, Fn - 1], device="cuda")])
    g, u = (w[i, 0].double().cpu().numpy() for i in (at, Fn + at))
    check_values(y[0, at].double().cpu().numpy(), FMT[amp.BF16], g / (1 + np.exp(-g)) * u, swiglu_err(g, u), "y")
    assert not torch.isnan(y).any()


def rows_and_columns(rng, n):
    return np.unique(np.concatenate([rng.integers(0, n, 24), [0, n - 1, n // 2]]))


@pytest.mark.parametrize("t,M,Fn,K", [(amp.BF16, 4100, 2056, 328), (amp.F16, 2048, 4096, 192)])
def test_large_tiles(t, M, Fn, K):
    """Outputs of enough tiles for 256 x 256 ones, ragged and whole, in sampled rows and columns."""
    g = torch.Generator(device="cuda").manual_seed(5)
    tt = torch.bfloat16 if t == amp.BF16 else torch.float16

    def normal(*s, k=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * k).to(tt)

    def v(a):
        return a.double().cpu().numpy()
    x, w, dy = normal(M, K), normal(2 * Fn, K, k=K ** -0.5), normal(M, Fn)
    y, gu, dgu, again = (torch.full((M, n), float("nan"), dtype=tt, device="cuda") for n in (Fn, 2 * Fn, 2 * Fn, 2 * Fn))
    dx, dw = torch.full((M, K), float("nan"), dtype=tt, device="cuda"), torch.full((2 * Fn, K), float("nan"), device="cuda")
    y2 = torch.full_like(y, float("nan"))
    area = torch.empty(amp.GEMM_SWIGLU_WORK, device="cuda")
    amp.amp_gemm_swiglu(M, Fn, K, x, t, K, w, K, y, Fn, gu, 2 * Fn)
    amp.amp_gemm_swiglu_backward(M, Fn, K, dy, t, Fn, x, K, w, K, None, 0, again, 2 * Fn, y2, Fn, dx, K, dw, amp.F32, K, area)
    amp.amp_gemm_swiglu_backward(M, Fn, K, dy, t, Fn, x, K, w, K, gu, 2 * Fn, dgu, 2 * Fn)
    for o in (y, gu, dgu, again, dx, dw, y2):
        assert not torch.isnan(o).any()
    assert torch.equal(y, y2)
    rng = np.random.default_rng(3)
    for rows, cols in ((rows_and_columns(rng, M), np.arange(Fn)), (np.arange(M), rows_and_columns(rng, Fn))):
        xs, ws = v(x[rows]), np.concatenate([v(w[cols]), v(w[Fn + cols])])
        wy, gg, uu, eg, eu = projections(xs, ws)
        check_values(v(y[rows][:, cols]), FMT[t], wy, y_err(gg, uu, eg, eu), "y")
        both = np.concatenate([cols, Fn + cols])
        check_values(v(gu[rows][:, both]), FMT[t], np.concatenate([gg, uu], 1), np.concatenate([eg, eu], 1), "gu")
        d = v(dy[rows][:, cols])
        check_values(v(again[rows][:, both]), FMT[t], O.activation_backward(d, gg, uu), dgu_err(d, gg, uu, eg, eu), "dgu again")
        kept = v(gu[rows][:, both])
        n = len(cols)
        check_values(v(dgu[rows][:, both]), FMT[t], O.activation_backward(d, kept[:, :n], kept[:, n:]),
                     np.concatenate(swiglu_back_err(d, kept[:, :n], kept[:, n:]), 1), "dgu kept")
    rows = rows_and_columns(rng, M)
    check_values(v(dx[rows]), FMT[t], v(again[rows]) @ v(w), sum_err(2 * Fn, v(again[rows]), v(w)), "dx")
    rows = rows_and_columns(rng, 2 * Fn)
    check_values(v(dw[rows]), FMT[amp.F32], v(again[:, rows]).T @ v(x), sum_err(M, v(again[:, rows]).T, v(x)), "dw")
