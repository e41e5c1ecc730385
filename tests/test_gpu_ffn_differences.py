"""Gradients of the gated feed-forward block against differences of the kernel's
own forward pass.

The loss is sum(dy y) of the y that the forward call returns, its steps are exact:
operands are multiples of a power of two, which is the step.  Every element of x
(or w) steps along the gradient's sign, so the loss moves by twice the step times
the gradient's absolute sum, which is large beside what the roundings can do.

What may remain, with h_g and h_u the step's effect on g and u (exact values):
  the third derivative, |silu'''| < 0.31 and |silu''| <= 0.5:
      |dy| (0.31 |h_g|^3 (|u| + |h_u|) + 3 0.5 h_g^2 |h_u|) / 3
  the roundings of y at both ends, half a step each, and the FP32 errors (y_err)
  the kept projections' rounding and dgu's FP32 errors (dgu_err), times |h_g|, |h_u|
  the rounding of dgu, half a step, times |h_g|, |h_u|
  the rounding of dx (dw is FP32) and the FP32 sums (sum_err), times the step."""
import numpy as np
import pytest
import torch

import mixed_precision_numerics_amd as amp
from oracle import ffn as O
from test_gpu_ffn import dgu_err, projections, sum_err, y_err

pytestmark = pytest.mark.gpu
TORCH = {amp.BF16: torch.bfloat16, amp.F16: torch.float16}


def v(a):
    return a.double().cpu().numpy()


def grid(rng, shape, size, step):
    """Normal values at multiples of `step`, few enough bits for BF16 a step up and down."""
    return np.clip(np.round(rng.standard_normal(shape) * size / step), -120, 120) * step


@pytest.mark.parametrize("t", [amp.F16, amp.BF16])
@pytest.mark.parametrize("saved", [True, False])
@pytest.mark.parametrize("which", ["x", "w"])
@pytest.mark.parametrize("M,Fn,K", [(1, 40, 64), (33, 48, 64), (200, 136, 72)])
def test_gradients_against_differences_of_the_forward_call(M, Fn, K, which, saved, t):
    tt, half = TORCH[t], torch.finfo(TORCH[t]).eps / 2
    rng = np.random.default_rng(7)
    hx, hw = 2.0 ** -5, 2.0 ** -8
    x, w = grid(rng, (M, K), 1.0, hx), grid(rng, (2 * Fn, K), K ** -0.5, hw)
    dy = v(torch.from_numpy(rng.standard_normal((M, Fn))).to(tt))

    def dev(a):
        d = torch.from_numpy(a).cuda().to(tt)
        assert np.array_equal(v(d), a)                           # exact
        return d

    def forward(x_, w_):
        y, gu = torch.empty(M, Fn, dtype=tt, device="cuda"), torch.empty(M, 2 * Fn, dtype=tt, device="cuda")
        amp.amp_gemm_swiglu(M, Fn, K, dev(x_), t, K, dev(w_), K, y, Fn, gu, 2 * Fn)
        return v(y), gu
    gu = forward(x, w)[1]
    dgu, dx, dw = torch.empty(M, 2 * Fn, dtype=tt, device="cuda"), torch.empty(M, K, dtype=tt, device="cuda"), torch.empty(2 * Fn, K, device="cuda")
    amp.amp_gemm_swiglu_backward(M, Fn, K, dev(dy), t, Fn, dev(x), K, dev(w), K, gu if saved else None, 2 * Fn, dgu, 2 * Fn, None, 0,
                                 dx, K, dw, amp.F32, K)
    grad = v(dx if which == "x" else dw)
    step = np.sign(grad) * (hx if which == "x" else hw)
    ends = [(x + s * step, w) if which == "x" else (x, w + s * step) for s in (1, -1)]
    up, down = (forward(*e)[0] for e in ends)
    moved, want = float((dy * (up - down)).sum()), 2 * float((grad * step).sum())

    _, g, u, eg, eu = projections(x, w)
    h = step @ w.T if which == "x" else x @ step.T
    hg, hu = np.abs(h[:, :Fn]), np.abs(h[:, Fn:])
    ady, au = np.abs(dy), np.abs(u)
    third = (ady * (0.31 * hg ** 3 * (au + hu) + 1.5 * hg ** 2 * hu) / 3).sum()
    ey = 0.0
    for e, got in zip(ends, (up, down)):
        _, g1, u1, eg1, eu1 = projections(*e)
        ey += (ady * (y_err(g1, u1, eg1, eu1) * (1 + half) + half * np.abs(g1 * u1) / (1 + np.exp(-g1)))).sum()
    if saved:
        eg, eu = eg * (1 + half) + half * np.abs(g), eu * (1 + half) + half * np.abs(u)
    ed = dgu_err(dy, g, u, eg, eu)
    exact = np.abs(O.activation_backward(dy, g, u))
    ed = ed * (1 + half) + half * exact
    egrad = 2 * (ed * np.concatenate([hg, hu], 1)).sum()
    d = v(dgu)
    if which == "x":
        es = sum_err(2 * Fn, d, w)
        es = es * (1 + half) + half * np.abs(d @ w)
    else:
        es = sum_err(M, d.T, x) * (1 + 2.0 ** -23) + 2.0 ** -24 * np.abs(d.T @ x)
    egrad += 2 * (es * np.abs(step)).sum()
    # (products of two such errors, and values below the types' normal range)
    slack = 1.01 * (third + ey + egrad) + 1e-3
    assert slack < 0.25 * want, "the step is too small to see the gradient"
    assert abs(moved - want) <= slack, (moved, want, slack)
