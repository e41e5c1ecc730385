"""The gated feed-forward block, its backward pass, the norm over all gradients
and their clipping as a training step runs them: against the formulas in float64
and against differences, captured, on two streams, with extreme values and with
offsets beyond 32 bits."""
import math

import numpy as np
import pytest
import torch

import mixed_precision_numerics_amd as amp
from oracle import ffn as O
from block_util import check_values, swiglu_back_err, swiglu_err
from gpu_util import empty, host
from test_gpu_block import FMT, Mat
from test_gpu_clip import check_coef
from test_gpu_ffn import projections, sum_err, y_err

pytestmark = pytest.mark.gpu


def v(t):
    return t.double().cpu().numpy()


class Step:
    """One block's step in BF16: forward, loss gradient as given, backward, norm, clip into FP32."""

    def __init__(self, M, Fn, K, seed=1):
        self.M, self.F, self.K = M, Fn, K
        bf = torch.bfloat16
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*s, k=1.0):
            return (torch.randn(*s, generator=g, device="cuda") * k).to(bf)

        def out(*s, t=bf):
            return torch.full(s, float("nan"), device="cuda", dtype=t)
        self.x, self.w, self.wd = normal(M, K), normal(2 * Fn, K, k=K ** -0.5), normal(K, Fn, k=Fn ** -0.5)
        self.do = normal(M, K, k=0.1)
        self.y, self.gu, self.o = out(M, Fn), out(M, 2 * Fn), out(M, K)
        self.dy, self.dgu, self.dx, self.dw, self.dwd = out(M, Fn), out(M, 2 * Fn), out(M, K), out(2 * Fn, K), out(K, Fn)
        self.area = out(amp.GEMM_SWIGLU_WORK, t=torch.float32)
        self.state, self.norm, self.res = empty(40), empty(amp.NORM_STATE_BYTES, 0xFF), out(2, t=torch.float32)
        amp.amp_scaler_init(self.state, 1.0)
        self.clipped = [out(2 * Fn, K, t=torch.float32), out(K, Fn, t=torch.float32)]
        self.grads = amp.TensorList([(t, t.numel(), amp.BF16) for t in (self.dw, self.dwd)])
        self.outs = amp.TensorList([(t, t.numel(), amp.F32) for t in self.clipped])

    def run(self):
        M, Fn, K, b = self.M, self.F, self.K, amp.BF16
        amp.amp_gemm_swiglu(M, Fn, K, self.x, b, K, self.w, K, self.y, Fn, self.gu, 2 * Fn)
        amp.amp_gemm(amp.OP_N, amp.OP_T, M, K, Fn, self.y, b, Fn, None, self.wd, b, Fn, None, self.o, b, K)
        amp.amp_gemm(amp.OP_N, amp.OP_N, M, Fn, K, self.do, b, K, None, self.wd, b, Fn, None, self.dy, b, Fn)
        amp.amp_gemm(amp.OP_T, amp.OP_N, K, Fn, M, self.do, b, K, None, self.y, b, Fn, None, self.dwd, b, Fn)
        amp.amp_gemm_swiglu_backward(M, Fn, K, self.dy, b, Fn, self.x, K, self.w, K, self.gu, 2 * Fn, self.dgu, 2 * Fn, None, 0,
                                     self.dx, K, self.dw, b, K, self.area)
        amp.amp_grad_norm_list(self.grads, True, self.state, self.norm, 0.5, self.res)
        amp.amp_grad_clip_list(self.grads, self.outs, self.state, self.res)

    def results(self):
        return [self.y, self.gu, self.o, self.dy, self.dgu, self.dx, self.dw, self.dwd, self.res, *self.clipped]


@pytest.mark.parametrize("M,Fn,K", [(5, 24, 40), (70, 136, 72), (300, 1024, 256)])
def test_a_whole_step_against_the_formulas(M, Fn, K):
    s = Step(M, Fn, K)
    s.run()
    x, w, bf = v(s.x), v(s.w), FMT[amp.BF16]
    wy, g, u, eg, eu = projections(x, w)
    check_values(v(s.y), bf, wy, y_err(g, u, eg, eu), "y")
    gu = v(s.gu)
    dgu = O.activation_backward(v(s.dy), gu[:, :Fn], gu[:, Fn:])
    check_values(v(s.dgu), bf, dgu, np.concatenate(swiglu_back_err(v(s.dy), gu[:, :Fn], gu[:, Fn:]), 1), "dgu")
    wx, ww = O.gradients(v(s.dgu), x, w)
    check_values(v(s.dx), bf, wx, sum_err(2 * Fn, v(s.dgu), w), "dx")
    check_values(v(s.dw), bf, ww, sum_err(M, v(s.dgu).T, x), "dw")
    sq = math.fsum((v(s.dw) ** 2).ravel().tolist() + (v(s.dwd) ** 2).ravel().tolist())
    check_coef(host(s.res, np.float32), sq, 3 * Fn * K, 0.5)
    coef = s.res[0]
    for c, t in zip(s.clipped, (s.dw, s.dwd)):
        assert torch.equal(c, t.float() * coef)


@pytest.mark.parametrize("again", [False, True])
def test_gradients_against_differences(again):
    """d sum(dy y) of the kernel's own forward pass along random directions, in FP16
    with every operand's step a power of two that FP16 adds exactly enough to see."""
    M, Fn, K = 33, 48, 64
    t, tt = amp.F16, torch.float16
    g = torch.Generator(device="cuda").manual_seed(3)

    def normal(*s, k=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * k).to(tt)
    x, w, dy = normal(M, K), normal(2 * Fn, K, k=K ** -0.5), normal(M, Fn)

    def loss(x_, w_):
        gu = O.forward(v(x_), v(w_))[0]                      # float64 of the same operands
        y = torch.empty(M, Fn, dtype=tt, device="cuda")
        amp.amp_gemm_swiglu(M, Fn, K, x_, t, K, w_, K, y, Fn)
        assert np.abs(v(y) - gu).max() <= 2.0 ** -10 * np.abs(gu).max()
        return float((gu * v(dy)).sum())
    gu, dgu = torch.empty(M, 2 * Fn, dtype=tt, device="cuda"), torch.empty(M, 2 * Fn, dtype=tt, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(2 * Fn, K, device="cuda")
    amp.amp_gemm_swiglu(M, Fn, K, x, t, K, w, K, None, 0, gu, 2 * Fn)
    amp.amp_gemm_swiglu_backward(M, Fn, K, dy, t, Fn, x, K, w, K, None if again else gu, 2 * Fn, dgu, 2 * Fn, None, 0, dx, K, dw, amp.F32, K)
    rng = np.random.default_rng(7)
    for which, grad in (("x", dx), ("w", dw)):
        for _ in range(3):
            base = x if which == "x" else w
            d = torch.from_numpy(rng.standard_normal(base.shape)).cuda() * (2.0 ** -7 if which == "x" else 2.0 ** -10)
            hi, lo = (base.double() + d).to(tt), (base.double() - d).to(tt)
            step = v(hi) - v(lo)                             # what the roundings left of it
            diff = loss(hi, w) - loss(lo, w) if which == "x" else loss(x, hi) - loss(x, lo)
            want = float((v(grad) * step).sum())
            # the central difference's third-order term and the 16-bit roundings of gu, dgu and dx (2^-11 each, in
            # quadrature over the terms' sizes, here bounded by their sum)
            slack = 3 * 2.0 ** -11 * float((np.abs(v(grad)) * np.abs(step)).sum()) + 2.0 ** -9 * abs(diff) + 1e-4
            assert abs(diff - want) <= slack, (which, diff, want, slack)


def test_captured_step_replayed():
    s = Step(130, 264, 136)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for k in range(4):
        n = Step(130, 264, 136, 10 + k)
        for a, b in ((s.x, n.x), (s.w, n.w), (s.wd, n.wd), (s.do, n.do)):
            a.copy_(b)
        for r in s.results():
            r.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        n.run()
        torch.cuda.synchronize()
        for a, b in zip(s.results(), n.results()):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    steps = [Step(600, 520, 264, k) for k in (1, 2)]
    want = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        want.append([r.clone() for r in s.results()])
        for r in s.results():
            r.fill_(float("nan"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        for a, b in zip(s.results(), w):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M", [9, 100, 300])
def test_a_token_that_is_not_finite_stays_alone(M):
    Fn, K, b, tt = 72, 136, amp.BF16, torch.bfloat16
    s = Step(M, Fn, K)
    bad = s.x.clone()
    bad[M // 2, 5], bad[M // 3, 7] = float("nan"), float("inf")
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[[M // 2, M // 3]] = False
    outs = []
    for x in (s.x, bad):
        y, gu, dgu, dx = (torch.zeros(M, n, dtype=tt, device="cuda") for n in (Fn, 2 * Fn, 2 * Fn, K))
        dy = s.do[:, :Fn].contiguous()
        amp.amp_gemm_swiglu(M, Fn, K, x, b, K, s.w, K, y, Fn, gu, 2 * Fn)
        amp.amp_gemm_swiglu_backward(M, Fn, K, dy, b, Fn, x, K, s.w, K, None, 0, dgu, 2 * Fn, None, 0, dx, K)
        outs.append((y, gu, dgu, dx))
    for a, c in zip(*outs):
        assert torch.equal(a[rest], c[rest]) and not torch.isnan(a).any()
        assert torch.isnan(c[M // 2]).all() and not torch.isfinite(c[M // 3]).all()


@pytest.mark.parametrize("t", [amp.BF16, amp.F16])
@pytest.mark.parametrize("M", [4, 40])
def test_gates_over_their_whole_range(t, M):
    """K == 1, one token's factor 1: g is the weight itself, from where the sigmoid is 0 to where it is 1."""
    Fn = 2048
    gv = np.linspace(-130.0, 130.0, Fn)
    x, w = Mat(M, 1, t, 7, np.ones((M, 1))), Mat(2 * Fn, 1, t, 7, np.concatenate([gv, np.ones(Fn)])[:, None])
    dy, y, dgu = Mat(M, Fn, t, 0, np.ones((M, Fn))), Mat(M, Fn, t), Mat(M, 2 * Fn, t)
    amp.amp_gemm_swiglu(M, Fn, 1, x.d, t, x.ld, w.d, w.ld, y.d, y.ld)
    g, u = np.tile(w.v[:Fn, 0], (M, 1)), np.ones((M, Fn))
    check_values(y.values(), FMT[t], g / (1 + np.exp(-g)), swiglu_err(g, u), "y")
    amp.amp_gemm_swiglu_backward(M, Fn, 1, dy.d, t, dy.ld, x.d, x.ld, w.d, w.ld, None, 0, dgu.d, dgu.ld)
    check_values(dgu.values(), FMT[t], O.activation_backward(dy.v, g, u), np.concatenate(swiglu_back_err(dy.v, g, u), 1), "dgu")


def test_offsets_beyond_32_bits():
    """2 F M > 2^31 elements: the last rows and columns hold what they should."""
    M, Fn, K, b, tt = 70_001, 16_384, 64, amp.BF16, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, K, generator=g, device="cuda").to(tt)
    w = (torch.randn(2 * Fn, K, generator=g, device="cuda") * K ** -0.5).to(tt)
    y, gu = torch.empty(M, Fn, dtype=tt, device="cuda"), torch.empty(M, 2 * Fn, dtype=tt, device="cuda")
    assert gu.numel() > 2 ** 31
    amp.amp_gemm_swiglu(M, Fn, K, x, b, K, w, K, y, Fn, gu, 2 * Fn)
    rows = [0, M // 2, M - 130, M - 1]
    wy, pg, pu, eg, eu = projections(v(x[rows]), v(w))
    check_values(v(y[rows]), FMT[b], wy, y_err(pg, pu, eg, eu), "y")
    check_values(v(gu[rows]), FMT[b], np.concatenate([pg, pu], 1), np.concatenate([eg, eu], 1), "gu")
    dx, dw = torch.empty(M, K, dtype=tt, device="cuda"), torch.empty(2 * Fn, K, device="cuda")
    kept = gu[rows].clone()
    dy = y                                                   # its values serve as a gradient
    amp.amp_gemm_swiglu_backward(M, Fn, K, dy, b, Fn, x, K, w, K, gu, 2 * Fn, gu, 2 * Fn, None, 0, dx, K, dw, amp.F32, K)
    d, k = v(dy[rows]), v(kept)
    check_values(v(gu[rows]), FMT[b], O.activation_backward(d, k[:, :Fn], k[:, Fn:]),
                 np.concatenate(swiglu_back_err(d, k[:, :Fn], k[:, Fn:]), 1), "dgu in place")
    check_values(v(dx[rows]), FMT[b], v(gu[rows]) @ v(w), sum_err(2 * Fn, v(gu[rows]), v(w)), "dx")
    cols = [0, Fn, 2 * Fn - 1]
    a = v(gu[:, cols]).T
    check_values(v(dw[cols]), FMT[amp.F32], a @ v(x), sum_err(M, a, v(x)), "dw")


def test_lists_of_tensors_beyond_32_bits():
    n = 2 ** 31 + 4099
    a = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    a[:2], a[2 ** 31 - 1:2 ** 31 + 1], a[-3:] = 3.0, 5.0, 7.0
    some = amp.TensorList([(a, n, amp.BF16), (a[-2:], 2, amp.BF16)])
    st, ns, out = empty(40), empty(amp.NORM_STATE_BYTES), torch.zeros(2, device="cuda")
    amp.amp_scaler_init(st, 1.0)
    amp.amp_grad_norm_list(some, True, st, ns, 1.0, out)
    want = 2 * 9 + 2 * 25 + 5 * 49
    assert host(ns, np.float64)[0] == want
    check_coef(host(out, np.float32), want, n)
    amp.amp_grad_clip_list(amp.TensorList([(a, n, amp.BF16)]), None, None, torch.full((1,), 0.5, device="cuda"))
    assert a[:3].tolist() == [1.5, 1.5, 0.0] and a[2 ** 31 - 2:2 ** 31 + 2].tolist() == [0.0, 2.5, 2.5, 0.0] and a[-4:].tolist() == [0.0, 3.5, 3.5, 3.5]
    assert float(a.float().sum()) == 2 * 1.5 + 2 * 2.5 + 3 * 3.5


def test_results_do_not_change_from_call_to_call():
    s = Step(2000, 520, 264)
    s.run()
    torch.cuda.synchronize()
    first = [r.clone() for r in s.results()]
    for _ in range(3):
        s.area.fill_(float("nan"))
        s.run()
        for a, b in zip(s.results(), first):
            assert torch.equal(a, b)


def test_operands_that_are_views_or_parameters():
    """Rows of larger tensors, a strided view, a parameter, a row whose one-element dimension has any stride."""
    M, Fn, K, b, tt = 7, 40, 64, amp.BF16, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(9)

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda").to(tt)
    big, w, wide = normal(M + 5, K), normal(2 * Fn, K), normal(M, 2 * K)
    want, got = torch.empty(M, Fn, dtype=tt, device="cuda"), torch.full((M + 2, Fn), float("nan"), dtype=tt, device="cuda")
    amp.amp_gemm_swiglu(M, Fn, K, big[3:3 + M].clone(), b, K, w, K, want, Fn)
    amp.amp_gemm_swiglu(M, Fn, K, big[3:3 + M], b, K, torch.nn.Parameter(w), K, got[1:1 + M], Fn)
    assert torch.equal(got[1:1 + M], want) and torch.isnan(got[[0, M + 1]]).all()
    amp.amp_gemm_swiglu(M, Fn, K, wide[:, K:].contiguous(), b, K, w, K, want, Fn)
    amp.amp_gemm_swiglu(M, Fn, K, wide[:, K:], b, 2 * K, w, K, got[1:1 + M], Fn)
    assert torch.equal(got[1:1 + M], want)
    amp.amp_gemm_swiglu(1, Fn, K, big[:1].clone(), b, K, w, K, want, Fn)
    amp.amp_gemm_swiglu(1, Fn, K, big.as_strided((1, K, 1), (12345, 1, 777)), b, K, w, K, got[1:2], Fn)
    assert torch.equal(got[1:2], want[:1])
    with pytest.raises(ValueError, match="x holds"):
        amp.amp_gemm_swiglu(M, Fn, K, big[6:], b, K, w, K, want, Fn)
    n = torch.nn.Parameter(torch.full((33,), 2.0, device="cuda"))
    st, ns, out = empty(40), empty(amp.NORM_STATE_BYTES), torch.zeros(2, device="cuda")
    amp.amp_scaler_init(st, 1.0)
    some = amp.TensorList([(n, 33, amp.F32), (torch.ones(4, device="cuda")[1:], 3, amp.F32)])
    amp.amp_grad_norm_list(some, True, st, ns, 1.0, out)
    assert host(ns, np.float64)[0] == 33 * 4 + 3
    n.data = torch.zeros(33, device="cuda")
    with pytest.raises(ValueError, match="has moved"):
        amp.amp_grad_norm_list(some, True, st, ns, 1.0, out)
