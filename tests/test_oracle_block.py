"""Pins for oracle/block.py: the norm and the gated activation against
PyTorch float64 functions, their gradients against float64 autograd and
central differences, and the tile scaling against oracle/blockwise.py."""
import numpy as np
import pytest
import torch

from oracle import block as B
from oracle import blockwise as BW
from oracle import formats as F
import synth


def _rand(seed, *shape, scale=1.0):
    return synth.rng(seed).standard_normal(shape) * scale


def test_norm_and_gradients_match_float64_autograd():
    h, gamma, dy = _rand(1, 7, 50, scale=2.0), 1 + _rand(2, 50, scale=0.1), _rand(3, 7, 50)
    eps = float(np.float32(1e-5))
    th = torch.tensor(h, requires_grad=True)
    tg = torch.tensor(gamma, requires_grad=True)
    ty = torch.nn.functional.rms_norm(th, (50,), tg, eps)
    ty.backward(torch.tensor(dy))
    y, r = B.rmsnorm(h, gamma, eps)
    dx, dgamma = B.rmsnorm_backward(dy, h, gamma, r)
    assert np.allclose(y, ty.detach().numpy(), rtol=1e-12, atol=0)
    assert np.allclose(dx, th.grad.numpy(), rtol=1e-10, atol=1e-12)
    assert np.allclose(dgamma, tg.grad.numpy(), rtol=1e-12, atol=1e-13)
    res = _rand(4, 7, 50)
    assert np.allclose(B.rmsnorm_backward(dy, h, gamma, r, res)[0], dx + res, rtol=0, atol=1e-14)


def test_gated_activation_and_gradients_match_float64_autograd():
    g, u, dy = _rand(5, 6, 40, scale=3.0), _rand(6, 6, 40), _rand(7, 6, 40)
    tg, tu = torch.tensor(g, requires_grad=True), torch.tensor(u, requires_grad=True)
    ty = torch.nn.functional.silu(tg) * tu
    ty.backward(torch.tensor(dy))
    dg, du = B.swiglu_backward(dy, g, u)
    assert np.allclose(B.swiglu(g, u), ty.detach().numpy(), rtol=1e-13, atol=0)
    assert np.allclose(dg, tg.grad.numpy(), rtol=1e-11, atol=1e-14)
    assert np.allclose(du, tu.grad.numpy(), rtol=1e-13, atol=0)


@pytest.mark.parametrize("which", ["norm", "swiglu"])
def test_gradients_match_central_differences(which):
    x, d = _rand(8, 3, 20), _rand(9, 3, 20)
    t = 1e-5
    if which == "norm":
        gamma, dy = 1 + _rand(10, 20, scale=0.1), _rand(11, 3, 20)
        f = lambda h: (B.rmsnorm(h, gamma, 1e-5)[0] * dy).sum()
        grad = B.rmsnorm_backward(dy, x, gamma, B.rmsnorm(x, gamma, 1e-5)[1])[0]
    else:
        dy = _rand(12, 3, 10)
        f = lambda h: (B.swiglu(h[:, :10], h[:, 10:]) * dy).sum()
        grad = np.concatenate(B.swiglu_backward(dy, x[:, :10], x[:, 10:]), axis=1)
    num = (f(x + t * d) - f(x - t * d)) / (2 * t)
    assert abs(num - (grad * d).sum()) < 1e-8 * np.abs(grad * d).sum()


@pytest.mark.parametrize("fmt", [F.E4M3, F.E5M2])
def test_tiles_are_those_of_the_blockwise_quantizer(fmt):
    x = synth.student_t_f32(13, (20, 300), 3.0, 2.0)
    x[3, :128] = 0.0
    codes, s = B.quantize(x, fmt)
    wq, ws = BW.quantize(synth.f32_bits(x), F.F32, fmt, block=False)
    assert np.array_equal(codes, wq) and np.array_equal(s, ws)
    assert np.array_equal(B.dequantize(codes, s, fmt), BW.dequantize(codes, s, fmt, False))


def test_scale_of_tiny_zero_and_non_finite_tiles_is_one():
    amax = np.array([[0.0, 1e-38, 1e-45, np.inf, np.nan, 1.0, 3.4e38]])
    sc = B.tile_scale(amax, F.E4M3)
    assert np.array_equal(sc[0, :5], np.ones(5)) and sc[0, 5] == 448.0 and 0 < sc[0, 6] < 1e-35


def test_dequantize_restarts_tiles_at_each_part():
    codes = np.full((1, 400), F.encode(np.array([1.0]), F.E4M3)[0])
    s = np.array([[1.0], [2.0], [3.0], [4.0]])
    v = B.dequantize(codes, s, F.E4M3, parts=2)[0]
    assert list(v[[0, 127, 128, 199, 200, 327, 328, 399]]) == [1, 1, 2, 2, 3, 3, 4, 4]
