"""Calls of the norm, gated-activation and requantization entry points at the
edges of what they allow, against oracle/block.py in float64."""
import numpy as np
import pytest
import torch

import mixed_precision_numerics_amd as amp
from oracle import block as B
from oracle import formats as F
from block_util import U, check_scaled, check_values, dx_err, norm_err, swiglu_back_err, swiglu_err
from gpu_util import dev, host
import test_gpu_block as plain
from test_gpu_block import FMT, NPT, TYPES, Mat, Tiles, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xt", TYPES)
@pytest.mark.parametrize("cols", [40, 512, 1536])
@pytest.mark.parametrize("rows", [1, 2, 3, 5, 1030])
def test_norm_without_eps_records_the_rows_maximum_alone(xt, rows, cols):
    """eps == 0 with no zero row: what the threads of a block hold past the last
    row (zeros, whose norm is 0 * inf) reaches no output, the amax among them."""
    x = Mat(rows, cols, xt, 3, rand(rows + cols, rows, cols))
    y, yq, rstd = Mat(rows, cols, amp.E4M3, 1), Tiles(rows, cols), Mat(1, rows, amp.F32)
    am, sc = torch.full((1,), 1e-3, device="cuda"), np.float32([16.0])
    amp.amp_rmsnorm(x.d, xt, rows, cols, x.ld, None, 0, None, 0, 0.0, None, 0, y.d, amp.E4M3, y.ld, dev(sc), am, yq.arg, None, rstd.d)
    wy, wr = B.rmsnorm(x.v, np.ones(cols), 0.0)
    e = norm_err(cols)
    err = np.abs(wy) * (e + 3 * U)
    check_values(am.cpu().numpy(), FMT[amp.F32], np.array([np.abs(wy).max()]), err.max(), "amax")
    check_values(rstd.values()[0], FMT[amp.F32], wr, e * wr, "rstd")
    check_scaled(y.codes(), FMT[amp.E4M3], wy, err, 16.0, 16.0, "y")
    yq.check(wy, err, "yq")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 40), (5, 4096), (64, 1000), (301, 96), (512, 512), (512, 2047), (513, 96), (700, 520), (600, 2048),
                                       (7, 5120), (40, 9000), (30, 20483), (5, 40003)])
def test_norm_backward_in_place_of_the_stored_input(dt, rows, cols):
    """dx replaces h, which the gamma gradient reads too, on every path by rows and by vectors."""
    hv, ones = rand(1, rows, cols), np.ones(cols)
    dy, dres = Mat(rows, cols, dt, 1, rand(2, rows, cols)), Mat(rows, cols, dt, 2, rand(3, rows, cols))
    for gradient in (True, False):
        h = Mat(rows, cols, dt, 5, hv)
        r = F.f32(B.rmsnorm(h.v, ones, 1e-5)[1])
        dgamma, work = Mat(1, cols, amp.F32), Mat(min(rows, amp.RMSNORM_PARTIALS), cols, amp.F32)
        amp.amp_rmsnorm_backward(dy.d, dt, rows, cols, dy.ld, h.d, h.ld, None, None, 0, dev(r.astype(np.float32)), dres.d, dres.ld,
                                 h.d, h.ld, dgamma.d if gradient else None, work.d)
        wx, wg = B.rmsnorm_backward(dy.v, h.v, ones, r, dres.v)
        check_values(h.values(), FMT[dt], wx, dx_err(dy.v, h.v, ones, r, dres.v, wx), "dx in place of h")
        work.codes()
        if gradient:
            check_values(dgamma.values()[0], FMT[amp.F32], wg, (rows + 8) * U * np.abs(dy.v * h.v * r[:, None]).sum(0), "dgamma")


@pytest.mark.parametrize("scale", [1.0, 2.0 ** 100])
def test_sigmoid_over_its_whole_range(scale):
    """s as the header bounds it, through du = dy s g with dy a power of two
    (FP32) and through y = g s u with u one (BF16, whose range is FP32's)."""
    rows, cols, dt = 5, 4096, amp.F32
    gv = np.linspace(-135.0, 100.0, rows * cols).reshape(rows, cols)
    x = Mat(rows, 2 * cols, dt, 1, np.concatenate([gv, np.full((rows, cols), scale)], 1))
    dy, dx, y = Mat(rows, cols, dt, 2, np.full((rows, cols), scale)), Mat(rows, 2 * cols, dt), Mat(rows, cols, amp.BF16)
    g = x.v[:, :cols]
    s, om = B.sigmoid(g), B.sigmoid(-g)
    # the header's bounds of s, and a rounding of the product with g (that with a power of two has none: where s is
    # normal dy s and g s u are, and below 2^-126 the absolute bound holds)
    es = np.where(g >= -87, s * (6 * U + om * np.abs(g) * 4 * U), 2.0 ** -125)
    err = np.abs(g) * scale * (es + U * s)
    amp.amp_swiglu_backward(dy.d, dt, rows, cols, dy.ld, x.d, x.ld, None, dx.d, dx.ld)
    amp.amp_swiglu(x.d, dt, rows, cols, x.ld, y.d, amp.BF16, y.ld)
    check_values(dx.values()[:, cols:], FMT[dt], g * s * scale, err, "du")
    check_values(y.values(), FMT[amp.BF16], g * s * scale, err, "y")


# ------------------------------------------- what lies behind an input's rows ---

class Hollow(Mat):
    """A Mat that, as an input, has NaN (all bits set in every type) behind its rows and its end."""

    def __init__(self, rows, cols, t, pad=0, v=None):
        super().__init__(rows, cols, t, pad, v)
        if v is not None:
            a = host(self.d, NPT[t]).copy()
            keep = self.codes().copy()
            a.view(np.uint8)[:] = self.fill = 0xFF
            a[:rows * self.ld].reshape(rows, self.ld)[:, :cols] = keep
            self.d = dev(a)


@pytest.fixture
def hollow(monkeypatch):
    monkeypatch.setattr(plain, "Mat", Hollow)


@pytest.mark.parametrize("xt", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (2, 129), (9, 511), (33, 2047), (1027, 1401), (2, 7001), (2, 20483), (3, 70003)])
def test_norm_reads_its_rows_alone(hollow, xt, rows, cols):
    plain.test_norm_every_output(xt, rows, cols)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("saved", ["stored", "checkpoint"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (2, 129), (33, 2047), (700, 41), (601, 515), (530, 1501), (4, 7001), (9, 25001), (2, 40003)])
def test_norm_backward_reads_its_rows_alone(hollow, dt, saved, rows, cols):
    plain.test_norm_backward(dt, saved, rows, cols)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (2, 129), (37, 201), (9, 2047), (3, 4101)])
def test_swiglu_and_its_backward_read_their_rows_alone(hollow, dt, rows, cols):
    plain.test_swiglu_every_output(dt, rows, cols)
    for saved in ("stored", "checkpoint"):
        plain.test_swiglu_backward_in_the_gradients_type(dt, saved, rows, cols)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("saved", ["stored", "checkpoint"])
@pytest.mark.parametrize("rows,cols", [(1, 128), (129, 256)])
def test_swiglu_backward_reads_its_rows_alone_for_every_fp8_operand(hollow, dt, saved, rows, cols):
    plain.test_swiglu_backward_every_fp8_operand(dt, saved, rows, cols)


@pytest.mark.parametrize("rows,cols", [(1, 3), (5, 7), (129, 201), (260, 333)])
def test_transposed_operands_read_their_rows_alone(hollow, rows, cols):
    plain.test_swiglu_backward_transposed_operands_at_odd_widths(rows, cols)
    plain.test_requantize(rows, cols, amp.E4M3, amp.E5M2, amp.BF16)
    plain.test_requantize(rows, cols, amp.E5M2, amp.E4M3, None)


# --------------------------------------- forms that the other tests do not combine ---

@pytest.mark.parametrize("xt", TYPES)
@pytest.mark.parametrize("gt", TYPES)
@pytest.mark.parametrize("rows,cols", [(3, 512), (5, 1003), (600, 520)])
def test_norm_with_gamma_of_another_type(xt, gt, rows, cols):
    x, dy = Mat(rows, cols, xt, 1, rand(1, rows, cols)), Mat(rows, cols, xt, 2, rand(2, rows, cols))
    gamma = Mat(1, cols, gt, 0, 1 + rand(3, 1, cols, scale=0.1))
    yq, rstd, dx, dgamma = Tiles(rows, cols), Mat(1, rows, amp.F32), Mat(rows, cols, xt), Mat(1, cols, amp.F32)
    work = Mat(min(rows, amp.RMSNORM_PARTIALS), cols, amp.F32)
    amp.amp_rmsnorm(x.d, xt, rows, cols, x.ld, None, 0, gamma.d, gt, 1e-5, yq=yq.arg, rstd=rstd.d)
    wy, _ = B.rmsnorm(x.v, gamma.v[0], 1e-5)
    yq.check(wy, np.abs(wy) * (norm_err(cols) + 3 * U), "yq")
    r = rstd.values()[0]
    amp.amp_rmsnorm_backward(dy.d, xt, rows, cols, dy.ld, x.d, x.ld, None, gamma.d, gt, rstd.d, None, 0, dx.d, dx.ld, dgamma.d, work.d)
    wx, wg = B.rmsnorm_backward(dy.v, x.v, gamma.v[0], r)
    check_values(dx.values(), FMT[xt], wx, dx_err(dy.v, x.v, gamma.v[0], r, None, wx), "dx")
    check_values(dgamma.values()[0], FMT[amp.F32], wg, (rows + 8) * U * np.abs(dy.v * x.v * r[:, None]).sum(0), "dgamma")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rows,cols", [(3, 5), (130, 201), (129, 256)])
def test_swiglu_backward_in_place_with_fp8_operands(dt, rows, cols):
    """dx replaces x while the same call writes the transposed operands."""
    x, dy = Mat(rows, 2 * cols, dt, 3, rand(1, rows, 2 * cols)), Mat(rows, cols, dt, 1, rand(2, rows, cols))
    g, u = x.v[:, :cols], x.v[:, cols:]
    dxqt, yqt = Tiles(2 * cols, rows, amp.E5M2, 3), Tiles(cols, rows, amp.E4M3, 5)
    amp.amp_swiglu_backward(dy.d, dt, rows, cols, dy.ld, x.d, x.ld, None, x.d, x.ld, None, dxqt.arg, yqt.arg)
    w, e = np.concatenate(B.swiglu_backward(dy.v, g, u), 1), np.concatenate(swiglu_back_err(dy.v, g, u), 1)
    check_values(x.values(), FMT[dt], w, e, "dx in place of x")
    dxqt.check(w.T, e.T, "dxqt")
    yqt.check(B.swiglu(g, u).T, swiglu_err(g, u).T, "yqt")
