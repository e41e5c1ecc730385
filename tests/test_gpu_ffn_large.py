"""Gated feed-forward block in tiles of 256 x 256 on the GPU: the forward call, the
recomputing backward pass and both gradient products, in sampled rows and columns
against float64, with the bounds of test_gpu_ffn.  test_ffn_choice shows that
these sizes take those tiles."""
import numpy as np
import pytest
import torch

import mixed_precision_numerics_amd as amp
from oracle import ffn as O
from block_util import check_values, swiglu_back_err
from ffn_shapes import LARGE
from test_gpu_block import FMT
from test_gpu_ffn import dgu_err, projections, sum_err, y_err

pytestmark = pytest.mark.gpu
TORCH = {amp.BF16: torch.bfloat16, amp.F16: torch.float16, amp.F32: torch.float32}


def v(a):
    return a.double().cpu().numpy()


class Padded:
    """A matrix of type t whose rows are `pad` elements apart, NaN between them and behind the last."""

    def __init__(self, rows, cols, t, pad, values=None):
        self.whole = torch.full((rows + 1, cols + pad), float("nan"), dtype=TORCH[t], device="cuda")
        self.d, self.ld, self.t = self.whole[:rows, :cols], cols + pad, t
        if values is not None:
            self.d.copy_(values)

    def written(self, what):
        rows, cols = self.d.shape
        assert not torch.isnan(self.d).any(), what
        assert torch.isnan(self.whole[:, cols:]).all() and torch.isnan(self.whole[rows]).all(), what + ": written outside"
        return self.d


def sample(rng, n):
    """Rows or columns to look at: the first and the last tile's ends, and some between."""
    ends = [0, 31, 32, 127, 128, 255, 256, n // 2, n - 257, n - 34, n - 2, n - 1]
    return np.unique(np.concatenate([rng.integers(0, n, 12), ends]))


@pytest.mark.parametrize("t", [amp.BF16, amp.F16])
@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("M,Fn,K", LARGE)
def test_large_tiles_of_every_product(M, Fn, K, pad, t):
    gen = torch.Generator(device="cuda").manual_seed(M + pad)

    def normal(*s, k=1.0):
        return torch.randn(*s, generator=gen, device="cuda") * k
    x, w = Padded(M, K, t, pad, normal(M, K)), Padded(2 * Fn, K, t, pad, normal(2 * Fn, K, k=K ** -0.5))
    dy = Padded(M, Fn, t, pad, normal(M, Fn, k=0.25))
    y, gu, y2, again, kept = (Padded(M, n, t, pad) for n in (Fn, 2 * Fn, Fn, 2 * Fn, 2 * Fn))
    dwt = t if pad else amp.F32
    dx, dw = Padded(M, K, t, pad), Padded(2 * Fn, K, dwt, pad)
    area = torch.full((amp.GEMM_SWIGLU_WORK,), float("nan"), device="cuda")

    def backward(gu, dgu, y, dx, dw):
        amp.amp_gemm_swiglu_backward(M, Fn, K, dy.d, t, dy.ld, x.d, x.ld, w.d, w.ld, gu and gu.d, gu.ld if gu else 0, dgu.d, dgu.ld,
                                     y and y.d, y.ld if y else 0, dx and dx.d, dx.ld if dx else 0, dw and dw.d, dwt, dw.ld if dw else 0, area)
    amp.amp_gemm_swiglu(M, Fn, K, x.d, t, x.ld, w.d, w.ld, y.d, y.ld, gu.d, gu.ld)
    backward(None, again, y2, dx, dw)
    backward(gu, kept, None, None, None)
    for what, o in dict(y=y, gu=gu, y2=y2, again=again, kept=kept, dx=dx, dw=dw).items():
        o.written(what)
    assert torch.equal(y.d, y2.d)
    rng = np.random.default_rng(3)
    rows, cols = sample(rng, M), sample(rng, Fn)
    hx, hw = v(x.d), v(w.d)
    for r, c in ((rows, np.arange(Fn)), (np.arange(M), cols)):
        two = np.concatenate([c, Fn + c])
        wy, g, u, eg, eu = projections(hx[r], hw[two])
        ri, ci, ti = (torch.from_numpy(i).cuda() for i in (r, c, two))

        def at(o, k):
            return v(o.d[ri][:, k])
        d = at(dy, ci)
        check_values(at(y, ci), FMT[t], wy, y_err(g, u, eg, eu), "y")
        check_values(at(gu, ti), FMT[t], np.concatenate([g, u], 1), np.concatenate([eg, eu], 1), "gu")
        check_values(at(again, ti), FMT[t], O.activation_backward(d, g, u), dgu_err(d, g, u, eg, eu), "dgu again")
        g, u = np.split(at(gu, ti), 2, axis=1)
        check_values(at(kept, ti), FMT[t], O.activation_backward(d, g, u), np.concatenate(swiglu_back_err(d, g, u), 1), "dgu kept")
    dg, kcols = v(again.d), sample(rng, K)
    frows = np.unique(np.concatenate([sample(rng, Fn), Fn + sample(rng, Fn)]))

    def check_dx(dx):
        got = v(dx.written("dx"))
        for r, c in ((rows, np.arange(K)), (np.arange(M), kcols)):
            check_values(got[r][:, c], FMT[t], dg[r] @ hw[:, c], sum_err(2 * Fn, dg[r], hw[:, c]), "dx")

    def check_dw(dw):
        got = v(dw.written("dw"))
        for r, c in ((frows, np.arange(K)), (np.arange(2 * Fn), kcols)):
            check_values(got[r][:, c], FMT[dwt], dg[:, r].T @ hx[:, c], sum_err(M, dg[:, r].T, hx[:, c]), "dw")
    check_dx(dx)
    check_dw(dw)
    # either gradient alone, the projections once more
    dgu, dx, dw = Padded(M, 2 * Fn, t, pad), Padded(M, K, t, pad), Padded(2 * Fn, K, dwt, pad)
    backward(None, dgu, None, dx, None)
    check_dx(dx)
    backward(None, dgu, None, None, dw)
    check_dw(dw)
    assert torch.equal(dgu.d, again.d)
