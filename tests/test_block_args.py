"""Refusals of the norm, gated-activation and requantization entry points: all
come before any device work, so they need no GPU."""
import os

import pytest
import torch

import mixed_precision_numerics_amd as amp

pytestmark = pytest.mark.skipif(not os.path.exists(amp.lib_path()), reason="libamp.so not built")
EINVAL, EUNSUP = -1, -2
P = 4096            # a pointer that no refused call follows


def tiles(ldq, lds, t=amp.E4M3, q=P, s=P):
    return amp.Fp8Tiles(q, s, ldq, lds, t)


def status(fn, *a):
    args = [amp.ctypes.addressof(x) if isinstance(x, amp.Fp8Tiles) else x for x in a]
    return getattr(amp.load(), fn)(*args)


def norm(**k):
    a = dict(x=P, xt=amp.BF16, rows=4, cols=300, ldx=300, res=None, ldr=0, gamma=P, gt=amp.F32, eps=1e-5, h=None, ldh=0, y=P,
             yt=amp.BF16, ldy=300, d_scale=None, d_amax=None, yq=None, ckpt=None, rstd=None)
    a.update(k)
    return status("amp_rmsnorm", *a.values(), None)


def norm_back(**k):
    a = dict(dy=P, dt=amp.BF16, rows=4, cols=300, lddy=300, h=P, ldh=300, ckpt=None, gamma=P, gt=amp.F32, rstd=P, dres=None, lddr=0,
             dx=2 * P, lddx=300, dgamma=P, d_work=P)
    a.update(k)
    return status("amp_rmsnorm_backward", *a.values(), None)


def gate(**k):
    a = dict(x=P, xt=amp.BF16, rows=4, cols=300, ldx=600, y=P, yt=amp.BF16, ldy=300, d_scale=None, d_amax=None, yq=None, ckpt=None)
    a.update(k)
    return status("amp_swiglu", *a.values(), None)


def gate_back(**k):
    a = dict(dy=P, dt=amp.BF16, rows=4, cols=300, lddy=300, x=P, ldx=600, ckpt=None, dx=2 * P, lddx=600, dxq=None, dxqt=None, yqt=None)
    a.update(k)
    return status("amp_swiglu_backward", *a.values(), None)


def requant(**k):
    a = dict(x=tiles(300, 4), rows=4, cols=300, d_row=None, col=None, ct=0, qt=tiles(4, 300))
    a.update(k)
    return status("amp_requantize_blockwise", *a.values(), None)



@pytest.mark.parametrize("call,bad", [
    (norm, dict(rows=-1)), (norm, dict(cols=-1)), (norm, dict(eps=-1e-5)), (norm, dict(eps=float("nan"))),
    (norm, dict(eps=float("inf"))), (norm, dict(x=None)), (norm, dict(y=None)), (norm, dict(ldx=299)),
    (norm, dict(res=P, ldr=299)), (norm, dict(h=2 * P, ldh=299)), (norm, dict(ldy=299)), (norm, dict(rstd=P + 2)),
    (norm, dict(d_amax=P + 1)), (norm, dict(d_scale=P + 2)), (norm, dict(yq=tiles(299, 4))), (norm, dict(yq=tiles(300, 3))),
    (norm, dict(ckpt=tiles(300, 4, q=None))), (norm, dict(ckpt=tiles(300, 4, s=None))), (norm, dict(ckpt=tiles(300, 4, s=P + 2))),
    (norm, dict(h=P, ldh=304)), (norm, dict(res=2 * P, ldr=300, h=2 * P, ldh=301)),
    (norm_back, dict(rows=-1)), (norm_back, dict(dy=None)), (norm_back, dict(rstd=None)), (norm_back, dict(h=None)),
    (norm_back, dict(ckpt=tiles(300, 4))), (norm_back, dict(h=None, ckpt=tiles(300, 3))), (norm_back, dict(d_work=None)),
    (norm_back, dict(dx=None, dgamma=None)), (norm_back, dict(lddy=299)), (norm_back, dict(ldh=299)), (norm_back, dict(lddx=299)),
    (norm_back, dict(dres=P, lddr=299)), (norm_back, dict(dgamma=P + 2)), (norm_back, dict(dx=P, lddx=301)),
    (norm_back, dict(dres=2 * P, lddr=301)),
    (gate, dict(rows=-1)), (gate, dict(cols=-2)), (gate, dict(x=None)), (gate, dict(y=None)), (gate, dict(ldx=599)),
    (gate, dict(ldy=299)), (gate, dict(yq=tiles(300, 3))), (gate, dict(ckpt=tiles(599, 4))), (gate, dict(d_scale=P + 1)),
    (gate_back, dict(rows=-1)), (gate_back, dict(dy=None)), (gate_back, dict(x=None)), (gate_back, dict(ckpt=tiles(600, 4))),
    (gate_back, dict(dx=None)), (gate_back, dict(lddy=299)), (gate_back, dict(ldx=599)), (gate_back, dict(lddx=599)),
    (gate_back, dict(dxqt=tiles(4, 599))), (gate_back, dict(dxqt=tiles(3, 600))), (gate_back, dict(yqt=tiles(4, 299))),
    (gate_back, dict(dx=P, lddx=601)),
    (requant, dict(rows=-1)), (requant, dict(x=None)), (requant, dict(qt=None)), (requant, dict(x=tiles(299, 4))),
    (requant, dict(x=tiles(300, 3))), (requant, dict(qt=tiles(3, 300))), (requant, dict(qt=tiles(4, 299))),
    (requant, dict(d_row=P + 2)),
])
def test_invalid_arguments(call, bad):
    assert call(**bad) == EINVAL


@pytest.mark.parametrize("call,bad", [
    (norm, dict(xt=amp.E4M3)), (norm, dict(gt=amp.E5M2)), (norm, dict(yt=amp.F32)), (norm, dict(yq=tiles(300, 4, amp.BF16))),
    (norm_back, dict(dt=amp.E4M3)), (norm_back, dict(gt=9)), (norm_back, dict(h=None, ckpt=tiles(300, 4, amp.E2M1X2))),
    (gate, dict(xt=7)), (gate, dict(yt=amp.E2M1X2)), (gate, dict(ckpt=tiles(600, 4, amp.F16))),
    (gate_back, dict(dt=amp.E5M2)), (gate_back, dict(dxq=tiles(600, 4))),    # 300 columns: a tile across the halves
    (requant, dict(col=P, ct=amp.E4M3)), (requant, dict(qt=tiles(4, 300, amp.F32))),
])
def test_unsupported_types_and_layouts(call, bad):
    assert call(**bad) == EUNSUP


def test_empty_work_is_accepted_without_pointers():
    assert norm(rows=0, x=None, y=None) == 0 and norm(cols=0, ldx=0) == 0
    assert gate(rows=0, x=None) == 0 and gate_back(cols=0, dy=None) == 0 and requant(rows=0, x=None) == 0
    assert norm_back(rows=0, dgamma=None) == 0 and norm_back(cols=0) == 0


def test_binding_refuses_tensors_smaller_than_the_call_spans():
    bf, u8 = torch.bfloat16, torch.uint8
    x, g = torch.zeros(4, 300, dtype=bf), torch.zeros(300)
    ok = amp.Fp8Tiles(torch.zeros(4, 300, dtype=u8), torch.zeros(3, 4), 300, 4)
    short_q = amp.Fp8Tiles(torch.zeros(1199, dtype=u8), torch.zeros(3, 4), 300, 4)
    short_s = amp.Fp8Tiles(torch.zeros(1200, dtype=u8), torch.zeros(11), 300, 4)

    def refused(what, fn, *a, **k):
        with pytest.raises(ValueError, match=what + " holds"):
            fn(*a, **k)
    refused("x", amp.amp_rmsnorm, x, amp.BF16, 4, 301, 301, None, 0, None, 0, 1e-5, yq=ok)
    refused("res", amp.amp_rmsnorm, x, amp.BF16, 4, 300, 300, x[1:], 300, None, 0, 1e-5, yq=ok)
    refused("gamma", amp.amp_rmsnorm, x, amp.BF16, 4, 300, 300, None, 0, g[1:], amp.F32, 1e-5, yq=ok)
    refused("yq.q", amp.amp_rmsnorm, x, amp.BF16, 4, 300, 300, None, 0, g, amp.F32, 1e-5, yq=short_q)
    refused("ckpt.s", amp.amp_rmsnorm, x, amp.BF16, 4, 300, 300, None, 0, g, amp.F32, 1e-5, ckpt=short_s)
    refused("rstd", amp.amp_rmsnorm, x, amp.BF16, 4, 300, 300, None, 0, g, amp.F32, 1e-5, rstd=torch.zeros(3))
    refused("d_work", amp.amp_rmsnorm_backward, x, amp.BF16, 4, 300, 300, x, 300, None, g, amp.F32, torch.zeros(4), None, 0, None, 0,
            g, torch.zeros(1199))
    refused("x", amp.amp_swiglu, x, amp.BF16, 4, 151, 302, yq=ok)
    refused("ckpt.s", amp.amp_swiglu, x, amp.BF16, 4, 150, 300, ckpt=ok)      # 2 halves of 2 tiles
    refused("dxqt.q", amp.amp_swiglu_backward, x, amp.BF16, 4, 150, 300, x, 300, None, dxqt=amp.Fp8Tiles(
        torch.zeros(1199, dtype=u8), torch.zeros(300), 4, 300))
    refused("d_row", amp.amp_requantize_blockwise, ok, 4, 300, torch.zeros(3), None, 0, amp.Fp8Tiles(
        torch.zeros(300, 4, dtype=u8), torch.zeros(300), 4, 300))
    refused("qt.s", amp.amp_requantize_blockwise, ok, 4, 300, None, None, 0, amp.Fp8Tiles(
        torch.zeros(300, 4, dtype=u8), torch.zeros(299), 4, 300))


def test_binding_refuses_tensors_that_are_not_on_the_current_gpu():
    """Big enough, but host memory: the kernel would fault."""
    x, g, r = torch.zeros(4, 300, dtype=torch.bfloat16), torch.zeros(300), torch.zeros(4)
    t = amp.Fp8Tiles(torch.zeros(4, 300, dtype=torch.uint8), torch.zeros(3, 4), 300, 4)
    tt = amp.Fp8Tiles(torch.zeros(300, 4, dtype=torch.uint8), torch.zeros(1, 300), 4, 300)
    gt = amp.Fp8Tiles(torch.zeros(4, 150, dtype=torch.uint8), torch.zeros(2, 4), 150, 4)
    for fn, a, k in ((amp.amp_rmsnorm, (x, amp.BF16, 4, 300, 300, None, 0, g, amp.F32, 1e-5), dict(yq=t)),
                     (amp.amp_rmsnorm_backward, (x, amp.BF16, 4, 300, 300, x, 300, None, g, amp.F32, r), dict(dx=x, lddx=300)),
                     (amp.amp_swiglu, (x, amp.BF16, 4, 150, 300), dict(yq=gt)),
                     (amp.amp_swiglu_backward, (x[:, :150], amp.BF16, 4, 150, 300, x, 300, None), dict(dx=x, lddx=300)),
                     (amp.amp_requantize_blockwise, (t, 4, 300, None, None, 0, tt), {})):
        with pytest.raises(ValueError, match="on cpu"):
            fn(*a, **k)


@pytest.mark.parametrize("call", [norm, norm_back, gate, gate_back, requant])
def test_columns_beyond_a_launch_are_refused(call):
    assert call(cols=(1 << 26) + 1) == EUNSUP


def test_binding_refuses_scalars_without_room():
    x, none = torch.zeros(2, 256, dtype=torch.bfloat16), torch.zeros(0)
    y = torch.zeros(2, 256, dtype=torch.bfloat16)
    for k in ("d_scale", "d_amax"):
        with pytest.raises(ValueError, match=k):
            amp.amp_rmsnorm(x, amp.BF16, 2, 256, 256, None, 0, None, 0, 1e-5, y=y, ldy=256, **{k: none})
        with pytest.raises(ValueError, match=k):
            amp.amp_swiglu(x, amp.BF16, 2, 128, 256, y=y, ldy=256, **{k: none})


def test_the_quick_module_takes_plain_operands_only():
    """Anything else gives None (the binding's own path decides), a plain call
    the entry point's status; every call here is refused before device work."""
    from mixed_precision_numerics_amd import _quick
    lib = amp.load()
    names = ("amp_rmsnorm", "amp_rmsnorm_backward", "amp_swiglu", "amp_swiglu_backward", "amp_requantize_blockwise")
    _quick.bind(torch.Tensor, amp.Fp8Tiles, *(amp.ctypes.cast(getattr(lib, n), amp.ctypes.c_void_p).value for n in names))
    x, g = torch.zeros(4, 300, dtype=torch.bfloat16), torch.zeros(300)
    q, s = torch.zeros(4, 300, dtype=torch.uint8), torch.zeros(3, 4)
    good = [x, amp.BF16, 4, 300, 300, None, 0, g, 9, 1e-5, None, 0, None, amp.BF16, 0, None, None, amp.Fp8Tiles(q, s, 300, 4), None, None, 0, -1]
    assert _quick.rmsnorm(*good) == EUNSUP              # gamma's type; all operands are plain

    def but(i, v):
        return _quick.rmsnorm(*good[:i], v, *good[i + 1:])
    for i, v in ((0, P), (0, x[:, :200]), (0, torch.zeros(4, 299, dtype=torch.bfloat16)), (2, 5), (2, "4"), (2, 1 << 70), (4, 400), (9, 1),
                 (16, torch.zeros(0)), (17, P), (17, q), (17, amp.Fp8Tiles(q, s[:2], 300, 4)), (17, amp.Fp8Tiles(q, s, 301, 4)),
                 (17, amp.Fp8Tiles(P, P, 300, 4)), (21, 0)):
        assert but(i, v) is None, (i, v)
    assert but(2, -1) == EINVAL and but(1, 7) == EUNSUP
    with pytest.raises(TypeError):
        _quick.rmsnorm(*good[:-1])
    dead = amp.Fp8Tiles(q, s, 300, 4)
    dead.tensors = (q.clone(), s)                       # not what the structure points to
    assert but(17, dead) is None


@pytest.mark.parametrize("part", [0, 1])
@pytest.mark.parametrize("how", ["resize_", "set_", "data", "field"])
def test_binding_refuses_tiles_that_no_longer_point_to_their_tensors(how, part):
    """The room is checked at the tensors, the kernel follows the structure."""
    def made(rows, nb):
        q, s = torch.zeros(rows, 512, dtype=torch.uint8), torch.zeros(nb, rows)
        t = amp.Fp8Tiles(q, s, 512, rows)
        v = t.tensors[part]
        if how == "resize_":
            v.resize_(64 * v.shape[0], v.shape[1])
        elif how == "set_":
            v.set_(torch.zeros_like(v))
        elif how == "data":
            v.data = torch.zeros_like(v)
        else:
            setattr(t, "qs"[part], getattr(t, "qs"[part]) + 16)
        return t

    x, r = torch.zeros(4, 600, dtype=torch.bfloat16), torch.zeros(4)
    good, tall = amp.Fp8Tiles(torch.zeros(4, 600, dtype=torch.uint8), torch.zeros(6, 4), 600, 4), made(300, 1)
    for what, fn, a, k in (("yq", amp.amp_rmsnorm, (x, amp.BF16, 4, 300, 600, None, 0, None, 0, 1e-5), dict(yq=made(4, 3))),
                           ("ckpt", amp.amp_rmsnorm, (x, amp.BF16, 4, 300, 600, None, 0, None, 0, 1e-5), dict(ckpt=made(4, 3))),
                           ("ckpt", amp.amp_rmsnorm_backward, (x, amp.BF16, 4, 300, 600, None, 0, made(4, 3), None, 0, r), dict(dx=x, lddx=600)),
                           ("yq", amp.amp_swiglu, (x, amp.BF16, 4, 300, 600), dict(yq=made(4, 3))),
                           ("ckpt", amp.amp_swiglu_backward, (x, amp.BF16, 4, 150, 600, None, 0, made(4, 4)), dict(dx=x, lddx=600)),
                           ("yqt", amp.amp_swiglu_backward, (x, amp.BF16, 4, 300, 600, x, 600, None), dict(yqt=tall)),
                           ("x", amp.amp_requantize_blockwise, (made(4, 3), 4, 300, None, None, 0, good), {}),
                           ("qt", amp.amp_requantize_blockwise, (good, 4, 300, None, None, 0, tall), {})):
        with pytest.raises(ValueError, match=what + r"\." + "qs"[part] + " has moved"):
            fn(*a, **k)


def test_tiles_of_addresses_follow_their_fields():
    """Without a tensor to compare with, the structure's fields are what a call takes."""
    t = amp.Fp8Tiles(P, P, 300, 4)
    t.q = 2 * P
    assert amp._tiles("f", "yq", t, 4, 300, [None]) == amp.ctypes.addressof(t)
    empty = amp.Fp8Tiles(torch.zeros(0, dtype=torch.uint8), torch.zeros(0), 300, 4)
    assert amp._tiles("f", "yq", empty, 0, 300, [-1]) == amp.ctypes.addressof(empty)


def test_norm_gradient_over_the_stored_input_needs_its_stride():
    assert norm_back(h=2 * P, ldh=301) == EINVAL and norm_back(h=2 * P, ldh=301, dgamma=None) == EINVAL


def test_every_finite_eps_is_accepted():
    top = float(torch.finfo(torch.float32).max)
    assert norm(eps=top, rows=0) == 0 and norm(eps=3.1e38, rows=0) == 0 and norm(eps=0.0, rows=0) == 0
    assert norm(eps=float("inf"), rows=0) == EINVAL and norm(eps=-0.5, rows=0) == EINVAL
