"""Refusals of the gated feed-forward block and of the calls over lists of
tensors: all come before any device work, so they need no GPU."""
import os

import pytest
import torch

import mixed_precision_numerics_amd as amp

pytestmark = pytest.mark.skipif(not os.path.exists(amp.lib_path()), reason="libamp.so not built")
EINVAL, EUNSUP = -1, -2
P = 4096            # a pointer that no refused call follows


def forward(**k):
    a = dict(M=4, F=24, K=40, x=P, t=amp.BF16, ldx=40, w=P, ldw=40, y=2 * P, ldy=24, gu=None, ldgu=0)
    a.update(k)
    return amp.load().amp_gemm_swiglu(*a.values(), None)


def backward(**k):
    a = dict(M=4, F=24, K=40, dy=P, t=amp.BF16, lddy=24, x=P, ldx=40, w=P, ldw=40, gu=P, ldgu=48, dgu=2 * P, lddgu=48, y=None, ldy=0,
             dx=3 * P, lddx=40, dw=4 * P, dwt=amp.BF16, lddw=40, d_work=5 * P)
    a.update(k)
    return amp.load().amp_gemm_swiglu_backward(*a.values(), None)


def tensors(*entries):
    a = (amp._Tensor * len(entries))()
    for t, (p, n, dt) in zip(a, entries):
        t.p, t.n, t.type = p, n, dt
    return a


def norm(entries=((P, 5, amp.F32),), count=None, grads=True, **k):
    arr = tensors(*entries)
    a = dict(grads=amp.ctypes.addressof(arr) if grads else None, count=len(entries) if count is None else count, first=1, d_state=P, d_norm=P,
             max_norm=1.0, d_out=P)
    a.update(k)
    return amp.load().amp_grad_norm_list(*a.values(), None)


def clip(entries=((P, 5, amp.F32),), outs=None, count=None, grads=True, **k):
    arr = tensors(*entries)
    o = tensors(*outs) if outs is not None else None
    a = dict(grads=amp.ctypes.addressof(arr) if grads else None, outs=amp.ctypes.addressof(o) if o is not None else None,
             count=len(entries) if count is None else count, d_state=P, d_coef=P)
    a.update(k)
    return amp.load().amp_grad_clip_list(*a.values(), None)


@pytest.mark.parametrize("call,bad", [
    (forward, dict(M=-1)), (forward, dict(F=-1)), (forward, dict(K=-1)), (forward, dict(x=None)), (forward, dict(w=None)),
    (forward, dict(y=None)), (forward, dict(ldx=39)), (forward, dict(ldw=39)), (forward, dict(ldy=23)), (forward, dict(gu=P, ldgu=47)),
    (forward, dict(x=P + 1)), (forward, dict(w=P + 1)), (forward, dict(y=P + 1)), (forward, dict(gu=P + 1, ldgu=48)),
    (backward, dict(M=-1)), (backward, dict(F=-1)), (backward, dict(K=-1)), (backward, dict(dy=None)), (backward, dict(dgu=None)),
    (backward, dict(x=None)), (backward, dict(w=None)), (backward, dict(y=6 * P, ldy=24)), (backward, dict(lddy=23)),
    (backward, dict(ldx=39)), (backward, dict(ldw=39)), (backward, dict(ldgu=47)), (backward, dict(lddgu=47)), (backward, dict(lddx=39)),
    (backward, dict(lddw=39)), (backward, dict(gu=None, y=6 * P, ldy=23)), (backward, dict(gu=2 * P, ldgu=56)),
    (backward, dict(gu=None, dw=None, x=None)), (backward, dict(gu=None, dx=None, w=None)), (backward, dict(dw=P + 1)),
    (backward, dict(dwt=amp.F32, dw=P + 2)), (backward, dict(d_work=P + 2)), (backward, dict(dy=P + 1)), (backward, dict(dgu=P + 1)),
    (backward, dict(dx=P + 1)), (backward, dict(M=0, dw=4 * P, lddw=39)),
    (norm, dict(count=-1)), (norm, dict(grads=False)), (norm, dict(d_state=None)), (norm, dict(d_norm=None)), (norm, dict(d_state=P + 4)),
    (norm, dict(d_norm=P + 4)), (norm, dict(d_out=P + 2)), (norm, dict(max_norm=0.0)), (norm, dict(max_norm=float("nan"))),
    (norm, dict(max_norm=float("inf"))), (norm, dict(entries=((P, -1, amp.F32),))), (norm, dict(entries=((None, 1, amp.F32),))),
    (norm, dict(entries=((P, 4, amp.F16), (P + 2, 1, amp.F32)))), (norm, dict(entries=((P + 1, 1, amp.BF16),))),
    (clip, dict(count=-1)), (clip, dict(grads=False)), (clip, dict(d_state=P + 4)), (clip, dict(d_coef=P + 1)),
    (clip, dict(outs=((2 * P, 4, amp.F32),))), (clip, dict(outs=((None, 5, amp.F32),))), (clip, dict(outs=((P, 5, amp.F16),))),
    (clip, dict(outs=((P + 2, 5, amp.F32),))),
])
def test_invalid_arguments(call, bad):
    assert call(**bad) == EINVAL


@pytest.mark.parametrize("call,bad", [
    (forward, dict(t=amp.F32)), (forward, dict(t=amp.E4M3)), (forward, dict(K=(1 << 26) + 1)), (forward, dict(F=(1 << 26) + 1)),
    (forward, dict(M=1 << 40)), (forward, dict(M=1 << 30, F=1 << 20)), (forward, dict(M=(1 << 63) - 1)),
    (backward, dict(t=amp.F32)), (backward, dict(dwt=amp.F16)), (backward, dict(F=1 << 26, K=1 << 26)), (backward, dict(M=(1 << 63) - 1)),
    (norm, dict(entries=((P, 5, amp.E4M3),))), (norm, dict(entries=((P, (1 << 37) + 1, amp.BF16),))), (norm, dict(count=65537)),
    (clip, dict(entries=((P, 5, 9),))), (clip, dict(outs=((2 * P, 5, amp.E5M2),))), (clip, dict(count=65537)),
])
def test_unsupported_types_and_sizes(call, bad):
    assert call(**bad) == EUNSUP


def test_empty_work_is_accepted_without_pointers():
    assert forward(M=0, x=None, y=None) == 0 and forward(F=0, w=None, y=None) == 0
    assert backward(M=0, dw=None, dy=None, dgu=None) == 0 and backward(F=0, dx=None, dy=None) == 0 and backward(M=0, F=0) == 0
    assert clip(entries=(), grads=False) == 0


def test_binding_refuses_tensors_smaller_than_the_call_spans():
    bf = torch.bfloat16
    x, w, y, gu = torch.zeros(4, 40, dtype=bf), torch.zeros(48, 40, dtype=bf), torch.zeros(4, 24, dtype=bf), torch.zeros(4, 48, dtype=bf)
    work = torch.zeros(16)

    def refused(what, fn, *a, **k):
        with pytest.raises(ValueError, match=what + " holds"):
            fn(*a, **k)
    refused("x", amp.amp_gemm_swiglu, 5, 24, 40, x, amp.BF16, 40, w, 40, torch.zeros(5, 24, dtype=bf), 24)
    refused("w", amp.amp_gemm_swiglu, 4, 24, 40, x, amp.BF16, 40, w[1:], 40, y, 24)
    refused("y", amp.amp_gemm_swiglu, 4, 24, 40, x, amp.BF16, 40, w, 40, y, 25)
    refused("gu", amp.amp_gemm_swiglu, 4, 24, 40, x, amp.BF16, 40, w, 40, y, 24, gu[1:], 48)

    def back(**k):
        a = dict(M=4, F=24, K=40, dy=y, t=amp.BF16, lddy=24, x=x, ldx=40, w=w, ldw=40, gu=gu, ldgu=48, dgu=gu.clone(), lddgu=48)
        a.update(k)
        return amp.amp_gemm_swiglu_backward(**a)
    refused("dy", back, dy=y[1:])
    refused("dgu", back, dgu=gu[1:])
    refused("dx", back, dx=x[1:], lddx=40)
    refused("dw", back, dw=w, dwt=amp.F32, lddw=40)
    refused("d_work", back, dw=w, lddw=40, d_work=work)
    refused("tensor 1", amp.TensorList, [(x, 160, amp.BF16), (x, 161, amp.BF16)])


def test_binding_refuses_tensors_that_are_not_on_the_current_gpu():
    bf = torch.bfloat16
    x, w, y, gu = torch.zeros(4, 40, dtype=bf), torch.zeros(48, 40, dtype=bf), torch.zeros(4, 24, dtype=bf), torch.zeros(4, 48, dtype=bf)
    some, st, ns = amp.TensorList([(x, 160, amp.BF16)]), torch.zeros(10), torch.zeros(1025, dtype=torch.float64)
    for fn, a, k in ((amp.amp_gemm_swiglu, (4, 24, 40, x, amp.BF16, 40, w, 40, y, 24), {}),
                     (amp.amp_gemm_swiglu_backward, (4, 24, 40, y, amp.BF16, 24, x, 40, w, 40, gu, 48, gu, 48), dict(dx=x, lddx=40)),
                     (amp.amp_grad_norm_list, (some, True, st, ns), {}), (amp.amp_grad_clip_list, (some,), {})):
        with pytest.raises(ValueError, match="on cpu"):
            fn(*a, **k)


@pytest.mark.parametrize("how", ["resize_", "set_", "data"])
def test_binding_refuses_lists_whose_tensors_have_moved(how):
    a, b = torch.zeros(100), torch.zeros(7)
    some, st, ns = amp.TensorList([(a, 100, amp.F32), (b, 7, amp.F32)]), torch.zeros(10), torch.zeros(1025, dtype=torch.float64)
    if how == "resize_":
        b.resize_(1 << 20)
    elif how == "set_":
        b.set_(torch.zeros(7))
    else:
        b.data = torch.zeros(7)
    for fn, args in ((amp.amp_grad_norm_list, (some, True, st, ns)), (amp.amp_grad_clip_list, (some,)),
                     (amp.amp_grad_clip_list, (amp.TensorList([(a, 100, amp.F32), (a, 7, amp.F32)]), some))):
        with pytest.raises(ValueError, match="has moved"):
            fn(*args)


def test_lists_that_do_not_fit_are_refused():
    a, b = torch.zeros(100), torch.zeros(7)
    with pytest.raises(ValueError, match="1 gradients, 2 outputs"):
        amp.amp_grad_clip_list(amp.TensorList([(a, 100, amp.F32)]), amp.TensorList([(a, 100, amp.F32), (b, 7, amp.F32)]))
    with pytest.raises(ValueError, match="tensor 0 is of type 3"):
        amp.TensorList([(a, 100, amp.E4M3)])
    assert len(amp.TensorList([])) == 0


def test_lists_that_are_written_to_hold_no_memory_twice():
    a, b = torch.zeros(100), torch.zeros(100)
    twice, over = [(a, 100, amp.F32), (a, 100, amp.F32)], [(a, 100, amp.F32), (a[99:], 1, amp.F32)]
    for entries in (twice, over):
        some = amp.TensorList(entries)
        with pytest.raises(ValueError, match="tensors of grads overlap"):
            amp.amp_grad_clip_list(some)
        with pytest.raises(ValueError, match="tensors of outs overlap"):
            amp.amp_grad_clip_list(amp.TensorList([(b, e[1], amp.F32) for e in entries]), some)
    assert amp.TensorList([(a[50:], 50, amp.F32), (a, 50, amp.F32), (a, 0, amp.F32)]).apart


def test_lists_of_elements_with_gaps_are_refused():
    a = torch.zeros(8, 8)
    for t in (a[:, :4], a[::2]):
        with pytest.raises(ValueError, match="tensor 1's elements are not one after another"):
            amp.TensorList([(a, 64, amp.F32), (t, 32, amp.F32)])
    assert len(amp.TensorList([(a.t(), 64, amp.F32), (a[:4], 32, amp.F32), (a[:, :1], 0, amp.F32)])) == 3
