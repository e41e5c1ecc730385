"""Lists of tensors on the CPU: what the binding refuses of them, on its Python
path and in the compiled module that plain operands take."""
import os

import pytest
import torch

import mixed_precision_numerics_amd as amp

pytestmark = pytest.mark.skipif(not os.path.exists(amp.lib_path()), reason="libamp.so not built")
EINVAL = -1


@pytest.fixture
def quick(monkeypatch):
    """The compiled module with the library's entry points, as once a GPU is in use."""
    pytest.importorskip("mixed_precision_numerics_amd._quick")
    amp.load()
    monkeypatch.setattr(amp, "_plain", None)
    monkeypatch.setattr(amp, "_current", lambda: (0, 0))
    amp._bind()
    return amp._plain


def takes(quick, some):
    """Whether the compiled module passes the list to the library, which refuses the call for its NULL state."""
    st = quick.norm_list(some, True, None, None, 1.0, None, 0, -1)
    assert st in (None, EINVAL)
    return st is not None


def moved_into(t, other):
    """t, a tensor at an address where memory of another size begins now."""
    t.set_(torch.from_dlpack(other))
    return t


@pytest.mark.parametrize("left", [7, 99])
def test_a_tensor_of_less_memory_at_the_same_address_is_refused(quick, left):
    """Storage that was given up may come back at the same address, and smaller."""
    buf = torch.zeros(100)
    t = torch.empty(0).set_(buf)
    some, st, ns = amp.TensorList([(torch.zeros(3), 3, amp.F32), (t, 100, amp.F32)]), torch.zeros(10), torch.zeros(1025, dtype=torch.float64)
    assert takes(quick, some)
    moved_into(t, buf[:left])
    assert t.data_ptr() == buf.data_ptr() and t.untyped_storage().nbytes() == 4 * left
    assert not takes(quick, some)
    for fn, args in ((amp.amp_grad_norm_list, (some, True, st, ns)), (amp.amp_grad_clip_list, (some,))):
        with pytest.raises(ValueError, match="a tensor of grads holds"):
            fn(*args)


def test_a_tensor_that_shrank_within_its_memory_is_taken():
    """Its elements are still there: the list's lengths count."""
    t = torch.zeros(100)
    some = amp.TensorList([(t, 100, amp.F32)])
    t.resize_(7)
    assert amp._listed("f", "grads", some, [-1])
    t.resize_(100)
    assert amp._listed("f", "grads", some, [-1])
