"""Gated feed-forward block: which sizes each call takes."""
import os

import pytest

import mixed_precision_numerics_amd as amp

pytestmark = pytest.mark.skipif(not os.path.exists(amp.lib_path()), reason="libamp.so not built")
EUNSUP, ENODEVICE = -2, -4
FAR = [1 << 48, 1 << 50, 1 << 52, 1 << 54, 1 << 56, 1 << 57]


@pytest.fixture(autouse=True)
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("accepted calls would run")


def forward(M, F, K):
    x, y, w = FAR[:3]
    return amp.load().amp_gemm_swiglu(M, F, K, x, amp.BF16, K, w, K, y, F, None, 0, None)


def backward(M, F, K):
    x, w, dy, dgu, dx, dw = FAR
    return amp.load().amp_gemm_swiglu_backward(M, F, K, dy, amp.BF16, F, x, K, w, K, None, 0, dgu, 2 * F, None, 0, dx, K, dw, amp.BF16, K, None, None)


# the product [M, 2F] alone has to fit the forward call: 2^22 tiles of 128 x 128
@pytest.mark.parametrize("M,F,K,forms,differentiates", [
    (1, 1 << 23, 8192, True, False), (1, 1 << 23, 1 << 12, True, True), (1 << 10, 1 << 20, 1 << 16, True, False),
    (1 << 29, 64, 64, True, True), ((1 << 29) + 1, 64, 64, False, False), (1 << 29, 64, 129, True, False),
    (1 << 23, 1 << 12, 64, True, True), (1 << 23, (1 << 12) + 1, 64, False, False), (512, 1 << 26, 4, True, True),
    (513, 1 << 26, 4, False, False), (1, 1 << 26, 1 << 26, True, False)])
def test_each_call_counts_the_products_that_it_forms(M, F, K, forms, differentiates):
    assert forward(M, F, K) == (ENODEVICE if forms else EUNSUP)
    assert backward(M, F, K) == (ENODEVICE if differentiates else EUNSUP)
