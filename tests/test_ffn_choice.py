"""Which kernel each size of the gated feed-forward block takes: the rule is
plain C++ and is asked here without a GPU, so that the tests which are meant for
a kernel are known to reach it."""
import ctypes
import os
import shutil
import subprocess

import pytest

import test_gpu_ffn as small
from ffn_shapes import LARGE

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixed_precision_numerics_amd", "csrc")
FEW, LARGE_TILES, RING, SMALL, STAGED = range(5)
WORK = 1 << 23
SOURCE = """
#include "ffn_choice.hpp"
extern "C" int gate(int64_t M, int64_t F, int64_t K, int fast, int gradient) { return amp::gate_form(M, F, K, fast, gradient); }
extern "C" void gradients(int64_t M, int64_t F, int64_t K, int fast, int64_t room, int dx, int dw, int* out) {
  const amp::GradientForm f = amp::gradient_form(dx ? M : 0, dx ? K : 0, 2 * F, dw ? 2 * F : 0, dw ? K : 0, M, fast, room);
  out[0] = f.wide; out[1] = f.split_x; out[2] = f.split_w; out[3] = f.dx_first;
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("choice")
    (d / "choice.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-fPIC", "-shared", "-I" + CSRC, str(d / "choice.cpp"), "-o", str(d / "choice.so")], check=True)
    lib = ctypes.CDLL(str(d / "choice.so"))
    lib.gate.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 2
    lib.gradients.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]

    class Rule:
        @staticmethod
        def gate(M, F, K, fast=True, gradient=False):
            return lib.gate(M, F, K, fast, gradient)

        @staticmethod
        def gradients(M, F, K, fast=True, room=WORK, dx=True, dw=True):
            out = (ctypes.c_int * 4)()
            lib.gradients(M, F, K, fast, room, dx, dw, out)
            return tuple(out)
    return Rule


@pytest.mark.parametrize("M,F,K", LARGE)
def test_the_large_shapes_take_large_tiles(rule, M, F, K):
    assert K % 8 == 0 and F % 4 == 0                            # the direct loads take them
    assert rule.gate(M, F, K) == rule.gate(M, F, K, gradient=True) == LARGE_TILES
    assert rule.gradients(M, F, K)[:3] == (1, 1, 1) and rule.gradients(M, F, K, room=0)[0]


def test_some_large_shape_takes_them_for_either_product_alone(rule):
    assert any(rule.gradients(*s, dw=False)[0] and rule.gradients(*s, dx=False)[0] for s in LARGE)


def test_the_small_shapes_take_every_other_form(rule):
    shapes = small.SHAPES + small.BACK_SHAPES + small.TILE_SHAPES + [(4100, 2056, 328), (2048, 4096, 192)]
    for gradient in (False, True):
        got = {rule.gate(*s, fast=fast, gradient=gradient) for s in shapes for fast in (False, True)}
        assert got >= {FEW, RING, SMALL, STAGED}
    forms = [rule.gradients(*s, fast=fast) for s in small.BACK_SHAPES for fast in (False, True)]
    assert any(f[1] > 1 for f in forms) and any(f[2] > 1 for f in forms) and {f[3] for f in forms} == {0, 1}


@pytest.mark.parametrize("M,F,K,form", [(1, 14336, 4096, FEW), (16, 14336, 4096, FEW), (33, 20480, 5120, SMALL), (64, 14336, 4096, RING),
                                        (65, 14336, 4096, RING), (1000, 14336, 4096, LARGE_TILES), (8192, 14336, 4096, LARGE_TILES),
                                        (1, 1 << 26, 1, SMALL)])
def test_forward_choices(rule, M, F, K, form):
    assert rule.gate(M, F, K) == form
    assert rule.gate(M, F, K, fast=False) == (FEW if form == FEW else STAGED)


def test_parts_stay_within_the_work_area(rule):
    for M in (1, 7, 100, 777, 4000, 1 << 20):
        for F in (1, 33, 2048, 14336):
            for K in (1, 72, 512, 4096):
                for room in (0, 1000, WORK):
                    wide, sx, sw, _ = rule.gradients(M, F, K, room=room)
                    assert (sx * M * K if sx > 1 else 0) + (sw * 2 * F * K if sw > 1 else 0) <= room
                    assert not wide or sx == sw == 1
