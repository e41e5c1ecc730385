"""Gated feed-forward block: outputs over inputs or over one another are
refused before any device work; operands that only lie between one another's
rows are taken."""
import itertools
import os

import pytest

import mixed_precision_numerics_amd as amp

pytestmark = pytest.mark.skipif(not os.path.exists(amp.lib_path()), reason="libamp.so not built")
EINVAL = -1
M, F, K, B = 6, 24, 40, 2
AREA = 4 * amp.GEMM_SWIGLU_WORK
# rows, columns, bytes of each operand
FORWARD = dict(x=(M, K, 2), w=(2 * F, K, 2), y=(M, F, 2), gu=(M, 2 * F, 2))
BACKWARD = dict(dy=(M, F, 2), x=(M, K, 2), w=(2 * F, K, 2), gu=(M, 2 * F, 2), dgu=(M, 2 * F, 2), y=(M, F, 2), dx=(M, K, 2), dw=(2 * F, K, 4),
                work=(1, amp.GEMM_SWIGLU_WORK, 4))
FAR = {n: (i + 1) << 28 for i, n in enumerate(BACKWARD)}       # places that are far apart


def forward(at, ld):
    return amp.load().amp_gemm_swiglu(M, F, K, at["x"], amp.BF16, ld["x"], at["w"], ld["w"], at.get("y"), ld["y"], at.get("gu"), ld["gu"], None)


def backward(at, ld):
    return amp.load().amp_gemm_swiglu_backward(
        M, F, K, at["dy"], amp.BF16, ld["dy"], at["x"], ld["x"], at["w"], ld["w"], at.get("gu"), ld["gu"], at["dgu"], ld["dgu"], at.get("y"), ld["y"],
        at.get("dx"), ld["dx"], at.get("dw"), amp.F32, ld["dw"], at.get("work"), None)


def call(operands, at, pad=0, **lds):
    ld = {n: c + pad for n, (_, c, _) in operands.items()}
    ld.update(lds)
    return (forward if operands is FORWARD else backward)(at, ld)


def places(operands, without=()):
    return {n: FAR[n] for n in operands if n not in without}


def taken(status):
    """Accepted by every check of the arguments: the next is for a GPU."""
    return status != EINVAL


@pytest.fixture(autouse=True)
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("accepted calls would run")


PAIRS = [(FORWARD, (), p) for p in (("y", "x"), ("y", "w"), ("gu", "x"), ("gu", "w"), ("gu", "y"))]
PAIRS += [(BACKWARD, ("y",), p) for p in itertools.product(("dgu", "dx", "dw", "work"), ("dy", "x", "w", "gu")) if p != ("dgu", "gu")]
PAIRS += [(BACKWARD, ("y",), p) for p in itertools.combinations(("dgu", "dx", "dw", "work"), 2)]
PAIRS += [(BACKWARD, ("gu",), ("y", n)) for n in ("dy", "x", "w", "dgu", "dx", "dw", "work")]


def span(operands, n, pad):
    r, c, b = operands[n]
    return ((r - 1) * (c + pad) + c) * b


@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("operands,without,pair", PAIRS, ids=["-".join(p) for _, _, p in PAIRS])
def test_overlap_is_refused_and_neighbours_are_not(operands, without, pair, pad):
    a, b = pair
    at = places(operands, without)
    assert taken(call(operands, at, pad))
    ea, eb = span(operands, a, pad), span(operands, b, pad)
    at[a] = at[b]
    assert call(operands, at, pad) == EINVAL or (pad and operands[a][1] * operands[a][2] != operands[b][1] * operands[b][2])
    whole = not pad or "work" in pair
    for off, ok in ((eb - 4, False), (eb, True), (4 - ea, False), (-ea, True)):
        at[a] = at[b] + off
        if "work" in pair and pad and not ok:
            # the one row ends inside the other's first or last: seen whatever the gaps
            assert call(operands, at, pad) == EINVAL
        elif ok or whole:
            assert taken(call(operands, at, pad)) == ok, off


@pytest.mark.parametrize("pair", [("y", "x"), ("gu", "y"), ("gu", "w")])
def test_rows_of_one_pitch_between_one_another(pair):
    """Columns of one buffer: any two that share no column are taken, in every order of their rows."""
    a, b = pair
    ra, ca, _ = FORWARD[a]
    rb, cb, _ = FORWARD[b]
    pitch = ca + cb + 6
    for rows in range(-ra - 1, rb + 2):
        for off in range(-ca - 3, cb + 4):
            at = places(FORWARD)
            at[a] = at[b] + 2 * (rows * pitch + off)
            lds = {a: pitch, b: pitch}
            # row i of a starts at column off of row rows + i of b, counted from where b's row starts
            meets = any(0 <= i + rows + k < rb and -ca < off - k * pitch < cb for i in range(ra) for k in (-1, 0, 1))
            assert taken(call(FORWARD, at, **lds)) == (not meets), (rows, off)


@pytest.mark.parametrize("which", ["y", "x"])
def test_one_without_gaps_beside_rows_with_gaps(which):
    """A whole matrix fits between two rows of another, to the element."""
    gap = M * (F if which == "y" else K) + 10
    other = "x" if which == "y" else "y"
    co = FORWARD[other][1]
    for off in range(-2 * gap, 8 * gap, 7):
        at = places(FORWARD, ("gu",))
        at[which] = at[other] + 2 * off
        mine = M * FORWARD[which][1]
        meets = any(off < i * (co + gap) + co and i * (co + gap) < off + mine for i in range(M))
        assert taken(call(FORWARD, at, **{other: co + gap})) == (not meets), off


def test_operands_that_the_call_does_not_read_may_be_anywhere():
    at = places(BACKWARD, ("y", "dw"))
    at["x"] = at["dx"]                                          # only dw would read x
    assert taken(call(BACKWARD, at))
    at = places(BACKWARD, ("y", "dx"))
    at["w"] = at["dw"]
    assert taken(call(BACKWARD, at))
    at = places(BACKWARD, ("y",))
    at["dgu"] = at["gu"]                                        # in place
    assert taken(call(BACKWARD, at))
    at["dgu"] += 4
    assert call(BACKWARD, at) == EINVAL


def test_different_pitches_with_gaps_are_not_compared():
    at = places(FORWARD, ("gu",))
    at["y"] = at["x"] + 2 * K
    assert taken(call(FORWARD, at, x=K + 100, y=F + 60))
    # ... but a single row has none
    assert amp.load().amp_gemm_swiglu(1, F, K, at["x"], amp.BF16, K + 100, at["w"], K, at["x"] + 2 * K - 2, F + 60, None, 0, None) == EINVAL


@pytest.mark.parametrize("tokens,features", [(0, F), (M, 0)])
@pytest.mark.parametrize("pad", [0, 8])
def test_inputs_of_a_call_that_reads_none_may_be_anything(tokens, features, pad):
    """Without tokens dw is zeros, without features dx is: inputs with no stride, over the outputs, are not looked at."""
    for ld in (0, 1, K):
        for off in (0, 2, 100):
            at = 1 << 28
            st = amp.load().amp_gemm_swiglu_backward(tokens, features, K, at + off, amp.BF16, ld, at + off, ld, at + off, ld, None, 0, at + off, ld,
                                                     None, 0, at if features == 0 else None, K + pad, at if tokens == 0 else None, amp.F32, K + pad,
                                                     None, None)
            assert taken(st)
