"""Global gradient norm and clipping over lists of tensors on the GPU, against
oracle/clip.py: the float64 sum of squares within n * 2^-52 of the exact one, the
coefficient as in test_gpu_clip, clipped values bit for bit."""
import math

import numpy as np
import pytest
import torch

import mixed_precision_numerics_amd as amp
from oracle import clip as OC
from oracle import formats as F
from gpu_util import dev, empty, host, scaler_state
from test_gpu_clip import GF, check_coef, grads

pytestmark = pytest.mark.gpu
EB = {amp.F32: 4, amp.F16: 2, amp.BF16: 2}
NPT = {amp.F32: np.uint32, amp.F16: np.uint16, amp.BF16: np.uint16}
INF = {amp.F16: 0x7C00, amp.BF16: 0x7F80, amp.F32: 0x7F800000}
NAN = {amp.F16: 0x7E00, amp.BF16: 0x7FC0, amp.F32: 0x7FC00000}


class Many:
    """Tensors of given lengths and types in one buffer, `gap` elements apart, all bits set between them."""

    def __init__(self, lengths, types, gap=0, codes=None):
        self.types, self.lengths = types, lengths
        self.at, size = [], 0
        for n, t in zip(lengths, types):
            size = -(-size // EB[t]) * EB[t]
            self.at.append(size)
            size += n * EB[t] + gap * EB[t]
        a = np.full(size + 16, 0xFF, np.uint8)
        for i, c in enumerate(codes or []):
            self.part(a, i)[:] = c
        self.d = dev(a)
        self.list = amp.TensorList([(self.d.data_ptr() + p, n, t) for p, n, t in zip(self.at, lengths, types)])

    def part(self, a, i):
        return a[self.at[i]:self.at[i] + self.lengths[i] * EB[self.types[i]]].view(NPT[self.types[i]])

    def read(self):
        a = host(self.d, np.uint8).copy()
        out = [self.part(a, i).copy() for i in range(len(self.lengths))]
        for i in range(len(self.lengths)):
            self.part(a, i)[:] = NPT[self.types[i]](~NPT[self.types[i]](0))
        assert np.all(a == 0xFF), "written between the tensors"
        return out


def state(S):
    st = empty(40)
    amp.amp_scaler_init(st, S)
    return st


def sums(m, codes, S):
    parts = [OC.norm_sq(c, GF[t], S) for c, t in zip(codes, m.types)]
    return math.fsum(p[0] for p in parts), any(p[1] for p in parts)


ALL = [amp.F32, amp.F16, amp.BF16]


def mixed(lengths, seed, types=None):
    types = types or [ALL[i % 3] for i in range(len(lengths))]
    return types, [grads(t, n, seed + i, 0.5 + i % 5) if n else np.zeros(0, NPT[t]) for i, (n, t) in enumerate(zip(lengths, types))]


# one element; nothing; ends inside a 16-byte piece, a chunk; more tensors than one launch takes; long next to short
LENGTHS = [[1], [0], [0, 0, 5, 0], [7, 8, 9, 4095, 4096, 4097, 12289], [3 + i % 11 for i in range(700)], [1, 300007, 2, 0, 70001],
           [(1 << 24) + 13, 5, (1 << 20) + 1], [0] * 200 + [33] + [0] * 200]


@pytest.mark.parametrize("S", [1.0, 1024.0])
@pytest.mark.parametrize("gap", [0, 1])
@pytest.mark.parametrize("lengths", LENGTHS, ids=[f"{len(x)}x{max(x)}" for x in LENGTHS])
def test_norm_of_a_list(lengths, gap, S):
    types, codes = mixed(lengths, 40)
    m = Many(lengths, types, gap, codes)
    st, ns, out = state(S), empty(amp.NORM_STATE_BYTES, 0xFF), torch.full((2,), -1.0, device="cuda")
    amp.amp_grad_norm_list(m.list, True, st, ns, 1.0, out)
    want, bad = sums(m, codes, S)
    n = sum(lengths)
    got = host(ns, np.float64)[0]
    assert not bad and int(scaler_state(st)["found_inf"]) == 0
    assert abs(got - want) <= n * 2.0 ** -52 * want, (got, want)
    check_coef(host(out, np.float32), want, max(n, 1))
    # once more, added to the first, bit for bit the same sum
    amp.amp_grad_norm_list(m.list, False, st, ns)
    assert host(ns, np.float64)[0] == got + got
    amp.amp_grad_norm_list(m.list, True, st, ns)
    assert host(ns, np.float64)[0] == got


@pytest.mark.parametrize("t", ALL)
@pytest.mark.parametrize("what", [INF, NAN])
@pytest.mark.parametrize("at", [(0, 0), (2, 4096), (2, 5000), (450, 2)])
def test_a_non_finite_element_anywhere_sets_the_flag(t, what, at):
    lengths = [9, 20, 5001] + [3] * 500
    types, codes = mixed(lengths, 60, [t] * len(lengths))
    codes[at[0]][at[1]] = what[t]
    m = Many(lengths, types, 1, codes)
    st, ns, out = state(8.0), empty(amp.NORM_STATE_BYTES), torch.zeros(2, device="cuda")
    amp.amp_grad_norm_list(m.list, True, st, ns, 1.0, out)
    want, bad = sums(m, codes, 8.0)
    assert bad and int(scaler_state(st)["found_inf"]) == 1
    assert abs(host(ns, np.float64)[0] - want) <= sum(lengths) * 2.0 ** -52 * want
    assert host(out, np.float32).tolist() == [1.0, math.inf]


def test_the_list_agrees_with_one_call_per_tensor():
    lengths = [5, 100003, 64, 0, 1 << 18]
    types, codes = mixed(lengths, 80)
    m = Many(lengths, types, 0, codes)
    st, a, b = state(4.0), empty(amp.NORM_STATE_BYTES), empty(amp.NORM_STATE_BYTES)
    out = torch.empty(2, 2, device="cuda")
    amp.amp_grad_norm_init(a)
    for p, n, t in zip(m.at, lengths, types):
        amp.amp_grad_norm_accumulate(m.d.data_ptr() + p, t, n, st, a)
    amp.amp_clip_coefficient(a, 0.25, st, out[0])
    amp.amp_grad_norm_list(m.list, True, st, b, 0.25, out[1])
    x, y = host(a, np.float64)[0], host(b, np.float64)[0]
    assert abs(x - y) <= 2 * sum(lengths) * 2.0 ** -53 * x
    want, _ = sums(m, codes, 4.0)
    for o in out:
        check_coef(host(o, np.float32), want, sum(lengths), 0.25)


def clipped(codes, t, o, S, coef):
    x = F.f32(F.decode(codes, GF[t]))
    with np.errstate(over="ignore", invalid="ignore"):
        v = F.f32(F.f32(x * float(F.f32(1.0 / S))) * float(np.float32(coef)))
        return F.encode(v, GF[o])


def same(got, want, o):
    """Equal codes, any NaN for a NaN."""
    return np.array_equal(F.decode(got, GF[o]), F.decode(want, GF[o]), equal_nan=True) and np.array_equal(
        np.signbit(F.decode(got, GF[o])[~np.isnan(F.decode(got, GF[o]))]), np.signbit(F.decode(want, GF[o])[~np.isnan(F.decode(want, GF[o]))]))


@pytest.mark.parametrize("o", ALL + [None])
@pytest.mark.parametrize("gap", [0, 1])
@pytest.mark.parametrize("lengths", LENGTHS[:6] + LENGTHS[7:], ids=[f"{len(x)}x{max(x)}" for x in LENGTHS[:6] + LENGTHS[7:]])
def test_clip_of_a_list(lengths, gap, o):
    types, codes = mixed(lengths, 90)
    for i, c in enumerate(codes):
        if c.size > 3:
            c[c.size // 2], c[c.size // 3] = INF[types[i]], NAN[types[i]]
    m = Many(lengths, types, gap, codes)
    kinds = [o] * len(lengths) if o is not None else types
    out = Many(lengths, kinds, 1 - gap)
    S, coef = 16.0, 0.3
    amp.amp_grad_clip_list(m.list, out.list, state(S), torch.full((1,), coef, device="cuda"))
    for got, c, t, k in zip(out.read(), codes, types, kinds):
        assert same(got, clipped(c, t, k, S, coef), k)
    for got, c in zip(m.read(), codes):
        assert np.array_equal(got, c)


@pytest.mark.parametrize("aliased", [False, True])
def test_clip_in_place(aliased):
    lengths = [1, 5000, 17, 0, 33333]
    types, codes = mixed(lengths, 120)
    m = Many(lengths, types, 1, codes)
    amp.amp_grad_clip_list(m.list, m.list if aliased else None, state(2.0), torch.full((1,), 0.7, device="cuda"))
    first = m.read()
    for got, c, t in zip(first, codes, types):
        assert same(got, clipped(c, t, t, 2.0, 0.7), t)
    # times one, by both factors or by none given: as it is
    amp.amp_grad_clip_list(m.list, None, state(1.0), torch.ones(1, device="cuda"))
    amp.amp_grad_clip_list(m.list)
    for a, b in zip(first, m.read()):
        assert np.array_equal(a, b)


def test_clipped_gradients_give_the_step_that_the_optimizer_forms_itself():
    """Norm, coefficient, clipping into FP32 and a plain step against the step with d_grad_mult."""
    n, S = 70001, 256.0
    codes = grads(amp.F16, n, 7, 3.0 * S)
    m = Many([n], [amp.F16], 0, [codes])
    st, ns, out = state(S), empty(amp.NORM_STATE_BYTES), torch.empty(2, device="cuda")
    amp.amp_grad_norm_list(m.list, True, st, ns, 1.0, out)
    assert host(out, np.float32)[0] < 1.0
    flat = Many([n], [amp.F32])
    amp.amp_grad_clip_list(m.list, flat.list, st, out)
    hp = amp.AdamWHParams(1e-3, 0.9, 0.999, 1e-8, 0.01)
    theta = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    res = []
    for g, t, S2, mult in ((m.d, amp.F16, st, out), (flat.d, amp.F32, state(1.0), None)):
        p, mo, v = theta.clone(), torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        amp.amp_optimizer_step_ex(p, mo, v, g, t, None, amp.F16, n, hp, S2, mult)
        res.append((p, mo, v))
    for a, b in zip(*res):
        assert torch.equal(a, b)


def test_captured_norm_and_clip_replayed():
    """A graph of the norm and the clipping that follows it, replayed on new gradients with eager work between."""
    lengths = [5, 4097, 100, 70001] + [50] * 300
    types, codes = mixed(lengths, 150)
    m, out = Many(lengths, types, 0, codes), Many(lengths, [amp.F32] * len(lengths))
    st, ns, res = state(4.0), empty(amp.NORM_STATE_BYTES), torch.zeros(2, device="cuda")

    def step():
        amp.amp_grad_norm_list(m.list, True, st, ns, 1.0, res)
        amp.amp_grad_clip_list(m.list, out.list, st, res)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        _, new = mixed(lengths, 200 + 10 * k)
        m.d.copy_(Many(lengths, types, 0, new).d)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got, sq, vals = res.clone(), host(ns, np.float64)[0], out.d.clone()
        out.d.fill_(0xFF)
        step()
        torch.cuda.synchronize()
        assert torch.equal(res, got) and host(ns, np.float64)[0] == sq and torch.equal(out.d, vals)
        want, _ = sums(m, new, 4.0)
        check_coef(host(got, np.float32), want, sum(lengths))
