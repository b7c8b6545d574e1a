"""AdamW over many tensors on the GPU against a 64-bit reference.

Tolerances. fp32 moments: each is a fused multiply-add of an exact old value and a product rounded once
(m) or twice (v), so it is within 2^-24 (|m'| + |(1 - beta1) g|) (m) and 3 * 2^-24 v' (v, all terms
positive; its factors in fp32 add 2 * 2^-24), and the fp32 betas add 2^-24 of either term: 4 * 2^-24
of |beta1 m| + |(1 - beta1) g| and 6 * 2^-24 of v' cover both. The step lr m / (sqrt(v) / root + eps)
is a short chain of at most 10 such roundings on top of the moments' own (m's of its terms, half of
v's): 20 * 2^-24 of lr (|beta1 m| + |(1 - beta1) g|) / (1 - beta1^t) / denominator; decay and
subtraction add 3 * 2^-24 (|p| + |step|), and the rounding to the param's type half an eps of the value.
8-bit moments are computed in fp64: codes and exponents have to be equal.
"""
import numpy as np
import pytest
import torch

from bcjr_soft_decoding_amd import bcjr
from tests import ops_reference as ref
from tests.gpu_helpers import log_case
from tests.test_gpu_ops import TYPES, exact64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
VALUES = ref.e4m3_values()


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bcjr.lib()


def hyper(**kw):
    return {**dict(step=3, lr=2e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.05, seed=11), **kw}


class Case:
    """Tensors, gradients and moments; check() runs a step and compares everything."""

    def __init__(self, sizes, pt, gt, bits, seed, offset=0):
        rng = np.random.default_rng(seed)
        self.sizes, self.bits = sizes, bits

        def tensor(n, t, scale):
            a = torch.from_numpy(scale * rng.standard_normal(n + offset)).to(TYPES[t]).cuda()
            return a[offset:]

        self.p = [tensor(n, pt, 1.0) for n in sizes]
        self.g = [tensor(n, gt, 0.01) for n in sizes]
        self.first = np.cumsum([0] + [-(-n // 32) * 32 for n in sizes])
        total = int(self.first[-1])
        if bits == 32:
            self.m = torch.from_numpy(0.01 * rng.standard_normal(total)).float().cuda()
            self.v = torch.from_numpy((0.01 * rng.standard_normal(total)) ** 2).float().cuda()
            self.ms = self.vs = None
        else:
            code = rng.integers(0, 127, total) | (rng.integers(0, 2, total) << 7)
            self.m = torch.from_numpy(code.astype(np.uint8)).cuda().view(torch.float8_e4m3fn)
            self.v = torch.from_numpy(rng.integers(0, 127, total).astype(np.uint8)).cuda().view(torch.float8_e4m3fn)
            self.ms = torch.from_numpy(rng.integers(105, 118, total // 32).astype(np.uint8)).cuda()
            self.vs = torch.from_numpy(rng.integers(105, 118, total // 32).astype(np.uint8)).cuda()

    def held(self):
        if self.bits == 32:
            return exact64(self.m), exact64(self.v)
        return VALUES[self.m.view(torch.uint8).cpu().numpy()], VALUES[self.v.view(torch.uint8).cpu().numpy()]

    def step(self, h):
        if self.bits == 32:
            h = {k: v for k, v in h.items() if k != "seed"}
        bcjr.bcjr_adamw_step(self.p, self.g, self.m, self.v, self.ms, self.vs, **h)

    @np.errstate(invalid="ignore")
    def check(self, h):
        before = [exact64(p) for p in self.p]
        m0, v0 = self.held()
        raw0 = [t.view(torch.uint8).cpu().numpy().copy() for t in (self.m, self.v)]
        sc0 = None if self.bits == 32 else [t.cpu().numpy().copy() for t in (self.ms, self.vs)]
        self.step(h)
        m1, v1 = self.held()
        raw1 = [t.view(torch.uint8).cpu().numpy() for t in (self.m, self.v)]
        b1, b2, t = h["beta1"], h["beta2"], h["step"]
        for i, n in enumerate(self.sizes):
            o = int(self.first[i])
            here = slice(o, o + n)
            g = exact64(self.g[i])
            size = 4 if self.bits == 32 else 1
            for a, b in zip(raw0, raw1):  # what lies behind the last element
                np.testing.assert_array_equal(a[size * (o + n):size * int(self.first[i + 1])],
                                              b[size * (o + n):size * int(self.first[i + 1])])
            if self.bits == 32:
                want, m, v = ref.adamw(before[i], g, m0[here], v0[here], h, 32)
                terms = np.abs(b1 * m0[here]) + np.abs((1 - b1) * g)
                for got, w, tol in ((m1[here], m, 4 * U * terms), (v1[here], v, 6 * U * v)):
                    fine = np.isfinite(w)
                    np.testing.assert_array_equal(got[~fine], w[~fine])
                    assert np.all(np.abs(got - w)[fine] <= (tol + 1e-44)[fine])
            else:
                sb = slice(o // 32, (o + n + 31) // 32)
                want, mv, rv, mb, rb = ref.adamw(before[i], g, m0[here], v0[here], h, 8, o, [s[sb] for s in sc0])
                np.testing.assert_array_equal(self.ms.cpu().numpy()[sb], mb)
                np.testing.assert_array_equal(self.vs.cpu().numpy()[sb], rb)
                np.testing.assert_array_equal(m1[here], mv)
                np.testing.assert_array_equal(v1[here], rv)
                blk = np.arange(n) // 32
                m = np.ldexp(m0[here], sc0[0][sb].astype(int)[blk] - 127)
                terms = np.abs(b1 * m) + np.abs((1 - b1) * g)
                v = b2 * np.ldexp(v0[here], sc0[1][sb].astype(int)[blk] - 127) ** 2 + (1 - b2) * g * g
            with np.errstate(all="ignore"):
                denom = np.sqrt(v / (1 - b2 ** t)) + h["eps"]
                move = h["lr"] * terms / (1 - b1 ** t) / denom
            tol = 20 * U * move + 3 * U * (np.abs(before[i]) + move) + np.abs(want) * torch.finfo(self.p[i].dtype).eps / 2
            if self.p[i].dtype == torch.float16:
                tol = tol + 2.0 ** -25  # its spacing is never below 2^-24
            got = exact64(self.p[i])
            bad = ~np.isfinite(want)
            assert np.array_equal(bad, ~np.isfinite(got))
            assert np.all(np.abs(got - want)[~bad] <= (tol + 1e-37)[~bad]), np.nanmax(np.abs(got - want) / tol)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pt,gt", [("fp32", "fp32"), ("fp32", "bf16"), ("fp32", "fp16"), ("bf16", "bf16"), ("fp16", "fp16"),
                                   ("bf16", "fp32"), ("fp16", "bf16")])
def test_steps(pt, gt, bits):
    sizes = [1, 31, 32, 33, 2047, 2048, 2049, 7, 0, 70001, 255, 4096]
    for offset in (0, 1):  # the second: params and grads that are not aligned to 16 bytes
        log_case(f"adamw {pt} {gt} bits={bits} offset={offset}")
        c = Case(sizes, pt, gt, bits, 1, offset)
        for step in (1, 2, 1000):
            c.check(hyper(step=step, seed=step * 77))


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_state_first_step_and_settings(bits):
    log_case(f"adamw zero state bits={bits}")
    for kw in (dict(), dict(beta1=0.0), dict(beta2=0.0), dict(weight_decay=0.0), dict(lr=0.0), dict(eps=1.0)):
        c = Case([100, 3], "fp32", "fp32", bits, 2)
        for t in (c.m, c.v, c.ms, c.vs):
            if t is not None:
                t.view(torch.uint8).zero_()
        for step in (1, 2, 3):
            c.check(hyper(step=step, **kw))


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(bits):
    """More tensors than one launch's table holds, empty ones among them."""
    log_case(f"adamw many bits={bits}")
    rng = np.random.default_rng(0)
    c = Case([int(n) for n in rng.integers(0, 90, 230)] + [5000], "fp32", "fp32", bits, 3)
    c.check(hyper())


@pytest.mark.parametrize("bits", [32, 8])
def test_extreme_gradients(bits):
    """Zeros, the smallest and largest numbers; 8-bit moments keep blocks of very different sizes."""
    log_case(f"adamw extremes bits={bits}")
    c = Case([32 * 40], "fp32", "fp32", bits, 4)
    g = c.g[0].view(40, 32)
    g[0] = 0.0
    g[1] = 1e-30
    g[2, ::2] = 1e-12
    g[3] *= 1e6
    g[4, 5] = 1e15
    g[5] *= 1e-9
    if bits == 8:  # the second moment's root is computed from fp64: no overflow at the ends
        g[6, 3], g[7, 4], g[8] = 3e38, 1e-45, 1e-45
        for s in (c.ms, c.vs):
            s[8:10] = 0
        c.m.view(torch.uint8)[8 * 32:10 * 32] = 0
        c.v.view(torch.uint8)[8 * 32:10 * 32] = 0
    for step in (1, 2):
        c.check(hyper(step=step, eps=1e-8))


@pytest.mark.parametrize("bits", [32, 8])
def test_non_finite_gradients_stay_in_their_element(bits):
    log_case(f"adamw non-finite bits={bits}")
    c = Case([96], "fp32", "fp32", bits, 5)
    bad = {3: float("nan"), 40: float("inf"), 77: float("-inf")}
    for i, b in bad.items():
        c.g[0][i] = b
    c.check(hyper())
    c.check(hyper(step=4))
    rest = [i for i in range(96) if i not in bad]
    assert bool(torch.isfinite(c.p[0][rest]).all())
    assert not bool(torch.isfinite(c.p[0][list(bad)]).any())


def test_eight_bits_follow_thirty_two():
    """Over 400 steps of noisy gradients the dithered moments estimate what fp32 ones hold, also where v
    has to fall to a sixteenth: a nearest rounding would leave it where it began. What the dither adds
    to v: a step moves r from its code by D = (1 - beta2) / 2 r (g^2 / v - 1), so the rounding's
    variance is at most |D| u with u <= r / 8, and v = r^2 is that much too large on average. Over the
    1 / (1 - beta2) steps that v remembers, relative to v: E|g^2 / v - 1| / 16 <= (E[g^2] / v + 1) / 16
    = 1 / 8. m's rounding is unbiased; its mean over 2^15 elements is held to 5 %."""
    log_case("adamw 400 steps")
    n = 1 << 15
    gen = torch.Generator(device="cuda").manual_seed(1)
    sig = torch.exp(torch.randn(n, generator=gen, device="cuda") * 0.3)
    p8, p32 = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    m8, v8 = (torch.zeros(n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ms, vs = (torch.zeros(n // 32, dtype=torch.uint8, device="cuda") for _ in range(2))
    m32, v32 = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    for step in range(1, 401):
        size = 1.0 if step <= 200 else 0.25  # the second half needs v to fall
        g = size * sig * (torch.randn(n, generator=gen, device="cuda") + 0.5)
        h = dict(step=step, lr=1e-3, beta1=0.9, beta2=0.98, eps=1e-8, weight_decay=0.0)
        bcjr.bcjr_adamw_step([p8], [g], m8, v8, ms, vs, seed=5, **h)
        bcjr.bcjr_adamw_step([p32], [g], m32, v32, **h)
        if step in (200, 400):
            r = torch.ldexp(v8.float().view(-1, 32), vs.int()[:, None] - 127).view(-1)
            ratio = (r.square() / v32)
            assert abs(float(ratio.mean()) - 1) < 0.125, step
            m = torch.ldexp(m8.float().view(-1, 32), ms.int()[:, None] - 127).view(-1)
            assert abs(float((m / sig).mean() / (m32 / sig).mean()) - 1) < 0.05
    assert float((p8 - p32).abs().mean()) < 0.1 * float(p32.abs().mean())


def test_agrees_with_the_formula_over_steps():
    """20 steps in fp32 against the definition in 64 bits carried along by itself."""
    log_case("adamw 20 steps fp32")
    c = Case([1000, 33], "fp32", "fp32", 32, 6)
    c.m.zero_(), c.v.zero_()
    p, m, v = [exact64(t) for t in c.p], [np.zeros(n) for n in c.sizes], [np.zeros(n) for n in c.sizes]
    gen = torch.Generator(device="cuda").manual_seed(3)
    for step in range(1, 21):
        c.g = [torch.randn(n, generator=gen, device="cuda") for n in c.sizes]
        h = hyper(step=step)
        c.step(h)
        for i in range(2):
            p[i], m[i], v[i] = ref.adamw(p[i], exact64(c.g[i]), m[i], v[i], h, 32)
    for i in range(2):
        # each step adds at most 3 * 2^-24 (|p| + move) + 20 * 2^-24 move, moves are at most about
        # lr (1 - beta1) / sqrt(1 - beta2) = 2 lr here; 20 steps of them with |p| < 6
        assert np.all(np.abs(exact64(c.p[i]) - p[i]) <= 20 * (3 * U * 6 + 23 * U * 4e-3))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_and_on_streams(bits):
    """Replays of a captured step with eager work between them, and steps on another stream, give
    bitwise what eager steps do."""
    log_case(f"adamw graph bits={bits}")
    sizes = [5000, 33, 1]
    a, b, d = (Case(sizes, "fp32", "fp32", bits, 7) for _ in range(3))
    h = hyper()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(h)
    for i in range(4):
        g = [torch.randn(n, device="cuda") for n in sizes]
        for c in (a, b, d):
            for t, src in zip(c.g, g):
                t.copy_(src)
        torch.cuda.synchronize()
        graph.replay()
        b.step(h)
        with torch.cuda.stream(side):
            d.step(h)
        torch.cuda.synchronize()
        for c in (b, d):
            for t, u in zip(a.p + [a.m.view(torch.uint8), a.v.view(torch.uint8)], c.p + [c.m.view(torch.uint8), c.v.view(torch.uint8)]):
                assert torch.equal(t, u)


def test_refused_calls_write_nothing():
    c = Case([100, 50], "fp32", "fp32", 32, 8)
    keep = [t.clone() for t in c.p + [c.m, c.v]]
    with pytest.raises(bcjr.BcjrError) as e:
        bcjr.bcjr_adamw_step([c.p[0], c.p[0]], [c.g[0], c.g[0]], torch.zeros(256, device="cuda"), torch.zeros(256, device="cuda"),
                             step=1, lr=1e-3)
    assert e.value.status == bcjr.BCJR_E_ARG
    for kw in (dict(step=0), dict(lr=-1.0), dict(beta1=1.0)):
        with pytest.raises(bcjr.BcjrError):
            c.step(hyper(**kw))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(keep, c.p + [c.m, c.v]))


def test_autograd_sees_the_update():
    p = torch.ones(8, device="cuda", requires_grad=True)
    y = (p * p).sum()
    bcjr.bcjr_adamw_step([p], [torch.ones(8, device="cuda")], torch.zeros(32, device="cuda"), torch.zeros(32, device="cuda"),
                         step=1, lr=1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@pytest.mark.parametrize("gt", ["bf16", "fp32"])
def test_moments_right_at_borders(gt):
    """Gradients that are small whole multiples of the block's unit: a moment is then often a power of two,
    or on a code's border, up to its last bit, and codes and exponents are the formula's all the same."""
    log_case(f"adamw borders {gt}")
    n = 1 << 18
    c = Case([n], "fp32", gt, 8, 9)
    rng = np.random.default_rng(10)
    unit = np.ldexp(1.0, c.ms.cpu().numpy().astype(int).repeat(32) - 127)
    g = torch.from_numpy(unit * rng.integers(-128, 129, n)).cuda()
    c.g[0].copy_(g)
    assert torch.equal(c.g[0].double(), g)
    c.vs.copy_(c.ms)
    for step in (3, 4):
        c.check(hyper(step=step, seed=step))
