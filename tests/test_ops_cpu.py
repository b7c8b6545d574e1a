"""The optimiser and quantised-linear entry points without a GPU: refusals of the C ABI and of the
binding (all before anything is enqueued), sizes, and the references the GPU tests go by."""
import ctypes

import numpy as np
import pytest
import torch

from bcjr_soft_decoding_amd import bcjr
from tests import ops_reference as ref
from tests.test_binding_cpu import raises

P = ctypes.c_void_p
ARG, SHAPE, UNSUPPORTED, OK = bcjr.BCJR_E_ARG, bcjr.BCJR_E_SHAPE, bcjr.BCJR_E_UNSUPPORTED, bcjr.BCJR_OK


@pytest.fixture(scope="module")
def lib():
    return bcjr.lib()


def _int4(lib, q=0x1000, s=0x2000, z=None, rows=4, cols=100, group=32, x=0x3000, tokens=2, xs=100,
          dt=0, y=0x4000, ys=4):
    return lib.bcjr_int4_matvec(P(q), P(s), P(z), rows, cols, group, P(x), tokens, xs, dt, P(y), ys, None)


def test_int4_matvec_refusals(lib):
    for kw, want in ((dict(q=0), ARG), (dict(s=0), ARG), (dict(x=0), ARG), (dict(y=0), ARG),
                     (dict(q=0x1008), ARG), (dict(x=0x3002), ARG), (dict(dt=2, x=0x3001), ARG),
                     (dict(dt=3), ARG), (dict(dt=-1), ARG), (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE),
                     (dict(group=0), SHAPE), (dict(group=16), SHAPE), (dict(group=48), SHAPE),
                     (dict(tokens=-1), SHAPE), (dict(xs=99), SHAPE), (dict(ys=3), SHAPE),
                     (dict(rows=1 << 31, cols=1 << 31, xs=1 << 31, ys=1 << 31), SHAPE),
                     (dict(tokens=1 << 40, xs=1 << 30), SHAPE),
                     (dict(rows=0, q=0, s=0, x=0, y=0), OK), (dict(tokens=0, q=0, x=0, y=0), OK)):
        assert _int4(lib, **kw) == want, kw


def _code(lib, n=8, k=2, v=1, cb=0x1000, code=0x2000, rows=4, cols=64, L=32, scales=None, x=0x3000,
          tokens=2, xs=64, dt=0, y=0x4000, ys=4):
    tr = bcjr.Trellis(n, k, v, cb)
    return lib.bcjr_code_matvec(ctypes.byref(tr), P(code), rows, cols, L, P(scales), P(x), tokens, xs, dt,
                                P(y), ys, None)


def test_code_matvec_refusals(lib):
    assert lib.bcjr_code_matvec(None, None, 0, 1, 1, None, None, 0, 1, 0, None, 1, None) == ARG
    for kw, want in ((dict(n=0), SHAPE), (dict(n=17), SHAPE), (dict(k=0), SHAPE), (dict(k=9), SHAPE),
                     (dict(v=2), UNSUPPORTED), (dict(cb=0), ARG), (dict(code=0), ARG), (dict(x=0), ARG),
                     (dict(y=0), ARG), (dict(dt=7), ARG), (dict(L=0), SHAPE), (dict(L=48), SHAPE),
                     (dict(L=128), SHAPE), (dict(xs=63), SHAPE), (dict(ys=1), SHAPE), (dict(rows=-2), SHAPE),
                     (dict(y=0x4002), ARG), (dict(rows=0, code=0, x=0, y=0, cb=0), OK),
                     (dict(tokens=0, x=0, y=0), OK)):
        assert _code(lib, **kw) == want, kw


def test_int4_quantize_refusals(lib):
    def call(w=0x1000, dt=0, rows=2, cols=40, group=32, q=0x2000, s=0x3000):
        return lib.bcjr_int4_quantize(P(w), dt, rows, cols, group, P(q), P(s), None, None)

    for kw, want in ((dict(w=0), ARG), (dict(q=0), ARG), (dict(s=0), ARG), (dict(q=0x2004), ARG), (dict(dt=4), ARG),
                     (dict(w=0x1002), ARG), (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(group=31), SHAPE),
                     (dict(rows=0, w=0, q=0, s=0), OK)):
        assert call(**kw) == want, kw
    assert lib.bcjr_int4_dequantize(P(0x1000), P(0), None, 1, 1, 32, P(0x2000), None) == ARG
    assert lib.bcjr_int4_dequantize(P(0x1000), P(0x2000), None, 1, 0, 32, P(0x2000), None) == SHAPE
    assert [lib.bcjr_int4_words(c) for c in (-1, 0, 1, 128, 129, 1 << 24, (1 << 24) + 1)] == [0, 0, 16, 16, 32, 1 << 21, 0]
    assert call(cols=(1 << 24) + 1) == SHAPE and _int4(lib, cols=(1 << 24) + 1, xs=1 << 25) == SHAPE


class Tensor(ctypes.Structure):
    _fields_ = [("param", P), ("grad", P), ("numel", ctypes.c_int64)]


def _adamw(lib, entries=((0x10000, 0x20000, 10),), pt=0, gt=0, bits=32, m=0x100000, v=0x200000, ms=None, vs=None,
           lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, step=1, count=None):
    t = (Tensor * max(1, len(entries)))(*[Tensor(*e) for e in entries])
    h = bcjr.Adamw(lr, b1, b2, eps, wd, step, 0)
    return lib.bcjr_adamw_step(t, len(entries) if count is None else count, pt, gt, bits, ctypes.byref(h), P(m), P(v),
                               P(ms), P(vs), None)


def test_adamw_refusals(lib):
    nan, inf = float("nan"), float("inf")
    for kw in (dict(lr=-1.0), dict(lr=nan), dict(lr=inf), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=nan),
               dict(eps=-1e-9), dict(eps=inf), dict(wd=-1.0), dict(wd=nan), dict(step=0), dict(step=-3), dict(pt=3),
               dict(gt=-1), dict(m=0), dict(v=0), dict(m=0x100008), dict(bits=8), dict(bits=8, ms=0x1000),
               dict(entries=((0, 0x20000, 10),)), dict(entries=((0x10000, 0, 10),)), dict(entries=((0x10002, 0x20000, 10),)),
               dict(entries=((0x10000, 0x20000, 10), (0x10000, 0x30000, 10))),    # the same tensor twice
               dict(entries=((0x10000, 0x20000, 10), (0x10024, 0x30000, 10))),    # an overlap by one element
               dict(entries=((0x10024, 0x20000, 10), (0x10000, 0x30000, 10)))):   # the other way round
        assert _adamw(lib, **kw) == ARG, kw
    assert _adamw(lib, bits=16) == UNSUPPORTED
    assert _adamw(lib, entries=((0x10000, 0x20000, -1),)) == SHAPE
    assert _adamw(lib, entries=((0x10000, 0x20000, (1 << 40) + 1),)) == SHAPE
    assert _adamw(lib, entries=((0x10000, 0x20000, 1 << 40), (0x10000, 0x20000, 1 << 40))) == SHAPE
    assert _adamw(lib, count=-1) == SHAPE
    assert _adamw(lib, entries=(), m=0, v=0) == OK
    assert _adamw(lib, entries=((0, 0, 0),), m=0, v=0) == OK
    assert lib.bcjr_adamw_step(None, 1, 0, 0, 32, None, None, None, None, None, None) == ARG


def test_adamw_state_numel(lib):
    t = (Tensor * 3)(Tensor(None, None, 1), Tensor(None, None, 0), Tensor(None, None, 33))
    assert lib.bcjr_adamw_state_numel(t, 3) == 96 == bcjr.bcjr_adamw_state_numel([1, 0, 33])
    assert lib.bcjr_adamw_state_numel(t, 0) == 0 and lib.bcjr_adamw_state_numel(None, 2) == 0
    t[0].numel = -1
    assert lib.bcjr_adamw_state_numel(t, 3) == 0


def test_binding_refusals_int4():
    x, q = torch.zeros(2, 100), torch.zeros(4, 16, dtype=torch.uint32)
    s, z = torch.zeros(4, 4), torch.zeros(4, 4, dtype=torch.uint8)
    f = lambda **kw: bcjr.bcjr_int4_matvec(**{**dict(x=x, q=q, scales=s, zeros=z, group=32), **kw})  # noqa: E731
    raises(lambda: f(x=x.double()), "x", "float32")
    raises(lambda: f(x=torch.zeros(100)), "x", "shape")
    raises(lambda: f(x=torch.zeros(100, 2).t()), "x", "contiguous rows")
    raises(lambda: f(x=torch.zeros(1, 100).expand(2, 100)), "x", "overlapping")
    raises(lambda: f(x=torch.zeros(2, 129)), "q", "words")
    raises(lambda: f(q=q.to(torch.int64)), "q", "uint32")
    raises(lambda: f(scales=torch.zeros(4, 3)), "scales", "shape")
    raises(lambda: f(scales=None), "scales")
    raises(lambda: f(scales=s.half()), "scales", "float32")
    raises(lambda: f(q=None), "q")
    raises(lambda: f(x=[1.0]), "x")
    raises(lambda: f(zeros=torch.zeros(4, 4)), "zeros", "uint8")
    raises(lambda: f(group=40), "group")
    raises(lambda: f(y=torch.zeros(2, 5)), "y", "shape")
    raises(lambda: f(y=torch.zeros(2, 4).half()), "y", "float32")
    raises(lambda: f(x=x.clone().requires_grad_()), "gradient")
    raises(lambda: f(), "CUDA")
    raises(lambda: bcjr.bcjr_int4_quantize(torch.zeros(4, 64).t(), 32), "contiguous")
    raises(lambda: bcjr.bcjr_int4_quantize(torch.zeros(4, 0), 32), "columns")
    raises(lambda: bcjr.bcjr_int4_quantize(torch.zeros(4, 8, dtype=torch.int32), 32), "float32")
    raises(lambda: bcjr.bcjr_int4_quantize(torch.zeros(4, 8), 20), "group")
    raises(lambda: bcjr.bcjr_int4_dequantize(q, s, z, 129, 32), "words")


def test_binding_refusals_code():
    x, code, c = torch.zeros(2, 64), torch.zeros(8, 3, dtype=torch.uint32), torch.zeros(256)
    f = lambda **kw: bcjr.bcjr_code_matvec(**{**dict(x=x, code=code, codebook=c, n=8, k=2, L=32), **kw})  # noqa: E731
    raises(lambda: f(code=torch.zeros(8, 2, dtype=torch.uint32)), "words")
    raises(lambda: f(code=torch.zeros(7, 3, dtype=torch.uint32)), "rows")
    raises(lambda: f(x=torch.zeros(2, 60)), "rows")
    raises(lambda: f(codebook=torch.zeros(255)), "codebook")
    raises(lambda: f(scales=torch.zeros(7)), "scales")
    raises(lambda: f(y=torch.zeros(4, 2).t()), "y", "contiguous")
    raises(lambda: f(y=torch.zeros(3, 4)), "y", "shape")
    raises(lambda: f(L=0), "words")
    raises(lambda: f(codebook=None), "codebook")
    raises(lambda: f(code=None), "code")
    raises(lambda: f(x=None), "x")
    raises(lambda: f(), "CUDA")


def test_binding_refusals_adamw():
    p, g, m, v = torch.zeros(40), torch.zeros(40), torch.zeros(64), torch.zeros(64)
    f = lambda ps=(p,), gs=(g,), **kw: bcjr.bcjr_adamw_step(  # noqa: E731
        ps, gs, **{**dict(exp_avg=m, exp_avg_sq=v, step=1, lr=1e-3), **kw})
    raises(lambda: f(gs=()), "1 params and 0 grads")
    raises(lambda: f(gs=(None,)), "grads")
    raises(lambda: f(gs=(torch.zeros(41),)), "shape")
    raises(lambda: f(ps=(p, p.half()), gs=(g, g)), "float16")
    raises(lambda: f(ps=(p, p), gs=(g, g.half())), "float16")
    raises(lambda: f(ps=(torch.zeros(8, 5).t(),), gs=(torch.zeros(5, 8),)), "contiguous")
    raises(lambda: f(ps=(p.double(),)), "float32")
    raises(lambda: f(exp_avg=torch.zeros(40)), "exp_avg", "shape")
    raises(lambda: f(exp_avg_sq=None), "exp_avg_sq")
    raises(lambda: f(avg_scale=torch.zeros(2, dtype=torch.uint8)), "avg_scale")
    m8 = torch.zeros(64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    raises(lambda: f(exp_avg=m8), "exp_avg_sq", "float8")
    raises(lambda: f(exp_avg=m8, exp_avg_sq=m8), "avg_scale")
    sc = torch.zeros(2, dtype=torch.uint8)
    raises(lambda: f(exp_avg=m8, exp_avg_sq=m8, avg_scale=sc, avg_sq_scale=sc[:1]), "avg_sq_scale")
    raises(lambda: f(), "CUDA")
    assert bcjr.bcjr_adamw_step([], [], m, v, step=1, lr=1e-3) is None


# ---- the references ------------------------------------------------------------------------------

def test_int4_layout_is_a_bijection():
    word, shift = ref.int4_place(256)
    assert sorted(zip(word, shift)) == [(w, 4 * i) for w in range(32) for i in range(8)]
    codes = np.random.default_rng(0).integers(0, 16, (3, 131))
    np.testing.assert_array_equal(ref.int4_unpack(ref.int4_pack(codes), 131), codes)


def test_dithered_rounding_is_unbiased():
    """The mean of many roundings of one value is that value: the dithers of different places and steps
    are spread evenly. 2^16 draws of a uniform dither have a mean off by at most 5 sigma
    = 5 u / sqrt(12 * 2^16), u the spacing."""
    for x, top in ((0.3, 1.0), (0.9999, 1.0), (0.0021, 1.0)):
        d = np.concatenate([ref.dithers(0, 1 << 15, t, 7)[i] for t, i in ((1, 0), (2, 1))])
        blocks = np.full((d.size // 31 + 1, 32), x)
        blocks[:, 0] = top
        dd = np.resize(d, blocks.shape)
        v, b = ref.encode(blocks, dd, 0)
        v = np.ldexp(v, b[:, None].astype(int) - 127)[:, 1:].reshape(-1)
        u = 2.0 ** (np.floor(np.log2(x)) - 3)
        assert np.abs(v - x).max() < u
        assert abs(v.mean() - x) < 5 * u / np.sqrt(12 * (1 << 15)) * 2


def test_dithers_of_steps_and_moments_are_unrelated():
    a, b = ref.dithers(0, 1 << 16, 1, 0)
    c, _ = ref.dithers(0, 1 << 16, 2, 0)
    for x, y in ((a, b), (a, c), (a[1:], a[:-1])):
        # the correlation of 2^16 independent pairs is off zero by less than 5 / sqrt(2^16)
        assert abs(np.corrcoef(x, y)[0, 1]) < 5 / 256
    for x in (a, b, c):
        assert abs(x.mean() - 0.5) < 5 / np.sqrt(12 * 65536)


def test_qat_options_are_checked_first():
    from bcjr_soft_decoding_amd import qat

    with pytest.raises(ValueError, match="optimizer"):
        qat.QATConfig(optimizer="adam").check()
    for kw in (dict(group=48), dict(group=0)):
        with pytest.raises(ValueError, match="serving"):
            qat.run(8, 512, 8, qat.QATConfig(), serve=True, **kw)
    with pytest.raises(ValueError, match="serving"):
        qat.run(8, 384, 8, qat.QATConfig(), serve=True)
    res = qat.QATResult(w=None, g_max=2.0)
    assert res.budget(qat.QATConfig(lr=0.5, steps=3)) == 3.0
    assert res.budget(qat.QATConfig(lr=1.0, steps=2, optimizer="adamw")) == pytest.approx(2 * 0.1 / (0.001 * (1 - 0.81 / 0.999)) ** 0.5)
    assert res.budget(qat.QATConfig(optimizer="adamw8", betas=(0.99, 0.9))) == float("inf")
