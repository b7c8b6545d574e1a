"""Products with quantised weights and rounding to 4 bits on the GPU against 64-bit references.

Tolerance of a product y = sum of n terms w x. The result is rounded once to its type: eps / 2 of
the value. The sum is fp32; each of its at most n + 8 roundings is at most 2^-24 of a partial sum,
which is at most A, the sum of the terms' magnitudes. Taken as independent with mean zero, they
together stay below lambda sqrt(n + 8) 2^-24 A but with a probability of 2 exp(-lambda^2 / 2); lambda
= 8 makes that 3e-14. A for 4-bit weights counts a term as 32 |scale x|, the most that a code and its
zero point may be summed as before they are subtracted (each at most 16 units). A codeword may be held
as two 16-bit parts for 16-bit x: 2^-16 of each term on top, worst case.
"""
import threading

import numpy as np
import pytest
import torch

from bcjr_soft_decoding_amd import bcjr
from tests import ops_reference as ref
from tests.gpu_helpers import dev, log_case

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bcjr.lib()


def exact64(t):
    return t.detach().double().cpu().numpy()


def assert_product(y, x, w, mags, what, parts=0.0):
    """y [tokens, rows] against x w^T; mags bounds the magnitude a weight is summed with."""
    x64 = exact64(x)
    want, got = x64 @ w.T, exact64(y)
    a = np.abs(x64) @ mags.T
    n = w.shape[1] + 8
    tol = np.abs(want) * torch.finfo(y.dtype).eps / 2 + a * (8 * np.sqrt(n) * 2.0 ** -24 + parts) + 1e-30
    if y.dtype == torch.float16:
        tol = tol + 2.0 ** -25  # half a spacing of its subnormals
    assert np.all(np.isfinite(got)), what
    worst = np.max(np.abs(got - want) / tol) if got.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} of the tolerance"


def make_x(tokens, cols, t, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((tokens, cols)) * np.exp(0.75 * rng.standard_normal(cols))
    return torch.from_numpy(x).to(TYPES[t]).cuda()


def make_int4(rows, cols, group, zeros, seed):
    rng = np.random.default_rng(seed)
    groups = -(-cols // group)
    codes = rng.integers(0, 16, (rows, cols))
    s = (0.005 * (0.5 + rng.random((rows, groups)))).astype(np.float32)
    s[rng.random(s.shape) < 0.2] *= -1  # any finite scale is allowed
    z = rng.integers(0, 16, (rows, groups)).astype(np.uint8) if zeros else None
    return codes, s, z


def int4_case(rows, cols, group, zeros, tokens, t, seed=0):
    codes, s, z = make_int4(rows, cols, group, zeros, seed)
    g = np.arange(cols) // group
    return (make_x(tokens, cols, t, seed + 1), dev(ref.int4_pack(codes)), dev(s), None if z is None else dev(z),
            ref.int4_weights(codes, s, z, group), 32 * np.abs(s.astype(np.float64))[:, g])


# ---- 4-bit weights -------------------------------------------------------------------------------

SHAPES = [(1, 1), (3, 7), (16, 32), (17, 33), (5, 127), (33, 128), (2, 129), (64, 500), (130, 1031), (47, 4099)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("group,zeros", [(32, False), (64, True), (96, False), (128, True), (512, False), (8192, True)])
def test_int4_matvec(rows, cols, group, zeros, t):
    for tokens in (1, 2, 3, 5, 8, 16, 17, 40):
        log_case(f"int4 {rows}x{cols} g{group} zeros={zeros} tokens={tokens} {t}")
        x, q, s, z, w, mags = int4_case(rows, cols, group, zeros, tokens, t, seed=rows + cols)
        assert_product(bcjr.bcjr_int4_matvec(x, q, s, z, group), x, w, mags, "int4")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows,cols,group,tokens", [(2048, 8192, 128, 1), (512, 16384, 64, 4), (1000, 5000, 32, 33),
                                                    (4, 70000, 256, 1), (20000, 64, 32, 2), (300, 2048, 128, 130)])
def test_int4_matvec_larger(rows, cols, group, tokens, t):
    log_case(f"int4 {rows}x{cols} g{group} tokens={tokens} {t}")
    rng = np.random.default_rng(3)
    q = torch.from_numpy(rng.integers(0, 1 << 32, (rows, bcjr.bcjr_int4_words(cols)), dtype=np.uint32)).cuda()
    s = torch.from_numpy((0.01 * rng.random((rows, -(-cols // group)))).astype(np.float32)).cuda()
    x = make_x(tokens, cols, t, 4)
    y = bcjr.bcjr_int4_matvec(x, q, s, None, group)
    # the nibbles behind the last column are not zero here: nothing may read a weight from them
    w = ref.int4_weights(ref.int4_unpack(q.cpu().numpy(), cols), s.cpu().numpy(), None, group)
    mags = 32 * np.abs(s.cpu().numpy().astype(np.float64))[:, np.arange(cols) // group]
    assert_product(y, x, w, mags, "int4")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("which", ["int4", "code"])
@pytest.mark.parametrize("tokens", [1, 3, 20])
def test_strided_and_unaligned(which, t, tokens):
    """x and y as slices of wider matrices at odd offsets; what lies between y's rows stays."""
    rows, cols, group = 37, 224, 32
    log_case(f"strided {which} tokens={tokens} {t}")
    call, w, mags, parts = product(which, rows, cols)
    for pad, off in ((0, 0), (3, 1), (8, 8), (16, 4)):
        wide = make_x(tokens, cols + pad + off, t, 9)
        x = wide[:, off:off + cols]
        out = torch.full((tokens, rows + 11), 7.0, dtype=TYPES[t], device="cuda")
        y = out[:, 5:5 + rows]
        assert call(x, y=y) is y
        assert_product(y, x, w, mags, which, parts)
        assert bool((out[:, :5] == 7).all()) and bool((out[:, 5 + rows:] == 7).all())


def product(which, rows, cols, seed=5):
    """(call(x, y=None), weights, magnitudes, parts) of either operator on fixed weights."""
    if which == "int4":
        codes, s, z = make_int4(rows, cols, 32, True, seed)
        q, sd, zd = dev(ref.int4_pack(codes)), dev(s), dev(z)
        mags = 32 * np.abs(s.astype(np.float64))[:, np.arange(cols) // 32]
        return (lambda x, y=None: bcjr.bcjr_int4_matvec(x, q, sd, zd, 32, y=y)), ref.int4_weights(codes, s, z, 32), mags, 0.0
    n, k, L = 8, 2, 32
    code, cb, s, w = make_code(rows, cols, n, k, L, True, seed)
    cd, cbd, sd = dev(code), dev(cb), dev(s)
    return (lambda x, y=None: bcjr.bcjr_code_matvec(x, cd, cbd, n, k, L, sd, y=y)), w, np.abs(w), 2.0 ** -16


@pytest.mark.parametrize("which", ["int4", "code"])
@pytest.mark.parametrize("t", TYPES)
def test_non_finite_x_stays_in_its_token(which, t):
    log_case(f"non-finite {which} {t}")
    call, w, mags, parts = product(which, 40, 192)
    for tokens in (1, 4, 18):
        for bad in (float("nan"), float("inf"), float("-inf")):
            x = make_x(tokens, 192, t, 3)
            x[tokens // 2, 77] = bad
            y = call(x)
            assert not bool(torch.isfinite(y[tokens // 2]).any()), bad
            others = [i for i in range(tokens) if i != tokens // 2]
            assert_product(y[others], x[others], w, mags, which, parts)


def test_non_finite_scales_stay_in_their_rows():
    log_case("non-finite scales")
    for t in TYPES:
        x, q, s, z, w, mags = int4_case(40, 192, 32, True, 5, t)
        s[7, 2] = float("nan")
        s[21, 5] = float("inf")
        y = bcjr.bcjr_int4_matvec(x, q, s, z, 32)
        rest = [r for r in range(40) if r not in (7, 21)]
        assert not bool(torch.isfinite(y[:, [7, 21]]).any())
        assert_product(y[:, rest], x, w[rest], mags[rest], "int4")
        code, cb, cs, w = make_code(40, 192, 8, 2, 32, True, 1)
        cs[6 * 9 + 1] = np.nan
        y = bcjr.bcjr_code_matvec(x, dev(code), dev(cb), 8, 2, 32, dev(cs))
        rest = [r for r in range(40) if r != 9]
        assert not bool(torch.isfinite(y[:, 9]).any())
        assert_product(y[:, rest], x, w[rest], np.abs(w[rest]), "code", 2.0 ** -16)


@pytest.mark.parametrize("which", ["int4", "code"])
def test_no_tokens_no_rows(which):
    call, _, _, _ = product(which, 4, 64)
    assert tuple(call(torch.zeros(0, 64, device="cuda")).shape) == (0, 4)
    if which == "int4":
        y = bcjr.bcjr_int4_matvec(torch.ones(2, 64, device="cuda"), torch.zeros(0, 16, dtype=torch.int32, device="cuda").view(torch.uint32),
                                  torch.zeros(0, 2, device="cuda"), None, 32)
    else:
        y = bcjr.bcjr_code_matvec(torch.ones(2, 64, device="cuda"), torch.zeros(0, 3, dtype=torch.int32, device="cuda").view(torch.uint32),
                                  torch.zeros(256, device="cuda"), 8, 2, 32)
    assert tuple(y.shape) == (2, 0)


@pytest.mark.parametrize("which", ["int4", "code"])
def test_captured_streams_and_repeats(which):
    """Bitwise the same: eager, on another stream, two streams at once, and replays of a graph with
    new inputs and eager work between them."""
    log_case(f"graph {which}")
    call, w, mags, parts = product(which, 260, 1056)
    for t in TYPES:
        xs = [make_x(3, 1056, t, 20 + i) for i in range(4)]
        eager = [call(x) for x in xs]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        other = []
        for i, x in enumerate(xs):
            with torch.cuda.stream(streams[i % 2]):
                other.append(call(x))
        torch.cuda.synchronize()
        xin, yout = xs[0].clone(), torch.empty_like(eager[0])
        call(xin, y=yout)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(xin, y=yout)
        for i, x in enumerate(xs):
            assert torch.equal(eager[i], other[i])
            xin.copy_(x)
            graph.replay()
            again = call(x)
            torch.cuda.synchronize()
            assert torch.equal(yout, eager[i]) and torch.equal(again, eager[i])
        assert_product(eager[1], xs[1], w, mags, which, parts)


def test_int4_offsets_beyond_32_bits():
    """Codes of 2^32 weights and more: the last rows are found (all others have scale 0)."""
    rows, cols, group = 66000, 65536, 128
    log_case(f"int4 {rows}x{cols}")
    q = torch.zeros((rows, bcjr.bcjr_int4_words(cols)), dtype=torch.int32, device="cuda")
    s = torch.zeros((rows, cols // group), device="cuda")
    codes, sl, _ = make_int4(3, cols, group, False, 8)
    q[-3:] = torch.from_numpy(ref.int4_pack(codes).view(np.int32)).cuda()
    s[-3:] = torch.from_numpy(sl).cuda()
    x = make_x(2, cols, "bf16", 1)
    y = bcjr.bcjr_int4_matvec(x, q.view(torch.uint32), s, None, group)
    assert bool((y[:, :-3] == 0).all())
    w = ref.int4_weights(codes, sl, None, group)
    assert_product(y[:, -3:], x, w, 32 * np.abs(sl.astype(np.float64))[:, np.arange(cols) // group], "int4")


# ---- rounding to 4 bits --------------------------------------------------------------------------

def check_quantize(w, group, zeros):
    q, s, z = bcjr.bcjr_int4_quantize(w, group, zeros)
    codes, s_ref, z_ref = ref.int4_quantize(exact64(w), group, zeros)
    np.testing.assert_array_equal(s.cpu().numpy(), s_ref)
    if zeros:
        np.testing.assert_array_equal(z.cpu().numpy(), z_ref)
    else:
        assert z is None
    np.testing.assert_array_equal(q.cpu().numpy(), ref.int4_pack(codes))
    back = bcjr.bcjr_int4_dequantize(q, s, z, w.shape[1], group)
    fine = ref.int4_weights(codes, s_ref, z_ref, group)
    np.testing.assert_array_equal(back.cpu().numpy(), fine.astype(np.float32))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows,cols,group", [(1, 1, 32), (3, 31, 32), (5, 129, 64), (7, 1000, 96), (9, 777, 128), (2, 5000, 2048),
                                             (33, 512, 512), (6, 640, 1024)])
def test_int4_quantize(rows, cols, group, zeros, t):
    log_case(f"quantize {rows}x{cols} g{group} zeros={zeros} {t}")
    rng = np.random.default_rng(rows * cols)
    w = 0.02 * rng.standard_normal((rows, cols)) + (0.01 if zeros else 0.0)
    check_quantize(torch.from_numpy(w).to(TYPES[t]).cuda(), group, zeros)
    # one sign only, ties between codes, and groups of zeros
    w = np.abs(w)
    check_quantize(torch.from_numpy(w).to(TYPES[t]).cuda(), group, zeros)
    ties = rng.integers(-14, 15, (rows, cols)) / 2.0
    ties[:, ::group] = 7.0
    check_quantize(torch.from_numpy(ties).to(TYPES[t]).cuda(), group, zeros)
    ties[0] = 0.0
    check_quantize(torch.from_numpy(ties).to(TYPES[t]).cuda(), group, zeros)


@pytest.mark.parametrize("zeros", [False, True])
def test_int4_quantize_extremes(zeros):
    rng = np.random.default_rng(2)
    for scale in (1e-45, 1e-40, 1e-30, 1e30, 1e38):
        log_case(f"quantize scale={scale}")
        w = np.clip(scale * rng.standard_normal((4, 200)), -3.4e38, 3.4e38).astype(np.float32)
        check_quantize(torch.from_numpy(w).cuda(), 64, zeros)
    w = rng.standard_normal((4, 200)).astype(np.float32)
    w[0, 3], w[1, 70], w[2, 199] = np.nan, np.inf, -np.inf
    q, s, z = bcjr.bcjr_int4_quantize(torch.from_numpy(w).cuda(), 64, zeros)
    codes, s_ref, z_ref = ref.int4_quantize(w, 64, zeros)
    np.testing.assert_array_equal(s.cpu().numpy(), s_ref)
    np.testing.assert_array_equal(q.cpu().numpy(), ref.int4_pack(codes))


# ---- trellis-coded weights -----------------------------------------------------------------------

def make_code(rows, cols, n, k, L, scales, seed):
    rng = np.random.default_rng(seed)
    chains, words = rows * cols // L, (n + k * (L - 1) + 31) // 32
    code = rng.integers(0, 1 << 32, (chains, words), dtype=np.uint32)
    tail = 32 * words - n - k * (L - 1)
    code[:, -1] &= np.uint32(0xFFFFFFFF ^ ((1 << tail) - 1))
    cb = rng.standard_normal(1 << n).astype(np.float32)
    s = (0.02 * (0.5 + rng.random(chains))).astype(np.float32) if scales else None
    w = cb.astype(np.float64)[ref.code_states(code, n, k, L)]
    if scales:
        w = w * s.astype(np.float64)[:, None]
    return code, cb, s, w.reshape(rows, cols)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,k", [(4, 1), (4, 4), (5, 3), (8, 2), (10, 1), (12, 2), (12, 4), (13, 3), (15, 2), (16, 2), (16, 16), (1, 1), (9, 8)])
def test_code_matvec(n, k, t):
    for rows, L, chains in ((1, 1, 1), (5, 33, 3), (18, 100, 2), (40, 128, 3), (70, 256, 8), (3, 1000, 1)):
        for tokens in (1, 2, 6, 16, 19):
            log_case(f"code n={n} k={k} rows={rows} L={L} chains={chains} tokens={tokens} {t}")
            scales = (rows + tokens) % 2 == 0
            code, cb, s, w = make_code(rows, L * chains, n, k, L, scales, rows + n)
            x = make_x(tokens, L * chains, t, 2)
            y = bcjr.bcjr_code_matvec(x, dev(code), dev(cb), n, k, L, None if s is None else dev(s))
            assert_product(y, x, w, np.abs(w), "code", 2.0 ** -16 if t != "fp32" else 0.0)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows,cols,n,k,L,tokens", [(2048, 8192, 12, 2, 256, 1), (512, 4096, 8, 2, 4096, 3), (1030, 2048, 16, 2, 256, 4),
                                                    (256, 16384, 12, 3, 128, 33), (4, 65536, 10, 2, 256, 1)])
def test_code_matvec_larger(rows, cols, n, k, L, tokens, t):
    log_case(f"code {rows}x{cols} n={n} k={k} L={L} tokens={tokens} {t}")
    code, cb, s, w = make_code(rows, cols, n, k, L, True, 6)
    x = make_x(tokens, cols, t, 7)
    y = bcjr.bcjr_code_matvec(x, dev(code), dev(cb), n, k, L, dev(s))
    assert_product(y, x, w, np.abs(w), "code", 2.0 ** -16 if t != "fp32" else 0.0)


def test_products_agree_with_the_decoder():
    """Viterbi, pack, product: the same as the decoder's own hard weights."""
    n, k, L, rows, cols = 8, 2, 256, 64, 1024
    log_case("decode, pack, product")
    rng = np.random.default_rng(1)
    w = dev(rng.standard_normal((rows * cols // L, L)).astype(np.float32))
    cb = dev(rng.standard_normal(1 << n).astype(np.float32))
    states, hard = bcjr.viterbi_decode(cb, w, n, k)
    code = bcjr.bcjr_pack_code(states, n, k)
    wh = exact64(hard).reshape(rows, cols)
    for t in TYPES:
        x = make_x(4, cols, t, 3)
        assert_product(bcjr.bcjr_code_matvec(x, code, cb, n, k, L), x, wh, np.abs(wh), "code", 2.0 ** -16)


# ---- the ends of the ranges ------------------------------------------------------------------------

@pytest.mark.parametrize("L,chains", [(8, 17), (9, 15), (12, 11), (31, 9), (32, 8), (64, 5), (96, 3), (100, 21), (136, 4)])
@pytest.mark.parametrize("t", TYPES)
def test_code_chains_against_blocks(L, chains, t):
    """Chains that begin anywhere within a lane's eight columns, and columns that are no multiple of eight."""
    for n, k in ((12, 2), (7, 3), (15, 4), (16, 1)):
        for tokens in (1, 2, 3, 5, 17):
            log_case(f"code n={n} k={k} L={L} chains={chains} tokens={tokens} {t}")
            code, cb, s, w = make_code(21, L * chains, n, k, L, tokens != 2, n + L)
            x = make_x(tokens, L * chains, t, 5)
            y = bcjr.bcjr_code_matvec(x, dev(code), dev(cb), n, k, L, None if s is None else dev(s))
            assert_product(y, x, w, np.abs(w), "code", 2.0 ** -16 if t != "fp32" else 0.0)


@pytest.mark.parametrize("L", [100, 128])
@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e4, 3e37])
def test_code_ranges(L, size):
    """Codewords far from 1, brought back by the scales: also beyond what a half holds."""
    for t in TYPES:
        log_case(f"code range {size} L={L} {t}")
        code, cb, s, w = make_code(33, 4 * L, 9, 2, L, True, 3)
        big = (cb.astype(np.float64) * size).astype(np.float32)
        s2 = (s.astype(np.float64) / size).astype(np.float32)
        w = big.astype(np.float64)[ref.code_states(code, 9, 2, L)] * s2.astype(np.float64)[:, None]
        w = w.reshape(33, 4 * L)
        x = make_x(4, 4 * L, t, 6)
        y = bcjr.bcjr_code_matvec(x, dev(code), dev(big), 9, 2, L, dev(s2))
        assert_product(y, x, w, np.abs(w), "code", 2.0 ** -16 if t != "fp32" else 0.0)


@pytest.mark.parametrize("L", [100, 256])
def test_non_finite_codewords_stay_in_their_rows(L):
    log_case(f"non-finite codewords L={L}")
    n, k, rows, cols = 10, 2, 24, 2 * L
    code, cb, s, w = make_code(rows, cols, n, k, L, True, 4)
    used = ref.code_states(code, n, k, L).reshape(rows, cols)
    for bad in (np.nan, np.inf):
        c2 = cb.copy()
        c2[used[5, 17]] = bad
        hit = (used == used[5, 17]).any(axis=1)
        for t in TYPES:
            x = make_x(3, cols, t, 8)
            y = bcjr.bcjr_code_matvec(x, dev(code), dev(c2), n, k, L, dev(s))
            assert not bool(torch.isfinite(y[:, hit]).any())
            assert_product(y[:, ~hit], x, w[~hit], np.abs(w[~hit]), "code", 2.0 ** -16)


@pytest.mark.parametrize("which", ["int4", "code"])
def test_rows_of_x_far_apart_and_very_many_tokens(which):
    call, w, mags, parts = product(which, 3, 96)
    far = (1 << 24) + 40
    for tokens in (2, 5):
        log_case(f"{which} x stride {far} tokens={tokens}")
        x = make_x(tokens, 96, "bf16", 2)
        wide = torch.zeros(((tokens - 1) * far + 96,), dtype=x.dtype, device="cuda")
        strided = wide.as_strided((tokens, 96), (far, 1))
        strided.copy_(x)
        assert_product(call(strided), x, w, mags, which, parts)
    tokens = 5 * 32768 + 3
    log_case(f"{which} tokens={tokens}")
    few = make_x(7, 96, "fp32", 3)
    y = call(few.repeat(tokens // 7 + 1, 1)[:tokens].contiguous())
    for at in (0, 70000, tokens - 14):
        at = at // 7 * 7
        assert_product(y[at:at + 7], few, w, mags, which, parts)


def test_longest_rows():
    """2^24 columns in 4 bits; a chain of more columns than the tiles take."""
    cols, group = 1 << 24, 1 << 20
    log_case("int4 2^24 columns")
    q = torch.zeros((2, bcjr.bcjr_int4_words(cols)), dtype=torch.int32, device="cuda")
    codes, s, _ = make_int4(2, 512, 512, False, 3)
    q[:, -64:] = torch.from_numpy(ref.int4_pack(codes).view(np.int32)).cuda()
    scales = torch.zeros((2, cols // group), device="cuda")
    scales[:, -1:] = torch.from_numpy(np.abs(s)).cuda()
    x = torch.zeros((1, cols), device="cuda")
    x[:, -512:] = make_x(1, 512, "fp32", 4)
    w = ref.int4_weights(codes, np.abs(s), None, 512)
    assert_product(bcjr.bcjr_int4_matvec(x, q.view(torch.uint32), scales, None, group), x[:, -512:], w, 32 * np.abs(s) * np.ones((2, 512)), "int4")
    L = (1 << 20) + 64
    log_case(f"code {L} columns")
    code, cb, sc, w = make_code(2, L, 10, 2, L, True, 4)
    for t in ("fp32", "bf16"):
        x = make_x(2, L, t, 4)
        assert_product(bcjr.bcjr_code_matvec(x, dev(code), dev(cb), 10, 2, L, dev(sc)), x, w, np.abs(w), "code", 2.0 ** -16 if t != "fp32" else 0.0)


@pytest.mark.parametrize("n,k,L,cols", [(12, 2, 256, 4096), (15, 2, 256, 4096), (15, 1, 100, 4100), (16, 2, 64, 4096)])
def test_captured_large_tables(n, k, L, cols):
    """Tables beyond 64 KiB of LDS, and in memory: eager, from two host threads at once, on their streams, and
    captured give the same bits."""
    rows = 2056
    code, cb, s, w = make_code(rows, cols, n, k, L, True, 8)
    cd, cbd, sd = dev(code), dev(cb), dev(s)
    call = lambda x, y=None: bcjr.bcjr_code_matvec(x, cd, cbd, n, k, L, sd, y=y)  # noqa: E731
    for t, tokens in (("bf16", 1), ("fp16", 5), ("fp32", 2)):
        log_case(f"large table n={n} k={k} L={L} {t} tokens={tokens}")
        xs = [make_x(tokens, cols, t, 30 + i) for i in range(3)]
        eager = [call(x) for x in xs]
        torch.cuda.synchronize()
        assert_product(eager[0], xs[0], w, np.abs(w), "code", 2.0 ** -16 if t != "fp32" else 0.0)
        results = [None, None]

        def work(i):
            with torch.cuda.stream(torch.cuda.Stream()):
                results[i] = [call(x) for x in xs]
                torch.cuda.current_stream().synchronize()

        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for th in threads:
            th.start()
        for th in threads:
            th.join()
        xin, yout = xs[0].clone(), torch.empty_like(eager[0])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(xin, y=yout)
        for i, x in enumerate(xs):
            assert all(torch.equal(r[i], eager[i]) for r in results)
            xin.copy_(x)
            graph.replay()
            again = call(x)
            torch.cuda.synchronize()
            assert torch.equal(yout, eager[i]) and torch.equal(again, eager[i])
