"""AdamW, the QAT driver with it, and layers served from their packed code or 4-bit weights: the
operators as they are used together."""
import json

import numpy as np
import pytest
import torch

from bcjr_soft_decoding_amd import bcjr, linear, optim, qat, synth
from oracle import qat as oqat
from tests import ops_reference as ref
from tests.gpu_helpers import RTOL_FWD, RTOL_GRAD, assert_normwise, assert_rel, dev, log_case
from tests.test_gpu_ops import TYPES, assert_product, exact64, make_x

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bcjr.lib()


def test_optimizer_matches_the_formula_and_resumes():
    log_case("optimizer class")
    for bits in (32, 8):
        gen = torch.Generator(device="cuda").manual_seed(0)
        sizes = [(17, 5), (3,), (64, 64)]
        p = [torch.randn(*s, generator=gen, device="cuda") for s in sizes]
        grads = [[0.1 * torch.randn(*s, generator=gen, device="cuda") for s in sizes] for _ in range(6)]
        q = [t.clone() for t in p]
        a = optim.AdamW(p, lr=1e-2, weight_decay=0.1, state_bits=bits, seed=3)
        for g in grads[:3]:
            a.step(g)
        # the formula in 64 bits gives the moments; in 8 bits they are its rounding
        m = sum(0.1 * 0.9 ** (2 - i) * exact64(grads[i][2]) for i in range(3))
        v = sum(0.001 * 0.999 ** (2 - i) * exact64(grads[i][2]) ** 2 for i in range(3))
        if bits == 32:
            got = a.moments(2)
            np.testing.assert_allclose(exact64(got[1]), v, rtol=20 * 2.0 ** -24)
            assert np.all(np.abs(exact64(got[0]) - m) <= 20 * 2.0 ** -24 * 3 * 0.1)
        # a second optimiser takes over the state and the tensors and goes on bit for bit
        b = optim.AdamW([t.clone() for t in p], state_bits=bits)
        state = a.state_dict()
        b.load_state_dict(state)
        for i, g in enumerate(grads[3:]):
            a.step(g)
            for t, gr in zip(b.params, g):
                t.grad = gr
            b.step()
        assert a.steps == b.steps == 6
        assert all(torch.equal(s, t) for s, t in zip(p, b.params))
        assert all(not torch.equal(s, t) for s, t in zip(p, q))
        with pytest.raises(ValueError):
            optim.AdamW(p, state_bits=40 - bits).load_state_dict(state)
        with pytest.raises(ValueError):
            optim.AdamW(p[:2], state_bits=bits).load_state_dict(state)


def test_optimizer_refusals():
    p = torch.zeros(8, device="cuda")
    for call in (lambda: optim.AdamW([]), lambda: optim.AdamW([p], state_bits=16), lambda: optim.AdamW([p, p.half()]),
                 lambda: optim.AdamW([p.cpu()]), lambda: optim.AdamW([torch.zeros(4, 4, device="cuda").t()[:, :2]]),
                 lambda: optim.AdamW([p]).step(), lambda: optim.AdamW([p]).step([None]), lambda: optim.AdamW([p]).step([])):
        with pytest.raises(ValueError):
            call()
    a = optim.AdamW([p])
    with pytest.raises(bcjr.BcjrError):
        optim.AdamW([p, p]).step([p.clone(), p.clone()])
    g = torch.ones(8, device="cuda")
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        with pytest.raises(RuntimeError, match="captured"):
            a.step([g])
        g.add_(1)
    assert a.steps == 0


def test_layers():
    log_case("layers")
    rng = np.random.default_rng(0)
    W = dev(rng.standard_normal((96, 512)).astype(np.float32))
    cb = dev(rng.standard_normal(256).astype(np.float32))
    coded = linear.CodedLinear.from_weights(W, cb, 8, 2, 128, dev((0.5 + rng.random(96 * 4)).astype(np.float32)))
    assert coded.nbytes() == 4 * 96 * 4 * ((8 + 2 * 127 + 31) // 32) + 4 * 96 * 4
    for layer, parts in ((coded, 2.0 ** -16), (linear.Int4Linear.from_weights(W, 64), 0.0), (linear.Int4Linear.from_weights(W, 96, True), 0.0)):
        w = exact64(layer.weights())
        assert w.shape == (96, 512)
        mags = np.abs(w) if layer is coded else np.full_like(w, 32 * float(layer.scales.max()))
        for t in TYPES:
            x = make_x(6, 512, t, 1)
            y = layer(x)
            # weights() rounds w to fp32 once more: 2^-24 of each term
            assert_product(y, x, w, mags, "layer", parts + 2.0 ** -24)
            y3 = layer(x.view(2, 3, 512))
            assert tuple(y3.shape) == (2, 3, 96) and torch.equal(y3.view(6, 96), y)
            y1 = layer(x[2])
            assert tuple(y1.shape) == (96,)
            assert_product(y1.view(1, 96), x[2:3], w, mags, "layer", parts + 2.0 ** -24)
            assert_product(layer(x.t().contiguous().t()), x, w, mags, "layer", parts + 2.0 ** -24)
        with pytest.raises(ValueError):
            layer(torch.zeros(1, 511, device="cuda"))
    with pytest.raises(ValueError):
        linear.CodedLinear.from_weights(W, cb, 8, 2, 100)


@pytest.mark.parametrize("optimizer", ["adamw", "adamw8"])
def test_annealed_adamw_matches_the_oracle(optimizer):
    """Each step from the driver's own weights: the oracle's gradient through the 64-bit AdamW. The first
    step of AdamW is lr sign(g) but where g is next to zero, so steps are compared in the moments and
    in the weights where |g| is over a thousandth of its RMS."""
    n, R, C, N, L = 8, 4, 512, 256, 128
    steps, lr, t0, t_end = 4, 1e-3, 0.3, 0.05
    log_case(f"qat {optimizer}")
    W, X, _, c = synth.qat_layer(R, C, N, n, seed=4)
    cfg = qat.QATConfig(n=n, k=2, L=L, t0=t0, t_end=t_end, steps=steps, lr=lr, optimizer=optimizer)
    res = qat.train(dev(W), dev(X), dev(c), cfg, log_every=1)
    assert res.drift_inf <= res.budget(cfg) * 1.25
    loss, g, _ = oqat.loss_and_grad(W, W, X, c, n, 2, L, t0)
    assert_rel(res.history[0]["soft_loss"], loss, RTOL_FWD, "loss")
    one = qat.train(dev(W), dev(X), dev(c), qat.QATConfig(n=n, k=2, L=L, t0=t0, t_end=t_end, steps=1, lr=lr, optimizer=optimizer))
    moved = exact64(one.w) - W
    big = np.abs(g) > 1e-3 * np.sqrt(np.mean(g * g))
    # g within RTOL_GRAD of its RMS: the sign is right where |g| is over that; |step| = lr then
    assert np.all(np.sign(moved[big]) == -np.sign(g[big]))
    assert np.all(np.abs(np.abs(moved[big]) - lr) <= 2.0 ** -22)


def test_train_and_serve():
    """The whole way: AdamW with 8-bit moments, Viterbi, packed code, products; the served error is the
    hard code's own, and the driver reports it beside the 4-bit baseline."""
    log_case("train and serve")
    rows, cols, N, n = 256, 1024, 512, 8
    cfg = qat.QATConfig(n=n, k=2, L=256, steps=10, lr=1e-3, optimizer="adamw8")
    r = qat.run(rows, cols, N, cfg, seed=0, serve=True, group=64)
    again = qat.run(rows, cols, N, cfg, seed=0, serve=True, group=64)
    for key in ("qat_loss_heldout", "drift_inf", "chains_with_new_code"):
        assert r[key] == again[key]
    assert r["served"] == again["served"]
    # two fp32 evaluations of one sum of squares of differences
    assert r["served"]["code_loss_heldout"] == pytest.approx(r["qat_loss_heldout"], rel=1e-4)
    assert r["served"]["code_bits_per_weight"] == pytest.approx(32 * 17 / 256)
    assert r["served"]["int4_bits_per_weight"] == pytest.approx(4 + 32 / 64)
    W, _, Xv, _ = qat.synthetic_layer(rows, cols, N, n, 0)
    q = ref.int4_quantize(exact64(W), 64, False)
    w4 = ref.int4_weights(*q, 64)
    d = exact64(Xv) @ (w4 - exact64(W)).T
    assert r["served"]["int4_loss_heldout"] == pytest.approx(np.sum(d * d) / N / (rows * cols), rel=1e-4)


def test_command(capsys):
    log_case("qat command")
    qat.main(["--rows", "64", "--cols", "512", "--samples", "64", "--steps", "3", "--t0", "0.3", "--optimizer", "adamw8", "--serve"])
    out = json.loads(capsys.readouterr().out.strip().splitlines()[-1])
    assert out["optimizer"] == "adamw8" and set(out["served"]) == {
        "code_loss_heldout", "code_bits_per_weight", "int4_loss_heldout", "int4_bits_per_weight"}
