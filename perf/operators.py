"""Cases of the optimiser and quantised-linear operators: what is timed and what they compute.

Four operators a quantisation-aware training run and the serving of its layers need:

* ``adamw``: one AdamW step over a list of tensors, first and second moments in fp32 or in 8 bits;
* ``int4_quantize``: weights to 4-bit codes with one fp32 scale (and optionally a zero point) for
  each group of columns;
* ``int4_matvec``: products of a few tokens with such weights;
* ``code_matvec``: products of a few tokens with trellis-coded weights (the packed hard code).

``run`` computes them in elementary torch operations, or, where ``own`` is true, by this package's
entry points. ``exact`` computes the definitions again in 64 bits.

The 8-bit moments are blocks of 32 elements: e4m3 codes and one power of two for each block, 2^(b - 127)
with b held in 8 bits. The first moment m is held as it is, the second as r = sqrt(v). A block's
power of two puts its largest magnitude in [128, 256). Rounding is up with the probability of what
is cut off, by a dither d that is a hash of the element's place in the state, the step and the seed:
code = floor(|y| / u + d) u, u the spacing of e4m3 at y, and at least one u where r > 0.

The 4-bit weights of a row lie in blocks of 128 columns, 16 words of 8 columns each: word 4 g + j of
a block holds its columns 32 j + 8 g .. + 7, and of a word's columns c = 0 .. 7 the even ones are the
nibbles c / 2 and the odd ones the nibbles 4 + (c - 1) / 2, counted from the low end. What a weight
stands for is (nibble - zero) * scale, with zero = 8 where none is given. Columns behind a row's last
are zero nibbles.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
MASK = 0xFFFFFFFF
BLOCK = 32


# ---- cases -------------------------------------------------------------------------------------

def listed():
    return [
        # the layer of the QAT command's defaults, one fp32 tensor: launch latency
        dict(name="adamw-layer", op="adamw", sizes="524288", param="fp32", grad="fp32", bits=32),
        # a model's ragged tensors in bf16 (odd matrices, vectors, single values), fp32 moments
        dict(name="adamw-ragged-bf16", op="adamw", param="bf16", grad="bf16", bits=32,
             sizes="4194304,2048,1000001,1,37,2048,4194304,777777,31,33,65536,2047,1049600,129,5,8388608"),
        # the latent weights of several 2048x8192 and 2048x2048 layers with their norms, 8-bit moments
        dict(name="adamw-model-8bit", op="adamw", param="fp32", grad="fp32", bits=8,
             sizes=",".join(["16777216", "16777216", "4194304", "4194304", "2048", "2048"] * 4)),
        # an odd layer with zero points and the smallest groups
        dict(name="int4-quantize-odd", op="int4_quantize", rows=1000, cols=4100, group=32, zeros=True, type="bf16"),
        # the 2048x8192 layer of the benchmark's Llama-shaped workload
        dict(name="int4-quantize-layer", op="int4_quantize", rows=2048, cols=8192, group=128, zeros=False, type="fp32"),
        # one token through the QAT command's default layer in the framework's own fp32
        dict(name="int4-token-small", op="int4_matvec", rows=512, cols=1024, group=32, zeros=False, tokens=1, type="fp32"),
        # one token through the 2048x8192 layer: decoding
        dict(name="int4-token-layer", op="int4_matvec", rows=2048, cols=8192, group=128, zeros=False, tokens=1, type="bf16"),
        # a few sequences decoded together, ragged rows and columns, zero points
        dict(name="int4-batch-odd", op="int4_matvec", rows=5000, cols=4097, group=64, zeros=True, tokens=7, type="fp16"),
        # a large layer and a full batch of sequences
        dict(name="int4-batch-large", op="int4_matvec", rows=16384, cols=16384, group=128, zeros=False, tokens=32, type="bf16"),
        # one token through the QAT command's default layer as the trellis code it exports
        dict(name="code-token-small", op="code_matvec", rows=512, cols=1024, n=8, k=2, L=256, scales=False, tokens=1, type="fp32"),
        # one token through the 2048x8192 layer of the S = 4096 workload, a scale for each chain
        dict(name="code-token-layer", op="code_matvec", rows=2048, cols=8192, n=12, k=2, L=256, scales=True, tokens=1, type="bf16"),
        # a batch of sequences through a large layer
        dict(name="code-batch-large", op="code_matvec", rows=8192, cols=8192, n=12, k=2, L=256, scales=True, tokens=16, type="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "int4_quantize", "int4_matvec", "int4_matvec", "code_matvec", "code_matvec"])
    t = rng.choice(["fp32", "bf16", "fp16"])
    if op == "adamw":
        count, total = _log(rng, 1, 24), _log(rng, 1 << 10, 1 << 26)
        share = [math.exp(rng.uniform(-6, 0)) for _ in range(count)]
        sizes = [max(1, int(total * s / sum(share))) for s in share]
        return dict(op=op, sizes=",".join(map(str, sizes)), param=t, grad=rng.choice(["fp32", t]), bits=rng.choice([8, 32]))
    if op == "int4_quantize":
        return dict(op=op, rows=_log(rng, 64, 8192), cols=_log(rng, 64, 8192), group=rng.choice([32, 64, 96, 128, 256]),
                    zeros=rng.random() < 0.5, type=t)
    if op == "int4_matvec":
        return dict(op=op, rows=_log(rng, 64, 16384), cols=_log(rng, 64, 16384), group=rng.choice([32, 64, 96, 128, 256]),
                    zeros=rng.random() < 0.5, tokens=_log(rng, 1, 32), type=t)
    n = rng.randint(4, 16)
    L = rng.choice([32, 64, 100, 128, 256, 256, 512])
    return dict(op=op, rows=_log(rng, 64, 8192), cols=L * _log(rng, 1, 8192 // L), n=n, k=rng.randint(1, 4), L=L,
                scales=rng.random() < 0.5, tokens=_log(rng, 1, 16), type=t)


def _sizes(case):
    return [int(s) for s in case["sizes"].split(",")]


def _padded(n):
    return -(-n // BLOCK) * BLOCK


def _words(case):
    return (case["n"] + case["k"] * (case["L"] - 1) + 31) // 32


def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(_sizes(case))
        state = 16 * n if case["bits"] == 32 else 4 * n + 4 * n // BLOCK
        return {"bytes": n * (2 * SIZE[case["param"]] + SIZE[case["grad"]]) + state, "flops": 14 * n}
    r, c = case["rows"], case["cols"]
    if op == "code_matvec":
        chains = r * c // case["L"]
        held = 4 * chains * _words(case) + 4 * (1 << case["n"]) + (4 * chains if case["scales"] else 0)
    else:
        groups = r * -(-c // case["group"])
        held = r * c // 2 + groups * (5 if case["zeros"] else 4)
    if op == "int4_quantize":
        return {"bytes": r * c * SIZE[case["type"]] + held, "flops": 4 * r * c}
    m = case["tokens"]
    return {"bytes": held + m * (r + c) * SIZE[case["type"]], "flops": 2 * m * r * c}


# ---- inputs ------------------------------------------------------------------------------------

def _channels(gen, c):
    """Scales of a layer's input channels: log-normal, as the outlier channels of activations."""
    return torch.exp(0.75 * torch.randn(c, generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    randn = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    rand = lambda *shape: torch.rand(*shape, generator=gen, device="cuda")  # noqa: E731
    s = dict(case)
    if case["op"] == "adamw":
        sizes = _sizes(case)
        s["params"] = [randn(n).to(DTYPES[case["param"]]) for n in sizes]
        s["grads"] = [(1e-3 * randn(n) * torch.exp(0.75 * randn(n))).to(DTYPES[case["grad"]]) for n in sizes]
        total = sum(_padded(n) for n in sizes)
        s["offsets"] = [sum(_padded(m) for m in sizes[:i]) for i in range(len(sizes))]
        s["hyper"] = dict(step=100, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
        if case["bits"] == 32:
            s["exp_avg"], s["exp_avg_sq"] = 3e-4 * randn(total), (1e-3 * randn(total)).square_()
        else:
            s["exp_avg"] = (30 * randn(total)).clamp_(-240, 240).to(torch.float8_e4m3fn)
            s["exp_avg_sq"] = (60 * randn(total)).abs_().clamp_(1, 240).to(torch.float8_e4m3fn)
            s["avg_scale"] = (108 + 4 * rand(total // BLOCK)).to(torch.uint8)
            s["avg_sq_scale"] = (109 + 3 * rand(total // BLOCK)).to(torch.uint8)
            s["hyper"]["seed"] = int(seed) & 0xFFFF
        return s
    r, c, t = case["rows"], case["cols"], DTYPES[case["type"]]
    if case["op"] == "int4_quantize":
        s["w"] = (0.02 * randn(r, c) * _channels(gen, c)).to(t)
        return s
    s["x"] = (randn(case["tokens"], c) * _channels(gen, c)).to(t)
    if case["op"] == "int4_matvec":
        groups = -(-c // case["group"])
        nibbles = torch.randint(0, 16, (r, c), generator=gen, device="cuda", dtype=torch.uint8)
        s["q"] = _pack_nibbles(nibbles)
        s["scales"] = 0.005 * (0.5 + rand(r, groups))
        s["zero_points"] = torch.randint(5, 11, (r, groups), generator=gen, device="cuda", dtype=torch.uint8) if case["zeros"] else None
        return s
    chains, tail = r * c // case["L"], 32 * _words(case) - case["n"] - case["k"] * (case["L"] - 1)
    code = torch.randint(0, 1 << 32, (chains, _words(case)), generator=gen, device="cuda", dtype=torch.int64)
    code[:, -1] &= MASK ^ ((1 << tail) - 1)
    s["code"] = code.to(torch.uint32)
    s["codebook"] = randn(1 << case["n"])
    s["chain_scales"] = 0.02 * (0.5 + rand(chains)) if case["scales"] else None
    return s


# ---- plain forms -------------------------------------------------------------------------------

def _pack_nibbles(nibbles):
    """Words [r, 16 blocks] (uint32) of codes [r, c] (uint8), laid out as the module says."""
    r, c = nibbles.shape
    blocks = -(-c // 128)
    x = torch.zeros(r, blocks * 128, dtype=torch.uint8, device=nibbles.device)
    x[:, :c] = nibbles
    x = x.view(r, blocks, 4, 4, 4, 2).permute(0, 1, 3, 2, 5, 4).to(torch.int64)  # block, g, j, odd, pair
    shifts = 4 * torch.arange(8, device=x.device)
    return (x.reshape(r, blocks * 16, 8) << shifts).sum(-1).to(torch.uint32)


def _unpack_nibbles(q, c):
    r, words = q.shape
    shifts = 4 * torch.arange(8, device=q.device)
    x = (q.to(torch.int64)[..., None] >> shifts) & 15
    x = x.view(r, words // 16, 4, 4, 2, 4).permute(0, 1, 3, 2, 5, 4)  # block, j, g, pair, odd
    return x.reshape(r, words * 8)[:, :c]


def _mix(x):
    """Multiply-xorshift mix of 32-bit values held in 64."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & MASK
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & MASK
    return x ^ (x >> 16)


def _dithers(first, count, step, seed):
    """The dithers in (0, 1) of the elements first .. first + count - 1 of the state, for m and for r."""
    key = int(_mix(torch.tensor((int(_mix(torch.tensor(seed & MASK))) + step) & MASK)))
    at = torch.arange(first, first + count, device="cuda", dtype=torch.int64)
    h = _mix(((at & MASK) * 0x9E3779B1 + (at >> 32) * 0x85EBCA6B + key) & MASK)
    return ((h & 0xFFFF).double() + 0.5) / 65536, ((h >> 16).double() + 0.5) / 65536


def _encode(x, dither, positive):
    """x [blocks, 32] fp64 -> e4m3 values and the exponents b of each block's scale 2^(b - 127)."""
    a = torch.where(x.abs() < math.inf, x.abs(), 0.0)
    top = a.amax(1, keepdim=True)
    b = torch.where(top > 0, (torch.frexp(top)[1] - 1 - 7 + 127).clamp(0, 254), 0)
    y = torch.ldexp(a, 127 - b)
    u = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=-6).double() - 3)
    n = torch.floor(y / u + dither)
    n = torch.where(y > 0, n.clamp(min=1) if positive else n, 0.0)
    code = torch.where(x.abs() < math.inf, torch.copysign(n * u, x), math.nan)
    return code.float().to(torch.float8_e4m3fn), b.to(torch.uint8)[:, 0]


def _blocks(x):
    return torch.nn.functional.pad(x.reshape(-1).double(), (0, _padded(x.numel()) - x.numel())).view(-1, BLOCK)


def _adamw8(p, g, first, s, step, lr, beta1, beta2, eps, weight_decay, seed):
    """One tensor's step with 8-bit moments, in 64 bits since a code's border decides it."""
    end = first + _padded(p.numel())
    here, scale_at = slice(first, end), slice(first // BLOCK, end // BLOCK)
    gd = _blocks(g)
    m = torch.ldexp(s["exp_avg"][here].double().view(-1, BLOCK), s["avg_scale"][scale_at].int()[:, None] - 127)
    r = torch.ldexp(s["exp_avg_sq"][here].double().view(-1, BLOCK), s["avg_sq_scale"][scale_at].int()[:, None] - 127)
    m = beta1 * m + (1 - beta1) * gd
    r = torch.sqrt(beta2 * r * r + (1 - beta2) * gd * gd)
    step_by = m / (1 - beta1**step) / (r / math.sqrt(1 - beta2**step) + eps)
    pd = p.double()
    p.copy_(pd - lr * weight_decay * pd - lr * step_by.view(-1)[: p.numel()])
    valid = (torch.arange(end - first, device="cuda") < p.numel()).view(-1, BLOCK)
    dm, dr = _dithers(first, end - first, step, seed)
    m_code, m_scale = _encode(torch.where(valid, m, 0.0), dm.view(-1, BLOCK), False)
    r_code, r_scale = _encode(torch.where(valid, r, 0.0), dr.view(-1, BLOCK), True)
    here = slice(first, first + p.numel())
    s["exp_avg"][here], s["avg_scale"][scale_at] = m_code.view(-1)[: p.numel()], m_scale
    s["exp_avg_sq"][here], s["avg_sq_scale"][scale_at] = r_code.view(-1)[: p.numel()], r_scale


def _adamw32(p, g, first, s, step, lr, beta1, beta2, eps, weight_decay):
    here = slice(first, first + p.numel())
    g, pf = g.float(), p.float()
    m = s["exp_avg"][here].mul_(beta1).add_((1 - beta1) * g)
    v = s["exp_avg_sq"][here].mul_(beta2).add_((1 - beta2) * g * g)
    step_by = (m / (1 - beta1**step)) / (v.sqrt() / math.sqrt(1 - beta2**step) + eps)
    p.copy_(pf - (lr * weight_decay) * pf - lr * step_by)


def _adamw(s):
    one = _adamw32 if s["bits"] == 32 else _adamw8
    [one(p, g, first, s, **s["hyper"]) for p, g, first in zip(s["params"], s["grads"], s["offsets"])]


def _quantize(s):
    w, group = s["w"], s["group"]
    r, c = w.shape
    groups = -(-c // group)
    x = torch.nn.functional.pad(w.double(), (0, groups * group - c)).view(r, groups, group)  # 64 bits: borders of codes
    if s["zeros"]:
        lo, hi = x.amin(-1).clamp(max=0.0), x.amax(-1).clamp(min=0.0)
        scale = ((hi - lo) / 15).float()
    else:
        scale = (x.abs().amax(-1) / 7).float()
    by = torch.where(scale > 0, scale.double(), 1.0)
    zero = torch.round(-lo / by).clamp(0, 15) if s["zeros"] else torch.full_like(by, 8.0)
    code = (torch.round(x / by[..., None]) + zero[..., None]).clamp(0, 15).view(r, -1)[:, :c].to(torch.uint8)
    return _pack_nibbles(code), scale, zero.to(torch.uint8) if s["zeros"] else None


def _int4_weights(s, cols):
    code = _unpack_nibbles(s["q"], cols).float()
    group = torch.arange(cols, device="cuda") // s["group"]
    zero = 8.0 if s["zero_points"] is None else s["zero_points"].float()[:, group]
    return (code - zero) * s["scales"][:, group]


def _code_weights(s, cols):
    """Every state is the n-bit window of its chain's code that starts at bit k t."""
    at = s["k"] * torch.arange(s["L"], device="cuda")
    words = torch.nn.functional.pad(s["code"].to(torch.int64), (0, 1))
    pair = (words[:, at >> 5] << 32) | words[:, (at >> 5) + 1]
    w = s["codebook"][(pair >> (64 - s["n"] - (at & 31))) & ((1 << s["n"]) - 1)]
    if s["chain_scales"] is not None:
        w = w * s["chain_scales"][:, None]
    return w.view(-1, cols)


# ---- the passes --------------------------------------------------------------------------------

def _own(s):
    from bcjr_soft_decoding_amd import bcjr

    if s["op"] == "adamw":
        bcjr.bcjr_adamw_step(s["params"], s["grads"], s["exp_avg"], s["exp_avg_sq"], s.get("avg_scale"),
                             s.get("avg_sq_scale"), **s["hyper"])
        return None
    if s["op"] == "int4_quantize":
        return bcjr.bcjr_int4_quantize(s["w"], s["group"], s["zeros"])
    if s["op"] == "int4_matvec":
        return bcjr.bcjr_int4_matvec(s["x"], s["q"], s["scales"], s["zero_points"], s["group"])
    return bcjr.bcjr_code_matvec(s["x"], s["code"], s["codebook"], s["n"], s["k"], s["L"], s["chain_scales"])


def _plain(s):
    if s["op"] == "adamw":
        return _adamw(s)
    if s["op"] == "int4_quantize":
        return _quantize(s)
    cols = s["x"].shape[1]
    w = _int4_weights(s, cols) if s["op"] == "int4_matvec" else _code_weights(s, cols)
    return (s["x"].float() @ w.t()).to(s["x"].dtype)


def run(state):
    y = _own(state) if own else _plain(state)
    if state["op"] == "adamw":
        return {k: state[k] for k in ("params", "exp_avg", "exp_avg_sq", "avg_scale", "avg_sq_scale") if k in state}
    if state["op"] == "int4_quantize":
        return {"q": y[0].view(torch.int32), "scales": y[1], "zeros": y[2]}
    return y


# ---- the definitions in 64 bits ----------------------------------------------------------------

def _exact_adamw(s):
    h = s["hyper"]
    b1, b2, t = h["beta1"], h["beta2"], h["step"]
    out = {"params": [], "exp_avg": s["exp_avg"].double(), "exp_avg_sq": s["exp_avg_sq"].double()}
    if s["bits"] == 8:
        out["avg_scale"], out["avg_sq_scale"] = s["avg_scale"].clone(), s["avg_sq_scale"].clone()
    for p, g, o in zip(s["params"], s["grads"], s["offsets"]):
        n = p.numel()
        p, g = p.double(), g.double()
        m, v = out["exp_avg"][o : o + n].clone(), out["exp_avg_sq"][o : o + n].clone()
        block = torch.arange(n, device="cuda") // BLOCK
        if s["bits"] == 8:
            here = slice(o // BLOCK, o // BLOCK + int(block[-1]) + 1)
            m *= 2.0 ** (s["avg_scale"][here].double()[block] - 127)
            v = (v * 2.0 ** (s["avg_sq_scale"][here].double()[block] - 127)) ** 2
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g**2
        out["params"].append((1 - h["lr"] * h["weight_decay"]) * p
                             - h["lr"] * (m / (1 - b1**t)) / ((v / (1 - b2**t)) ** 0.5 + h["eps"]))
        if s["bits"] == 8:
            dithers = _dithers(o, n, t, h["seed"])
            for x, d, codes, scale, least in ((m, dithers[0], "exp_avg", "avg_scale", 0), (v**0.5, dithers[1], "exp_avg_sq", "avg_sq_scale", 1)):
                top = torch.zeros(int(block[-1]) + 1, dtype=torch.float64, device="cuda").scatter_reduce_(0, block, x.abs(), "amax")
                e = torch.floor(torch.log2(top))
                e = torch.where(2.0**e > top, e - 1, torch.where(2.0 ** (e + 1) <= top, e + 1, e))  # log2 next to a power of two
                b = torch.where(top > 0, (e + 120).clamp(0, 254), 0.0)
                y = x.abs() / 2.0 ** (b[block] - 127)
                e = torch.floor(torch.log2(y))
                e = torch.where(2.0**e > y, e - 1, torch.where(2.0 ** (e + 1) <= y, e + 1, e)).clamp(min=-6)
                k = torch.floor(y * 2.0 ** (3 - e) + d).clamp(min=least)
                out[codes][o : o + n] = torch.where(y > 0, k * 2.0 ** (e - 3) * torch.sign(x), 0.0)
                out[scale][here] = b.to(torch.uint8)
        else:
            out["exp_avg"][o : o + n], out["exp_avg_sq"][o : o + n] = m, v
    return out


def _exact_quantize(s):
    w, group = s["w"].double(), s["group"]
    scales, zeros, codes = [], [], []
    for at in range(0, w.shape[1], group):
        x = w[:, at : at + group]
        lo, hi = x.min(1)[0].clamp(max=0), x.max(1)[0].clamp(min=0)
        exact = (hi - lo) / 15 if s["zeros"] else torch.maximum(hi, -lo) / 7
        scale = exact.float().double()  # the codes go by the scale that is kept
        safe = torch.where(scale == 0, torch.ones_like(scale), scale)
        zero = (-lo / safe).round().clamp(0, 15) if s["zeros"] else torch.full_like(lo, 8)
        codes.append(((x / safe[:, None]).round() + zero[:, None]).clamp(0, 15))
        scales.append(exact)
        zeros.append(zero)
    codes = torch.cat(codes, 1).long()
    r, c = codes.shape
    q = torch.zeros(r, -(-c // 128) * 16, dtype=torch.int64, device="cuda")
    for col in range(c):
        block, i = divmod(col, 128)
        j, i = divmod(i, 32)
        g, i = divmod(i, 8)
        q[:, block * 16 + 4 * g + j] |= codes[:, col] << (4 * (i // 2 + 4 * (i % 2)))
    return {"q": q.to(torch.uint32).view(torch.int32), "scales": torch.stack(scales, 1),
            "zeros": torch.stack(zeros, 1).to(torch.uint8) if s["zeros"] else None}


def _exact_int4(s, cols):
    col = torch.arange(cols, device="cuda")
    word = col // 128 * 16 + 4 * (col % 32 // 8) + col % 128 // 32
    shift = 4 * (col % 8 // 2 + 4 * (col % 2))
    w = ((s["q"].to(torch.int64)[:, word] >> shift) % 16).double()
    w -= 8 if s["zero_points"] is None else s["zero_points"].double().repeat_interleave(s["group"], 1)[:, :cols]
    return w * s["scales"].double().repeat_interleave(s["group"], 1)[:, :cols]


def _exact_code(s, cols):
    code, n = s["code"].to(torch.int64), s["n"]
    state = torch.zeros(code.shape[0], s["L"], dtype=torch.int64, device="cuda")
    for i in range(n):  # bit by bit, the most significant first
        bit = s["k"] * torch.arange(s["L"], device="cuda") + i
        state = 2 * state + ((code[:, bit // 32] >> (31 - bit % 32)) & 1)
    w = s["codebook"].double()[state]
    if s["chain_scales"] is not None:
        w *= s["chain_scales"].double()[:, None]
    return w.reshape(-1, cols)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "adamw":
        return _exact_adamw(s)
    if s["op"] == "int4_quantize":
        return _exact_quantize(s)
    cols = s["x"].shape[1]
    w = _exact_int4(s, cols) if s["op"] == "int4_matvec" else _exact_code(s, cols)
    return s["x"].double() @ w.t()
