"""GPU parity of the linear layers (llvq_linear, llvq_linear_grouped) against the definition in 64 bits.

The weight comes from the CPU oracle's decode (72 and 96 bits: the library's own decode, which the parity
tests pin to the oracle) and the gains; the layer's formula is evaluated in fp64.

Tolerances.  With u the half step of the output type (fp16 2^-11, bf16 2^-8):
  * each decoded weight is within 2^-11 of w (one rounding to 11 bits), every product is exact in fp32, and
    the fp32 sums of nk 16-column steps and up to 74 split parts lose at most 2^-23 of the running sum each, so
    |dz| <= (2^-11 + (nk + 90) 2^-23) sum |w x| + 2^-22 |z| (bias and scales);
  * |act'| <= 1.13 for every activation here, and its evaluation is off by a few fp32 steps;
  * y is rounded once: u |y|, or half of the least subnormal.
`bound` adds these up per output.  A second check holds the RMS: independent roundings of the weights give
var(dz) <= 2^-22 / 3 sum (w x)^2 (each uniform within its half step), and y's own rounding at most u^2 / 3 y^2;
1.25 covers the spread of the estimate over a few hundred outputs (fewer: not checked).
"""
import numpy as np
import pytest

import oracle
from codebook_free_lattice_b200 import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
LIP = 1.13


@pytest.fixture(scope="module")
def codecs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import codebook_free_lattice_b200 as L
    made = {}

    def get(bits):
        if bits not in made:
            made[bits] = (L.Codec(bits), oracle.Codec(48) if bits == 48 else None)
        return made[bits]
    yield get
    for g, _ in made.values():
        g.close()


class Layer:
    """A compressed weight [rows, cols] on the GPU and its fp64 values."""

    def __init__(self, codecs, bits, rows, cols, gain="table", seed=0, pitch=None, scale=None, bad=0):
        g, o = codecs(bits)
        self.codec, self.rows, self.cols = g, rows, cols
        nb = -(-cols // 24)
        pitch = nb if pitch is None else pitch
        rng = np.random.default_rng([seed, rows, cols])
        lo, hi = synth.uniform_indices(rng, rows * pitch, g.n_points, bits)
        if bad:                                       # some indices past the coded points
            lo[rng.choice(rows * pitch, bad, replace=False)] = np.uint64(2 ** 48 - 1)
        codes = rng.integers(0, 256, rows * pitch, dtype=np.uint8)
        words = synth.pack_words(lo, hi, codes if gain == "table" else None, bits)
        n = rows * pitch
        if bits == 48:
            ok = lo < np.uint64(o.n_points)
            v = np.zeros((n, 24), np.int8)
            v[ok] = o.decode_batch(lo[ok])
        else:
            out = torch.empty((n, 24), dtype=torch.int8, device="cuda")
            g.decode(torch.from_numpy(words.view(np.int64)).cuda(), out)
            v = out.cpu().numpy()
        v = v.astype(np.float64).reshape(rows, pitch, 24)[:, :nb]
        spread = (rng.uniform(0.5, 2.0, (rows, 1)) if scale is None else np.asarray(scale).reshape(rows, 1)) / np.sqrt(cols)
        if gain == "table":
            table = (spread * np.sort(np.sqrt(rng.chisquare(24, (rows, 256))), axis=1)).astype(np.float16)
            self.gains = table
            gv = np.take_along_axis(table.astype(np.float64), codes.reshape(rows, pitch)[:, :nb].astype(np.int64), 1)
            norm = np.sqrt((v ** 2).sum(2))
            gv = gv / np.where(norm == 0, 1, norm)
        else:
            self.gains = (spread * rng.uniform(0.2, 0.5, (rows, nb))).astype(np.float16)
            gv = self.gains.astype(np.float64)
        self.dense = torch.from_numpy((v * gv[..., None]).reshape(rows, nb * 24)[:, :cols].copy()).cuda()
        self.words_d = torch.from_numpy(words.view(np.int64)).cuda()
        self.gains_d = torch.from_numpy(self.gains.view(np.int16)).cuda()
        import codebook_free_lattice_b200 as L
        mode = L.LLVQ_GAIN_U8_TABLE if gain == "table" else L.LLVQ_GAIN_FP16_DIRECT
        self.weight = g.weight(self.words_d, self.gains_d, rows, cols, mode, pitch)


def activate(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3))
    return z


def expected(dense, x, act="none", gated=False, bias=None, residual=None):
    """(y, worst-case error before y's rounding, its variance) in fp64."""
    x = x.double()
    z = x @ dense.t()
    mass = x.abs() @ dense.abs().t()
    var = (2.0 ** -22 / 3) * ((x ** 2) @ (dense ** 2).t())
    if bias is not None:
        z = z + bias.double()
    nk = -(-dense.shape[1] // 16)
    dz = (2.0 ** -11 + (nk + 90) * 2.0 ** -23) * mass + 2.0 ** -22 * z.abs()
    if gated:
        f = z.shape[1] // 2
        a, up = activate(z[:, :f], act), z[:, f:]
        y = a * up
        da = LIP * dz[:, :f] + 2.0 ** -20 * z[:, :f].abs()
        dy = up.abs() * da + a.abs() * dz[:, f:] + da * dz[:, f:]
        vy = up ** 2 * LIP ** 2 * var[:, :f] + a ** 2 * var[:, f:]
    else:
        y = activate(z, act)
        dy = LIP * dz + 2.0 ** -20 * z.abs()
        vy = LIP ** 2 * var
    if residual is not None:
        y = y + residual.double()
    return y, dy, vy


def check(got, y, dy, vy):
    u = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).tiny * u
    err = (got.double() - y).abs()
    bound = dy * (1 + u) + u * y.abs() + tiny
    assert bool((err <= bound).all()), f"worst error {float((err / bound).max()):.3g} of its bound"
    if y.numel() >= 400:
        rms = float(err.pow(2).mean().sqrt())
        allowed = 1.25 * float((vy + u * u / 3 * y ** 2).mean().sqrt()) + tiny
        assert rms <= allowed, f"RMS error {rms:.3g}, allowed {allowed:.3g}"


def tokens_of(seed, tokens, cols, dtype):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(tokens, cols, device="cuda", generator=g)
    x[:, torch.randint(0, cols, (1 + cols // 64,), device="cuda", generator=g)] *= 9
    return x.to(dtype)


def random(seed, shape, dtype):
    return torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(dtype)


def number(act):
    import codebook_free_lattice_b200 as L
    return getattr(L, "LLVQ_ACT_" + act.upper())


# tokens, rows, cols, dtype, act, gated, bias, residual, gain
CASES = [
    (1, 1, 1, "float16", "none", False, False, False, "table"),
    (1, 2, 24, "bfloat16", "silu", True, False, False, "table"),
    (1, 300, 1000, "float16", "none", False, False, True, "table"),
    (1, 300, 1000, "bfloat16", "gelu", False, True, True, "direct"),
    (2, 130, 2005, "float16", "silu", True, True, True, "table"),
    (3, 513, 25, "float16", "relu", False, True, False, "direct"),
    (5, 64, 23, "bfloat16", "gelu_tanh", False, False, True, "table"),
    (16, 256, 1024, "float16", "gelu_tanh", False, True, True, "table"),
    (17, 127, 999, "float16", "gelu", False, True, True, "table"),
    (32, 600, 130, "bfloat16", "silu", True, False, True, "direct"),
    (33, 258, 520, "bfloat16", "none", False, True, False, "table"),
    (64, 1026, 776, "float16", "relu", True, True, False, "table"),
    (255, 257, 320, "float16", "silu", False, False, False, "table"),
    (257, 384, 1111, "bfloat16", "gelu", True, True, True, "table"),
    (300, 5, 4000, "float16", "none", False, True, True, "direct"),
    (700, 1000, 264, "bfloat16", "relu", False, False, True, "table"),
    (1500, 520, 96, "float16", "gelu_tanh", True, False, True, "table"),
]


@pytest.mark.parametrize("tokens,rows,cols,dtype,act,gated,bias,residual,gain", CASES)
def test_linear(codecs, tokens, rows, cols, dtype, act, gated, bias, residual, gain):
    dtype = getattr(torch, dtype)
    layer = Layer(codecs, 48, rows, cols, gain, seed=tokens)
    outs = rows // 2 if gated else rows
    x = tokens_of(1, tokens, cols, dtype)
    b = random(2, (rows,), dtype) if bias else None
    r = random(3, (tokens, outs), dtype) if residual else None
    y = torch.full((tokens, outs), float("nan"), dtype=dtype, device="cuda")
    layer.codec.linear(layer.weight, x, y, bias=b, activation=number(act), gated=gated, residual=r)
    check(y, *expected(layer.dense, x, act, gated, b, r))
    assert layer.codec.get_error() == 0


def shares(kind, tokens, experts, seed):
    rng = np.random.default_rng([seed, tokens, experts])
    if kind == "one":                                  # every token to one expert
        counts = np.zeros(experts, int)
        counts[experts // 2] = tokens
    elif kind == "ends":                               # the first and the last expert have none
        counts = np.bincount(rng.integers(1, experts - 1, tokens), minlength=experts)
    elif kind == "each":                               # at most one token each
        counts = (np.arange(experts) < tokens).astype(int)
        rng.shuffle(counts)
    else:
        p = rng.exponential(1, experts) * (rng.random(experts) > 0.3) + 1e-6
        counts = np.bincount(rng.choice(experts, tokens, p=p / p.sum()), minlength=experts)
    return counts


# tokens, experts, rows, cols, dtype, act, gated, bias, residual, gain, kind, rows of x before and behind
GROUPED = [
    (1, 1, 40, 100, "float16", "none", False, True, False, "table", "uneven", 0, 0),
    (1, 7, 64, 48, "bfloat16", "silu", True, True, True, "table", "one", 0, 3),
    (9, 40, 130, 333, "float16", "gelu", False, True, True, "table", "each", 2, 1),
    (16, 64, 96, 512, "bfloat16", "silu", True, False, False, "table", "uneven", 0, 0),
    (77, 5, 331, 1000, "float16", "gelu", False, True, True, "direct", "ends", 0, 19),
    (300, 3, 258, 200, "bfloat16", "relu", False, False, True, "table", "one", 5, 0),
    (700, 9, 514, 130, "float16", "gelu_tanh", True, True, True, "table", "uneven", 1, 40),
    (1200, 33, 70, 72, "bfloat16", "none", False, True, False, "direct", "uneven", 0, 8),
    (600, 700, 24, 50, "float16", "relu", False, False, False, "table", "uneven", 0, 0),
]


def grouped_case(codecs, bits, tokens, experts, rows, cols, dtype, act, gated, bias, residual, gain, kind, before, behind):
    dtype = getattr(torch, dtype)
    layer = Layer(codecs, bits, experts * rows, cols, gain, seed=tokens)
    outs, room = rows // 2 if gated else rows, before + tokens + behind
    counts = shares(kind, tokens, experts, 5)
    edges = np.concatenate(([0], np.cumsum(counts))) + before
    x = tokens_of(1, room, cols, dtype)
    x[:before], x[room - behind:] = float("nan"), float("nan")
    b = random(2, (experts, rows), dtype) if bias else None
    r = random(3, (room, outs), dtype) if residual else None
    y = random(4, (room, outs), dtype)
    kept = y.clone()
    layer.codec.linear_grouped(layer.weight, experts, x, torch.tensor(edges, dtype=torch.int32, device="cuda"), y,
                               bias=b, activation=number(act), gated=gated, residual=r)
    parts = []
    for e in range(experts):
        lo, hi = edges[e], edges[e + 1]
        if lo < hi:
            parts.append(expected(layer.dense[e * rows:(e + 1) * rows], x[lo:hi], act, gated,
                                  None if b is None else b[e], None if r is None else r[lo:hi]))
    check(y[before:before + tokens], *(torch.cat(t) for t in zip(*parts)))
    assert torch.equal(y[:before], kept[:before]) and torch.equal(y[before + tokens:], kept[before + tokens:])
    assert layer.codec.get_error() == 0


@pytest.mark.parametrize("tokens,experts,rows,cols,dtype,act,gated,bias,residual,gain,kind,before,behind", GROUPED)
def test_grouped(codecs, tokens, experts, rows, cols, dtype, act, gated, bias, residual, gain, kind, before, behind):
    grouped_case(codecs, 48, tokens, experts, rows, cols, dtype, act, gated, bias, residual, gain, kind, before, behind)
