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
    (1, 50, 24001, "bfloat16", "silu", True, True, True, "table"),
    (2, 33, 30000, "float16", "none", False, False, True, "direct"),
    (3, 20, 30000, "bfloat16", "none", False, True, False, "table"),
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
    (16, 70, 34, 2500, "float16", "silu", True, True, True, "table", "uneven", 0, 0),
    (4, 12, 20, 19001, "bfloat16", "gelu", False, False, False, "direct", "uneven", 4, 7),
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


# ---- larger budgets ------------------------------------------------------------------------------
@pytest.mark.parametrize("tokens,rows,cols,dtype,gated,gain", [
    (1, 70, 500, "bfloat16", True, "table"), (3, 130, 96, "float16", False, "direct"), (40, 200, 1000, "float16", True, "table"),
    (300, 129, 250, "bfloat16", False, "direct")])
def test_72_bits(codecs, tokens, rows, cols, dtype, gated, gain):
    dtype = getattr(torch, dtype)
    layer = Layer(codecs, 72, rows, cols, gain, seed=tokens)
    x = tokens_of(1, tokens, cols, dtype)
    y = torch.empty(tokens, rows // 2 if gated else rows, dtype=dtype, device="cuda")
    layer.codec.linear(layer.weight, x, y, activation=number("silu"), gated=gated)
    check(y, *expected(layer.dense, x, "silu", gated))
    assert layer.codec.get_error() == 0


def test_72_bits_grouped(codecs):
    grouped_case(codecs, 72, 90, 6, 66, 180, "float16", "gelu", True, True, True, "table", "uneven", 3, 4)
    grouped_case(codecs, 72, 4, 9, 40, 100, "bfloat16", "none", False, True, False, "table", "uneven", 0, 0)


def test_96_bits(codecs):
    """One codec (its tables take seconds and 23.6 GB), both forms, both gain modes, groups."""
    for tokens, gain, dtype in ((2, "table", torch.float16), (50, "direct", torch.bfloat16)):
        layer = Layer(codecs, 96, 130, 300, gain, seed=tokens)
        x = tokens_of(1, tokens, 300, dtype)
        y = torch.empty(tokens, 65, dtype=dtype, device="cuda")
        layer.codec.linear(layer.weight, x, y, activation=number("gelu_tanh"), gated=True)
        check(y, *expected(layer.dense, x, "gelu_tanh", True))
    grouped_case(codecs, 96, 60, 5, 40, 100, "float16", "relu", False, True, True, "table", "uneven", 2, 3)
    layer.codec.close()


# ---- layouts -------------------------------------------------------------------------------------
@pytest.mark.parametrize("tokens", (1, 2, 33, 300))
@pytest.mark.parametrize("dtype", ("float16", "bfloat16"))
def test_strides_and_addresses(codecs, tokens, dtype):
    """x, residual and y as columns of wider matrices, at odd addresses; words with a pitch."""
    dtype = getattr(torch, dtype)
    layer = Layer(codecs, 48, 90, 203, pitch=13, seed=tokens)
    wide = tokens_of(1, tokens, 350, dtype)
    for at, width in ((0, 350), (1, 350), (2, 350), (8, 344)):
        x = wide[:, :width][:, at:at + 203]
        out = random(5, (tokens, 101), dtype)
        kept, r = out.clone(), random(6, (tokens, 97), dtype)
        y = out[:, 3:93]
        layer.codec.linear(layer.weight, x, y, residual=r[:, 5:95], activation=number("silu"))
        check(y.contiguous(), *expected(layer.dense, x, "silu", residual=r[:, 5:95]))
        assert torch.equal(out[:, :3], kept[:, :3]) and torch.equal(out[:, 93:], kept[:, 93:])


@pytest.mark.parametrize("tokens,cols,dtype,grouped", [
    (2100, 1001, "bfloat16", False), (2200, 1000, "bfloat16", True), (2200, 999, "float16", False), (70, 33000, "bfloat16", False)])
def test_many_values_restated(codecs, tokens, cols, dtype, grouped):
    """Enough activations for the kernel that restates them by itself; rows beyond what its threads hold, too."""
    dtype = getattr(torch, dtype)
    layer = Layer(codecs, 48, 48, cols, seed=7)
    x = tokens_of(3, tokens, cols, dtype)
    x = (x.double() * torch.tensor([1.0, 2.0 ** -60 if dtype is torch.bfloat16 else 2.0 ** -6], device="cuda", dtype=torch.float64)
         [torch.arange(tokens, device="cuda") % 2, None]).to(dtype)
    if grouped:
        x[:30], x[-40:] = float("nan"), float("inf")
        edges = [30, 700, 700, tokens - 40]
        y = random(1, (tokens, 16), dtype)
        kept = y.clone()
        layer.codec.linear_grouped(layer.weight, 3, x, torch.tensor(edges, dtype=torch.int32, device="cuda"), y)
        parts = [expected(layer.dense[16 * e:16 * e + 16], x[edges[e]:edges[e + 1]]) for e in (0, 2)]
        want = [torch.cat(t) for t in zip(*parts)]
        assert torch.equal(y[:30], kept[:30]) and torch.equal(y[-40:], kept[-40:])
        y = y[30:-40]
    else:
        y = torch.empty(tokens, 48, dtype=dtype, device="cuda")
        layer.codec.linear(layer.weight, x, y)
        want = expected(layer.dense, x)
    for k in range(2):
        check(y[k::2].contiguous(), *(t[k::2] for t in want))
    assert layer.codec.get_error() == 0


@pytest.mark.parametrize("tokens", (1, 64, 400))
@pytest.mark.parametrize("gated", (False, True))
def test_residual_in_place_and_broadcast(codecs, tokens, gated):
    layer = Layer(codecs, 48, 260, 192, seed=3)
    outs = 130 if gated else 260
    x = tokens_of(1, tokens, 192, torch.float16)
    y = random(2, (tokens, outs), torch.float16)
    want = expected(layer.dense, x, "silu", gated, residual=y.clone())
    layer.codec.linear(layer.weight, x, y, activation=number("silu"), gated=gated, residual=y)
    check(y, *want)
    row = random(4, (outs,), torch.float16)
    layer.codec.linear(layer.weight, x, y, activation=number("silu"), gated=gated, residual=row)
    check(y, *expected(layer.dense, x, "silu", gated, residual=row[None].expand(tokens, outs)))


# ---- values --------------------------------------------------------------------------------------
@pytest.mark.parametrize("tokens", (2, 40))
@pytest.mark.parametrize("gain", ("table", "direct"))
def test_rows_of_very_different_scales(codecs, tokens, gain):
    """Rows whose gains are near fp16's subnormals, ordinary and near its largest values: no row loses precision to
    another, and none overflows before the output does."""
    rows = 66
    scale = np.array([[2.0 ** -9, 1.0, 2.0 ** 9][r % 3] for r in range(rows)])
    layer = Layer(codecs, 48, rows, 240, gain, seed=1, scale=scale)
    x = tokens_of(1, tokens, 240, torch.bfloat16)
    y = torch.empty(tokens, rows, dtype=torch.bfloat16, device="cuda")
    layer.codec.linear(layer.weight, x, y)
    want = expected(layer.dense, x)
    for k in range(3):                                  # each scale by itself, or the largest hides the others
        check(y[:, k::3].contiguous(), *(t[:, k::3] for t in want))


@pytest.mark.parametrize("tokens", (3, 70))
def test_bf16_range(codecs, tokens):
    """Tokens of 2^-120, 1, 2^100 and with subnormals: the restatement in fp16 keeps every one of them."""
    layer = Layer(codecs, 48, 96, 120, seed=2)
    x = tokens_of(1, tokens, 120, torch.bfloat16)
    x = (x.double() * torch.tensor([2.0 ** -120, 1.0, 2.0 ** 100], device="cuda", dtype=torch.float64)
         [torch.arange(tokens, device="cuda") % 3, None]).to(torch.bfloat16)
    x[0, :60] = 2.0 ** -133
    y = torch.empty(tokens, 96, dtype=torch.bfloat16, device="cuda")
    layer.codec.linear(layer.weight, x, y)
    want = expected(layer.dense, x)
    for k in range(3):
        check(y[k::3].contiguous(), *(t[k::3] for t in want))


@pytest.mark.parametrize("tokens", (3, 40))
@pytest.mark.parametrize("dtype", ("float16", "bfloat16"))
def test_infinities_and_nan_stay_where_they_are(codecs, tokens, dtype):
    """A NaN or an infinity in one token or in one row's gains reaches that token's or that row's outputs only."""
    dtype = getattr(torch, dtype)
    layer = Layer(codecs, 48, 130, 150, seed=4)
    x = tokens_of(1, tokens, 150, dtype)
    y, z = (torch.empty(tokens, 130, dtype=dtype, device="cuda") for _ in range(2))
    layer.codec.linear(layer.weight, x, y)
    x[1, 7], x[2, 3] = float("nan"), float("inf")
    layer.codec.linear(layer.weight, x, z)
    assert bool(torch.isnan(z[1]).all())
    hit = layer.dense[:, 3] != 0
    assert bool((z[2, hit] == torch.sign(layer.dense[hit, 3]).to(dtype) * float("inf")).all()) and bool(torch.isnan(z[2, ~hit]).all())
    rest = [t for t in range(tokens) if t not in (1, 2)]
    assert torch.equal(z[rest], y[rest])
    layer.gains_d.view(torch.float16)[5] = float("nan")
    layer.codec.linear(layer.weight, tokens_of(1, tokens, 150, dtype), z)
    others = [r for r in range(130) if r != 5]
    assert bool(torch.isnan(z[:, 5]).all()) and torch.equal(z[:, others], y[:, others])


@pytest.mark.parametrize("tokens", (2, 30))
def test_zero_gains_and_uncoded_indices(codecs, tokens):
    import codebook_free_lattice_b200 as L
    layer = Layer(codecs, 48, 40, 100, seed=5, bad=20)
    layer.gains_d.view(torch.float16)[7] = 0
    layer.dense[7] = 0
    b = random(1, (40,), torch.float16)
    x = tokens_of(1, tokens, 100, torch.float16)
    y = torch.empty(tokens, 40, dtype=torch.float16, device="cuda")
    layer.codec.get_error()
    layer.codec.linear(layer.weight, x, y, bias=b)
    check(y, *expected(layer.dense, x, bias=b))
    assert torch.equal(y[:, 7], b[7].expand(tokens))
    assert layer.codec.get_error() == L.LLVQ_FLAG_INDEX_RANGE


def test_rare_classes_only(codecs):
    """Every block from the classes that neither fast decode takes (odd with five magnitudes, even off the tables):
    more than the list that keeps them holds."""
    g, o = codecs(48)
    rare, start = [], 0
    for c in o.classes():
        off_tables = not c.odd and c.k not in (8, 12, 16)
        if (c.odd and len(c.vals) > 4) or off_tables:
            rare.append((start, c.size))
        start += c.size
    assert len(rare) > 5
    rng = np.random.default_rng(1)
    rows, nb = 200, 40
    pick = rng.integers(0, len(rare), rows * nb)
    lo = np.array([rare[k][0] + int(rng.integers(0, rare[k][1])) for k in pick], np.uint64)
    gains = (rng.uniform(0.5, 1, (rows, nb)) / 14 / np.sqrt(nb)).astype(np.float16)
    dense = torch.from_numpy((o.decode_batch(lo).astype(np.float64).reshape(rows, nb, 24) * gains.astype(np.float64)[..., None])
                             .reshape(rows, nb * 24)).cuda()
    words, gd = torch.from_numpy(lo.view(np.int64)).cuda(), torch.from_numpy(gains.view(np.int16)).cuda()
    import codebook_free_lattice_b200 as L
    w = g.weight(words, gd, rows, nb * 24, L.LLVQ_GAIN_FP16_DIRECT)
    for tokens in (1, 20):
        x = tokens_of(1, tokens, nb * 24, torch.float16)
        y = torch.empty(tokens, rows, dtype=torch.float16, device="cuda")
        g.linear(w, x, y)
        check(y, *expected(dense, x))


# ---- groups --------------------------------------------------------------------------------------
@pytest.mark.parametrize("tokens", (6, 60))
@pytest.mark.parametrize("bad", ([0, 3, 2, 6], [-1, 2, 4, 6], [0, 2, 4, 61], [5, 0, 0, 0]))
def test_offsets_out_of_order_write_nothing(codecs, tokens, bad):
    import codebook_free_lattice_b200 as L
    layer = Layer(codecs, 48, 3 * 32, 72, seed=6)
    x = tokens_of(1, tokens, 72, torch.float16)
    y = random(1, (tokens, 32), torch.float16)
    kept = y.clone()
    layer.codec.get_error()
    layer.codec.linear_grouped(layer.weight, 3, x, torch.tensor(bad, dtype=torch.int32, device="cuda"), y)
    assert layer.codec.get_error() == L.LLVQ_FLAG_OFFSETS
    assert torch.equal(y, kept)


@pytest.mark.parametrize("tokens", (4, 50))
def test_no_tokens_in_any_group(codecs, tokens):
    layer = Layer(codecs, 48, 3 * 32, 72, seed=6)
    x, y = tokens_of(1, tokens, 72, torch.float16), random(1, (tokens, 32), torch.float16)
    kept = y.clone()
    layer.codec.linear_grouped(layer.weight, 3, x, torch.full((4,), 2, dtype=torch.int32, device="cuda"), y)
    assert torch.equal(y, kept) and layer.codec.get_error() == 0
    layer.codec.linear(Layer(codecs, 48, 32, 72).weight, x[:0], y[:0])


def test_groups_equal_their_layers(codecs):
    """A group's outputs are those of a layer of its own over its own tokens: the same weights, the same sums."""
    layer = Layer(codecs, 48, 4 * 96, 400, seed=8)
    counts = [40, 0, 7, 81]
    edges = np.concatenate(([0], np.cumsum(counts)))
    x = tokens_of(1, 128, 400, torch.bfloat16)
    y = torch.empty(128, 96, dtype=torch.bfloat16, device="cuda")
    layer.codec.linear_grouped(layer.weight, 4, x, torch.tensor(edges, dtype=torch.int32, device="cuda"), y, activation=number("silu"))
    nb = -(-400 // 24)
    for e in range(4):
        if counts[e]:
            w = layer.codec.weight(layer.words_d[e * 96 * nb:], layer.gains_d[e * 96:], 96, 400, 1)
            own = torch.empty(counts[e], 96, dtype=torch.bfloat16, device="cuda")
            layer.codec.linear(w, x[edges[e]:edges[e + 1]], own, activation=number("silu"))
            # the two may split K differently: equal up to the order of fp32 sums
            assert float((own.double() - y[edges[e]:edges[e + 1]].double()).norm() / own.double().norm()) < 2.0 ** -8


# ---- streams, graphs, workspaces -----------------------------------------------------------------
@pytest.mark.parametrize("tokens", (1, 48, 600))
def test_same_results_every_time(codecs, tokens):
    layer = Layer(codecs, 48, 700, 1500, seed=9)
    x = tokens_of(1, tokens, 1500, torch.float16)
    first = torch.empty(tokens, 700, dtype=torch.float16, device="cuda")
    ws = layer.codec.linear(layer.weight, x, first)
    for _ in range(20):
        ws.fill_(0xFF)                                 # nothing of an earlier call is used
        y = torch.empty_like(first)
        assert layer.codec.linear(layer.weight, x, y, workspace=ws) is ws
        assert torch.equal(y, first)


def test_two_streams_at_once(codecs):
    layer = Layer(codecs, 48, 600, 900, seed=10)
    xs = [tokens_of(k, n, 900, torch.bfloat16) for k, n in ((1, 1), (2, 200))]
    want = []
    for x in xs:
        y = torch.empty(x.shape[0], 600, dtype=torch.bfloat16, device="cuda")
        layer.codec.linear(layer.weight, x, y)
        want.append(y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got, ws = [[], []], [None, None]
    for _ in range(10):
        for k, (x, s) in enumerate(zip(xs, streams)):
            y = torch.full_like(want[k], float("nan"))
            s.wait_stream(torch.cuda.current_stream())
            ws[k] = layer.codec.linear(layer.weight, x, y, workspace=ws[k], stream=s)
            got[k].append(y)
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(y, want[k]) for y in got[k])


@pytest.mark.parametrize("tokens,experts", ((1, 0), (40, 0), (6, 8), (90, 4)))
def test_captured_and_replayed(codecs, tokens, experts):
    """A captured call, replayed with other activations and other offsets in the same buffers."""
    rows, cols = 96, 360
    layer = Layer(codecs, 48, max(experts, 1) * rows, cols, seed=11)
    x = tokens_of(1, tokens, cols, torch.float16)
    y = torch.empty(tokens, rows, dtype=torch.float16, device="cuda")
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")

    def run(ws=None):
        if experts:
            return layer.codec.linear_grouped(layer.weight, experts, x, offsets, y, activation=number("gelu"), workspace=ws)
        return layer.codec.linear(layer.weight, x, y, activation=number("gelu"), workspace=ws)

    ws = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(ws)
    for seed in (2, 3, 4):
        x.copy_(tokens_of(seed, tokens, cols, torch.float16))
        counts = shares("uneven", tokens, experts, seed) if experts else [tokens]
        edges = np.concatenate(([0], np.cumsum(counts)))
        if experts:
            offsets.copy_(torch.tensor(edges, dtype=torch.int32))
        graph.replay()
        parts = [expected(layer.dense[e * rows:(e + 1) * rows], x[edges[e]:edges[e + 1]], "gelu")
                 for e in range(len(counts)) if counts[e]]
        check(y, *(torch.cat(t) for t in zip(*parts)))


@pytest.mark.parametrize("tokens", (1, 30))
def test_waits_give_up_then_recover(codecs, tokens):
    """The table copy's and the product's bounded waits, made to give up at once: the flag is raised, the kernels
    return, and the next call is right."""
    import codebook_free_lattice_b200 as L
    layer = Layer(codecs, 48, 512, 480, seed=12)
    g = layer.codec
    x = tokens_of(1, tokens, 480, torch.float16)
    y = torch.empty(tokens, 512, dtype=torch.float16, device="cuda")
    g.get_error()
    for polls in ((0, 0xFFFFFFFF),) if tokens == 1 else ((0, 0xFFFFFFFF), (0xFFFFFFFF, 0)):
        L.llvq_set_wait_polls(*polls)
        try:
            g.linear(layer.weight, x, y)
            assert g.get_error() == L.LLVQ_FLAG_WAIT_TIMEOUT
        finally:
            L.llvq_set_wait_polls()
        g.linear(layer.weight, x, y)
        check(y, *expected(layer.dense, x))
        assert g.get_error() == 0


# ---- a run of them -------------------------------------------------------------------------------
@pytest.mark.parametrize("tokens", (1, 5, 130))
def test_feed_forward_blocks_in_a_row(codecs, tokens):
    """A dense gated feed-forward block (gate and up, then down onto the stream in place), then one over experts with
    two experts per token: the tokens sorted by expert, both products grouped, the weighted sum."""
    g, _ = codecs(48)
    width, inner, experts, dtype = 240, 336, 6, torch.bfloat16
    up, down = Layer(codecs, 48, 2 * inner, width, seed=1), Layer(codecs, 48, width, inner, seed=2)
    ups = Layer(codecs, 48, experts * 2 * inner, width, seed=3)
    downs = Layer(codecs, 48, experts * width, inner, seed=4)
    x = tokens_of(1, tokens, width, dtype)
    x = x / x.double().norm(dim=1, keepdim=True).to(dtype) * 15
    stream, silu = x.clone(), number("silu")
    h = torch.empty(tokens, inner, dtype=dtype, device="cuda")
    ws = g.linear(up.weight, stream, h, activation=silu, gated=True)
    ws = g.linear(down.weight, h, stream, residual=stream, workspace=ws)
    score = random(7, (tokens, experts), torch.float32)
    top, chosen = score.softmax(1).topk(2, 1)
    order = chosen.reshape(-1).argsort(stable=True)
    offsets = torch.cat((torch.zeros(1, device="cuda"), chosen.reshape(-1).bincount(minlength=experts).cumsum(0))).int()
    xe = stream[order // 2]
    he = torch.empty(2 * tokens, inner, dtype=dtype, device="cuda")
    ye = torch.empty(2 * tokens, width, dtype=dtype, device="cuda")
    ws = g.linear_grouped(ups.weight, experts, xe, offsets, he, activation=silu, gated=True, workspace=ws)
    ws = g.linear_grouped(downs.weight, experts, he, offsets, ye, workspace=ws)
    back = torch.empty_like(ye)
    back[order] = ye
    out = stream + (back.reshape(tokens, 2, width) * top.to(dtype)[..., None]).sum(1)
    assert g.get_error() == 0

    def mlp(u, d, v):
        z = v @ u.t()
        return (activate(z[:, :inner], "silu") * z[:, inner:]) @ d.t()

    want = x.double() + mlp(up.dense, down.dense, x.double())
    dense = want.clone()
    for e in range(experts):
        part = mlp(ups.dense[2 * e * inner:2 * (e + 1) * inner], downs.dense[e * width:(e + 1) * width], dense)
        want += part * torch.where(chosen == e, top, 0).sum(1, keepdim=True).double()
    # six roundings to bf16 follow one another (h, stream, he, ye, their product, the sum), each off by at most
    # 2^-8 of values no larger than a few times the result, and partly independent: 6 2^-8
    assert float((out.double() - want).norm() / want.norm()) < 6 * 2.0 ** -8
