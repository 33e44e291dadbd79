"""How near the linear layers come to the definition in 64 bits where a bound per output (test_gpu_linear.py) does not
show it: the precision of gated layers, the tails of the activations, infinite gains."""
import pytest

from tests.test_gpu_linear import Layer, activate, codecs, number, random, shares, tokens_of  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def rms(v):
    return float(v.double().pow(2).mean().sqrt())


def definition(layer, x, act, rows=None):
    z = x.double() @ (layer.dense if rows is None else layer.dense[rows]).t()
    half = z.shape[1] // 2
    return activate(z[:, :half], act) * z[:, half:]


# The output's own rounding is the yardstick: its RMS error is measured on the same outputs.  The weights' 22 bits are
# off by 2^-21 at most, which is nothing beside it.  What is left are the fp32 sums: each of the at most 2 x 63 steps
# of 16 columns (1000 columns, two parts) takes at most 2^-23 of the running sum, so each of the two sums is off by
# 2^-16, their product by 2^-15.5 = 2.2e-5, a tenth of the rounding's 2e-4; independent of it, that adds less than 1%.
# Weights of 11 bits would give 1.7.
MARGIN = 1.05


@pytest.mark.parametrize("bits,tokens,rows,cols,act,gain", [
    (48, 6, 600, 700, "silu", "table"), (48, 7, 600, 700, "silu", "table"), (48, 40, 300, 1000, "silu", "direct"), (48, 300, 520, 480, "gelu_tanh", "table"),
    (72, 50, 130, 300, "none", "table")])
def test_gated_fp16_is_as_good_as_its_rounding(codecs, bits, tokens, rows, cols, act, gain):
    layer = Layer(codecs, bits, rows, cols, gain, seed=tokens)
    x = tokens_of(1, tokens, cols, torch.float16)
    y = torch.empty(tokens, rows // 2, dtype=torch.float16, device="cuda")
    layer.codec.linear(layer.weight, x, y, activation=number(act), gated=True)
    want = definition(layer, x, act)
    assert rms(y - want) <= MARGIN * rms(want.half() - want)
    assert layer.codec.get_error() == 0


def test_gated_fp16_experts_are_as_good_as_their_rounding(codecs):
    experts, rows, cols, tokens = 4, 264, 400, 90
    layer = Layer(codecs, 48, experts * rows, cols, "table", seed=3)
    x = tokens_of(1, tokens, cols, torch.float16)
    y = torch.empty(tokens, rows // 2, dtype=torch.float16, device="cuda")
    counts = shares("uneven", tokens, experts, 5).tolist()
    edges = [sum(counts[:e]) for e in range(experts + 1)]
    layer.codec.linear_grouped(layer.weight, experts, x, torch.tensor(edges, dtype=torch.int32, device="cuda"), y,
                               activation=number("silu"), gated=True)
    want = torch.cat([definition(layer, x[edges[e]:edges[e + 1]], "silu", slice(e * rows, (e + 1) * rows)) for e in range(experts)])
    assert rms(y - want) <= MARGIN * rms(want.half() - want)
    assert layer.codec.get_error() == 0


@pytest.mark.parametrize("gain", ("table", "direct"))
@pytest.mark.parametrize("tokens,cols", ((40, 150), (600, 4001)))
def test_infinities_in_a_gated_fp16_layer(codecs, tokens, cols, gain):
    """Where the definition has an infinity, a NaN or a number, so has the layer: x with infinities and a NaN, a row
    with a NaN among its gains (its last block, beyond whose columns the layer has none)."""
    layer = Layer(codecs, 48, 130, cols, gain, seed=4)
    x = tokens_of(1, tokens, cols, torch.float16)
    x[1, 7], x[2, 3], x[3, cols - 1] = float("nan"), float("inf"), -float("inf")
    y = torch.empty(tokens, 65, dtype=torch.float16, device="cuda")
    layer.codec.linear(layer.weight, x, y, gated=True)
    want = definition(layer, x, "none")
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.isinf(), want.isinf())
    assert torch.equal(y[want.isinf()] > 0, want[want.isinf()] > 0)
    assert bool(want.isinf().any()) and layer.codec.get_error() == 0
    g = layer.gains_d.view(torch.float16)
    g[5] = float("nan")
    x = tokens_of(1, tokens, cols, torch.float16)
    layer.codec.linear(layer.weight, x, y, gated=True)
    assert bool(y[:, 5].isnan().all()) and int(y.isnan().sum()) == tokens


@pytest.mark.parametrize("gain", ("table", "direct"))
@pytest.mark.parametrize("tokens,dtype,gated", ((2, "float16", False), (40, "float16", False), (40, "bfloat16", False), (40, "float16", True)))
def test_infinite_gains(codecs, tokens, dtype, gated, gain):
    """A row with an infinite gain at one block: the layer has an infinity where the definition has one (the products
    of the block all of one sign), of the same sign, and a NaN where it has one."""
    dtype = getattr(torch, dtype)
    layer = Layer(codecs, 48, 64, 60, gain, seed=9)         # 2.5 blocks per row
    row = next(r for r in range(32) if bool((layer.dense[r, :24] != 0).all()))       # an odd block: no coordinate is zero
    x = tokens_of(1, tokens, 60, dtype)
    sign = torch.sign(layer.dense[row, :24]).to(dtype)
    x[0, :24], x[1, :24] = sign * x[0, :24].abs(), -sign * x[1, :24].abs()
    infinite = torch.zeros(64, 60, dtype=torch.float64, device="cuda")
    g = layer.gains_d.view(torch.float16)
    if gain == "direct":
        g[row, 0] = float("inf")
    else:
        code = int(layer.words_d.reshape(64, -1)[row, 0] >> 48) & 255
        g[row, code] = float("inf")
        assert all(int(w >> 48) & 255 != code for w in layer.words_d.reshape(64, -1)[row, 1:])
    infinite[row, :24] = float("inf")
    layer.dense = torch.where(infinite > 0, torch.sign(layer.dense) * infinite, layer.dense)
    y = torch.empty(tokens, 32 if gated else 64, dtype=dtype, device="cuda")
    layer.codec.linear(layer.weight, x, y, gated=gated)
    want = definition(layer, x, "none") if gated else x.double() @ layer.dense.t()
    assert bool(want[:2, row].isinf().all())
    finite = want.isfinite()
    assert torch.equal(y.isfinite(), finite)
    some = want.isinf()
    assert torch.equal(y[some].double(), want[some])


@pytest.mark.parametrize("dtype", ("float16", "bfloat16"))
@pytest.mark.parametrize("tokens", (1, 40))
@pytest.mark.parametrize("gated", (False, True))
@pytest.mark.parametrize("act,low", (("silu", -88.0), ("gelu_tanh", -9.75), ("gelu", -12.5)))
def test_tails_of_the_activations(codecs, act, low, gated, tokens, dtype):
    """z from the bias alone (every gain is zero), so that it is exact: the activation is as good as its rounding, relative
    to its value, as far as the type goes; a gated layer's factor of 512 brings more of an fp16 tail back.

    The evaluation, with fp32's half step h = 2^-24 and |u| <= 88.5 the exponent: the exponential is off by 2 h (2 + 1.16
    |u|) <= 2^-16.2; its argument's three roundings by 3 h |u| <= 2^-15.9 more (gelu: erfc by 8 h, and its argument's by
    2 h z^2 / 2 <= 2^-16.7); the rest are a few h.  Together below 2^-14.9; 2^-14 is allowed."""
    dtype = getattr(torch, dtype)
    values = 400
    layer = Layer(codecs, 48, values * (2 if gated else 1), 30, seed=1)
    layer.gains_d.zero_()
    z = torch.linspace(low, 8, values, device="cuda").to(dtype)
    bias = torch.cat((z, torch.full_like(z, 512))) if gated else z
    x = tokens_of(1, tokens, 30, dtype)
    y = torch.empty(tokens, values, dtype=dtype, device="cuda")
    layer.codec.linear(layer.weight, x, y, bias=bias, activation=number(act), gated=gated)
    # (1 + erf) / 2, or ndtr where it is computed so, has no tail in 64 bits either; erfc has
    want = z.double() * torch.special.erfc(z.double() / -2 ** 0.5) / 2 if act == "gelu" else activate(z.double(), act)
    want *= 512 if gated else 1
    u = torch.finfo(dtype).eps / 2
    err = (y.double() - want).abs()
    bound = (u + 2.0 ** -14) * want.abs() + torch.finfo(dtype).tiny * u
    assert bool((err <= bound).all()), f"worst error {float((err / bound).max()):.3g} of its bound at z = {float(z[(err / bound).amax(0).argmax()])}"


def test_uncoded_indices_in_a_gated_fp16_layer(codecs):
    """They contribute nothing to either part of a weight, whatever the workspace held."""
    import codebook_free_lattice_b200 as L
    layer = Layer(codecs, 48, 40, 100, seed=5, bad=20)
    layer.gains_d.view(torch.float16)[7] = 0
    layer.dense[7] = 0
    x = tokens_of(1, 30, 100, torch.float16)
    y = torch.empty(30, 20, dtype=torch.float16, device="cuda")
    layer.codec.get_error()
    ws = layer.codec.linear(layer.weight, x, y, gated=True)
    ws.fill_(0xFF)
    layer.codec.linear(layer.weight, x, y, gated=True, workspace=ws)
    want = definition(layer, x, "none")
    assert rms(y - want) <= MARGIN * rms(want.half() - want) and bool((y[:, 7] == 0).all())
    assert layer.codec.get_error() == L.LLVQ_FLAG_INDEX_RANGE
