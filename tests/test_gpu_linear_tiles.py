"""Layers of the sizes at which the product takes its large tiles, several per pair of CTAs, in bands of row tiles, with the
last ones split (test_linear_tiles.py shows that they do), against the definition in 64 bits."""
import pytest

from tests.test_gpu_linear import Layer, check, codecs, expected, number, random, tokens_of  # noqa: F401
from tests.test_linear_tiles import TILES

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("tokens,rows,cols,dtype,act,gated,bias,residual", TILES)
def test_large_tiles(codecs, tokens, rows, cols, dtype, act, gated, bias, residual):
    dtype = getattr(torch, dtype)
    experts, before, behind = len(tokens), 5, 9
    layer = Layer(codecs, 48, experts * rows, cols, seed=3)
    outs, room = rows // 2 if gated else rows, before + sum(tokens) + behind
    x = tokens_of(1, room, cols, dtype)
    b = random(2, (experts, rows), dtype) if bias else None
    r = random(3, (room, outs), dtype) if residual else None
    y = random(4, (room, outs), dtype)
    kept = y.clone()
    edges = [before + sum(tokens[:e]) for e in range(experts + 1)]
    if experts > 1:
        x[:before], x[room - behind:] = float("nan"), float("inf")
        layer.codec.linear_grouped(layer.weight, experts, x, torch.tensor(edges, dtype=torch.int32, device="cuda"), y, bias=b,
                                   activation=number(act), gated=gated, residual=r)
    else:
        used = slice(before, room - behind)
        layer.codec.linear(layer.weight, x[used], y[used], bias=b, activation=number(act), gated=gated,
                           residual=None if r is None else r[used])
    assert layer.codec.get_error() == 0
    for e in range(experts):
        lo, hi = edges[e], edges[e + 1]
        if lo < hi:
            check(y[lo:hi], *expected(layer.dense[e * rows:(e + 1) * rows], x[lo:hi], act, gated, None if b is None else b[e],
                                      None if r is None else r[lo:hi]))
    assert torch.equal(y[:before], kept[:before]) and torch.equal(y[room - behind:], kept[room - behind:])
