"""The product's bounded waits made to give up while copies and products are under way: the kernel ends, says so, leaves
nothing behind (no copy, no tensor memory), and the next call has the same results as the first."""
import pytest

from tests.test_gpu_linear import Layer, codecs, tokens_of  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


# few long tiles split over the pairs; several tiles per pair, each longer than the fewest polls last
@pytest.mark.parametrize("tokens,rows,cols,dtype,gated", [
    (40, 600, 24000, "float16", False), (20, 130, 40000, "float16", True), (700, 4500, 6000, "bfloat16", False)])
def test_waits_that_give_up_under_way(codecs, tokens, rows, cols, dtype, gated):
    import codebook_free_lattice_b200 as L
    dtype = getattr(torch, dtype)
    layer = Layer(codecs, 48, rows, cols, seed=1)
    x = tokens_of(1, tokens, cols, dtype)
    outs = rows // 2 if gated else rows
    first = torch.empty(tokens, outs, dtype=dtype, device="cuda")
    ws = layer.codec.linear(layer.weight, x, first, gated=gated)
    assert layer.codec.get_error() == 0
    gave_up = 0
    for polls in (1, 2, 4, 0):
        for _ in range(3):
            L.llvq_set_wait_polls(0xFFFFFFFF, polls)
            try:
                y = torch.empty_like(first)
                layer.codec.linear(layer.weight, x, y, gated=gated, workspace=ws)
                flags = layer.codec.get_error()
            finally:
                L.llvq_set_wait_polls()
            assert flags in (0, L.LLVQ_FLAG_WAIT_TIMEOUT)
            gave_up += flags != 0
            assert flags or torch.equal(y, first)
            y = torch.empty_like(first)
            layer.codec.linear(layer.weight, x, y, gated=gated, workspace=ws)
            assert layer.codec.get_error() == 0 and torch.equal(y, first)
    assert gave_up >= 3                                # no polls at all cannot succeed
