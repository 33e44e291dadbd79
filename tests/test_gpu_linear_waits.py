"""The product's bounded waits made to give up while copies and products are under way: the kernel ends, says so, leaves
nothing behind (no copy, no tensor memory), and the next call has the same results as the first."""
import pytest

from tests.test_gpu_linear import codecs, tokens_of  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


# Long tiles split over the pairs; several tiles per pair; and four per pair, each longer than the fewest polls last, so
# that the epilogue of the first gives up while the later ones are loaded and multiplied.
@pytest.mark.parametrize("tokens,rows,cols,dtype,gated", [
    (40, 600, 24000, "float16", False), (20, 130, 40000, "float16", True), (700, 4500, 6000, "bfloat16", False),
    (64, 75776, 12000, "bfloat16", False)])
def test_waits_that_give_up_under_way(codecs, tokens, rows, cols, dtype, gated):
    import codebook_free_lattice_b200 as L
    dtype = getattr(torch, dtype)
    codec, _ = codecs(48)
    g = torch.Generator("cuda").manual_seed(1)
    words = torch.randint(0, 1 << 40, (rows, -(-cols // 24)), device="cuda", generator=g)
    gains = torch.rand(rows, 256, device="cuda", generator=g).half()
    w = codec.weight(words, gains, rows, cols, L.LLVQ_GAIN_U8_TABLE)
    x = tokens_of(1, tokens, cols, dtype)
    outs = rows // 2 if gated else rows
    first = torch.empty(tokens, outs, dtype=dtype, device="cuda")
    ws = codec.linear(w, x, first, gated=gated)
    assert codec.get_error() == 0
    gave_up = 0
    for polls in (1, 2, 4, 0):
        for _ in range(3):
            L.llvq_set_wait_polls(0xFFFFFFFF, polls)
            try:
                y = torch.empty_like(first)
                codec.linear(w, x, y, gated=gated, workspace=ws)
                flags = codec.get_error()
            finally:
                L.llvq_set_wait_polls()
            assert flags in (0, L.LLVQ_FLAG_WAIT_TIMEOUT)
            gave_up += flags != 0
            assert flags or torch.equal(y, first)
            y = torch.empty_like(first)
            codec.linear(w, x, y, gated=gated, workspace=ws)
            assert codec.get_error() == 0 and torch.equal(y, first)
    assert gave_up >= (6 if rows > 70000 else 3)       # no polls at all cannot succeed, one poll not on the longest
