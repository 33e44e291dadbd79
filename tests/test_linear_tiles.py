"""Which tiles the product of the linear layers takes (the rule's times compiled from its header, the choice restated),
and that the layers of test_gpu_linear_tiles.py reach the forms that only large layers have."""
import ctypes as C
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "codebook_free_lattice_b200", "csrc")
PAIRS = 74                                            # of CTAs on 148 SMs

# tokens (per expert where there are several), weight rows of a matrix, columns, dtype, activation, gated, bias, residual
TILES = [
    ([785], 4802, 1986, "float16", "gelu", False, True, True),
    ([971], 4612, 2527, "float16", "none", False, False, False),
    ([1038], 3596, 2024, "bfloat16", "silu", True, True, False),
    ([1568], 5396, 2040, "bfloat16", "relu", False, False, True),
    ([1574], 5516, 1958, "float16", "silu", True, False, True),
    ([1300], 3300, 700, "float16", "gelu_tanh", True, True, True),
    ([606, 0, 42, 590], 2578, 2074, "bfloat16", "none", False, True, False),
]


@pytest.fixture(scope="module")
def cost(tmp_path_factory):
    from codebook_free_lattice_b200 import build
    d = tmp_path_factory.mktemp("tiles")
    (d / "tiles.cu").write_text('#include "codec.h"\n#include "linear_product.cuh"\nextern "C" int cost(int tiles, int cap, int pairs, int nk, int *split) '
                                '{ return llvq::lp_cost(tiles, cap, pairs, nk, *split); }\n')
    so = str(d / "tiles.so")
    subprocess.run([build.NVCC, "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "--expt-relaxed-constexpr", "-I", CSRC,
                    "-Xcompiler", "-fPIC", "-shared", "-o", so, str(d / "tiles.cu")], check=True, capture_output=True)
    return C.CDLL(so).cost


def schedule(cost, tokens, rows, cols, dtype, gated):
    """The tiles of a call: tokens of a tile (most; by group), of the groups' last tiles, row tiles, whole tiles, tiles
    split over the pairs that are left, ways of each, K stages, units of the busiest pair."""
    blocks = -(-cols // 24)
    nk = -(-(48 * blocks if gated and dtype == "float16" else cols) // 64)
    row_tiles, best = -(-rows // 256), None
    for cap in range(32, 257, 32):
        tiles, split = row_tiles * sum(-(-t // cap) for t in tokens), C.c_int()
        ns = cost(tiles, cap, PAIRS, nk, C.byref(split))
        if best is None or ns <= best[0]:
            best = (ns, cap, tiles, split.value)
    _, cap, tiles, split = best
    rest = tiles % PAIRS
    sizes, last = [], []
    for t in tokens:
        if t:
            n = -(-t // cap)
            sizes.append((-(-t // n) + 31) // 32 * 32)
            last.append((t - (n - 1) * sizes[-1] + 31) // 32 * 32)
    return {"sizes": sizes, "last": last, "row_tiles": row_tiles, "whole": tiles - rest, "rest": rest, "split": split, "nk": nk,
            "units": -(-(tiles - rest + rest * split) // PAIRS)}


def test_the_large_layers_reach_every_form(cost):
    plans = [schedule(cost, t, r, c, dtype, gated) for t, r, c, dtype, _, gated, _, _ in TILES]
    tiles = {n for p in plans for n in p["sizes"] + p["last"]}
    assert {64, 96, 128, 160, 192, 224, 256} <= tiles            # a tile's halves: every sum of boxes of 128 .. 16 tokens but the least
    for p in plans:
        assert p["row_tiles"] > 8 and p["row_tiles"] % 8          # a band of row tiles and part of one
        assert p["whole"] > 0 and p["units"] >= 2 and p["nk"] > 8
    assert sum(p["split"] > 1 for p in plans) >= 5               # whole tiles and split ones in a call
    assert any(p["units"] >= 3 and max(p["sizes"]) >= 224 for p in plans)
    assert any(len(set(p["sizes"])) > 1 for p in plans)
