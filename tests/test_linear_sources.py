"""What the sources of the linear layers have to hold to, checked by reading them."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "codebook_free_lattice_b200", "csrc")


def arguments_of(function, text):
    for m in re.finditer(r"\b" + function + r"\(", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        yield text[m.end():at - 1]


def test_only_constant_data_is_read_by_non_coherent_loads():
    """The kernels overlap the ones before them on the stream, whose outputs (the workspace, and x, residual and
    offsets where another layer wrote them) therefore take coherent loads: __ldg is for the weight and the tables."""
    constant = (r"a\.gains \+ ", r"word_at\(", r"d\.tabC \+ ", r"g \+ j$", r"reinterpret_cast<const uint4 \*>\(g\) \+ lane$")
    found = 0
    for f in sorted(glob.glob(os.path.join(CSRC, "linear*.cuh"))):
        text = re.sub(r"//[^\n]*", "", open(f).read())
        for argument in arguments_of("__ldg", text):
            found += 1
            assert any(re.match(p, argument) for p in constant), (os.path.basename(f), argument)
    assert found >= 8


def test_the_erfc_of_gelu():
    """The coefficients in the source against scipy's scaled complementary error function, in relative terms: 1e-6 from
    zero to where erfc leaves fp32's range."""
    import numpy as np
    special = __import__("pytest").importorskip("scipy.special")
    text = open(os.path.join(CSRC, "linear_common.cuh")).read()
    body = text[text.index("const float t = __fdividef(1.f, fmaf("):text.index("const float tail")]
    p, *_ = re.findall(r"fmaf\(([0-9.]+)f, x", body)
    q = [float(v) for v in re.findall(r"(-?\d\.\d+)f, t,", body)] + [float(v) for v in re.findall(r", t, (-?\d\.\d+)f\)", body)]
    assert len(q) == 7
    x = np.linspace(0, 10, 100001)
    t = 1 / (1 + float(p) * x)
    assert np.abs(np.polyval(q, t) * t / special.erfcx(x) - 1).max() < 1e-6
