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
