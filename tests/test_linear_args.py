"""Refusals and workspace sizes of the linear layers, on the CPU: every refused call returns before any CUDA
call, so a codec object made by hand (no device, no tables) is enough."""
import ctypes as C
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "codebook_free_lattice_b200", "csrc")

torch = pytest.importorskip("torch")

SOURCE = """
#include "codec.h"
extern "C" llvq_codec *bare_codec(int bits) {
    llvq_codec *c = new llvq_codec;
    c->index_bits = bits;
    c->device = 0;
    c->num_sms = 148;
    c->pairs = 74;
    return c;
}
extern "C" size_t call_bytes() { return sizeof(llvq_linear_call); }
"""


@pytest.fixture(scope="module")
def L():
    from codebook_free_lattice_b200 import build
    build.build()
    import codebook_free_lattice_b200 as L
    L.lib()
    return L


@pytest.fixture(scope="module")
def bare(tmp_path_factory):
    from codebook_free_lattice_b200 import build
    d = tmp_path_factory.mktemp("bare")
    (d / "bare.cu").write_text(SOURCE)
    so = str(d / "bare.so")
    subprocess.run([build.NVCC, "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "--expt-relaxed-constexpr", "-I", CSRC,
                    "-Xcompiler", "-fPIC", "-shared", "-o", so, str(d / "bare.cu")], check=True, capture_output=True)
    lib = C.CDLL(so)
    lib.bare_codec.restype = C.c_void_p
    lib.call_bytes.restype = C.c_size_t
    return {"bytes": lib.call_bytes(), **{bits: C.c_void_p(lib.bare_codec(bits)) for bits in (48, 72, 96)}}


ADDRESS = 1 << 20                                     # an aligned address that no refused call looks at


def weight(L, rows=64, cols=100, bits=48, **other):
    nb = -(-cols // 24)
    w = L.llvq_weight(rows, cols, nb, bits, 8 if bits == 48 else 16, L.LLVQ_GAIN_U8_TABLE, nb, ADDRESS, ADDRESS)
    for k, v in other.items():
        setattr(w, k, v)
    return w


def call(L, tokens=5, rows=64, cols=100, **other):
    q = L.llvq_linear_call(tokens, L.LLVQ_DTYPE_FP16, L.LLVQ_ACT_NONE, 0, 0, ADDRESS, cols, None, None, 0, 2 * ADDRESS, rows, None)
    for k, v in other.items():
        setattr(q, k, v)
    return q


REFUSED = [
    (dict(tokens=-1), {}), (dict(dtype=2), {}), (dict(activation=5), {}), (dict(activation=-1), {}), (dict(gated=2), {}),
    (dict(experts=2), {}), (dict(x_stride=99), {}), (dict(y_stride=63), {}), (dict(residual=ADDRESS, residual_stride=63), {}),
    (dict(residual=ADDRESS, residual_stride=-64), {}), (dict(x=ADDRESS + 1), {}), (dict(y=ADDRESS + 1), {}),
    (dict(bias=ADDRESS + 1), {}), (dict(residual=ADDRESS + 1), {}), (dict(x=None), {}), (dict(y=None), {}),
    (dict(y=ADDRESS), {}), (dict(tokens=(1 << 30) + 1), {}),
    (dict(offsets=ADDRESS), {}), ({}, dict(cols=0, blocks_per_row=0)), ({}, dict(rows=-1)), ({}, dict(words=None)),
    ({}, dict(index_bits=72)), ({}, dict(row_pitch_words=4)), ({}, dict(gains=ADDRESS + 1)), ({}, dict(words=ADDRESS + 4)),
    (dict(gated=1), dict(rows=63)),
]


@pytest.mark.parametrize("changed,of_weight", REFUSED)
def test_linear_refuses(L, bare, changed, of_weight):
    w, q = weight(L, **of_weight), call(L, **changed)
    need = 1 << 40
    assert L.lib().llvq_linear(bare[48], C.byref(w), C.byref(q), C.c_void_p(ADDRESS), need, None) == L.LLVQ_ERR_ARG
    assert L.lib().llvq_last_error_message()


GROUPED_REFUSED = [(dict(experts=0), 1), (dict(experts=5), 1), (dict(offsets=None), 1), (dict(offsets=ADDRESS + 2), 1),
                   (dict(experts=2049), 2), (dict(gated=1, experts=64), 1)]


@pytest.mark.parametrize("changed,status", GROUPED_REFUSED)
def test_grouped_refuses(L, bare, changed, status):
    w, q = weight(L, rows=2049 * 64 if changed.get("experts") == 2049 else 64), call(L, **{"experts": 4, "offsets": ADDRESS, **changed})
    assert L.lib().llvq_linear_grouped(bare[48], C.byref(w), C.byref(q), C.c_void_p(ADDRESS), 1 << 40, None) == status
    assert L.lib().llvq_last_error_message()


def test_null_and_workspace(L, bare):
    w, q = weight(L), call(L)
    lib = L.lib()
    need = lib.llvq_linear_workspace(bare[48], C.byref(w), C.byref(q))
    assert need > 0
    for workspace, size in ((None, need), (ADDRESS, need - 1), (ADDRESS + 128, need)):
        assert lib.llvq_linear(bare[48], C.byref(w), C.byref(q), C.c_void_p(workspace), size, None) == L.LLVQ_ERR_ARG
    assert lib.llvq_linear(None, C.byref(w), C.byref(q), C.c_void_p(ADDRESS), need, None) == L.LLVQ_ERR_ARG
    assert lib.llvq_linear(bare[48], None, C.byref(q), C.c_void_p(ADDRESS), need, None) == L.LLVQ_ERR_ARG
    assert lib.llvq_linear(bare[48], C.byref(w), None, C.c_void_p(ADDRESS), need, None) == L.LLVQ_ERR_ARG
    assert lib.llvq_linear_grouped(None, None, None, None, 0, None) == L.LLVQ_ERR_ARG
    assert lib.llvq_linear_workspace(None, None, None) == 0
    q.dtype = 7
    assert lib.llvq_linear_workspace(bare[48], C.byref(w), C.byref(q)) == 0


@pytest.mark.parametrize("tokens,stride,refused", ((5, 0, True), (5, 65, True), (1, 0, False), (5, 64, False)))
def test_a_residual_at_y_has_its_stride(L, bare, tokens, stride, refused):
    """Rows of y may be the residual's, in place; one of them added to all, or rows between them, would change under the
    call.  (A call that passes this check is stopped by its workspace.)"""
    w, q = weight(L), call(L, tokens=tokens, residual=2 * ADDRESS, residual_stride=stride)
    assert L.lib().llvq_linear(bare[48], C.byref(w), C.byref(q), None, 0, None) == L.LLVQ_ERR_ARG
    assert (b"residual" in L.lib().llvq_last_error_message()) == refused


def test_nothing_to_do_is_ok_without_pointers(L, bare):
    lib = L.lib()
    w, q = weight(L), call(L, tokens=0, x=None, y=None)
    assert lib.llvq_linear(bare[48], C.byref(w), C.byref(q), None, 0, None) == L.LLVQ_OK
    w, q = weight(L, rows=0), call(L)
    assert lib.llvq_linear(bare[48], C.byref(w), C.byref(q), None, 0, None) == L.LLVQ_OK
    w, q = weight(L), call(L, tokens=0, experts=4, offsets=ADDRESS)
    assert lib.llvq_linear_grouped(bare[48], C.byref(w), C.byref(q), None, 0, None) == L.LLVQ_OK


def test_sizes_beyond_the_kernels_fields(L, bare):
    lib = L.lib()
    w = weight(L, cols=24 * 65536)
    q = call(L, cols=24 * 65536)
    assert lib.llvq_linear(bare[48], C.byref(w), C.byref(q), C.c_void_p(ADDRESS), 1 << 60, None) == L.LLVQ_ERR_UNSUPPORTED
    w, q = weight(L, rows=148 * 65536, cols=24), call(L, rows=148 * 65536, cols=24)
    assert lib.llvq_linear(bare[48], C.byref(w), C.byref(q), C.c_void_p(ADDRESS), 1 << 60, None) == L.LLVQ_ERR_UNSUPPORTED


def up256(n):
    return -(-n // 256) * 256


@pytest.mark.parametrize("bits", (48, 72, 96))
def test_workspace_sizes(L, bare, bits):
    """The decoded weight (rows of whole 128-byte lines), its row scales, the split tiles' counters and partial
    sums; restated activations only for bf16 and unaligned x; a few tokens need the blocks' dot products alone."""
    lib = L.lib()

    def need(rows, cols, tokens, **other):
        w, q = weight(L, rows, cols, bits), call(L, tokens, rows, cols, **other)
        return lib.llvq_linear_workspace(bare[bits], C.byref(w), C.byref(q))

    def base(held, cols):
        return up256(held * -(-(-(-cols // 24) * 24) // 64) * 128) + up256(held * 4) + up256(74 * 128 * 4) + 74 * 2 * 256 * 128 * 4

    assert need(4096, 4096, 64) == base(4096, 4096)
    assert need(1000, 999, 64, x_stride=1000) == base(1000, 999)
    assert need(1000, 999, 64) == base(1000, 999) + 64 * 1024 * 2                           # rows of 999 values
    assert need(1000, 1000, 64, x=ADDRESS + 2) == base(1000, 1000) + 64 * 1024 * 2
    assert need(1000, 1000, 64, dtype=1) == base(1000, 1000) + 64 * 1024 * 2 + 256
    assert need(4096, 4096, 3) == 3 * 4096 * 171 * 4
    assert need(4096, 4096, 1, dtype=1) == 4096 * 171 * 4
    if bits == 48:                                     # ... and what does not fit in shared memory, restated
        assert need(64, 28672, 2) == up256(2 * 64 * 1195 * 4) + up256(2 * 1195 * 48) + 256
        assert need(64, 28672, 3) == base(64, 28672)
    # experts: as many as can have a token are decoded
    assert need(64 * 100, 8192, 20, experts=64) == base(20 * 100, 8192)
    assert need(64 * 100, 8192, 1000, experts=64) == base(64 * 100, 8192)
    assert need(64 * 100, 240, 4, experts=64) == up256(4 * 4 * 100 * 10 * 4)


def test_binding_checks(L, bare):
    """Types, places and shapes that the binding refuses by itself."""
    codec = object.__new__(L.Codec)
    codec._h, codec.index_bits, codec.word_bytes, codec.device = C.c_void_p(), 48, 8, torch.device("cuda", 0)
    w = weight(L)
    half = dict(dtype=torch.float16)
    x, y = torch.zeros(5, 100, **half), torch.zeros(5, 64, **half)
    with pytest.raises(TypeError, match="float32"):
        codec.linear(w, x.float(), y)
    with pytest.raises(ValueError, match="x is"):
        codec.linear(w, x[:, :99], y)
    with pytest.raises(ValueError, match="x is"):
        codec.linear(w, x[0], y)
    with pytest.raises(ValueError, match="y is"):
        codec.linear(w, x, y[:4])
    with pytest.raises(ValueError, match="y is"):
        codec.linear(w, x, y, gated=True)
    with pytest.raises(ValueError, match="y is"):
        codec.linear_grouped(w, 4, x, torch.zeros(5, dtype=torch.int32), y)
    with pytest.raises(TypeError, match="cpu"):
        codec.linear(w, x, y)


def test_binding_matches_the_header(L, bare):
    import re
    src = open(os.path.join(ROOT, "include", "llvq.h")).read()
    values = dict(re.findall(r"#define\s+(LLVQ_(?:DTYPE|ACT|FLAG)_\w+)\s+(0x[0-9a-fA-F]+|\d+)", src))
    assert {"LLVQ_DTYPE_BF16", "LLVQ_ACT_SILU", "LLVQ_FLAG_OFFSETS"} <= set(values)
    for name, value in values.items():
        assert getattr(L, name) == int(value, 0), name
    assert C.sizeof(L.llvq_linear_call) == bare["bytes"]


@pytest.mark.parametrize("bits", (48, 72, 96))
def test_workspace_of_a_gated_fp16_layer(L, bare, bits):
    """Its decoded weight has two fp16 values per weight, and so have its activations; a gated bf16 layer's has one, and
    a few tokens need the dot products alone."""
    lib = L.lib()

    def need(**other):
        w, q = weight(L, 200, 1000, bits), call(L, rows=100, cols=1000, gated=1, **{"tokens": 64, **other})
        return lib.llvq_linear_workspace(bare[bits], C.byref(w), C.byref(q))

    rest = up256(200 * 4) + up256(74 * 128 * 4) + 74 * 2 * 256 * 128 * 4
    assert need() == need(x_stride=1003) == need(experts=4) == 200 * 2048 * 2 + rest + 64 * 2048 * 2      # 42 blocks of 48
    assert need(dtype=1) == 200 * 1024 * 2 + rest + 64 * 1024 * 2 + 256
    assert need(tokens=2) == up256(2 * 200 * 42 * 4)
    assert need(tokens=6) == up256(6 * 200 * 42 * 4) and need(tokens=7) > 200 * 2048 * 2
    assert need(tokens=6, dtype=1) > 200 * 1024 * 2
    assert need(tokens=6, experts=2) == up256(6 * 200 * 42 * 4) and need(tokens=15, experts=5) == up256(15 * 200 * 42 * 4)
    assert need(tokens=16, experts=5) > 200 * 2048 * 2


def test_a_failed_setup_is_reported(L, tmp_path):
    """Kernels whose limits cannot be set (here: there is no device) fail the codec's creation, not a later launch."""
    if torch.cuda.is_available():
        pytest.skip("a device is present")
    from codebook_free_lattice_b200 import build
    (tmp_path / "setup.cu").write_text('#include "codec.h"\nextern "C" int setup() { llvq_codec c; c.num_sms = 148; '
                                       'return (int)llvq::set_linear_attrs(&c); }\n')
    so = str(tmp_path / "setup.so")
    subprocess.run([build.NVCC, "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "--expt-relaxed-constexpr", "-I", CSRC,
                    "-Xcompiler", "-fPIC", "-shared", "-o", so, str(tmp_path / "setup.cu"), L.LIB_PATH], check=True, capture_output=True)
    assert C.CDLL(so).setup() != 0


def test_a_codec_is_made_without_torch(L, monkeypatch):
    """A codec needs no torch before its first call with tensors; it knows its device from the library."""
    import sys
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: {"llvq_codec_device": 3}.get(name, made.append(name) or 0)

    monkeypatch.setattr(L, "_lib", Library())
    with monkeypatch.context() as m:
        m.setitem(sys.modules, "torch", None)
        codec = L.Codec(48)
    assert codec.device == torch.device("cuda", 3) and "llvq_codec_create" in made
    codec.close()
    assert codec.device == torch.device("cuda", 3)


def test_device_of_a_codec(L, bare):
    assert L.lib().llvq_codec_device(bare[48]) == 0 and L.lib().llvq_codec_device(None) == -1


def test_current_stream_without_the_private_accessor(L, monkeypatch):
    """The layers take the current stream's handle by a name of torch that is not public only where torch has it."""
    device = torch.device("cuda", 2)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    assert L._current_raw_stream(device) == 102
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: type("S", (), {"cuda_stream": 7 + d.index}))
    assert L._current_raw_stream(device) == 9
