"""An output over any input is refused before anything is launched.  No GPU: the handle is a block of
host memory that starts with the descriptor, as the library's own do, and goes on with a device number
that is never current, so that a call that is not refused ends at the device check."""

import ctypes

import pytest

from compressed_index_matmul_b200 import _binding as B
from compressed_index_matmul_b200 import build as libbuild


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return B.load()


def fake(desc):
    buf = ctypes.create_string_buffer(bytes(desc) + b"\xff" * 4096)
    return buf, ctypes.cast(buf, ctypes.c_void_p)


MB = 1 << 20
# Addresses that are never read, far apart
AT = {n: (i + 1) << 30 for i, n in enumerate(("x", "y", "signs", "lo", "hi4", "s2", "idx16", "idx8", "cb1", "cb2", "cbr0", "cbr1",
                                              "cb8", "scales", "bias", "mul", "residual", "corr_rows", "corr_cols",
                                              "corr_vals", "rows", "offsets"))}
N, K, M, E = 264, 576, 3, 5
G = K // 8
FORMATS = {
    "12+4": (B.VQ_FMT_RVQ12_4, 64, {}, dict(lo=N * G, hi4=N * G // 2, s2=N * G // 2, scales=2 * N * 9), dict(cb1=65536, cb2=256)),
    "12 per row": (B.VQ_FMT_RVQ12, K, {}, dict(lo=N * G, hi4=N * G // 2, scales=2 * N), dict(cb1=65536)),
    "16": (B.VQ_FMT_VQ16, 64, {}, dict(idx16=2 * N * G, scales=2 * N * 9), dict(cb1=MB)),
    "ladder": (B.VQ_FMT_VQ16_RVQ, 64, dict(n16=3, n8=1, mult=(0.5, 0.25, 0.125)),
               dict(idx16=6 * N * G, idx8=N * G, scales=2 * N * 9), dict(cb1=MB, cbr0=MB, cbr1=MB, cb8=4096)),
}
CASES = [(f, name) for f, (_, _, _, planes, books) in FORMATS.items() for name in (*planes, *books)]


def pointers(names):
    p = {n: AT[n] if n in names else None for n in AT}
    planes = B.make_planes(p["lo"], p["hi4"], p["s2"], p["idx16"], p["idx8"], p["corr_rows"], p["corr_cols"], p["corr_vals"])
    return planes, B.make_codebooks(p["cb1"], p["cb2"], [c for c in (p["cbr0"], p["cbr1"]) if c], p["cb8"])


def places(name, size, ybytes):
    """y with its last 16 bytes on the input's first, and its first on the input's last."""
    return AT[name] - (ybytes - 1) // 16 * 16, AT[name] + (size - 1) // 16 * 16


def epilogue(lib, fmt, y, names, signs=None, corr=0, bias=None):
    f, sg, extra, *_ = FORMATS[fmt]
    buf, h = fake(B.make_desc(N, K, f, sg, B.VQ_F16, M, corr=corr, **extra))
    planes, books = pointers(names)
    st = lib.vq_linear_forward_epilogue(h, AT["x"], signs, planes, books, AT["scales"], B.make_epilogue(bias=bias), y, M, N, K, None)
    return st, lib.vq_last_error().decode()


@pytest.mark.parametrize("fmt", FORMATS)
def test_an_output_of_its_own_gets_to_the_device(lib, fmt):
    names = (*FORMATS[fmt][3], *FORMATS[fmt][4])
    st, msg = epilogue(lib, fmt, AT["y"], names, signs=AT["signs"])
    assert st != B.VQ_OK and "overlap" not in msg and ("device" in msg.lower() or "cuda" in msg.lower())


@pytest.mark.parametrize("fmt,name", CASES)
def test_forward_over_its_weights(lib, fmt, name):
    _, _, _, planes, books = FORMATS[fmt]
    for y in places(name, {**planes, **books}[name], 2 * M * N):
        st, msg = epilogue(lib, fmt, y, (*planes, *books))
        assert st == B.VQ_ERR_INVALID_ARG and "y overlaps" in msg, (hex(y), msg)


@pytest.mark.parametrize("name,size", [("signs", K), ("corr_rows", 4 * (N + 1)), ("corr_cols", 4), ("corr_vals", 2), ("bias", 2 * N),
                                       ("x", 2 * M * K)])
def test_forward_over_its_other_inputs(lib, name, size):
    names = ["lo", "hi4", "s2", "cb1", "cb2"] + (["corr_rows", "corr_cols", "corr_vals"] if "corr" in name else [])
    for y in places(name, size, 2 * M * N):
        st, msg = epilogue(lib, "12+4", y, names, signs=AT["signs"] if name == "signs" else None, corr=int("corr" in name),
                           bias=AT["bias"] if name == "bias" else None)
        assert st == B.VQ_ERR_INVALID_ARG and "y overlaps" in msg, (hex(y), msg)


def experts(lib, fmt, y, shared, names, T=7, rows=True, bias=True):
    f, sg, extra, *_ = FORMATS[fmt]
    desc = B.vq_experts_desc(B.make_desc(N, K, f, sg, B.VQ_F16, 16, **extra), E, shared, 0, 0, 1)
    buf, h = fake(desc)
    planes, books = pointers(names)
    st = lib.vq_experts_forward(h, AT["x"], 4, AT["rows"], AT["offsets"], planes, books, AT["scales"], AT["bias"], y, T, None)
    return st, lib.vq_last_error().decode()


@pytest.mark.parametrize("shared", [0, 1])
@pytest.mark.parametrize("fmt,name", CASES)
def test_experts_over_their_weights(lib, fmt, name, shared):
    """The planes and scales of all experts count, the codebooks' sets too unless there is one."""
    _, _, _, planes, books = FORMATS[fmt]
    size = planes[name] * E if name in planes else books[name] * (1 if shared else E)
    st, msg = experts(lib, fmt, AT["y"], shared, (*planes, *books))
    assert st != B.VQ_OK and "overlap" not in msg
    for y in places(name, size, 2 * 7 * N):
        st, msg = experts(lib, fmt, y, shared, (*planes, *books))
        assert st == B.VQ_ERR_INVALID_ARG and "y overlaps" in msg, (hex(y), msg)
    # the first byte behind a shared codebook is free
    if shared and name in books:
        st, msg = experts(lib, fmt, AT[name] + books[name], shared, (*planes, *books))
        assert "overlap" not in msg


@pytest.mark.parametrize("name,size", [("x", 2 * 4 * K), ("rows", 4 * 7), ("offsets", 4 * (E + 1)), ("bias", 2 * E * N)])
def test_experts_over_their_other_inputs(lib, name, size):
    for y in places(name, size, 2 * 7 * N):
        st, msg = experts(lib, "12+4", y, 0, ("lo", "hi4", "s2", "cb1", "cb2"))
        assert st == B.VQ_ERR_INVALID_ARG and "y overlaps" in msg, (hex(y), msg)
