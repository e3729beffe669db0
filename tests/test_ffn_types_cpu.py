"""VQExperts looks at its arrays' types, not only at their sizes (refused before any handle is made)."""

import numpy as np
import pytest
import torch

from compressed_index_matmul_b200 import VQ_BF16, VQ_FMT_RVQ12_4, VQ_FMT_VQ16_RVQ, VQExperts

E, N, K = 2, 16, 64
G = K // 8


class Made(Exception):
    pass


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    """Arguments that pass end here instead of at the GPU."""
    class Here:
        def __init__(self, *a):
            raise Made

    monkeypatch.setattr(torch.cuda, "device", Here)


def arrays(fmt):
    if fmt == VQ_FMT_RVQ12_4:
        return dict(lo=torch.zeros((E, N * G), dtype=torch.uint8), hi4=torch.zeros((E, N * G // 2), dtype=torch.uint8),
                    s2=torch.zeros((E, N * G // 2), dtype=torch.uint8), cb1=torch.zeros((E, 4096, 8), dtype=torch.float16),
                    cb2=torch.zeros((E, 16, 8), dtype=torch.float16), scales=torch.zeros((E, N), dtype=torch.float16))
    return dict(idx16=torch.zeros((E, 2 * N * G), dtype=torch.int16), idx8=torch.zeros((E, N * G), dtype=torch.uint8),
                cb1=torch.zeros((1, 65536, 8), dtype=torch.float16), cbr=torch.zeros((1, 1, 65536, 8), dtype=torch.float16),
                cb8=torch.zeros((1, 256, 8), dtype=torch.float16), scales=torch.zeros((E, N), dtype=torch.float16),
                mult=[0.5, 0.25])


def make(fmt, **change):
    VQExperts(E, N, K, fmt, 64, VQ_BF16, 4, {**arrays(fmt), **change}, shared_codebooks=fmt == VQ_FMT_VQ16_RVQ, device="cpu")


CASES = [(f, n) for f in (VQ_FMT_RVQ12_4, VQ_FMT_VQ16_RVQ) for n in arrays(f) if n != "mult"]


@pytest.mark.parametrize("fmt,name", CASES)
def test_types(fmt, name):
    t = arrays(fmt)[name]
    with pytest.raises(Made):
        make(fmt)
    # the bits of a half or an index in a 16-bit container, numpy as a layer's file has them, signed bytes
    for good in ([t.view(torch.int16), t.view(torch.uint16)] if t.element_size() == 2 else [t.view(torch.int8)]):
        with pytest.raises(Made):
            make(fmt, **{name: good})
    with pytest.raises(Made):
        make(fmt, **{name: t.numpy()})
    if t.element_size() == 2:
        with pytest.raises(Made):
            make(fmt, **{name: t.numpy().view(np.uint16)})
    # the same size, another meaning; the values in a wider type
    bad = [t.view(torch.bfloat16), t.float()] if t.element_size() == 2 else [t.bool(), t.view(torch.float8_e4m3fn), t.int()]
    if name.startswith("idx16"):
        bad.append(t.view(torch.float16))
    for b in bad:
        with pytest.raises(ValueError, match=f"{name} must"):
            make(fmt, **{name: b})


@pytest.mark.parametrize("mult", [[], [0.5], [0.5, 0.25, 0.125]])
def test_a_multiplier_for_every_residual_stage(mult):
    """Two 16-bit stages and an 8-bit one have two residual stages."""
    with pytest.raises(ValueError, match="mult must have 2"):
        make(VQ_FMT_VQ16_RVQ, mult=mult)
