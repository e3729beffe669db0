"""Host-side checks of the feed-forward entry points that need no GPU."""

import ctypes
import os
import subprocess

import pytest
import torch

from compressed_index_matmul_b200 import _binding as B
from compressed_index_matmul_b200 import build as libbuild
from compressed_index_matmul_b200.layer import VQLinear, check_tensor

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return B.load()


def c_layout(tmp_path, structs):
    """sizeof and offsetof of the ABI structs as gcc lays them out from the header."""
    src = ["#include <stddef.h>", "#include <stdio.h>", '#include "vqlinear_ffn.h"', "int main(void) {"]
    for st, fs in structs.items():
        src.append(f'  printf("{st} sizeof %zu\\n", sizeof({st}));')
        src += [f'  printf("{st} {f} %zu\\n", offsetof({st}, {f}));' for f in fs]
    (tmp_path / "o.c").write_text("\n".join(src + ["  return 0;\n}"]))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(tmp_path / "o.c"), "-o",
                    str(tmp_path / "o")], check=True)
    out = subprocess.run([str(tmp_path / "o")], capture_output=True, text=True, check=True).stdout
    return {(a, b): int(c) for a, b, c in (ln.split() for ln in out.splitlines())}


def same_layout(tmp_path, names):
    structs = {n: [f for f, _ in getattr(B, n)._fields_] for n in names}
    got = c_layout(tmp_path, structs)
    for st, fs in structs.items():
        cls = getattr(B, st)
        assert got[(st, "sizeof")] == ctypes.sizeof(cls), st
        for f in fs:
            assert got[(st, f)] == getattr(cls, f).offset, (st, f)


def test_structs_match_the_header(tmp_path):
    same_layout(tmp_path, ["vq_epilogue", "vq_experts_desc", "vq_router_desc"])


def test_epilogue_rejects_a_null_handle(lib):
    e = B.make_epilogue()
    cb, pl = B.make_codebooks(16, 16), B.make_planes(16, 16, 16)
    assert lib.vq_linear_forward_epilogue(None, 16, None, pl, cb, 16, e, 16, 1, 64, 64, None) == B.VQ_ERR_INVALID_ARG
    assert b"handle" in lib.vq_last_error()


def test_long_messages_are_cut_not_lost(lib):
    assert lib.vq_rht_apply(16, 16, 16, 1, 100, 0, None) == B.VQ_ERR_INVALID_ARG
    assert 0 < len(lib.vq_last_error()) < 512


def test_check_tensor():
    cpu = torch.device("cpu")
    t = torch.zeros((4, 8), dtype=torch.float16)
    check_tensor(t, "t", (4, 8), torch.float16, cpu)
    for bad in (t[:, ::2], t.t(), t.float(), t[:3]):
        with pytest.raises(ValueError, match="t must be a contiguous"):
            check_tensor(bad, "t", (4, 8), torch.float16, cpu)
    with pytest.raises(ValueError):
        check_tensor(t, "t", (4, 8), torch.float16, torch.device("meta"))


def test_fused_forward_checks_its_tensors_before_the_library():
    """No handle is needed to refuse a tensor of another shape, type or layout."""
    L = VQLinear.__new__(VQLinear)
    L.N, L.K, L.act_dtype, L.device, L.handle = 16, 64, B.VQ_F16, torch.device("cpu"), None
    x = torch.zeros((2, 64), dtype=torch.float16)
    y = torch.zeros((2, 16), dtype=torch.float16)
    for kw, name in ((dict(bias=y), "bias"), (dict(mul=y[:1]), "mul"), (dict(residual=y.float()), "residual"),
                     (dict(y=y.t()), "y"), (dict(signs=y[0]), "signs")):
        with pytest.raises(ValueError, match=f"{name} must be"):
            L.forward_fused(x, **kw)
    with pytest.raises(ValueError, match="x must be"):
        L.forward_fused(x[:, :32])


@pytest.mark.parametrize("E,k,max_T,renorm,status", [
    (0, 1, 1, 0, 1), (4, 0, 1, 0, 1), (4, 5, 1, 0, 1), (513, 1, 1, 0, 2), (64, 33, 1, 0, 2), (4, 1, 0, 0, 1),
    (4, 1, 1, 2, 1), (64, 32, 1 << 26, 0, 1),
    (1, 1, (1 << 30) + 1, 0, 1),
])
def test_router_rejects_bad_descriptors(lib, E, k, max_T, renorm, status):
    h = ctypes.c_void_p(1)
    assert lib.vq_router_create(B.vq_router_desc(E, k, renorm, max_T), ctypes.byref(h)) == status
    assert h.value is None and lib.vq_last_error()


def test_router_null_arguments(lib):
    assert lib.vq_router_create(None, None) == B.VQ_ERR_INVALID_ARG
    h = ctypes.c_void_p()
    assert lib.vq_router_create(None, ctypes.byref(h)) == B.VQ_ERR_INVALID_ARG
    assert lib.vq_router_forward(None, 16, 0, 16, 16, 16, 16, 16, 1, None) == B.VQ_ERR_INVALID_ARG
    assert lib.vq_router_destroy(None) == B.VQ_OK


P, Q = 1 << 20, 1 << 24  # addresses that are never read


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(y_rows=-1), 1), (dict(k=0), 1), (dict(k=33), 1), (dict(N=0), 1), (dict(N=12), 2), (dict(N=1 << 25), 2),
    (dict(dtype=2), 1), (dict(y=None), 1), (dict(w=None), 1), (dict(slots=None), 1), (dict(out=None), 1), (dict(y=P + 8), 1),
    (dict(res=Q + 16), 1),       # overlaps out, and is not out
    (dict(out=P + 64), 1),       # inside y
    (dict(out=P - 16), 1),       # runs into y
    (dict(w=Q + 16), 1), (dict(slots=Q), 1),
])
def test_combine_rejects_bad_arguments(lib, kw, status):
    a = dict(y=P, y_rows=8, w=1 << 12, slots=1 << 13, res=None, out=Q, T=4, k=2, N=64, dtype=1)
    a.update(kw)
    assert lib.vq_experts_combine(a["y"], a["y_rows"], a["w"], a["slots"], a["res"], a["out"], a["T"], a["k"], a["N"],
                                  a["dtype"], None) == status


def test_combine_of_no_tokens(lib):
    assert lib.vq_experts_combine(None, 0, None, None, None, None, 0, 2, 64, 1, None) == B.VQ_OK


def test_combine_checks_its_tensors():
    import compressed_index_matmul_b200 as vq

    with pytest.raises(ValueError, match="float16 or bfloat16"):
        vq.combine(torch.zeros(4, 8), None, None)
    with pytest.raises(ValueError, match="current CUDA device"):
        vq.combine(torch.zeros((4, 8), dtype=torch.float16), torch.zeros(2, 2), torch.zeros((2, 2), dtype=torch.int32))


@pytest.mark.parametrize("kw,status", [
    (dict(E=0), 1), (dict(E=1025), 2), (dict(gather=2), 1), (dict(glu=2), 1), (dict(act=5), 1), (dict(act=-1), 1), (dict(shared_codebooks=3), 1),
    (dict(N=12), 2), (dict(N=72, glu=1), 2), (dict(K=72), 1), (dict(K=80), 2), (dict(fmt=9), 1), (dict(max_rows=0), 1),
    (dict(rht=1), 2), (dict(corr=1), 2), (dict(N=1 << 17, K=1 << 17), 2), (dict(N=1 << 24, max_rows=1 << 20, E=1024), 2),
    (dict(fmt=B.VQ_FMT_VQ16_RVQ, n16=5), 1),
])
def test_experts_reject_bad_descriptors(lib, kw, status):
    a = dict(E=4, N=64, K=128, fmt=B.VQ_FMT_RVQ12_4, scale_group=64, act_dtype=B.VQ_BF16, max_rows=16)
    a.update(kw)
    with pytest.raises(B.VQError) as ei:
        B.vq_experts_create(**a)
    assert ei.value.status == status


def test_experts_null_arguments(lib):
    h = ctypes.c_void_p(1)
    assert lib.vq_experts_create(None, None) == B.VQ_ERR_INVALID_ARG
    assert lib.vq_experts_create(None, ctypes.byref(h)) == B.VQ_ERR_INVALID_ARG and h.value is None
    cb, pl = B.make_codebooks(16, 16), B.make_planes(16, 16, 16)
    assert lib.vq_experts_forward(None, 16, 1, None, 16, pl, cb, 16, None, 16, 1, None) == B.VQ_ERR_INVALID_ARG
    assert lib.vq_experts_set_path(None, 0) == B.VQ_ERR_INVALID_ARG
    assert lib.vq_experts_plan(None, 1, None) == B.VQ_ERR_INVALID_ARG
    assert lib.vq_experts_check(None, None) == B.VQ_ERR_INVALID_ARG
    assert lib.vq_experts_destroy(None) == B.VQ_OK
