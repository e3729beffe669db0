"""GPU tests of the tensor-core forward, plain, with the sparse correction and with the fused epilogue, at every
kind of K split and token tile (the shapes and their splits: test_tc_splits_cpu.py)."""

import numpy as np
import pytest
import torch

import compressed_index_matmul_b200 as vq
from synth import DT_BF16, FMT_VQ16_RVQ, LayerSpec, make_correction, make_layer, make_x
from tests.ffn_util import ACTS, epilogue64, epilogue_bound, product_bound
from tests.gpu_util import dev, layer_on_gpu, require_gpu
from tests.test_tc_splits_cpu import CASES, case_id

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def randn(shape, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16 if dt == DT_BF16 else torch.float16).cuda()


def to64(t, cols=slice(None)):
    return None if t is None else t.double().cpu().numpy()[..., cols]


def within(y, want, bound):
    bad = ~(np.abs(y - want) <= bound)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside; first {np.argwhere(bad)[0]}: {y[bad][0]} for {want[bad][0]} "
                           f"+- {np.broadcast_to(bound, y.shape)[bad][0]}")


# the correction is not defined for the ladder
RUNS = [(c, corr) for c in CASES for corr in (False, True) if not (corr and c[2] == FMT_VQ16_RVQ)]


@pytest.mark.parametrize("case,corr", RUNS, ids=[case_id(c) + ("corr" if corr else "") for c, corr in RUNS])
def test_every_split(oracle, case, corr):
    N, K, fmt, bpw, dt, M, splits, ctas = case
    layer = make_layer(LayerSpec(N, K, fmt, 64, bpw=bpw or 2), cfg_id=320, tensor_id=N + M)
    rows = np.sort(np.random.default_rng(N + M).choice(N, size=min(N, 192), replace=False))
    w0, _ = oracle.dequant(layer, rows=rows)
    w = w0
    if corr:
        layer["corr"] = make_correction(N, K, density=0.01, cfg_id=320, tensor_id=N + M)
        w, _ = oracle.dequant(layer, rows=rows)
    L = layer_on_gpu(layer, dt, M)
    L.set_path(vq.VQ_PATH_TC)
    p = L.plan(M)
    assert (p["splits"], p["ctas"]) == (splits, ctas)
    x = dev(make_x(M, K, dt, cfg_id=321, seed=M)).view(torch.bfloat16 if dt == DT_BF16 else torch.float16)
    x64 = to64(x)
    f = x64 @ w.T
    # W is rounded to the type, the correction is not; its sum is taken in fp32
    tol = product_bound(x64, w0, dt) + 2.0 ** -20 * np.abs(x64) @ np.abs(w - w0).T

    y = L.forward(x)
    within(to64(y, rows), f, epilogue_bound(tol, f, "none", dt))
    assert torch.equal(L.forward(x).view(torch.int16), y.view(torch.int16)), "not bit-identical from run to run"
    assert torch.equal(L.forward_fused(x).view(torch.int16), y.view(torch.int16)), "an empty epilogue changes the result"

    parts = dict(bias=randn((N,), dt, 1), mul=randn((M, N), dt, 2), residual=randn((M, N), dt, 3))
    for act, which in (("gelu", "bias mul residual"), ("silu", "mul"), ("gelu_tanh", "bias residual"), ("none", "residual")):
        some = {k: v for k, v in parts.items() if k in which}
        y = L.forward_fused(x, act=ACTS[act], **some)
        b, m, r = (to64(some.get(k), rows) for k in ("bias", "mul", "residual"))
        within(to64(y, rows), epilogue64(f, act, b, m, r), epilogue_bound(tol, f, act, dt, b, m, r))
        assert torch.equal(L.forward_fused(x, act=ACTS[act], **some).view(torch.int16), y.view(torch.int16))
        for name in some:
            if name != "bias":  # in place
                out = some[name].clone()
                L.forward_fused(x, act=ACTS[act], **{**some, name: out}, y=out)
                assert torch.equal(out.view(torch.int16), y.view(torch.int16)), name
    vq.vq_linear_check(L.handle)
