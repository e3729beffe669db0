"""GPU tests of the fused epilogue: y = act(x . W^T + bias) * mul + residual on every forward
path, against the oracle's fp64 product and the epilogue in 64 bits."""

import numpy as np
import pytest
import torch

import compressed_index_matmul_b200 as vq
from synth import (DT_BF16, DT_F16, FMT_RVQ12, FMT_RVQ12_4, FMT_VQ16, FMT_VQ16_RVQ, LayerSpec, make_correction,
                   make_layer, make_signs, make_x)
from tests.ffn_util import ACTS, epilogue64, epilogue_bound
from tests.gpu_util import dev, host_bits, layer_on_gpu, require_gpu, widen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def tdt(act):
    return torch.bfloat16 if act == DT_BF16 else torch.float16


def rand(shape, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(tdt(dt)).cuda()


def to64(t):
    return None if t is None else t.double().cpu().numpy()


def check(oracle, layer, L, x_bits, dt, f64, tol, act, parts, **kw):
    x = dev(x_bits).view(tdt(dt))
    y = L.forward_fused(x, act=ACTS[act], **parts, **kw)
    torch.cuda.synchronize()
    vq.vq_linear_check(L.handle)
    b, m, r = (to64(parts.get(k)) for k in ("bias", "mul", "residual"))
    got, want = to64(y), epilogue64(f64, act, b, m, r)
    bound = epilogue_bound(tol, f64, act, dt, b, m, r)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside; first {np.argwhere(bad)[0]}: {got[bad][0]} for "
                           f"{want[bad][0]} +- {np.broadcast_to(bound, got.shape)[bad][0]}")
    return y


PATHS = [
    # (N, K, fmt, scale_group, act dtype, M, path)
    (512, 1024, FMT_RVQ12_4, 64, DT_BF16, 1, vq.VQ_PATH_LUT),       # grid barrier, quads of rows
    (256, 128, FMT_RVQ12, 64, DT_F16, 1, vq.VQ_PATH_LUT),           # one slice
    (520, 1024, FMT_RVQ12, 1024, DT_F16, 1, vq.VQ_PATH_LUT),        # a scale per row
    (201, 576, FMT_RVQ12_4, 64, DT_F16, 3, vq.VQ_PATH_GEMV),        # odd N
    (576, 1536, FMT_RVQ12_4, 64, DT_BF16, 16, vq.VQ_PATH_GEMV),     # split-K tickets
    (129, 64, FMT_VQ16, 64, DT_BF16, 1, vq.VQ_PATH_GEMV),           # one split, one block of K
    (256, 512, FMT_RVQ12_4, 64, DT_BF16, 64, vq.VQ_PATH_TC),        # one split, bulk stores
    (2040, 512, FMT_RVQ12_4, 64, DT_BF16, 300, vq.VQ_PATH_TC),      # a K pair over a cluster
    (131, 576, FMT_RVQ12_4, 64, DT_F16, 21, vq.VQ_PATH_TC),         # odd N: stores per element
    (256, 8192, FMT_RVQ12_4, 64, DT_BF16, 33, vq.VQ_PATH_TC),       # several splits, last block sums
    (384, 512, FMT_VQ16, 512, DT_F16, 100, vq.VQ_PATH_TC),
    (512, 2048, FMT_VQ16, 2048, DT_F16, 1, vq.VQ_PATH_GATHER),
    (516, 1024, FMT_VQ16, 64, DT_BF16, 5, vq.VQ_PATH_GATHER),
]


@pytest.mark.parametrize("case", PATHS, ids=lambda c: f"{c[0]}x{c[1]}f{c[2]}a{c[4]}M{c[5]}p{c[6]}")
@pytest.mark.parametrize("act,which", [("silu", "bmr"), ("gelu", "b"), ("gelu_tanh", "m"), ("relu", "r"), ("none", "mr"),
                                       ("silu", "")])
def test_every_path(oracle, case, act, which):
    N, K, fmt, sg, dt, M, path = case
    layer = make_layer(LayerSpec(N, K, fmt, sg), cfg_id=300, tensor_id=N + M)
    L = layer_on_gpu(layer, dt, M)
    L.set_path(path)
    x = make_x(M, K, dt, cfg_id=301, seed=M)
    w, _ = oracle.dequant(layer)
    f = oracle.forward(layer, x, dt)
    parts = dict(bias=rand((N,), dt, 1) if "b" in which else None, mul=rand((M, N), dt, 2) if "m" in which else None,
                 residual=rand((M, N), dt, 3) if "r" in which else None)
    tol = oracle.tolerance(x, dt, w)
    y = check(oracle, layer, L, x, dt, f, tol, act, parts)
    again = L.forward_fused(dev(x).view(tdt(dt)), act=ACTS[act], **parts)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16)), "not bit-identical from run to run"
    # mul and residual may be the output
    for name in ("mul", "residual"):
        if parts[name] is not None:
            out = parts[name].clone()
            got = L.forward_fused(dev(x).view(tdt(dt)), act=ACTS[act], **{**parts, name: out}, y=out)
            assert got is out and torch.equal(y.view(torch.int16), out.view(torch.int16)), name


@pytest.mark.parametrize("case", PATHS, ids=lambda c: f"{c[0]}x{c[1]}f{c[2]}a{c[4]}M{c[5]}p{c[6]}")
def test_empty_epilogue_is_the_forward(case):
    N, K, fmt, sg, dt, M, path = case
    L = layer_on_gpu(make_layer(LayerSpec(N, K, fmt, sg), cfg_id=302, tensor_id=N), dt, M)
    L.set_path(path)
    x = dev(make_x(M, K, dt, cfg_id=303)).view(tdt(dt))
    assert np.array_equal(host_bits(L.forward(x)), host_bits(L.forward_fused(x)))


@pytest.mark.parametrize("bpw", [3, 5, 8])
@pytest.mark.parametrize("M", [1, 9, 40])
def test_residual_ladder(oracle, bpw, M):
    layer = make_layer(LayerSpec(264, 384, FMT_VQ16_RVQ, 64, bpw=bpw), cfg_id=304, tensor_id=bpw)
    L = layer_on_gpu(layer, DT_F16, M)
    x = make_x(M, 384, DT_F16, cfg_id=305)
    w, _ = oracle.dequant(layer)
    parts = dict(bias=rand((264,), DT_F16, 4), residual=rand((M, 264), DT_F16, 5))
    check(oracle, layer, L, x, DT_F16, oracle.forward(layer, x, DT_F16), oracle.tolerance(x, DT_F16, w), "silu", parts)


@pytest.mark.parametrize("fmt,N,K,M", [(FMT_RVQ12_4, 520, 1024, 1), (FMT_RVQ12, 200, 576, 7), (FMT_VQ16, 256, 512, 33)])
def test_with_the_sparse_correction(oracle, fmt, N, K, M):
    """The correction's term enters before the bias and the activation."""
    layer = make_layer(LayerSpec(N, K, fmt, 64), cfg_id=306, tensor_id=M)
    layer["corr"] = make_correction(N, K, density=0.02, cfg_id=306, tensor_id=M)
    L = layer_on_gpu(layer, DT_BF16, M)
    x = make_x(M, K, DT_BF16, cfg_id=307)
    w, _ = oracle.dequant(layer)
    parts = dict(bias=rand((N,), DT_BF16, 6), mul=rand((M, N), DT_BF16, 7))
    check(oracle, layer, L, x, DT_BF16, oracle.forward(layer, x, DT_BF16), oracle.tolerance(x, DT_BF16, w), "gelu", parts)


@pytest.mark.parametrize("fmt,K,M", [(FMT_VQ16, 1024, 1), (FMT_VQ16, 384, 4), (FMT_RVQ12_4, 576, 1), (FMT_RVQ12_4, 512, 20)])
def test_rotated_input(oracle, fmt, K, M):
    """signs given: the rotated forward's result goes through the epilogue (fused rotation and not)."""
    N = 256
    layer = make_layer(LayerSpec(N, K, fmt, 64), cfg_id=308, tensor_id=M)
    L = vq.VQLinear(N, K, fmt, 64, DT_F16, M, layer, rht=1)
    xb = make_x(M, K, DT_F16, cfg_id=309)
    signs = make_signs(K, cfg_id=309)
    x = dev(xb).view(torch.float16)
    st = torch.from_numpy(signs).cuda()
    parts = dict(bias=rand((N,), DT_F16, 8), residual=rand((M, N), DT_F16, 9))
    y = to64(L.forward_fused(x, act=ACTS["silu"], signs=st, **parts))
    xr = oracle.rht(xb, DT_F16, signs)
    w, _ = oracle.dequant(layer)
    # the unfused route rounds the rotated x to the type: at most half a step of each element
    tol = 2e-3 * np.linalg.norm(xr, axis=1, keepdims=True) * np.abs(w).max() + 2.0 ** -11 * np.abs(xr) @ np.abs(w).T
    f = xr @ w.T
    b, r = to64(parts["bias"]), to64(parts["residual"])
    assert (np.abs(y - epilogue64(f, "silu", b, None, r)) <= epilogue_bound(tol, f, "silu", DT_F16, b, None, r)).all()


SPECIAL = [1e30, -1e30, 0.0, -0.0, 1.0, -1.0, 3.5, -3.5, -4.0, 9.0, -9.0, 20.0, -20.0, 87.0, -87.0, 100.0, -100.0, 6e4, -6e4,
           2.0 ** -20, -2.0 ** -20, 0.3, -0.7, float("inf"), float("nan")]


@pytest.mark.parametrize("dt", [DT_F16, DT_BF16])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("M", [1, 2, 20])
def test_activation_values(act, dt, M):
    """x = 0 makes the product 0, so y = act(bias): every activation at small, large and special
    values, within the fp32 steps and the rounding of the type."""
    N = 32
    L = layer_on_gpu(make_layer(LayerSpec(N, 128, FMT_RVQ12_4, 64), cfg_id=310), dt, M)
    vals = (SPECIAL + [0.5] * N)[:N]
    bias = torch.tensor(vals).to(tdt(dt)).cuda()
    x = torch.zeros((M, 128), dtype=tdt(dt), device="cuda")
    y = to64(L.forward_fused(x, act=ACTS[act], bias=bias))
    b = to64(bias)
    want = np.broadcast_to(epilogue64(np.zeros((M, N)), act, b), (M, N))
    # values beyond the type's range round to infinity
    want = np.where(np.abs(want) >= (65520.0 if dt == DT_F16 else 3.4e38), np.copysign(np.inf, want), want)
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(want), np.isnan(y)) and np.array_equal(want[~fin & ~np.isnan(want)], y[~fin & ~np.isnan(want)])
    bound = epilogue_bound(0.0, np.zeros((M, N)), act, dt, np.where(np.isfinite(b), b, 0.0))
    # below 2^-126 / 2^-24 fp32 and the formulas may flush: |act(-87)| < 2^-118
    assert (np.abs(y[fin] - want[fin]) <= np.broadcast_to(bound, (M, N))[fin] + 2.0 ** -110).all()


def test_special_values_in_mul_and_residual():
    """Infinities and NaN in mul and residual reach exactly their own elements."""
    N, K, M = 264, 128, 19
    L = layer_on_gpu(make_layer(LayerSpec(N, K, FMT_RVQ12_4, 64), cfg_id=311), DT_BF16, M)
    x = dev(make_x(M, K, DT_BF16, cfg_id=312)).view(torch.bfloat16)
    mul, res = rand((M, N), DT_BF16, 1), rand((M, N), DT_BF16, 2)
    base = L.forward_fused(x, mul=mul, residual=res)
    mul2, res2 = mul.clone(), res.clone()
    mul2[3, 7], res2[18, 263], res2[0, 0] = float("nan"), float("inf"), float("-inf")
    y = L.forward_fused(x, mul=mul2, residual=res2)
    assert torch.isnan(y[3, 7]) and y[18, 263] == float("inf") and y[0, 0] == float("-inf")
    same = torch.ones_like(y, dtype=torch.bool)
    same[3, 7] = same[18, 263] = same[0, 0] = False
    assert torch.equal(y[same], base[same])


@pytest.mark.parametrize("M", [1, 16, 70])
def test_captured_and_replayed_on_another_stream(M):
    N, K = 512, 1024
    L = layer_on_gpu(make_layer(LayerSpec(N, K, FMT_RVQ12_4, 64), cfg_id=313), DT_BF16, M)
    x = dev(make_x(M, K, DT_BF16, cfg_id=314)).view(torch.bfloat16)
    bias, mul, res = rand((N,), DT_BF16, 1), rand((M, N), DT_BF16, 2), rand((M, N), DT_BF16, 3)
    want = L.forward_fused(x, act=2, bias=bias, mul=mul, residual=res)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = torch.zeros_like(want)
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            L.forward_fused(x, act=2, bias=bias, mul=mul, residual=res, y=y)
        g.replay()
    side.synchronize()
    assert torch.equal(y, want)
    x.mul_(-1.0)
    res.add_(1.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g.replay()
    side.synchronize()
    assert torch.equal(y, L.forward_fused(x, act=2, bias=bias, mul=mul, residual=res))
    # an explicit stream
    out = torch.zeros_like(want)
    L.forward_fused(x, act=2, bias=bias, mul=mul, residual=res, y=out, stream=side)
    side.synchronize()
    assert torch.equal(out, y)


def test_refusals():
    N, K, M = 256, 128, 8
    L = layer_on_gpu(make_layer(LayerSpec(N, K, FMT_RVQ12_4, 64), cfg_id=315), DT_BF16, M)
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    good = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    assert L.forward_fused(x[:0]).shape == (0, N)
    for kw in (dict(act=5), dict(act=-1)):
        with pytest.raises(vq.VQError, match="VQ_ACT"):
            L.forward_fused(x, **kw)
    big = torch.zeros((2 * M, N), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(vq.VQError, match="partially overlaps"):
        L.forward_fused(x, residual=big[1:M + 1], y=big[:M])
    with pytest.raises(vq.VQError, match="partially overlaps"):
        L.forward_fused(x, mul=big[M - 1:2 * M - 1], y=big[:M])
    with pytest.raises(vq.VQError, match="overlaps epi->bias"):
        L.forward_fused(x, bias=good[3], y=good)
    sq = layer_on_gpu(make_layer(LayerSpec(K, K, FMT_RVQ12_4, 64), cfg_id=315), DT_BF16, M)
    with pytest.raises(vq.VQError, match="y"):
        sq.forward_fused(x, y=x)
    for name, t in (("bias", torch.zeros(N + 1, dtype=torch.bfloat16, device="cuda")), ("mul", good.float()),
                    ("residual", good.t()), ("mul", good.cpu()), ("residual", good[:, ::2]),
                    ("signs", torch.ones(K, device="cuda"))):
        with pytest.raises(ValueError, match=name):
            L.forward_fused(x, **{name: t})
    with pytest.raises(ValueError, match="x must be"):
        L.forward_fused(x.half())
    with pytest.raises(vq.VQError, match="16-byte"):
        L.forward_fused(x, bias=torch.zeros(N + 8, dtype=torch.bfloat16, device="cuda")[1:N + 1])
    with pytest.raises(vq.VQError, match="M="):
        L.forward_fused(torch.zeros((M + 1, K), dtype=torch.bfloat16, device="cuda"))
    rc = vq.load().vq_linear_forward_epilogue(L.handle, x.data_ptr(), None, L.planes, L.codebooks,
                                              L.t["scales"].data_ptr(), None, good.data_ptr(), M, N, K, None)
    assert rc == 1
    torch.cuda.synchronize()
    vq.vq_linear_check(L.handle)
