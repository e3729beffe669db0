"""GPU tests of the products grouped by expert (vq_experts_forward) against the oracle's weights
and the definition in 64 bits, on both kernels."""

import numpy as np
import pytest
import torch

import compressed_index_matmul_b200 as vq
from compressed_index_matmul_b200 import _binding as B
from synth import DT_BF16, DT_F16, FMT_RVQ12, FMT_RVQ12_4, FMT_VQ16, FMT_VQ16_RVQ, LayerSpec, make_layer
from tests.ffn_util import ACTS, epilogue64, epilogue_bound, glu64, glu_bound, product_bound
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

GEMV, TC = vq.VQ_PATH_GEMV, vq.VQ_PATH_TC
BOOKS = ("cb1", "cb2", "cbr", "cb8", "mult")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def tdt(dt):
    return torch.bfloat16 if dt == DT_BF16 else torch.float16


def randn(shape, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(tdt(dt)).cuda()


def to64(t):
    return t.double().cpu().numpy()


def make_experts(E, N, K, fmt, sg, seed, shared=False, bpw=2):
    """E layers and their arrays with a leading dimension E."""
    layers = [make_layer(LayerSpec(N, K, fmt, sg or K, bpw=bpw), cfg_id=400, layer=e, tensor_id=seed) for e in range(E)]
    for l in layers:
        for k in BOOKS:
            if k in layers[0] and (shared or k == "mult"):  # the multipliers are the handle's
                l[k] = layers[0][k]
    arrays = {}
    for k in ("lo", "hi4", "s2", "idx16", "idx8", "scales"):
        if layers[0].get(k) is not None:
            arrays[k] = np.stack([l[k] for l in layers])
    for k in ("cb1", "cb2", "cb8"):
        if layers[0].get(k) is not None:
            arrays[k] = np.stack([l[k] for l in (layers[:1] if shared else layers)])
    if "cbr" in layers[0]:
        arrays["cbr"] = np.stack([l["cbr"] for l in (layers[:1] if shared else layers)], axis=1)
    if "mult" in layers[0]:
        arrays["mult"] = layers[0]["mult"]
    return layers, arrays


def offsets_of(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)).cuda()


def check(oracle, layers, X, x, offsets, rows, y, act, glu, bias, dt):
    """Every written row of y against the definition."""
    at = np.maximum.accumulate(np.clip(offsets.cpu().numpy().astype(np.int64), 0, y.shape[0]))
    x64, y64 = to64(x), to64(y)
    idx = np.arange(y.shape[0]) if rows is None else rows.cpu().numpy().astype(np.int64)
    for e, layer in enumerate(layers):
        if at[e] == at[e + 1]:
            continue
        w, _ = oracle.dequant(layer)
        sel = idx[at[e]:at[e + 1]]
        ok = (sel >= 0) & (sel < len(x64))
        xe = np.where(ok[:, None], x64[np.where(ok, sel, 0)], 0.0)
        f, tol = xe @ w.T, product_bound(xe, w, dt)
        b = None if bias is None else to64(bias[e])
        got = y64[at[e]:at[e + 1]]
        want = glu64(f, act, b) if glu else epilogue64(f, act, b)
        bound = glu_bound(tol, f, act, dt, b) if glu else epilogue_bound(tol, f, act, dt, b)
        bad = ~(np.abs(got - want) <= bound)
        assert not bad.any(), (f"expert {e}: {bad.sum()} of {bad.size} outside, first {np.argwhere(bad)[0]}: {got[bad][0]} for "
                               f"{want[bad][0]} +- {bound[bad][0]}")


def run(oracle, E, N, K, fmt, sg, dt, counts, path, act="none", glu=False, bias=False, gather=True, shared=False, bpw=2,
        seed=1, x_rows=None):
    layers, arrays = make_experts(E, N, K, fmt, sg, seed, shared, bpw)
    T = int(np.sum(counts))
    b = randn((E, N), dt, seed) if bias else None
    X = vq.VQExperts(E, N, K, fmt, sg or K, dt, T, arrays, act=ACTS[act], glu=glu, bias=b, shared_codebooks=shared)
    X.set_path(path)
    assert X.plan(T)["path"] == (path or X.plan(T)["path"])
    rows = None
    n = T
    if gather:
        n = x_rows or max(1, T // 2)
        rows = torch.from_numpy(np.random.default_rng(seed).integers(0, n, size=T).astype(np.int32)).cuda()
    x = randn((n, K), dt, seed + 1)
    off = offsets_of(counts)
    y = X.forward(x, off, rows=rows)
    torch.cuda.synchronize()
    vq.vq_experts_check(X.handle)
    check(oracle, layers, X, x, off, rows, y, act, glu, b, dt)
    again = X.forward(x, off, rows=rows)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16)), "not bit-identical from run to run"
    return X, x, off, rows, y


SHAPES = [
    # (E, N, K, fmt, scale group (0: per row), dtype, rows per expert)
    (1, 8, 64, FMT_RVQ12_4, 64, DT_BF16, [1]),
    (1, 128, 128, FMT_RVQ12, 64, DT_F16, [5]),
    (3, 136, 192, FMT_RVQ12_4, 64, DT_BF16, [0, 9, 0]),          # 64-wide last slice, ragged row tile
    (4, 256, 576, FMT_RVQ12_4, 64, DT_F16, [1, 0, 16, 17]),
    (5, 264, 320, FMT_RVQ12, 0, DT_BF16, [33, 1, 0, 0, 2]),
    (8, 128, 1024, FMT_RVQ12_4, 0, DT_BF16, [3, 70, 0, 1, 128, 129, 15, 0]),
    (2, 512, 2048, FMT_RVQ12_4, 64, DT_BF16, [300, 40]),
    (6, 72, 256, FMT_VQ16, 64, DT_BF16, [2, 0, 31, 8, 0, 64]),
    (3, 136, 448, FMT_VQ16, 0, DT_F16, [18, 257, 1]),
    # more slices of K than index slots, block scales: a slot is refilled while its neighbours decode
    (4, 512, 1280, FMT_VQ16, 64, DT_F16, [128, 128, 128, 128]),
    (3, 528, 1472, FMT_VQ16, 64, DT_BF16, [200, 60, 100]),
    (4, 512, 1472, FMT_RVQ12, 64, DT_F16, [128, 64, 128, 20]),
    (4, 512, 1280, FMT_RVQ12_4, 64, DT_F16, [128, 128, 128, 128]),
    (40, 48, 128, FMT_RVQ12_4, 64, DT_BF16, [i % 4 for i in range(40)]),  # a block meets many experts
]


@pytest.mark.parametrize("path", [GEMV, TC])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"E{s[0]}N{s[1]}K{s[2]}f{s[3]}")
def test_plain(oracle, shape, path):
    run(oracle, *shape, path)


@pytest.mark.parametrize("path", [GEMV, TC])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("act", list(ACTS))
def test_epilogues(oracle, act, gather, path):
    run(oracle, 4, 200, 256, FMT_RVQ12_4, 64, DT_BF16, [7, 0, 40, 18], path, act=act, bias=True, gather=gather)


@pytest.mark.parametrize("path", [GEMV, TC])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("shape", [
    (3, 32, 64, FMT_RVQ12_4, 64, DT_BF16, [2, 0, 19]),
    (2, 16, 128, FMT_RVQ12, 64, DT_F16, [1, 3]),
    (4, 272, 576, FMT_RVQ12_4, 64, DT_BF16, [17, 16, 15, 90]),       # 136 outputs: ragged 64-row halves
    (2, 400, 320, FMT_VQ16, 0, DT_F16, [5, 140]),
    (2, 1024, 1024, FMT_RVQ12_4, 0, DT_BF16, [260, 3]),
], ids=lambda s: f"E{s[0]}N{s[1]}K{s[2]}f{s[3]}")
def test_gated(oracle, shape, bias, path):
    run(oracle, *shape, path, act="silu", glu=True, bias=bias)


@pytest.mark.parametrize("path", [GEMV, TC])
@pytest.mark.parametrize("fmt,bpw", [(FMT_RVQ12, 2), (FMT_RVQ12_4, 2), (FMT_VQ16, 2), (FMT_VQ16_RVQ, 5)])
def test_shared_codebooks(oracle, fmt, bpw, path):
    run(oracle, 7, 80, 320, fmt, 64, DT_F16, [2, 0, 5, 33, 1, 0, 12], path, shared=True, bpw=bpw, act="gelu", bias=True)


@pytest.mark.parametrize("path", [GEMV, TC])
@pytest.mark.parametrize("bpw", [2, 3, 4, 5, 6, 7, 8])
def test_residual_ladder(oracle, bpw, path):
    run(oracle, 3, 136, 192, FMT_VQ16_RVQ, 64, DT_F16, [4, 0, 21], path, bpw=bpw)


@pytest.mark.parametrize("path", [GEMV, TC])
def test_gated_ladder(oracle, path):
    run(oracle, 2, 96, 256, FMT_VQ16_RVQ, 0, DT_BF16, [40, 3], path, bpw=3, act="silu", glu=True)


@pytest.mark.parametrize("path", [GEMV, TC])
def test_many_experts_with_few_rows(oracle, path):
    rng = np.random.default_rng(7)
    run(oracle, 300, 64, 64, FMT_RVQ12_4, 64, DT_BF16, rng.integers(0, 3, size=300), path, shared=True)
    run(oracle, 200, 32, 128, FMT_RVQ12, 64, DT_BF16, rng.integers(0, 2, size=200), path)  # one block, several codebooks


def test_automatic_choice(oracle):
    for counts in ([1] * 4, [100, 200, 3, 0]):
        X, *_ = run(oracle, 4, 128, 256, FMT_RVQ12_4, 64, DT_BF16, counts, vq.VQ_PATH_AUTO)
    assert X.plan(1)["path"] == GEMV and X.plan(56)["path"] == GEMV and X.plan(57)["path"] == TC and X.plan(303)["path"] == TC


@pytest.mark.parametrize("path", [GEMV, TC])
def test_rows_outside_the_offsets_stay_as_they_were(path):
    E, N, K = 3, 136, 128
    _, arrays = make_experts(E, N, K, FMT_RVQ12_4, 64, 3)
    X = vq.VQExperts(E, N, K, FMT_RVQ12_4, 64, DT_BF16, 100, arrays)
    X.set_path(path)
    x = randn((100, K), DT_BF16, 1)
    full = X.forward(x, offsets_of([40, 20, 40]))
    y = torch.full((100, N), 7.0, dtype=torch.bfloat16, device="cuda")
    X.forward(x, offsets_of([35, 20, 13], first=5), y=y)
    assert (y[:5] == 7.0).all() and (y[73:] == 7.0).all()
    assert torch.equal(y[5:40], full[5:40]) and torch.equal(y[40:60], full[40:60]) and torch.equal(y[60:73], full[60:73])
    y.fill_(7.0)
    X.forward(x, offsets_of([0, 0, 0]), y=y)
    X.forward(x, offsets_of([0, 0, 0], first=100), y=y)
    X.forward(x[:0], offsets_of([0, 0, 0]), y=y[:0])
    assert (y == 7.0).all()
    vq.vq_experts_check(X.handle)


@pytest.mark.parametrize("path", [GEMV, TC])
def test_a_row_does_not_depend_on_the_others(path):
    """Bit for bit, whatever the other rows and experts hold, NaN included."""
    E, N, K = 4, 256, 576
    _, arrays = make_experts(E, N, K, FMT_RVQ12_4, 64, 5)
    X = vq.VQExperts(E, N, K, FMT_RVQ12_4, 64, DT_BF16, 300, arrays)
    X.set_path(path)
    x = randn((300, K), DT_BF16, 2)
    ref = X.forward(x, offsets_of([70, 70, 70, 90]))
    x2 = x.clone()
    x2[:100] = float("nan")
    x2[101:160] = float("inf")
    assert torch.equal(X.forward(x2, offsets_of([70, 70, 70, 90]))[100], ref[100])
    one = torch.tensor([100], dtype=torch.int32, device="cuda")
    assert torch.equal(X.forward(x, offsets_of([0, 1, 0, 0]), rows=one)[0], ref[100])
    assert torch.equal(X.forward(x, offsets_of([0, 300, 0, 0]))[70:140], ref[70:140])


@pytest.mark.parametrize("path", [GEMV, TC])
@pytest.mark.parametrize("glu", [False, True])
def test_row_numbers_out_of_range_read_as_zeros(oracle, path, glu):
    E, N, K = 2, 96, 192
    layers, arrays = make_experts(E, N, K, FMT_RVQ12_4, 64, 6)
    b = randn((E, N), DT_F16, 6)
    X = vq.VQExperts(E, N, K, FMT_RVQ12_4, 64, DT_F16, 40, arrays, act=ACTS["silu"], glu=glu, bias=b)
    X.set_path(path)
    x = randn((9, K), DT_F16, 3)
    x[0] = float("nan")  # row 0 is only ever read where it is named
    rows = torch.randint(1, 9, (40,), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    rows[3], rows[17], rows[18], rows[39] = -1, 9, 2 ** 31 - 1, -2 ** 31
    off = offsets_of([19, 21])
    y = X.forward(x, off, rows=rows)
    x0 = x.clone()
    x0[0] = 0.0
    check(oracle, layers, X, x0, off, rows, y, "silu", glu, b, DT_F16)
    vq.vq_experts_check(X.handle)


@pytest.mark.parametrize("path", [GEMV, TC])
@pytest.mark.parametrize("bad", [[-5, 10, 30], [0, 500, 40], [20, 5, 40], [2 ** 31 - 1, -2 ** 31, 17], [0, 40, 0], [-9, -3, -1]])
def test_bad_offsets_stay_in_range(oracle, path, bad):
    """Clamped into [0, T] and to at least the ones before; rows that no expert has are not written."""
    E, N, K, T = 2, 72, 128, 40
    layers, arrays = make_experts(E, N, K, FMT_RVQ12_4, 64, 8)
    X = vq.VQExperts(E, N, K, FMT_RVQ12_4, 64, DT_BF16, T, arrays)
    X.set_path(path)
    x = randn((T, K), DT_BF16, 4)
    off = torch.tensor(np.array(bad, dtype=np.int64).astype(np.int32)).cuda()
    guard = torch.full((T + 64, N), 7.0, dtype=torch.bfloat16, device="cuda")
    y = X.forward(x, off, y=guard[:T])
    torch.cuda.synchronize()
    check(oracle, layers, X, x, off, None, y, "none", False, None, DT_BF16)
    at = np.maximum.accumulate(np.clip(np.array(bad), 0, T))
    keep = [r for r in range(T) if not (at[0] <= r < at[-1])]
    assert (guard[T:] == 7.0).all() and (y[keep] == 7.0).all()


@pytest.mark.parametrize("path", [GEMV, TC])
def test_captured_and_replayed_with_other_offsets(oracle, path):
    E, N, K, T = 4, 192, 256, 120
    layers, arrays = make_experts(E, N, K, FMT_RVQ12_4, 64, 9)
    X = vq.VQExperts(E, N, K, FMT_RVQ12_4, 64, DT_BF16, T, arrays, act=ACTS["relu"])
    X.set_path(path)
    x = randn((T, K), DT_BF16, 5)
    rows = torch.arange(T, dtype=torch.int32, device="cuda")
    off = offsets_of([30, 30, 30, 30])
    y = X.forward(x, off, rows=rows)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        X.forward(x, off, rows=rows, y=y)
    for counts, seed in (([0, 120, 0, 0], 1), ([1, 2, 3, 114], 2), ([50, 0, 1, 69], 3)):
        off.copy_(offsets_of(counts))
        rows.copy_(torch.randperm(T, generator=torch.Generator().manual_seed(seed)).to(torch.int32))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check(oracle, layers, X, x, off, rows, y, "relu", False, None, DT_BF16)
    side2 = torch.cuda.Stream()
    out = torch.zeros_like(y)
    X.forward(x, off, rows=rows, y=out, stream=side2)
    side2.synchronize()
    assert torch.equal(out, y)


@pytest.mark.parametrize("path", [GEMV, TC])
def test_two_handles_on_two_streams(path):
    made = []
    for seed in (1, 2):
        _, arrays = make_experts(4, 512, 512, FMT_RVQ12_4, 64, seed)
        X = vq.VQExperts(4, 512, 512, FMT_RVQ12_4, 64, DT_BF16, 200, arrays)
        X.set_path(path)
        x = randn((200, 512), DT_BF16, seed)
        made.append((X, x, X.forward(x, offsets_of([50, 0, 100, 50]))))
    off = offsets_of([50, 0, 100, 50])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(20):
        for i, (X, x, _) in enumerate(made):
            with torch.cuda.stream(streams[i]):
                outs[i].append(X.forward(x, off))
    torch.cuda.synchronize()
    for i, (_, _, want) in enumerate(made):
        assert all(torch.equal(o, want) for o in outs[i])


@pytest.mark.parametrize("path", [GEMV, TC])
def test_x_rows_past_32_bits(path):
    """Row number times K passes 2^31 elements (4.3 GB of x)."""
    E, N, K, n = 1, 64, 4096, (1 << 19) + 8
    _, arrays = make_experts(E, N, K, FMT_RVQ12_4, 64, 11)
    X = vq.VQExperts(E, N, K, FMT_RVQ12_4, 64, DT_BF16, 32, arrays)
    X.set_path(path)
    x = torch.zeros((n, K), dtype=torch.bfloat16, device="cuda")
    tail = randn((32, K), DT_BF16, 6)
    x[n - 32:] = tail
    rows = torch.arange(n - 32, n, dtype=torch.int32, device="cuda")
    assert torch.equal(X.forward(x, offsets_of([32]), rows=rows), X.forward(tail, offsets_of([32])))


@pytest.mark.parametrize("path", [GEMV, TC])
def test_planes_past_32_bits(path):
    """The last of 1024 experts starts past 2^32 index bytes."""
    E, N, K = 1024, 4096, 8256
    n = N * K // 8
    one, arrays = make_experts(1, N, K, FMT_RVQ12_4, 64, 12)
    big = {"cb1": torch.from_numpy(arrays["cb1"].view(np.int16)).cuda(), "cb2": torch.from_numpy(arrays["cb2"].view(np.int16)).cuda()}
    for k, size, dt in (("lo", n, torch.uint8), ("hi4", n // 2, torch.uint8), ("s2", n // 2, torch.uint8),
                        ("scales", N * K // 64, torch.int16)):
        big[k] = torch.zeros((E, size), dtype=dt, device="cuda")
        src = torch.from_numpy(arrays[k].view(np.int16) if dt == torch.int16 else arrays[k])
        big[k][E - 1] = src[0].cuda()
    assert (E - 1) * n > 2 ** 32
    X = vq.VQExperts(E, N, K, FMT_RVQ12_4, 64, DT_BF16, 20, big, shared_codebooks=True)
    eight = {k: v if k in ("cb1", "cb2") else np.concatenate([v] * 8) for k, v in arrays.items()}
    Y = vq.VQExperts(8, N, K, FMT_RVQ12_4, 64, DT_BF16, 20, eight, shared_codebooks=True)
    X.set_path(path)
    Y.set_path(path)
    x = randn((20, K), DT_BF16, 7)
    assert torch.equal(X.forward(x, offsets_of([0] * (E - 1) + [20])), Y.forward(x, offsets_of([0] * 7 + [20])))


@pytest.mark.parametrize("tokens", [1, 5, 200])
def test_a_whole_block(oracle, tokens):
    """Routing, the gated products, the down products and the sum, each against its definition on
    what it was given, eagerly and captured."""
    E, k, H, I, dt = 8, 2, 256, 192, DT_BF16
    up_l, up_a = make_experts(E, 2 * I, H, FMT_RVQ12_4, 64, 13)
    dn_l, dn_a = make_experts(E, H, I, FMT_RVQ12_4, 64, 14)
    R = vq.VQRouter(E, k, tokens, renorm=True)
    U = vq.VQExperts(E, 2 * I, H, FMT_RVQ12_4, 64, dt, tokens * k, up_a, act=ACTS["silu"], glu=True)
    D = vq.VQExperts(E, H, I, FMT_RVQ12_4, 64, dt, tokens * k, dn_a)
    x, logits = randn((tokens, H), dt, 1), randn((tokens, E), dt, 2)
    if tokens > 1:
        logits[1] = float("-inf")  # a padded token: no expert takes it

    def block():
        r = R.forward(logits)
        h = U.forward(x, r.offsets, rows=r.rows)
        d = D.forward(h, r.offsets)
        return r, h, d, vq.combine(d, r.weights, r.slots, residual=x)

    block()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        static = block()
    x.copy_(randn((tokens, H), dt, 3))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    for r, h, d, out in (block(), static):
        n = int(r.offsets[-1])
        assert n == k * (tokens - (1 if tokens > 1 else 0))
        check(oracle, up_l, U, x, r.offsets, r.rows, h[:n], "silu", True, None, dt)
        check(oracle, dn_l, D, h, r.offsets, None, d[:n], "none", False, None, dt)
        s = r.slots.long().clamp(min=0)
        terms = torch.where((r.slots >= 0).unsqueeze(2), r.weights.double().unsqueeze(2) * d[:max(n, 1)].double()[s], 0.0)
        want = terms.sum(1) + x.double()
        bound = 2.0 ** -8 * want.abs() + 2.0 ** -20 * (terms.abs().sum(1) + x.double().abs())
        assert ((out.double() - want).abs() <= bound).all()
        if tokens > 1:
            assert torch.equal(out[1], x[1])
    assert torch.equal(block()[3], static[3])


def test_refusals():
    E, N, K, T = 2, 64, 128, 16
    _, arrays = make_experts(E, N, K, FMT_RVQ12_4, 64, 15)
    X = vq.VQExperts(E, N, K, FMT_RVQ12_4, 64, DT_BF16, T, arrays)
    x, off = randn((T, K), DT_BF16, 1), offsets_of([8, 8])
    rows = torch.zeros(T, dtype=torch.int32, device="cuda")
    for kw, name in ((dict(x=x.half()), "x"), (dict(x=x[:, ::2]), "x"), (dict(offsets=off[:2]), "offsets"),
                     (dict(offsets=off.long()), "offsets"), (dict(rows=rows.long()), "rows"), (dict(y=x), "y"),
                     (dict(offsets=off.cpu()), "offsets")):
        with pytest.raises(ValueError, match=f"{name} must be"):
            X.forward(**{**dict(x=x, offsets=off), **kw})
    with pytest.raises(vq.VQError, match="max_M"):
        X.forward(randn((T + 1, K), DT_BF16, 1), off)
    with pytest.raises(vq.VQError, match="x_rows"):
        X.forward(x[:0], off, rows=rows)
    flat = torch.zeros(4 * T * K, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(vq.VQError, match="y overlaps x"):
        X.forward(flat[:T * K].view(T, K), off, y=flat[T * K // 2:T * K // 2 + T * N].view(T, N))
    with pytest.raises(vq.VQError, match="16-byte"):
        X.forward(flat[4:4 + T * K].view(T, K), off)
    with pytest.raises(vq.VQError, match="gather"):
        vq.VQExperts(E, N, K, FMT_RVQ12_4, 64, DT_BF16, T, arrays, gather=False).forward(x, off, rows=rows)
    with pytest.raises(vq.VQError, match="VQ_PATH"):
        X.set_path(vq.VQ_PATH_LUT)
    with pytest.raises(ValueError, match="must have"):
        vq.VQExperts(E + 1, N, K, FMT_RVQ12_4, 64, DT_BF16, T, arrays)
    with pytest.raises(ValueError, match="bias must be"):
        vq.VQExperts(E, N, K, FMT_RVQ12_4, 64, DT_BF16, T, arrays, bias=torch.zeros(N, device="cuda"))
    torch.cuda.synchronize()
    vq.vq_experts_check(X.handle)


def test_allocation_failure(monkeypatch):
    monkeypatch.setenv("VQ_TEST_FAIL_ALLOC", "1")
    with pytest.raises(vq.VQError) as ei:
        vq.vq_experts_create(2, 64, 128, FMT_RVQ12_4, 64, DT_BF16, 16)
    assert ei.value.status == B.VQ_ERR_NOMEM
    with pytest.raises(vq.VQError) as ei:
        vq.vq_router_create(8, 2, 16)
    assert ei.value.status == B.VQ_ERR_NOMEM
    monkeypatch.delenv("VQ_TEST_FAIL_ALLOC")
    vq.vq_router_destroy(vq.vq_router_create(8, 2, 16))


def test_results_come_from_the_memory_of_the_given_stream():
    """A result for another stream is not put where the current stream's freed blocks are: work on
    the current stream may still use those."""
    E, N, K, T = 2, 64, 128, 16
    _, arrays = make_experts(E, N, K, FMT_RVQ12_4, 64, 21)
    X = vq.VQExperts(E, N, K, FMT_RVQ12_4, 64, DT_BF16, T, arrays)
    L = vq.VQLinear(N, K, FMT_RVQ12_4, 64, DT_BF16, T, {k: v[0] for k, v in arrays.items()})
    R = vq.VQRouter(E, 1, T)
    x, off, logits = randn((T, K), DT_BF16, 1), offsets_of([8, 8]), torch.zeros((T, E), device="cuda")
    r, side = R.forward(logits), torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in (lambda s: X.forward(x, off, stream=s), lambda s: L.forward_fused(x, stream=s),
                 lambda s: R.forward(logits, stream=s).weights, lambda s: vq.combine(x, r.weights, r.slots, stream=s)):
        here = call(None)
        at = here.data_ptr()
        del here
        for s in (side, side.cuda_stream):
            assert call(s).data_ptr() != at
    torch.cuda.synchronize()
