"""GPU tests of the routing (vq_router_forward) and of the weighted sum back (vq_experts_combine)."""

import numpy as np
import pytest
import torch

import compressed_index_matmul_b200 as vq
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


DTYPES = [torch.float16, torch.bfloat16, torch.float32]


def route64(logits, k, renorm):
    """The definition, row by row: ids, weights (64 bits), offsets, rows, slots."""
    v = logits.double().cpu().numpy()
    T, E = v.shape
    ids, w, slots = np.full((T, k), -1), np.zeros((T, k)), np.full((T, k), -1)
    for t in range(T):
        ok = [e for e in range(E) if v[t, e] > -np.inf]  # NaN compares false
        best = sorted(ok, key=lambda e: (-v[t, e], e))[:k]
        if not best:
            continue
        mx = v[t, best[0]]
        p = {e: 1.0 if v[t, e] == mx else np.exp(v[t, e] - mx) for e in ok}
        total = sum(p[e] for e in (best if renorm else ok))
        ids[t, :len(best)] = best
        w[t, :len(best)] = [p[e] / total for e in best]
    pairs = sorted((ids[t, j], t, j) for t in range(T) for j in range(k) if ids[t, j] >= 0)
    for at, (_, t, j) in enumerate(pairs):
        slots[t, j] = at
    offsets = np.searchsorted([p[0] for p in pairs], np.arange(E + 1))
    return ids, w, offsets, np.array([p[1] for p in pairs], dtype=np.int64), slots


def check(r, logits, k, renorm):
    ids, w, offsets, rows, slots = route64(logits, k, renorm)
    E = logits.shape[1]
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.rows.cpu().numpy()[:len(rows)], rows)
    assert np.array_equal(r.slots.cpu().numpy(), slots)
    got = r.weights.cpu().numpy().astype(np.float64)
    # each exponential is within 2 units of 2^-23 and its argument's subtraction is off by
    # half a unit of |l - max| <= 88 (beyond, the weight is below 2^-126); the E terms of the
    # sum are each off by at most E / 2 units, the quotient by one
    span = np.abs(np.nan_to_num(logits.double().cpu().numpy(), nan=0.0, posinf=0.0, neginf=0.0)).max()
    rel = 2.0 ** -23 * (2 * (2 + min(88.0, 2 * span) / 2) + E / 2 + 1)
    assert (np.abs(got - w) <= rel * w + 2.0 ** -125).all(), np.abs(got / np.where(w > 0, w, 1) - 1).max()


def logits_of(T, E, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return (3.0 * torch.randn((T, E), generator=g)).to(dt).cuda()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (2, 5, 5), (3, 33, 2), (7, 512, 32), (63, 64, 6), (64, 128, 8),
                                   (65, 100, 3), (128, 8, 2), (129, 8, 2), (193, 256, 8), (1000, 60, 4), (4097, 16, 2)])
@pytest.mark.parametrize("dt", DTYPES)
def test_routing(T, E, k, dt):
    for renorm in (False, True):
        R = vq.VQRouter(E, k, T, renorm=renorm)
        x = logits_of(T, E, dt, T + E)
        r = R.forward(x)
        check(r, x, k, renorm)
        again = R.forward(x)
        assert all(torch.equal(a, b) for a, b in zip(r, again))


def test_many_tokens():
    T, E, k = 20000, 96, 6
    x = logits_of(T, E, torch.bfloat16, 5)  # bfloat16: many equal logits
    check(vq.VQRouter(E, k, T).forward(x), x, k, False)


@pytest.mark.parametrize("T", [5, 300])
def test_equal_logits_go_to_the_lowest_expert(T):
    x = torch.zeros((T, 70), device="cuda")
    x[:, 40:] = -0.0  # equal to +0
    r = vq.VQRouter(70, 5, T).forward(x)
    assert torch.equal(r.ids, torch.arange(5, dtype=torch.int32, device="cuda").expand(T, 5))
    assert torch.allclose(r.weights, torch.full_like(r.weights, 1 / 70), rtol=1e-6)
    check(r, x, 5, False)


@pytest.mark.parametrize("T", [8, 200])
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("renorm", [False, True])
def test_masked_logits(T, dt, renorm):
    """-inf and NaN are never chosen; rows with fewer than k left, with none, with +inf, and with the
    type's lowest value, which is a number and can be chosen."""
    E, k = 40, 4
    x = logits_of(T, E, dt, 9)
    x[0] = float("-inf")
    x[1] = float("nan")
    x[2, 2:] = float("-inf")
    x[3] = float("-inf")
    x[3, 17] = -2.0
    x[4, 3] = x[4, 30] = float("inf")
    x[5] = torch.finfo(dt).min
    x[6] = float("-inf")
    x[6, 1:3] = torch.finfo(dt).min
    x[7, ::2] = float("nan")
    r = vq.VQRouter(E, k, T, renorm=renorm).forward(x)
    check(r, x, k, renorm)
    assert r.ids[0].tolist() == [-1] * 4 and r.weights[1].tolist() == [0.0] * 4
    assert r.weights[3].tolist() == [1.0, 0.0, 0.0, 0.0] and r.weights[4].tolist() == [0.5, 0.5, 0.0, 0.0]
    assert int(r.offsets[-1]) == int((r.ids >= 0).sum()) < T * k


def test_rows_behind_the_last_pair_stay_as_they_were():
    x = logits_of(200, 16, torch.float32, 3)
    x[50:150] = float("-inf")
    R = vq.VQRouter(16, 2, 200)
    r = R.forward(x)
    r.rows.fill_(-7)
    r = R.forward(x, out=r)
    assert (r.rows[200:] == -7).all() and (r.rows[:200] >= 0).all()


def test_all_rows_to_one_expert():
    x = logits_of(500, 32, torch.float32, 4)
    x[:, 13] = 50.0
    check(vq.VQRouter(32, 2, 500).forward(x), x, 2, False)


def test_fewer_tokens_than_the_handle_was_made_for():
    R = vq.VQRouter(64, 8, 4096)
    for T in (4096, 1, 700, 128, 129, 0):
        x = logits_of(T, 64, torch.float32, T)
        r = R.forward(x)
        if T:
            check(r, x, 8, False)
        else:
            assert r.offsets.tolist() == [0] * 65


@pytest.mark.parametrize("T", [4, 1000])
def test_captured_and_replayed(T):
    R = vq.VQRouter(64, 4, T)
    x = logits_of(T, 64, torch.bfloat16, 1)
    out = R.forward(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
        R.forward(x, out=out)
    for seed in (2, 3):
        x.copy_(logits_of(T, 64, torch.bfloat16, seed))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check(out, x, 4, False)


def test_router_refusals():
    R = vq.VQRouter(16, 2, 8)
    with pytest.raises(ValueError, match="float16, bfloat16 or float32"):
        R.forward(torch.zeros((4, 16), device="cuda", dtype=torch.float64))
    for bad in (torch.zeros((4, 17), device="cuda"), torch.zeros((4, 32), device="cuda")[:, ::2], torch.zeros((4, 16))):
        with pytest.raises(ValueError, match="logits must be"):
            R.forward(bad)
    with pytest.raises(vq.VQError, match="max_T"):
        R.forward(torch.zeros((9, 16), device="cuda"))
    with pytest.raises(ValueError, match="ids must be"):
        R.forward(torch.zeros((4, 16), device="cuda"), out=R.forward(torch.zeros((5, 16), device="cuda")))
    with pytest.raises(vq.VQError, match="16-byte"):
        R.forward(torch.zeros(4 * 16 + 1, device="cuda")[1:].view(4, 16))
    r = R.forward(torch.zeros((4, 16), device="cuda"))
    logits = torch.zeros((4, 16), device="cuda")
    for out, names in ((r._replace(slots=r.ids), "slots overlaps ids"), (r._replace(rows=r.ids.view(-1)), "rows overlaps ids"),
                       (r._replace(weights=logits.view(-1)[8:16].view(4, 2)), "weights overlaps logits")):
        with pytest.raises(vq.VQError, match=names):
            R.forward(logits, out=out)


def test_no_tokens():
    r = vq.VQRouter(16, 2, 8).forward(torch.zeros((0, 16), device="cuda"))
    assert r.ids.shape == (0, 2) and r.rows.shape == (0,) and r.offsets.tolist() == [0] * 17


# ------------------------------------------------------------------------------------ combine


@pytest.mark.parametrize("T,k,N", [(1, 1, 8), (1, 8, 2048), (5, 2, 24), (33, 3, 576), (100, 32, 64), (257, 6, 1000), (64, 9, 4096)])
@pytest.mark.parametrize("dt", DTYPES[:2])
@pytest.mark.parametrize("res", [False, True])
def test_combine(T, k, N, dt, res):
    g = torch.Generator().manual_seed(T + k)
    rows = T * k
    y = torch.randn((rows, N), generator=g).to(dt).cuda()
    w = torch.randn((T, k), generator=g).cuda()
    slots = torch.randperm(rows, generator=g).view(T, k).to(torch.int32).cuda()
    r = torch.randn((T, N), generator=g).to(dt).cuda() if res else None
    out = vq.combine(y, w, slots, residual=r)
    terms = w.double().unsqueeze(2) * y.double()[slots.long()]
    want, size = terms.sum(1), terms.abs().sum(1)
    if res:
        want, size = want + r.double(), size + r.double().abs()
    # k fused steps and the residual's addition in fp32, one rounding to the type
    bound = (k + 1) * 2.0 ** -24 * size + torch.finfo(dt).eps / 2 * (want.abs() + (k + 1) * 2.0 ** -24 * size) + 2.0 ** -25
    assert ((out.double() - want).abs() <= bound).all()
    if res:  # in place
        got = vq.combine(y, w, slots, residual=r, out=r)
        assert got is r and torch.equal(out, r)


def test_slots_out_of_range_add_nothing():
    """Their weights are not used, whatever they hold; the rows they would name are not read."""
    y = torch.randn((6, 64), device="cuda").half()
    y[5] = float("nan")
    w = torch.ones((4, 3), device="cuda")
    slots = torch.tensor([[0, -1, 2], [-1, -1, -1], [6, 1, 2 ** 31 - 1], [-2 ** 31, 4, 3]], dtype=torch.int32, device="cuda")
    w[slots < 0] = float("nan")
    w[slots >= 6] = float("inf")
    out = vq.combine(y, w, slots)
    want = torch.stack([y[0].float() + y[2].float(), torch.zeros(64, device="cuda"), y[1].float(), y[4].float() + y[3].float()])
    assert torch.equal(out, want.half())
    same = vq.combine(y, torch.ones((4, 1), device="cuda"), torch.tensor([[3]] * 4, dtype=torch.int32, device="cuda"))
    assert torch.equal(same, y[3].expand(4, 64))  # the same row for every token
    none = vq.combine(y[:0], w, slots, residual=y[:4])
    assert torch.equal(none, y[:4])


def test_infinities_reach_their_token_only():
    y = torch.zeros((4, 16), device="cuda", dtype=torch.bfloat16)
    y[1, 3], y[2, 5] = float("inf"), float("nan")
    out = vq.combine(y, torch.ones((2, 2), device="cuda"), torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda"))
    assert out[0, 3] == float("inf") and torch.isnan(out[1, 5]) and int((out == 0).sum()) == 30


def test_combine_many_rows_past_32_bits():
    """Row times width passes 2^31 elements."""
    N, n = 1 << 14, (1 << 17) + 64
    y = torch.zeros((n, N), dtype=torch.float16, device="cuda")  # 4.3 GB
    y[n - 1] = 3.0
    y[n - 2] = 5.0
    out = vq.combine(y, torch.ones((2, 2), device="cuda"), torch.tensor([[n - 1, 0], [n - 2, n - 1]], dtype=torch.int32, device="cuda"))
    assert (out[0] == 3.0).all() and (out[1] == 8.0).all()


def test_combine_refusals():
    y = torch.zeros((4, 16), dtype=torch.float16, device="cuda")
    w, s = torch.zeros((2, 2), device="cuda"), torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    for kw, name in ((dict(weights=w.half()), "weights"), (dict(slots=s.long()), "slots"), (dict(residual=y), "residual"),
                     (dict(out=y[:2].float()), "out")):
        with pytest.raises(ValueError, match=f"{name} must be"):
            vq.combine(**{**dict(y=y, weights=w, slots=s), **kw})
    with pytest.raises(vq.VQError, match="out overlaps y"):
        vq.combine(y, w, s, out=y[2:])
    with pytest.raises(vq.VQError, match="multiple of 8"):
        vq.combine(torch.zeros((4, 12), dtype=torch.float16, device="cuda"), w, s)
