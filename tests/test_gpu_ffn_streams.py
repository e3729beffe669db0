"""GPU test: a result for the default stream, given explicitly, lies in the default stream's memory."""

import pytest
import torch

import compressed_index_matmul_b200 as vq
from synth import DT_BF16, FMT_RVQ12_4
from tests.gpu_util import require_gpu
from tests.test_gpu_experts import make_experts, offsets_of, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def test_the_default_stream_given_from_another_stream():
    """A block just freed on the default stream is the next result's, whichever stream is current; a
    block freed on the current one is not."""
    E, N, K, T = 2, 64, 128, 16
    _, arrays = make_experts(E, N, K, FMT_RVQ12_4, 64, 22)
    X = vq.VQExperts(E, N, K, FMT_RVQ12_4, 64, DT_BF16, T, arrays)
    L = vq.VQLinear(N, K, FMT_RVQ12_4, 64, DT_BF16, T, {k: v[0] for k, v in arrays.items()})
    R = vq.VQRouter(E, 1, T)
    x, off, logits = randn((T, K), DT_BF16, 1), offsets_of([8, 8]), torch.zeros((T, E), device="cuda")
    r, side = R.forward(logits), torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in (lambda s: X.forward(x, off, stream=s), lambda s: L.forward_fused(x, stream=s),
                 lambda s: R.forward(logits, stream=s).weights, lambda s: vq.combine(x, r.weights, r.slots, stream=s)):
        first = call(None)
        at = first.data_ptr()
        del first
        with torch.cuda.stream(side):
            here = call(None)
            assert here.data_ptr() != at
            side_at = here.data_ptr()
            del here
            for s in (torch.cuda.default_stream(), 0):
                got = call(s)
                assert got.data_ptr() == at and got.data_ptr() != side_at
                del got
            again = call(side)
            assert again.data_ptr() == side_at
            del again
        torch.cuda.synchronize()


def test_plain_forwards_for_another_stream():
    N, K, T = 64, 128, 16
    _, arrays = make_experts(1, N, K, FMT_RVQ12_4, 64, 23)
    L = vq.VQLinear(N, K, FMT_RVQ12_4, 64, DT_BF16, T, {k: v[0] for k, v in arrays.items()}, rht=1)
    x, signs, side = randn((T, K), DT_BF16, 1), torch.ones(K, dtype=torch.int8, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in (lambda s: L.forward(x, stream=s), lambda s: L.forward_rotated(x, signs, stream=s)):
        here = call(None)
        at = here.data_ptr()
        del here
        for s in (side, side.cuda_stream):
            assert call(s).data_ptr() != at
        with torch.cuda.stream(side):
            for s in (torch.cuda.default_stream(), 0):
                assert call(s).data_ptr() == at
        torch.cuda.synchronize()


@pytest.mark.parametrize("tokens", [1, 40, 600])
def test_operators_of_several_streams_at_once(tokens):
    """Blocks of experts on two streams (handles of their own) beside dense fused forwards on a third, none waiting
    for another: the results of the calls one after another, bit for bit."""
    E, k, H, I = 16, 4, 512, 384
    made = []
    for seed in (31, 32):
        _, up = make_experts(E, 2 * I, H, FMT_RVQ12_4, 64, seed)
        _, down = make_experts(E, H, I, FMT_RVQ12_4, 64, seed + 10)
        R = vq.VQRouter(E, k, tokens, renorm=True)
        U = vq.VQExperts(E, 2 * I, H, FMT_RVQ12_4, 64, DT_BF16, tokens * k, up, act=vq.VQ_ACT_SILU, glu=True)
        D = vq.VQExperts(E, H, I, FMT_RVQ12_4, 64, DT_BF16, tokens * k, down)
        x, logits = randn((tokens, H), DT_BF16, seed), randn((tokens, E), DT_BF16, seed + 1)

        def block(s, R=R, U=U, D=D, x=x, logits=logits):
            r = R.forward(logits, stream=s)
            h = U.forward(x, r.offsets, rows=r.rows, stream=s)
            return vq.combine(D.forward(h, r.offsets, stream=s), r.weights, r.slots, residual=x, stream=s)

        made.append(block)
    _, arrays = make_experts(1, 2048, 1024, FMT_RVQ12_4, 64, 51)
    L = vq.VQLinear(2048, 1024, FMT_RVQ12_4, 64, DT_BF16, 600, {n: v[0] for n, v in arrays.items()})
    xs = [randn((M, 1024), DT_BF16, M) for M in (1, 9, 64, 600)]
    made.append(lambda s: torch.cat([L.forward_fused(x, act=vq.VQ_ACT_GELU, stream=s) for x in xs]))
    torch.cuda.synchronize()
    want = [call(None) for call in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = [[] for _ in made]
    for _ in range(25):
        for i, call in enumerate(made):
            with torch.cuda.stream(streams[i]):
                got[i].append(call(streams[i] if i % 2 else None))
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        assert all(torch.equal(y.view(torch.int16), w.view(torch.int16)) for y in many)
    vq.vq_linear_check(L.handle)
