"""GPU tests of the grouped products where a block goes on: from tile to tile over several slices of K,
from expert to expert with codebooks of their own, on both kernels, against the definition in 64 bits."""

import numpy as np
import pytest
import torch

import compressed_index_matmul_b200 as vq
from synth import DT_BF16, DT_F16, FMT_RVQ12, FMT_RVQ12_4, FMT_VQ16, FMT_VQ16_RVQ
from tests.gpu_util import require_gpu
from tests.test_gpu_experts import offsets_of, randn, run

pytestmark = pytest.mark.gpu

GEMV, TC = vq.VQ_PATH_GEMV, vq.VQ_PATH_TC


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def pair_tiles(N, glu, counts, rows):
    """Tiles of the tensor-core kernel: 256 rows of W (glu: of the two halves together) by up to `rows`."""
    return -(-N // 256) * sum(-(-c // rows) for c in counts)


# (E, N, K, fmt, scale group (0: per row), dtype, rows per expert, rows of a tile, glu, shared)
PAIRS = [
    # Two accumulators (up to 128 rows a tile), 3 and 5 slices of K, more than two tiles a pair
    (24, 1792, 320, FMT_RVQ12_4, 64, DT_BF16, [50, 0, 64, 37] * 6, 128, False, False),
    (24, 2048, 576, FMT_RVQ12, 0, DT_F16, [33, 90, 64, 1] * 6, 128, True, False),
    # One accumulator (up to 256 rows), plain and gated
    (6, 2304, 576, FMT_RVQ12_4, 64, DT_BF16, [300, 257, 513, 0, 90, 300], 256, False, False),
    (6, 2064, 448, FMT_RVQ12_4, 64, DT_F16, [300, 257, 513, 0, 90, 300], 256, True, False),
    (6, 2304, 320, FMT_RVQ12, 64, DT_BF16, [300, 257, 513, 0, 90, 300], 256, True, True),
    # 16-bit indices and the ladder, an 8-bit stage of its own per expert among them
    (5, 2560, 704, FMT_VQ16, 64, DT_BF16, [300, 257, 513, 90, 300], 256, False, False),
    (5, 2560, 320, FMT_VQ16_RVQ, 64, DT_F16, [300, 257, 513, 90, 300], 256, True, False),
    # A tile an expert, four and more experts a pair: the codebook is replaced again and again
    (300, 256, 320, FMT_RVQ12_4, 64, DT_BF16, [(7 * i) % 31 for i in range(300)], 128, False, False),
    (300, 256, 192, FMT_RVQ12, 0, DT_F16, [(7 * i) % 31 for i in range(300)], 128, True, False),
    (300, 144, 64, FMT_RVQ12_4, 64, DT_BF16, [(7 * i) % 31 for i in range(300)], 128, False, False),  # one slice
]


@pytest.mark.parametrize("case", PAIRS, ids=lambda c: f"E{c[0]}N{c[1]}K{c[2]}f{c[3]}T{c[7]}g{int(c[8])}")
def test_a_pair_goes_on_to_further_tiles(oracle, case):
    E, N, K, fmt, sg, dt, counts, tile_rows, glu, shared = case
    X, x, off, rows, y = run(oracle, E, N, K, fmt, sg, dt, counts, TC, act="silu" if glu else "none", glu=glu, bias=True,
                             shared=shared, bpw=3)
    pairs, T = X.plan(len(y))["ctas"] // 2, sum(counts)
    assert tile_rows == (128 if T <= 64 * min(E, T) else 256)
    tiles = pair_tiles(N, glu, counts, tile_rows)
    assert tiles > 1.2 * pairs and (E < 300 or tiles > 3.5 * pairs), (tiles, pairs)
    # the same rows in order, without `rows`
    direct = X.forward(x[rows.long()], off)
    assert torch.equal(direct.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("K,wk", [(64, 1), (320, 2), (2048, 16)])
@pytest.mark.parametrize("fmt,sg,dt", [(FMT_RVQ12_4, 64, DT_BF16), (FMT_RVQ12, 0, DT_F16)])
def test_a_block_replaces_its_codebooks(oracle, fmt, sg, dt, K, wk):
    """The few-row kernel keeps two codebooks a block; 600 busy experts give each block four or more, with
    one, two and sixteen warps a tile (wk)."""
    E, counts = 600, [1 + i % 2 for i in range(600)]
    X, *_ = run(oracle, E, 32, K, fmt, sg, dt, counts, GEMV, bias=True)
    assert E >= 4 * X.plan(len(counts))["ctas"]


def test_a_block_replaces_its_8_bit_codebooks(oracle):
    run(oracle, 330, 48, 192, FMT_VQ16_RVQ, 64, DT_F16, [1 + i % 2 for i in range(330)], GEMV, bpw=3)


@pytest.mark.parametrize("path", [GEMV, TC])
def test_one_long_expert_among_many_short_ones(oracle, path):
    """Blocks of one long expert's tiles beside blocks that meet dozens of experts; experts without rows between."""
    counts = [0, 1, 2, 0, 3] * 60
    counts[37] = 1500
    run(oracle, 300, 64, 320, FMT_RVQ12_4, 64, DT_BF16, counts, path, bias=True)


@pytest.mark.parametrize("glu", [False, True])
def test_many_tiles_many_times(glu):
    """The same calls again and again, other calls between, give the same bits (the rings' steady state)."""
    E, N, K, T = 24, 1792, 576, 1500
    g = np.random.default_rng(3)
    arrays = {"lo": g.integers(0, 256, (E, N * K // 8), dtype=np.uint8), "hi4": g.integers(0, 256, (E, N * K // 16), dtype=np.uint8),
              "s2": g.integers(0, 256, (E, N * K // 16), dtype=np.uint8),
              "cb1": g.standard_normal((E, 4096, 8)).astype(np.float16), "cb2": g.standard_normal((E, 16, 8)).astype(np.float16),
              "scales": g.uniform(0.01, 0.03, (E, N * K // 64)).astype(np.float16)}
    X = vq.VQExperts(E, N, K, FMT_RVQ12_4, 64, DT_BF16, T, arrays, glu=glu)
    X.set_path(TC)
    x = randn((T, K), DT_BF16, 4)
    calls = []
    for seed, skew in ((1, 0.0), (2, 2.0), (3, 6.0)):
        p = np.exp(skew * np.random.default_rng(seed).standard_normal(E))
        off = offsets_of(np.random.default_rng(seed).multinomial(T, p / p.sum()))
        rows = torch.randperm(T, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
        calls.append((off, rows, X.forward(x, off, rows=rows)))
    for _ in range(60):
        for off, rows, want in calls:
            assert torch.equal(X.forward(x, off, rows=rows).view(torch.int16), want.view(torch.int16))
    vq.vq_experts_check(X.handle)
