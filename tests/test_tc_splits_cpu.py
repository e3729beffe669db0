"""The tensor-core forward's K splits at the shapes that test_gpu_tc_splits.py runs: a change of the
plan that moves one of them to another branch of the kernel's epilogue fails here first."""

import pytest

import compressed_index_matmul_b200 as vq
from compressed_index_matmul_b200 import build as libbuild
from synth import DT_BF16, DT_F16, FMT_RVQ12, FMT_RVQ12_4, FMT_VQ16, FMT_VQ16_RVQ

LADDER = {5: dict(n16=2, n8=1, mult=(0.5, 0.25))}

# (N, K, fmt, bits per weight of a ladder, dtype, M, splits, CTAs).  A CTA sums 128 rows of W by up to 256 tokens.
CASES = [
    # Token tiles of 64 and more, one CTA per SM
    (2040, 512, FMT_RVQ12_4, 0, DT_BF16, 300, 1, 32),     # one split: y by bulk stores, ragged rows and tokens
    (1003, 576, FMT_RVQ12, 0, DT_F16, 100, 1, 8),         # one split, odd N: y per element
    (2048, 2048, FMT_RVQ12_4, 0, DT_BF16, 256, 2, 32),    # a pair over a cluster
    (384, 512, FMT_VQ16, 0, DT_F16, 100, 2, 6),
    (1024, 14336, FMT_RVQ12_4, 0, DT_BF16, 128, 7, 56),   # partial sums, the last CTA of a tile adds them
    (2048, 8192, FMT_RVQ12, 0, DT_F16, 100, 5, 80),
    (1003, 4096, FMT_RVQ12_4, 0, DT_BF16, 100, 4, 32),    # the same with odd N
    (300, 14336, FMT_RVQ12_4, 0, DT_F16, 300, 4, 24),     # two token tiles, 44 tokens in the second, ragged rows
    (1024, 8192, FMT_VQ16, 0, DT_BF16, 100, 8, 64),
    (1003, 4096, FMT_VQ16_RVQ, 5, DT_F16, 70, 8, 64),
    (264, 384, FMT_VQ16_RVQ, 5, DT_BF16, 100, 2, 6),      # the ladder as a pair
    (4096, 4096, FMT_RVQ12_4, 0, DT_F16, 64, 4, 128),     # 64 tokens, too many splits for two CTAs per SM
    # 64 tokens, two CTAs per SM, three x stages
    (14336, 2048, FMT_RVQ12_4, 0, DT_BF16, 64, 2, 224),   # a pair
    (256, 1024, FMT_RVQ12, 0, DT_F16, 64, 2, 4),
    (14336, 1024, FMT_RVQ12_4, 0, DT_F16, 64, 1, 112),    # one split
    (1003, 1024, FMT_RVQ12_4, 0, DT_BF16, 64, 1, 8),      # odd N
    # 16 to 48 tokens, two CTAs per SM
    (136, 2048, FMT_RVQ12_4, 0, DT_F16, 48, 2, 4),
    (256, 8192, FMT_RVQ12_4, 0, DT_BF16, 33, 8, 16),
    (1003, 8192, FMT_RVQ12, 0, DT_F16, 48, 8, 64),
    # 16-bit indices, 16 to 48 tokens, one CTA per SM
    (1024, 8192, FMT_VQ16, 0, DT_F16, 24, 8, 64),
    (264, 1024, FMT_VQ16, 0, DT_BF16, 40, 2, 6),
    (264, 2048, FMT_VQ16_RVQ, 5, DT_BF16, 40, 8, 24),
]


def case_id(c):
    return f"{c[0]}x{c[1]}f{c[2]}M{c[5]}S{c[6]}"


@pytest.mark.parametrize("case", CASES, ids=case_id)
def test_splits_on_a_b200(case):
    libbuild.build()
    N, K, fmt, bpw, dt, M, splits, ctas = case
    p = vq.vq_plan_for_device(N, K, fmt, 64, dt, M, M, path=vq.VQ_PATH_TC, **LADDER.get(bpw, {}))
    assert (p["path"], p["launches"], p["splits"], p["ctas"]) == (vq.VQ_PATH_TC, 1, splits, ctas)


# (N, K, fmt, bits per weight, M, fewest splits): us with those splits or more / with 2.
@pytest.mark.parametrize("N,K,fmt,bpw,M,fewest", [
    (288, 8896, FMT_VQ16_RVQ, 6, 279, 7),     # 106 / 271
    (840, 5696, FMT_VQ16_RVQ, 6, 216, 6),     # 80 / 182
    (2592, 2432, FMT_VQ16_RVQ, 8, 79, 7),     # 38 / 78
    (1184, 1472, FMT_VQ16_RVQ, 6, 36, 6),     # 20 / 32
    (160, 768, FMT_VQ16_RVQ, 8, 18, 6),       # 19 / 26
    (1144, 2816, FMT_VQ16_RVQ, 4, 600, 3),    # 65 / 68
    (168, 8896, FMT_VQ16, 2, 545, 5),         # 59 / 86
])
def test_a_slower_decode_keeps_more_splits(N, K, fmt, bpw, M, fewest):
    """A residual stage is one more gather per group: what a split saves grows with the stages, what the sum
    over the splits costs does not."""
    libbuild.build()
    ladder = dict(n16=bpw // 2, n8=bpw % 2, mult=(0.5,) * (bpw // 2 + bpw % 2 - 1)) if fmt == FMT_VQ16_RVQ else {}
    p = vq.vq_plan_for_device(N, K, fmt, 64, DT_F16, M, M, path=vq.VQ_PATH_TC, **ladder)
    assert p["splits"] >= fewest
