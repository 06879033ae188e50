"""The rules that choose a kernel for the bf16 and int8 products: every kernel is reached, and what they say at
sizes whose best kernel is known."""
import pytest

import product_choice as choice


@pytest.mark.parametrize("c", choice.cases(), ids=choice.label)
def test_every_kernel_is_reached(c):
    bytes_, kind, name, past = c
    for behind in (0, 7):
        found = choice.case(name, past, bytes_, kind, behind)
        assert found is not None, choice.label(c)
        counts, N, K = found
        assert choice.product(counts, N, K, bytes_, kind, behind) == (name, past)


def test_known_sizes():
    # many rows, a tile's rows, few rows, few tiles
    assert choice.product([4096] * 8, 7168, 4096) == ("256x256", False)
    assert choice.product([500] * 8, 4096, 7168) == ("256x256", False)
    assert choice.product([500] * 7 + [600], 4096, 7168) == ("256x256 last in quarters", False)
    assert choice.product([500] * 2 + [600] * 6, 4096, 7168) == ("256x256 last in halves", False)
    assert choice.product([600] * 7 + [800], 4096, 7168) == ("256x256", False)
    assert choice.product([128] * 16, 2816, 4096) == ("256x128", True)
    assert choice.product([64] * 16, 2816, 4096) == ("256x64", True)
    assert choice.product([8] * 8, 4096, 7168) == ("128x64", True)
    assert choice.product([8], 4096, 7168)[0] == "narrow 32x32"
    assert choice.product([8] * 4, 2048, 4096)[0] == "narrow 32x32"


def test_uneven_rows():
    """One expert with more rows than a tile takes the tile that holds them."""
    assert choice.product([32] * 8, 4096, 7168, 1) == ("128x64", True)
    assert choice.product([94, 47, 31, 24, 19, 16, 13, 12], 4096, 7168, 1) == ("128x128", True)


def test_past_the_caches():
    """Only whole lines, large weights and rows that one tile holds."""
    assert choice.product([8] * 8, 4096, 7168) == ("128x64", True)
    assert choice.product([8] * 8, 4096, 7160) == ("128x64", False)             # rows of k off the lines
    assert choice.product([8] * 8, 4096, 7160, kind="transposed") == ("128x64", True)
    assert not choice.product([8] * 8, 512, 7168)[1]                              # 59 MB
    assert not choice.product([200] * 8, 4096, 7168)[1]


@pytest.mark.parametrize("E", [1, 3, 64, 1024])
def test_any_size_has_a_kernel(E):
    known = choice.KERNELS + list(choice.TAILS.values())
    for rows in (1, 2, 63, 1000, 1 << 19):
        for N in (8, 16, 1000, 1 << 17):
            for K in (8, 16, 1000, 1 << 17):
                for kind in ("plain", "gated"):
                    assert choice.product([rows] * E, N, K, kind=kind)[0] in known
