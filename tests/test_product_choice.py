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
        got = choice.product(sum(counts) + behind, N, K, len(counts), bytes_, kind == "gated",
                             kind == "transposed")
        assert got == (name, past)


def test_known_sizes():
    # rows, columns, K, experts: many rows, a tile's rows, few rows, few tiles
    assert choice.product(32768, 7168, 4096, 8) == ("256x256", False)
    assert choice.product(4000, 4096, 7168, 8) == ("256x256", False)
    assert choice.product(16 * 48, 2816, 4096, 16) == ("256x64", True)
    assert choice.product(64, 4096, 7168, 8) == ("128x64", True)
    assert choice.product(8, 4096, 7168, 1)[0] == "narrow 32x32"
    assert choice.product(32, 2048, 4096, 4)[0] == "narrow 32x32"


def test_past_the_caches():
    """Only whole lines, large weights and rows that one tile holds."""
    assert choice.product(64, 4096, 7168, 8) == ("128x64", True)
    assert choice.product(64, 4096, 7160, 8) == ("128x64", False)             # rows of k off the lines
    assert choice.product(64, 4096, 7160, 8, transposed=True) == ("128x64", True)
    assert not choice.product(64, 512, 7168, 8)[1]                              # 59 MB
    assert not choice.product(8 * 200, 4096, 7168, 8)[1]


@pytest.mark.parametrize("E", [1, 3, 64, 1024])
def test_any_size_has_a_kernel(E):
    for S in (1, 2, 63, 1000, (1 << 30) - 1):
        for N in (8, 16, 1000, 1 << 17):
            for K in (8, 16, 1000, 1 << 17):
                for gated in (False, True):
                    assert choice.product(S, N, K, E, 2, gated)[0] in choice.KERNELS
