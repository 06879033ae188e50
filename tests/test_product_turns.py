"""Every shape of the products' persistent kernel is reached with several tiles for a workgroup, at lengths of k on both
sides of how far its loads are ahead."""
import pytest

import product_choice as choice
import product_turns as turns

SHAPES = [c for c in choice.cases() if c[2] in turns.STAGES]


@pytest.mark.parametrize("c", SHAPES, ids=choice.label)
def test_every_shape_has_several_turns(c):
    bytes_, kind, name, past = c
    lengths = {"long"}
    if not past and name not in choice.TAILS.values():
        lengths |= {"short", "ahead"}                # a last round in pieces, and weights past the caches: where found
    for n in lengths:
        found = turns.case(c + (n,))
        assert found is not None, (choice.label(c), n)
    for n in ("short", "ahead", "long"):
        if (found := turns.case(c + (n,))) is not None:
            counts, N, K = found
            assert choice.product(counts, N, K, bytes_, kind, turns.BEHIND) == (name, past)
            assert turns.turns(name, counts, N, kind) >= 2 and turns.length(name, K, bytes_) == n


def test_turns():
    """Counted by hand: 8 shares of 32 workgroups."""
    assert turns.turns("128x128", [128] * 64, 512, "plain") == 1        # 256 tiles
    assert turns.turns("128x128", [129] * 64, 512, "plain") == 2        # 512
    assert turns.turns("128x128", [128] * 64, 520, "plain") == 2        # 320
    assert turns.turns("128x128", [128] * 64, 512, "gated") == 2        # 512
    assert turns.turns(choice.TAILS[1], [256] * 40, 4096, "plain") == 2  # 640 tiles: two rounds and half of one
    assert [turns.length("128x64", k, 2) for k in (64, 128, 136, 192, 193)] == ["short", "short", "ahead", "ahead",
                                                                               "long"]
    assert [turns.length("256x64", k, 1) for k in (128, 144, 256, 272)] == ["short", "ahead", "ahead", "long"]
