"""Sizes at which a workgroup of the bf16 and int8 products' persistent kernel works through several tiles, found by the
library's own rules: the loads that run on into the next tile, the stores of the one before that are counted in the
first wait, and the stage that the epilogue leaves to the next loads."""
import functools

import product_choice as choice
from expert_choice import CUS

STAGES = {"256x256": 3, choice.TAILS[1]: 3, choice.TAILS[2]: 3, "256x128": 3, "128x128": 4, "256x64": 3,
          "128x64": 4}
BEHIND = 7                   # rows behind the last segment


def blocks(K, bytes_):
    return -(-K * bytes_ // 128)


def turns(name, counts, N, kind):
    """Tiles that the busiest workgroup has, whole ones."""
    weights, tokens = (int(v) for v in name.split()[0].split("x"))
    columns = weights // 2 if kind == "gated" else weights
    share = -(-sum(-(-c // tokens) for c in counts) * -(-N // columns) // 8)
    slots = CUS // 8
    return share // slots if name in choice.TAILS.values() else -(-share // slots)


def length(name, K, bytes_):
    """'short': a tile has fewer blocks of k than its loads are ahead; 'ahead': as many; 'long': more."""
    n, ahead = blocks(K, bytes_), STAGES[name] - 1
    return "short" if n < ahead else "ahead" if n == ahead else "long"


def _segments():
    for E in (1, 2, 4, 8, 16, 24, 40, 64, 100, 200):
        for rows in (1, 20, 40, 60, 64, 90, 120, 128, 140, 190, 250, 300, 400, 600, 1000, 1700, 3000, 5000):
            if E * rows <= 100_000:
                yield [rows + i % 3 if rows > 2 else rows for i in range(E)]


_COLUMNS = (16, 80, 128, 144, 208, 272, 400, 528, 784, 1040, 1408, 2064, 4096)
_LENGTHS = {2: (16, 64, 80, 128, 144, 192, 208, 272, 400, 528, 1040, 2048, 4096),
            1: (16, 64, 128, 144, 256, 272, 384, 400, 528, 1040, 2064, 4096)}


@functools.lru_cache(maxsize=None)
def _found():
    best = {}
    for bytes_, kind in ((2, "plain"), (2, "transposed"), (2, "gated"), (1, "plain"), (1, "gated")):
        for counts in _segments():
            E, S = len(counts), sum(counts)
            for N in _COLUMNS:
                for K in _LENGTHS[bytes_]:
                    cost = (S + BEHIND) * (N + K) + E * N * K * (2 if kind == "gated" else 1)
                    if cost > 1 << 30:
                        continue
                    name, past = choice.product(counts, N, K, bytes_, kind, BEHIND)
                    if name not in STAGES or turns(name, counts, N, kind) < 2:
                        continue
                    key = bytes_, kind, name, past, length(name, K, bytes_)
                    if key not in best or cost < best[key][0]:
                        best[key] = cost, (counts, N, K)
    return {k: v[1] for k, v in best.items()}


def case(c):
    """The least size of a key: (rows of each expert, columns, K); None where there is none."""
    return _found().get(c)


def cases():
    """(bytes, kind, kernel, past the caches, length) of everything found."""
    return sorted(_found())


def label(c):
    return f"{choice.label(c[:4])}-{c[4]}"
