"""The library's choice of kernel for the bf16 and int8 products (csrc/experts/expert_choice.h), compiled for
the host: tests use it to know that their sizes reach the kernel they are for."""
import ctypes
import functools
import os
import subprocess
import tempfile

from expert_choice import CUS, HEADER

TAILS = {1: "256x256 last in halves", 2: "256x256 last in quarters"}
KERNELS = ["256x256", "256x128", "128x128", "256x64", "128x64", "narrow 64x64", "narrow 32x32",
           "narrow 32x32 paired"]
# tokens of the tiles that may read the weights past the caches
TOKENS = {"256x256": 256, TAILS[1]: 256, TAILS[2]: 256, "256x128": 128, "128x128": 128, "256x64": 64,
          "128x64": 64}

SHIM = f"""
#include "{HEADER}"
extern "C" int product(long long S, long long N, long long row_bytes, long long E, int gated, long long cus) {{
    return ep::choose_product(S, N, row_bytes, E, gated != 0, cus);
}}
extern "C" int tile(int t64, int t128, int t256, int N, int blocks, int gated, int cus) {{
    return ep::choose_product_tile(t64, t128, t256, N, blocks, gated != 0, cus);
}}
extern "C" int tail(int rest, int slots) {{ return ep::product_tail(rest, slots); }}
extern "C" int whole(long long N, long long row_bytes, long long E, int gated, long long line) {{
    return ep::product_whole_lines(N, row_bytes, E, gated != 0, line);
}}
extern "C" int past(int row_tiles, int used, int whole) {{
    return ep::product_past_caches(row_tiles, used, whole != 0);
}}
"""


@functools.lru_cache(maxsize=None)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, lib = os.path.join(d, "shim.cpp"), os.path.join(d, "shim.so")
        with open(src, "w") as f:
            f.write(SHIM)
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", "-o", lib, src],
                       check=True)
        h = ctypes.CDLL(lib)
    h.product.argtypes = [ctypes.c_longlong] * 4 + [ctypes.c_int, ctypes.c_longlong]
    h.whole.argtypes = [ctypes.c_longlong] * 3 + [ctypes.c_int, ctypes.c_longlong]
    return h


def product(counts, N, K, bytes_=2, kind="plain", behind=0):
    """(kernel's name, whether its weights go past the caches) for so many rows of each expert and `behind` of
    none.  N: columns of the result."""
    h, E, S, gated = _lib(), len(counts), sum(counts) + behind, int(kind == "gated")
    k = h.product(S, N, K * bytes_, E, gated, CUS)
    if KERNELS[k].startswith("narrow"):
        return KERNELS[k], False
    tiles = {t: sum(-(-c // t) for c in counts) for t in (64, 128, 256)}
    name = KERNELS[h.tile(tiles[64], tiles[128], tiles[256], N, -(-K * bytes_ // 128), gated, CUS)]
    if name == "256x256":
        slots, all_ = CUS // 8, -(-tiles[256] * -(-N // (128 if gated else 256)) // 8)
        if all_ > slots and all_ % slots:
            name = TAILS.get(h.tail(all_ % slots, slots), name)
    line = (N if kind == "transposed" else K) * bytes_
    whole = h.whole(N, K * bytes_, E, gated, line)
    return name, name in TOKENS and bool(h.past(tiles[TOKENS[name]], sum(c > 0 for c in counts), whole))


# Segments (rows of each expert), columns and lengths of k that between them reach every kernel
_SEGMENTS = ([5, 9, 3], [1, 0, 2], [1000, 0, 1], [500, 0, 400, 3], [250] * 4, [1] * 8 + [0] * 8, [10] * 8, [64] * 8,
             [96] * 8, [100, 0, 90, 1], [60] * 16, [11] * 15 + [100], [128] * 16, [45] * 18, [130] * 30,
             [3000, 0, 4000, 1, 2999], [4] * 64, [300] * 70, [2] * 100, [60] * 44,
             [3000, 700, 0, 800], [1100, 1300, 1200, 900], [700] * 7 + [2000], [250] * 35, [250] * 18)
_COLUMNS = (80, 144, 208, 264, 272, 520, 528, 784, 1040, 1408, 2064, 2816, 4096)
_LENGTHS = (80, 144, 272, 336, 400, 528, 1040, 1152, 2064, 4096, 7168)


@functools.lru_cache(maxsize=None)
def case(name, past, bytes_, kind, behind=0):
    """The least case that reaches a kernel: (rows of each expert, columns, K); None if there is none."""
    best = None
    for counts in _SEGMENTS:
        for N in _COLUMNS:
            for K in _LENGTHS:
                E, S = len(counts), sum(counts) + behind
                if bytes_ == 1 and (N % 16 or K % 16):
                    continue
                cost = E * N * K * (2 if kind == "gated" else 1) + S * (N + K)
                if best is not None and cost >= best[0]:
                    continue
                if product(counts, N, K, bytes_, kind, behind) == (name, past):
                    best = (cost, (counts, N, K))
    return best[1] if best else None


def cases():
    """(bytes, kind, kernel, past the caches) of everything that a call can launch."""
    return [(b, kind, name, past) for b in (2, 1) for kind in ("plain", "transposed", "gated")
            if (b, kind) != (1, "transposed") for name in KERNELS + list(TAILS.values())
            for past in (False, True)
            if not past or name in TOKENS]


def label(c):
    return f"{'bf16' if c[0] == 2 else 'int8'} {c[1]} {c[2]}{' past' if c[3] else ''}".replace(" ", "-")
