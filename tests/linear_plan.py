"""What nm_linear launches for a call, worked out apart from the library: which kernel, which instance of
it, in how many reduction ranges.  The estimate's constants are read from the source; the rest repeats
plan_linear, few_plan and mid_plan, and test_linear_cpu.py holds it against the workspace that the
library asks for."""
import math
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "semi_structured_sparse_amd", "csrc")


def _up(v, m):
    return -(-v // m)


def _constants():
    with open(os.path.join(SRC, "linear_tile.hip")) as f:
        text = f.read()

    def numbers(name):
        body = re.search(r"\b%s(?:\[\d+\])+ = (\{\{.*?\}\}|\{[^{}]*\})" % name, text).group(1)
        rows = [[{"true": True, "false": False}.get(v.strip()) if v.strip() in ("true", "false") else float(v)
                 for v in r.split(",")] for r in re.findall(r"\{([^{}]*)\}", body)]
        return rows if body.startswith("{{") else rows[0]

    return {n: numbers(n) for n in ("kBM", "kBN", "kRanges", "kChunk", "kAlone")}


K = _constants()


def mid_plan(t, o, k, sparse):
    """(tile shape, reduction ranges) of k_lin_tile."""
    chunks = _up(k, 64)
    stream = float(o) * float(k) * (1.125 if sparse else 2.0) / 5.0e6
    best, least = (3, 1), 0.0
    for sh in (3, 2, 1, 0):
        tiles = float(_up(o, int(K["kBM"][sh]))) * float(_up(t, int(K["kBN"][sh])))
        for r in (int(v) for v in K["kRanges"]):
            if r > 1 and (chunks < 8 * r or tiles * r > 1024):
                break
            full = tiles * r / 256
            rounds = 1.0 if full <= 1.0 else math.ceil(full) if K["kAlone"][sparse][sh] else full
            us = float(_up(chunks, r)) * K["kChunk"][sparse][sh] * rounds
            us = max(us, stream)
            if r > 1:
                us += 2.8 + float(r) * float(t) * float(o) * 8 / 3.2e6
            if (sh == 3 and r == 1) or us < least:
                least, best = us, (sh, r)
    return best


def few_plan(t, o, k, sparse):
    """(blocks of 16 tokens, blocks of 16 rows, waves, reduction ranges) of k_lin_few."""
    tb = 1 if t <= 16 else 2 if t <= 32 else 4
    steps = _up(k, 64 if sparse else 32)
    gy = _up(t, 16 * tb)
    rw = 1 if tb > 2 else 2 if tb == 2 else 4
    while rw > 1 and _up(o, 16 * rw) * gy < 200:
        rw //= 2
    blocks = _up(o, 16 * rw) * gy
    waves = 4 if blocks >= 192 else 8
    s = min(256 // blocks, steps // (4 * waves))
    if steps <= 8 * waves:
        s = 1
    splits = 1 if s < 2 else min(s, 16)
    if blocks <= 32 and splits == 1 and tb < 4 and steps >= 32:
        waves = 16
    return tb, rw, waves, splits


def plan(t, o, k, sparse, route=None):
    """('few', tb, rw, waves, ranges), ('tile', shape, ranges) or ('large',); route: None, 'few_stream',
    'few_tile' or 'tile_lds'."""
    sparse = bool(sparse)
    if route == "few_stream" or (route is None and t <= 16 and o < 8192 and t * k <= (16384 if sparse else 32768)):
        return ("few", *few_plan(t, o, k, sparse))
    if route == "tile_lds" or (route is None and _up(o, 256) * _up(t, 256) >= 160):
        return ("large",)
    return ("tile", *mid_plan(t, o, k, sparse))


def workspace(t, o, k, sparse, route=None):
    p = plan(t, o, k, sparse, route)
    return 0 if p[-1] in ("large", 1) else p[-1] * t * (_up(o, 4) * 4) * 4


def instance(p, sparse):
    """What of a plan is compiled or launched apart: the kernel's instance, split or whole."""
    return (bool(sparse), "large") if p[0] == "large" else (bool(sparse), *p[:-1], p[-1] > 1)


# (tokens, outputs, reduction, route): rows that end inside a piece, tiles and blocks that the tokens and
# outputs do not fill.  Together they run every instance.
DENSE = [(1, 33, 995, None), (3, 3165, 1033, None), (5, 37, 209, None), (7, 33, 2231, None), (2, 6769, 219, None),
         (9, 12797, 213, "few_stream"), (19, 33, 1031, "few_stream"), (31, 3169, 213, "few_stream"),
         (25, 41, 209, "few_stream"), (29, 35, 2325, "few_stream"), (17, 6371, 241, "few_stream"),
         (67, 1631, 215, "few_stream"), (50, 65, 333, "few_stream"), (45, 33, 2381, "few_stream"),
         (1, 4096, 4096, None), (129, 11077, 213, None), (1567, 65, 9375, None), (67, 12273, 215, None),
         (67, 887, 8161, None), (777, 1025, 1999, None), (257, 385, 6001, None), (40, 300, 259, None),
         (100, 385, 6001, None), (600, 4096, 4095, None), (16, 4096, 4096, None)]
SPARSE = [(1, 33, 1996, None), (3, 3109, 1028, None), (5, 37, 212, None), (3, 33, 4708, None), (2, 6441, 212, None),
          (9, 12875, 216, "few_stream"), (19, 33, 1996, "few_stream"), (31, 3309, 212, "few_stream"),
          (25, 41, 228, "few_stream"), (29, 35, 4572, "few_stream"), (17, 6519, 212, "few_stream"),
          (67, 1677, 216, "few_stream"), (50, 65, 332, "few_stream"), (45, 35, 4428, "few_stream"),
          (1, 4096, 4096, None), (135, 10991, 232, None), (1513, 133, 7048, None), (67, 11355, 212, None),
          (33, 1899, 6420, None), (101, 7037, 216, None), (33, 2529, 4916, None), (40, 300, 260, None),
          (257, 385, 6004, None), (128, 4096, 4100, None), (16, 4096, 4096, None)]
# 17 x 18 tiles of 256 x 256: over a round of the chip, the last band of the tile order not whole
LARGE = [(4200, 4400, 1024), (4200, 4400, 200)]
