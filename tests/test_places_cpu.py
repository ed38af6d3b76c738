"""The bound on a request's places in attention's list of work (csrc/places.cuh) against the tiles counted one by one:
never below them, and for windows not growing with the context."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_rejection_spec_gb300", "csrc")
LIMIT = 2 ** 31 - 1
ROWS, TILE = 256, 128
BEGIN, COST = 14, 5  # of a row block and of a tile, at most


@pytest.fixture(scope="module")
def places(tmp_path_factory):
    where = tmp_path_factory.mktemp("places")
    source, library = where / "places.cpp", where / "places.so"
    source.write_text('#include "places.cuh"\n'
                      'extern "C" int64_t places(int64_t r, int64_t k, int b, int t, int n) '
                      '{ return specrej::most_places(r, k, b, t, n); }\n'
                      'extern "C" int64_t keys(int64_t c, int64_t t, int64_t w, int64_t s, int b) '
                      '{ return specrej::most_window_keys(c, t, w, s, b); }\n')
    subprocess.check_call(["g++", "-std=c++17", "-shared", "-fPIC", "-w", "-I", CSRC, str(source), "-o", str(library)])
    lib = ctypes.CDLL(str(library))
    lib.places.restype, lib.places.argtypes = ctypes.c_int64, [ctypes.c_int64] * 2 + [ctypes.c_int] * 3
    lib.keys.restype, lib.keys.argtypes = ctypes.c_int64, [ctypes.c_int64] * 4 + [ctypes.c_int]
    return lib


def bound(lib, n, group, length, window=None, sinks=0, box=8, tree=False, shared=0):
    """What the kernel compares with the limit."""
    keys = length + n - shared
    if window is not None:
        keys = lib.keys(keys, n if tree else min(n, ROWS // group + 2), window, sinks, box)
    return lib.places(-(-n * group // ROWS), keys, BEGIN, COST, TILE)


def counted(n, group, length, window=None, sinks=0, box=8, tree=False, shared=0):
    """The places of every row block, its keys found as the sinks', the window's of its first row, and its own, in whole
    copies of `box` keys."""
    total = 0
    for m in range(0, n * group, ROWS):
        end = length + (min(m + ROWS, n * group) - 1) // group + 1
        keys = end - shared
        if window is not None:
            low = max(length + (0 if tree else m // group) - window + 1, 0) // box * box
            keys = end if low <= -(-sinks // box) * box else end - low + -(-sinks // box) * box
        total += BEGIN + COST * -(-keys // TILE)
    return total


@pytest.mark.parametrize("tree", [False, True])
def test_no_row_block_is_counted_short(places, tree):
    rng = random.Random(tree)
    for _ in range(3000):
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 71, 127, 128])
        n = rng.randrange(1, 129 if tree else 2000)
        length = rng.randrange(0, 1 << rng.randrange(1, 20))
        kw = dict(tree=tree, box=rng.choice([8, 16, 32, 64, 128]))
        if rng.randrange(4):
            kw.update(window=rng.randrange(1, 1 << rng.randrange(1, 20)), sinks=rng.choice([0, 1, 5, 129, 100000, 2 ** 30 - 1]))
        else:
            kw.update(shared=rng.randrange(0, length + 1))
        exact, most = counted(n, group, length, **kw), bound(places, n, group, length, **kw)
        assert exact <= most, (n, group, length, kw)


def test_long_prompts_over_a_window_are_within_the_limit(places):
    for n, group in ((185000, 128), (524000, 16), (2 ** 20, 128)):
        assert bound(places, n, group, 0, window=1024) <= LIMIT
        assert counted(n, group, 0, window=1024) <= LIMIT
    for length in (0, 10 ** 6, 2 ** 30 - 70000):  # whatever the context
        assert bound(places, 66000, 128, length, window=1024, sinks=4) <= 66000 // 2 * (BEGIN + COST * 12)
    assert bound(places, 66, 128, 2 ** 29, shared=2 ** 29 - 4096) <= 33 * (BEGIN + COST * 34)


def test_the_bound_does_not_wrap(places):
    """The largest sizes that pass the host's checks."""
    rows = (2 ** 30 - 1) // ROWS + 1
    assert places.places(rows, 2 ** 30 - 1, BEGIN, COST, TILE) == rows * (BEGIN + COST * 2 ** 23) > LIMIT
    assert places.keys(2 ** 30 - 1, 2 ** 30 - 1, 2 ** 30 - 1, 2 ** 30 - 1, 128) == 2 ** 30 - 1
