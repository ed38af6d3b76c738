"""Where the join of shared prefixes reads the parts of a row block (csrc/parts.cuh): inside of the workspace whatever
the description of the row block holds, as after a wait that gave up it was never written."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_rejection_spec_gb300", "csrc")
EDGES = [-2 ** 31, -2 ** 31 + 1, -2, -1, 0, 1, 2, 2 ** 31 - 2, 2 ** 31 - 1]


@pytest.fixture(scope="module")
def parts(tmp_path_factory):
    where = tmp_path_factory.mktemp("parts")
    source, library = where / "parts.cpp", where / "parts.so"
    source.write_text('#include "parts.cuh"\nextern "C" bool within(int32_t f, int32_t n, int32_t b) '
                      '{ return specrej::parts_within(f, n, b); }\n'
                      'extern "C" int64_t place(int32_t f, int32_t j, int32_t m, int32_t row) '
                      '{ return specrej::part_place(f, j, m, row); }\n')
    subprocess.check_call(["g++", "-std=c++17", "-shared", "-fPIC", "-w", "-I", CSRC, str(source), "-o", str(library)])
    lib = ctypes.CDLL(str(library))
    lib.within.restype, lib.within.argtypes = ctypes.c_bool, [ctypes.c_int32] * 3
    lib.place.restype, lib.place.argtypes = ctypes.c_int64, [ctypes.c_int32] * 4
    return lib


@pytest.mark.parametrize("blocks", [1, 2, 152, 160])
def test_whatever_stands_there_stays_inside(parts, blocks):
    rng = random.Random(blocks)
    near = [x + d for x in (0, blocks) for d in (-2, -1, 0, 1, 2)]
    pairs = [(f, n) for f in EDGES + near for n in EDGES + near]
    pairs += [(rng.randrange(-2 ** 31, 2 ** 31), rng.randrange(-2 ** 31, 2 ** 31)) for _ in range(2000)]
    pairs += [(rng.randrange(-3, blocks + 3), rng.randrange(-3, blocks + 3)) for _ in range(2000)]
    for first, count in pairs:
        fits = count == 0 or (count > 0 and first >= 0 and first + count <= blocks)
        assert parts.within(first, count, blocks) == fits, (first, count)
        if fits and count:
            for max_rows in (1, 36, 256):
                places = {parts.place(first, j, max_rows, row) for j in range(count) for row in (0, max_rows - 1)}
                assert min(places) >= 0 and max(places) < blocks * 2 * max_rows


def test_places_of_a_row_block_cut_in_three(parts):
    """The tail of the share of block 4, then the heads of 5's and 6's."""
    assert [parts.place(4, j, 100, 7) for j in range(3)] == [907, 1007, 1207]


def test_the_join_looks_before_it_reads():
    """Both descriptions of a row pass the check before anything is read from where they point."""
    src = open(os.path.join(CSRC, "attention.cuh")).read()
    body = src[src.index("join_shared_kernel(CacheView"):src.index("// Host")]
    look = body.index("parts_within")
    assert body.count("parts_within(") == 2 and look < body.index("place(k") and look < body.index("row_ml")
