"""The cache's kernels compiled for the host (tests/emulated: a block's threads are host threads) on memory that ends
where they may read no further: rows of padding are not read, by rotated append no table columns behind the pages held,
and rows land where they belong."""
import json
import os
import re
import shutil
import subprocess
import sys

import pytest

TESTS = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(TESTS)
CSRC = os.path.join(ROOT, "speculative_decoding_rejection_spec_gb300", "csrc")
CUDA = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    where = tmp_path_factory.mktemp("emulated")
    shutil.copy(os.path.join(TESTS, "emulated", "common.cuh"), where)
    for name in ("cache.cuh", "cache.cu", "rotate.cu"):
        source = open(os.path.join(CSRC, name)).read()
        source = re.sub(r'asm volatile\("griddepcontrol[^;]*;"[^;]*;', "", source)
        source = re.sub(r'asm volatile\("ld\.global.*?\(p\)\);', "r = *static_cast<const uint4 *>(p);", source, flags=re.S)
        assert "asm" not in source, name
        (where / name.replace(".cu", ".cpp") if name.endswith(".cu") else where / name).write_text(source)
    path = str(where / "emulated.so")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-w", "-shared", "-fPIC", "-pthread", "-I",
                           os.path.join(ROOT, "include"), "-isystem", CUDA, str(where / "cache.cpp"),
                           str(where / "rotate.cpp"), "-o", path])
    return path


def run(library, entry, **kw):
    p = subprocess.run([sys.executable, os.path.join(TESTS, "emulated", "reads.py"), library, entry, json.dumps(kw)],
                       capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, (p.returncode, p.stderr[-2000:])


@pytest.mark.parametrize("entry", ["append", "rotated"])
def test_rows_of_padding_are_not_read(library, entry):
    run(library, entry, n=[3, 5, 1], ctx=[10, 30, 0], held=[1, 3, 1], pad=60)
    if entry == "rotated":
        run(library, entry, n=[3, 5, 1], ctx=[10, 30, 0], held=[1, 3, 1], pad=60, interleaved=True, turn=32, tree=True)


def test_table_columns_behind_the_pages_held_are_not_read(library):
    """The last request's new tokens lie behind its pages, the first ones or all: those rows are skipped."""
    run(library, "rotated", n=[3, 5, 4], ctx=[10, 30, 30], held=[1, 3, 2], error=[32, 2])
    run(library, "rotated", n=[3, 5, 4], ctx=[10, 30, 32], held=[1, 3, 2], error=[32, 2])


def test_every_pass_of_a_warp_over_its_heads(library):
    """One, two and eight warps a token (two multiprocessors are made believe) and more heads than a pass takes."""
    for n, heads in (([20, 3, 30], 20), ([9, 0, 10], 40), ([1, 1, 1], 130)):
        run(library, "rotated", n=n, ctx=[10, 30, 0], held=[2, 3, 2], heads=heads, group=1, pad=2)
    run(library, "rotated", n=[20, 3, 30], ctx=[10, 30, 0], held=[2, 3, 2], heads=20, group=1, dim=40, turn=24, tree=True,
        interleaved=True)
