"""The paged cache without a GPU: exported symbols, the host's argument checks, the scratch sizes, and
the oracle of the bookkeeping on hand-made cases."""
import ctypes
import os
import re

import numpy as np
import pytest

import __graft_entry__ as G
from oracle import cache as oracle_cache
from speculative_decoding_rejection_spec_gb300 import cache

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 4096  # never dereferenced: the host checks fail first


@pytest.fixture(scope="module")
def lib():
    G.build()
    return cache.load()


def declared_functions():
    src = open(os.path.join(ROOT, "include", "spec_cache.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(spec_(?:cache|attention)\w*)\s*\(", src)))


def test_header_binding_and_library_agree(lib):
    assert set(cache.EXPORTED) == set(declared_functions())
    for name in declared_functions():
        assert hasattr(lib, name), f"{name} not exported"


def test_constants_match_the_header():
    src = open(os.path.join(ROOT, "include", "spec_cache.h")).read()
    define = lambda name: int(re.search(rf"#define {name} (\d+)", src).group(1))
    assert define("SPEC_CACHE_MAX_TREE") == cache.MAX_TREE
    assert define("SPEC_ATTENTION_MAX_HEAD_DIM") == cache.ATTENTION_MAX_HEAD_DIM
    assert (define("SPEC_DEVERR_PAGE"), define("SPEC_DEVERR_CAPACITY"), define("SPEC_DEVERR_LENGTH"),
            define("SPEC_DEVERR_FORK")) == (cache.DEVERR_PAGE, cache.DEVERR_CAPACITY, cache.DEVERR_LENGTH,
                                            cache.DEVERR_FORK)


def struct(**kw):
    f = dict(k=FAKE, v=FAKE, dtype=cache.BF16, num_layers=2, num_pages=10, page_size=16, num_kv_heads=2, head_dim=64,
             layer_stride=20480, page_stride=2048, token_stride=128, head_stride=64, page_table=FAKE, table_stride=4,
             num_requests=3, max_pages=4, lens=FAKE, held=FAKE, ref_counts=FAKE, free_pages=FAKE, num_free=FAKE,
             error=FAKE, scratch=FAKE)
    f.update(kw)
    return cache.SpecCache(**f)


BAD_STRUCTS = [
    (dict(k=None), 1), (dict(v=None), 1), (dict(dtype=0), 1), (dict(dtype=7), 1), (dict(num_layers=0), 1),
    (dict(num_pages=0), 1), (dict(page_size=0), 1), (dict(num_kv_heads=0), 1), (dict(head_dim=0), 1),
    (dict(head_dim=60), 1), (dict(head_dim=1032), 1), (dict(layer_stride=0), 1), (dict(page_stride=-2048), 1),
    (dict(token_stride=4), 1), (dict(head_stride=68), 1), (dict(table_stride=3), 1), (dict(num_requests=0), 1),
    (dict(max_pages=0), 1), (dict(k=FAKE + 8), 1), (dict(v=FAKE + 2), 1), (dict(scratch=FAKE + 4), 1),
    (dict(lens=None), 1), (dict(held=None), 1), (dict(ref_counts=None), 1), (dict(free_pages=None), 1),
    (dict(num_free=None), 1), (dict(error=None), 1), (dict(scratch=None), 1), (dict(page_table=None), 1),
    (dict(lens=FAKE + 1), 1), (dict(max_pages=2 ** 28, table_stride=2 ** 28), 2),
]


@pytest.mark.parametrize("kw,status", BAD_STRUCTS)
def test_every_entry_checks_the_cache(lib, kw, status):
    s = ctypes.byref(struct(**kw))
    P = ctypes.c_void_p(FAKE)
    assert lib.spec_cache_init(s, None) == status
    assert lib.spec_cache_reserve(s, P, 1, None) == status
    assert lib.spec_cache_append(s, 0, P, 128, 64, P, 128, 64, P, 1, 4, None) == status
    assert lib.spec_cache_commit(s, P, 1, 4, P, None, None, None, None) == status
    assert lib.spec_cache_fork(s, P, P, 1, None) == status
    assert lib.spec_cache_release(s, None, 1, None) == status
    assert lib.spec_attention(s, 0, P, 128, 64, 2, P, 1, 4, None, 1.0, P, 128, 64, None, P, 1 << 40, None) == status
    assert lib.spec_attention_workspace_size(s, 2, 1, 4) == 0


def test_null_cache(lib):
    P = ctypes.c_void_p(FAKE)
    assert lib.spec_cache_init(None, None) == 1
    assert lib.spec_cache_reserve(None, P, 1, None) == 1
    assert lib.spec_cache_error(None, None, None, None) == 1


def test_unit_dimensions_need_no_stride(lib):
    """The stride of a dimension of size 1 is not looked at: the call gets as far as its own checks."""
    s = ctypes.byref(struct(num_layers=1, layer_stride=0, num_kv_heads=1, head_stride=3, num_requests=1,
                            table_stride=0))
    assert lib.spec_attention_workspace_size(s, 4, 1, 4) > 0


def test_argument_checks(lib):
    s = ctypes.byref(struct())
    P, odd = ctypes.c_void_p(FAKE), ctypes.c_void_p(FAKE + 8)
    assert lib.spec_cache_reserve(s, None, 1, None) == 1
    assert lib.spec_cache_reserve(s, P, 4, None) == 1  # more requests than the table has
    assert lib.spec_cache_reserve(s, P, -1, None) == 1
    append = lambda layer=0, k=P, kt=128, kh=64, v=P, vt=128, vh=64, cu=P, B=1, N=4: lib.spec_cache_append(
        s, layer, k, kt, kh, v, vt, vh, cu, B, N, None)
    for kw in (dict(layer=2), dict(layer=-1), dict(k=None), dict(v=None), dict(k=odd), dict(kt=0), dict(kt=100),
               dict(vh=4), dict(cu=None), dict(B=4), dict(N=-1)):
        assert append(**kw) == 1, kw
    assert append(N=2 ** 31) == 2
    commit = lambda cu=P, B=1, N=4, acc=P, par=None, last=None, out=None: lib.spec_cache_commit(
        s, cu, B, N, acc, par, last, out, None)
    for kw in (dict(cu=None), dict(acc=None), dict(par=P), dict(last=P), dict(B=4), dict(N=-1),
               dict(out=ctypes.c_void_p(FAKE + 2))):
        assert commit(**kw) == 1, kw
    assert lib.spec_cache_fork(s, None, P, 1, None) == 1
    assert lib.spec_cache_fork(s, P, P, -1, None) == 1
    assert lib.spec_cache_release(s, P, 4, None) == 1


def test_attention_argument_checks(lib):
    s = ctypes.byref(struct())
    P, odd = ctypes.c_void_p(FAKE), ctypes.c_void_p(FAKE + 8)

    def call(cache_struct=s, layer=0, q=P, qt=256, qh=64, H=4, cu=P, B=1, N=4, parent=None, scale=1.0, out=P, ot=256,
             oh=64, lse=None, ws=P, wsb=1 << 40):
        return lib.spec_attention(cache_struct, layer, q, qt, qh, H, cu, B, N, parent, scale, out, ot, oh, lse, ws,
                                  wsb, None)

    for kw in (dict(layer=2), dict(q=None), dict(q=odd), dict(out=None), dict(out=odd), dict(qt=0), dict(qt=60),
               dict(qh=-64), dict(ot=0), dict(oh=3), dict(H=0), dict(H=3), dict(cu=None), dict(B=4), dict(B=-1),
               dict(N=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
               dict(ws=None), dict(lse=ctypes.c_void_p(FAKE + 2)), dict(parent=ctypes.c_void_p(FAKE + 2))):
        assert call(**kw) == 1, kw
    assert call(wsb=0) == 3
    assert call(H=2 * 129) == 2
    assert call(cache_struct=ctypes.byref(struct(page_size=12, page_stride=2048))) == 2
    assert call(cache_struct=ctypes.byref(struct(head_dim=136, head_stride=136, token_stride=272)), qh=136, qt=544,
                oh=136, ot=544) == 2
    assert call(N=2 ** 30) == 2


def test_scratch_size(lib):
    assert lib.spec_cache_scratch_size(0, 5) == 0 and lib.spec_cache_scratch_size(5, 0) == 0
    assert 0 < lib.spec_cache_scratch_size(1, 1) < lib.spec_cache_scratch_size(1000, 1 << 20)


def test_oracle_shared_page_is_copied_until_one_holder_is_left():
    b = oracle_cache.Book(3, 4, 8, 16)
    assert b.reserve([20, 0, 0]) == []
    assert b.table[0].tolist() == [7, 6, -1, -1] and b.num_free == 6
    b.commit([20, 0, 0], [19, -1, -1])
    b.fork([0, 0], [1, 2])
    assert b.ref.tolist() == [0] * 6 + [3, 3]
    # all three write into the shared page 6: the first two copy, the last keeps it
    assert b.reserve([1, 1, 13]) == [(6, 5, 4), (6, 4, 4)]
    assert b.table[:, :3].tolist() == [[7, 5, -1], [7, 4, -1], [7, 6, 3]]
    assert b.ref.tolist() == [0, 0, 0, 1, 1, 1, 1, 3]
    b.release([0, 20, 0])
    assert b.ref.tolist() == [0, 0, 0, 0, 1, 0, 0, 1] and b.free[:b.num_free].tolist() == [0, 1, 2, 3, 5, 6]
    assert b.take_error() == (0, -1)


def test_oracle_rollback_matches_the_pages(golden_dir):
    """After k drafts with a of them accepted the next step starts a + 1 positions further."""
    import json
    g = json.load(open(os.path.join(golden_dir, "rollback.json")))
    for case in g["cases"]:
        b = oracle_cache.Book(1, 4, 4, 16)
        b.reserve([g["k"] + 1])
        b.commit([g["k"] + 1], [case["num_accepted"]])
        assert b.lens[0] == case["advance"]


def test_oracle_tree_moves():
    b = oracle_cache.Book(1, 2, 2, 16)
    b.reserve([6])
    #        0
    #      1   2
    #    3    4 5
    parent = [-1, 0, 0, 1, 2, 2]
    assert b.commit([6], [2], [parent], [5]) == [(0, 2, 1), (0, 5, 2)]
    assert b.lens[0] == 3
    assert b.commit([6], [1], [parent], [5]) == [] and b.take_error() == (oracle_cache.TREE, 0)


def test_oracle_attention_sees_ancestors_only():
    seen = oracle_cache.visible(4, 2, [-1, 0, 0, 2])
    assert seen.astype(int).tolist() == [[1, 1, 1, 0, 0, 0], [1, 1, 1, 1, 0, 0], [1, 1, 1, 0, 1, 0],
                                         [1, 1, 1, 0, 1, 1]]
    rng = np.random.default_rng(0)
    k, v, q = rng.standard_normal((6, 8)), rng.standard_normal((6, 8)), rng.standard_normal((4, 2, 8))
    out, lse, _, _ = oracle_cache.attention(q, k, v, seen, 0.3)
    keep = [0, 1, 2, 4]  # node 2's view alone
    s = np.exp(q[2, 1] @ k[keep].T * 0.3)
    assert np.allclose(out[2, 1], s @ v[keep] / s.sum()) and np.isclose(lse[2, 1], np.log(s.sum()))


def test_pages_past_32_bits_are_refused(lib):
    """The vectors of a page (of one layer, keys or values) are numbered in 32 bits: 2^30 are refused."""
    wide = dict(max_pages=1, page_size=2 ** 23, num_kv_heads=16, head_dim=64)
    s = struct(**wide, token_stride=1024, head_stride=64, page_stride=2 ** 33, layer_stride=2 ** 40)
    assert lib.spec_cache_reserve(ctypes.byref(s), ctypes.c_void_p(FAKE), 1, None) == 2
    s.page_size = 2 ** 23 - 8
    assert lib.spec_attention_workspace_size(ctypes.byref(s), 16, 1, 4) > 0


def test_oracle_commits_only_what_the_pages_hold():
    """A step whose reserve found no room leaves the length as it was, and finds its room later."""
    b = oracle_cache.Book(2, 4, 3, 16)
    b.reserve([30, 10])
    b.commit([30, 10], [29, 9])
    b.reserve([5, 5])
    assert b.take_error() == (oracle_cache.CAPACITY, 0)
    b.commit([5, 5], [4, 4])
    assert b.take_error() == (oracle_cache.LENGTH, 0) and b.lens.tolist() == [30, 15]
    b.release([30, 0])
    b.reserve([5, 0])
    b.commit([5, 0], [4, 0])
    assert b.take_error() == (0, -1) and b.lens.tolist() == [35, 0]
