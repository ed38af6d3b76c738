"""Requests with bad data: nothing of theirs is written, and the others are as if they were alone."""
import numpy as np
import pytest

from speculative_decoding_rejection_spec_gb300 import binding, cache
from test_gpu_attention import Case, built, dev  # noqa: F401 (built: the module's fixture)
from test_gpu_cache import Pair

pytestmark = pytest.mark.gpu


# narrow row blocks, whole; wide ones, one and several of a request; both cut over many blocks
TREES = [([9, 20, 9], [100, 10, 20], 4, 128, "bf16"), ([64, 100, 3, 128], [300, 0, 77, 40], 4, 64, "f16"),
         ([33, 7, 2], [9000, 5000, 1], 1, 128, "bf16"), ([100, 64], [7000, 3000], 4, 128, "bf16")]


@pytest.mark.parametrize("n,ctx,group,dim,dtype", TREES)
@pytest.mark.parametrize("where,parent", [(0, 0), (0, -2), (1, 1), (1, -1), (-1, 500), (-1, -7), (-1, None)])
def test_rows_of_a_bad_tree_are_not_written(n, ctx, group, dim, dtype, where, parent):
    """One bad parent, of a node that may be nobody's ancestor, leaves all of its request's rows alone
    (parent None: the node itself)."""
    for bad in (0, 1):
        c = Case(n, ctx, group=group, dim=dim, dtype=dtype, tree=True, seed=4, poison=max(ctx) < 1000)
        node = where % n[bad]
        c.parents[bad] = c.parents[bad].copy()
        c.parents[bad][node] = node if parent is None else parent
        out, lse = c.run()
        c.check(out, lse, error=(5, binding.DEVERR_TREE, bad), skip=(bad,))


def test_the_first_bad_tree_is_named():
    c = Case([9, 20, 9, 5], [100, 10, 20, 700], tree=True, seed=4)
    for r in (3, 1):
        c.parents[r] = c.parents[r].copy()
        c.parents[r][2] = 2
    c.check(*c.run(), error=(5, binding.DEVERR_TREE, 1), skip=(1, 3))


@pytest.mark.parametrize("n,ctx", [([3, 4, 5, 2], [100, 200, 300, 50]), ([3, 300, 5, 2], [100, 200, 9000, 50])])
def test_attention_leaves_out_requests_without_their_pages(n, ctx):
    """Tokens behind the pages held: columns from held[r] on are not read, whatever stands there."""
    c = Case(n, ctx, seed=4, poison=False)
    held = c.c.held.clone()
    columns = c.table.shape[1]
    for r in (1, 2):
        for count in (int(held[r]) - 1, 0, -1, columns + 1):
            c.c.held[r] = count
            c.check(*c.run(), error=(5, cache.DEVERR_LENGTH, r), skip=(r,))
        c.c.held[r] = columns  # more than they need is theirs
        c.check(*c.run())
        c.c.held.copy_(held)


@pytest.mark.parametrize("tree", [False, True])
def test_a_step_without_room_commits_nothing(tree):
    """Reserve runs out of pages and the loop goes on: the request keeps its length and finds its room later."""
    import torch
    p = Pair(3, 8, 6, 16, layers=1, heads=2, dim=64)
    p.reserve([48, 33, 0])
    p.append([48, 33, 0])
    p.commit([48, 33, 0], [47, 32, 0])
    p.check()
    n, cu = [5, 3, 0], dev([0, 5, 8, 8])
    p.reserve(n)
    p.check((cache.DEVERR_CAPACITY, 0))
    rows = torch.randn((8, 2, 64), generator=p.gen).bfloat16()
    cache.append(p.c, 0, rows.cuda(), rows.cuda(), cu)
    for i in range(3):
        page, row = p.book.slot(1, 33 + i)
        p.k[0, page, row] = p.v[0, page, row] = rows[5 + i]
    assert cache.last_error(p.c) == (5, cache.DEVERR_PAGE, 0)
    q = torch.randn((8, 4, 64), generator=p.gen).bfloat16().cuda()
    out = torch.full_like(q, 7.0)
    parents = [np.array([-1, 0, 1, 2, 3], np.int32), np.array([-1, 0, 1], np.int32), np.zeros(0, np.int32)]
    cache.attention(p.c, 0, q, cu, parent=dev(np.concatenate(parents)) if tree else None, out=out)
    assert cache.last_error(p.c) == (5, cache.DEVERR_LENGTH, 0)
    assert (out[:5] == 7).all() and not (out[5:] == 7).any()
    if tree:
        p.commit(n, [4, 2, 0], parents, [4, 2, 0])
    else:
        p.commit(n, [4, 2, 0])
    assert p.book.lens.tolist() == [48, 36, 0]
    p.check((cache.DEVERR_LENGTH, 0))
    p.release([48, 20, 0])
    p.reserve(n)
    p.append(n)
    p.commit(n, [4, 2, 0])
    p.check()


@pytest.mark.parametrize("requests", [900, 1500])
def test_a_skipped_request_among_many_gets_nothing(requests):
    """A table that names a free page, which the same call hands to another request: the request is skipped and
    no page goes to two requests."""
    p = Pair(requests, 4, 8000, 8, layers=1, heads=1, dim=8)
    n, bad = [5] * requests, requests - 100
    p.reserve(n)
    p.append(n)
    p.commit(n, [4] * requests)
    p.check()
    p.book.table[bad, 0] = p.book.free[p.book.num_free - 1]  # goes to request 0
    p.c.page_table.copy_(dev(p.book.table))
    p.reserve([8] * requests)
    p.check((cache.DEVERR_PAGE, bad))
    pages = p.book.table[:, :2][np.arange(requests) != bad]
    assert len(np.unique(pages)) == pages.size
