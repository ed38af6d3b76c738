"""GPU attention of requests that share the pages of a prefix, and the plan that says which do, against the 64-bit
oracle (test_gpu_attention's bound: two partial sums of fp32 joined by a few more roundings lie within its 2^-20) and
against the attention that shares nothing."""
import types

import numpy as np
import pytest

from oracle import cache as oracle_cache
from speculative_decoding_rejection_spec_gb300 import binding, cache
from test_gpu_attention import Case, built, dev  # noqa: F401 (built: the module's fixture)
from test_gpu_cache_calls import BUSY

pytestmark = pytest.mark.gpu


class Grouped(Case):
    """A case whose requests share pages: groups of (first, end, pages); `ctx` is behind the shared tokens."""

    def __init__(self, groups, n, ctx, page=16, **kw):
        ctx = list(ctx)
        for a, b, pages in groups:
            for r in range(a, b):
                ctx[r] += pages * page
        super().__init__(n, ctx, page=page, **kw)
        self.plan = np.array([(r, r + 1, 0, 0) for r in range(len(n))], np.int32)
        for a, b, pages in groups:
            self.table[a:b, :pages] = self.table[a, :pages]
            self.plan[a:b] = a, b, pages * page, 0
        self.c.page_table.copy_(dev(self.table))

    def run(self, **kw):
        return super().run(shared=kw.pop("shared", dev(self.plan)), **kw)

    def apart(self):
        """The same without sharing."""
        return Case.run(self)


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("n", [1, 2, 9, 33])
@pytest.mark.parametrize("pages", [1, 7, 8, 9, 40])
def test_prefixes_around_the_tiles(dtype, dim, n, pages):
    groups = [(0, 5, pages), (5, 7, 1), (8, 11, 3 * pages)]
    c = Grouped(groups, [n] * 12, [0, 1, 127, 128, 300, 5, 64, 200, 129, 0, 16, 50], dim=dim, dtype=dtype, seed=n + pages)
    c.check(*c.run())


@pytest.mark.parametrize("dim", [8, 40, 72, 96, 120])
def test_odd_head_dims(dim):
    c = Grouped([(0, 3, 9), (3, 5, 20)], [1, 5, 0, 17, 2], [30, 3, 50, 260, 0], dim=dim, heads=3, group=2, seed=dim)
    c.check(*c.run())


@pytest.mark.parametrize("heads,group", [(1, 1), (3, 1), (2, 3), (1, 7), (1, 71), (1, 128)])
def test_head_groups(heads, group):
    c = Grouped([(0, 4, 11)], [1, 4, 0, 3], [40, 129, 5, 0], heads=heads, group=group, dim=64, seed=group)
    c.check(*c.run())


@pytest.mark.parametrize("page", [8, 24, 40, 64, 128, 192, 1000])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "hpn"])
def test_page_sizes(page, layout):
    c = Grouped([(1, 4, 2)], [3, 1, 40, 2], [50, 127, 77, 1], page=page, layout=layout, layers=2, layer=1, seed=page)
    c.check(*c.run())


@pytest.mark.parametrize("dtype,group,n", [("bf16", 4, [1, 31, 64, 65, 100, 0, 128, 2]), ("f16", 1, [128, 127, 20]),
                                           ("bf16", 7, [64, 40, 33, 128])])
def test_trees(dtype, group, n):
    rng = np.random.default_rng(len(n))
    c = Grouped([(0, len(n) - 1, 13)], n, rng.integers(0, 200, len(n)), group=group, dim=64, dtype=dtype, tree=True,
                seed=group)
    c.check(*c.run())


@pytest.mark.parametrize("n,ctx,group", [([200, 3], [0, 0], 1), ([300, 64, 1], [100, 0, 5], 4), ([129, 257], [0, 127], 5)])
def test_prompt_chunks_behind_a_prefix(n, ctx, group):
    c = Grouped([(0, len(n), 21)], n, ctx, heads=2, group=group, page=32, pad=3, seed=sum(n))
    c.check(*c.run())


def test_many_requests_of_one_token():
    """The rows of a group fill several row blocks."""
    rng = np.random.default_rng(5)
    n = rng.integers(0, 3, 300)
    c = Grouped([(3, 200, 30), (200, 290, 2)], n, rng.integers(0, 100, 300), heads=2, group=4, seed=9, poison=False)
    c.check(*c.run())


def test_many_groups():
    rng = np.random.default_rng(6)
    groups = [(a, a + int(rng.integers(2, 6)), int(rng.integers(0, 30))) for a in range(0, 600, 6)]
    n = rng.integers(0, 4, 600)
    c = Grouped(groups, n, rng.integers(0, 60, 600), heads=2, group=2, dim=64, dtype="f16", seed=10, poison=False)
    c.check(*c.run())


@pytest.mark.parametrize("n,heads,pages", [([1, 1], 1, 200), ([6, 1, 9], 2, 300), ([33, 2], 1, 120)])
def test_long_prefixes(n, heads, pages):
    """Row blocks of the group cut into the parts of many blocks."""
    c = Grouped([(0, len(n), pages)], n, [30] * len(n), heads=heads, page=64, seed=pages, poison=False)
    c.check(*c.run())


def test_long_contexts_behind_a_prefix():
    c = Grouped([(0, 3, 10)], [5, 1, 70], [9000, 20, 4000], heads=1, page=64, seed=2, poison=False)
    c.check(*c.run())


def test_the_same_as_without_sharing():
    """Within the bound of both, with a plan and with one of no group."""
    c = Grouped([(0, 4, 30)], [9] * 6, [100, 20, 3, 0, 700, 40], seed=1)
    c.check(*c.run())
    c.check(*c.apart())
    c.plan[:4] = [(r, r + 1, 0, 0) for r in range(4)]
    c.check(*c.run())


def test_repeated_calls_are_bit_identical():
    import torch
    c = Grouped([(0, 30, 60), (30, 40, 9)], [9] * 40, np.random.default_rng(0).integers(0, 300, 40), page=32, seed=1,
                poison=False)
    out, lse = c.run()
    for _ in range(3):
        again, lse2 = c.run()
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("entry", [
    (0, 5, 480, 0), (-1, 4, 480, 0), (0, 9, 480, 0), (1, 4, 480, 0), (0, 4, 470, 0), (0, 4, -16, 0), (0, 4, 2 ** 30, 0),
    (0, 4, 560, 0), (3, 4, 480, 0), (2 ** 31 - 1, -2 ** 31, 2 ** 31 - 16, 0), (0, 2 ** 31 - 1, 480, 0),
    (-2 ** 31, 4, 480, 0), (0, 1, 480, 0)])
@pytest.mark.parametrize("where", [0, 1, 3, 5])
def test_plans_that_do_not_fit_share_nothing(entry, where):
    """An entry that its request or its group's first one does not fit: the requests concerned read their own pages."""
    c = Grouped([(0, 4, 30)], [9] * 6, [100, 20, 3, 0, 700, 40], heads=1, group=2, dim=64, seed=1)
    c.plan[where] = entry
    c.check(*c.run())


def test_a_plan_that_was_outlived():
    """Requests shorter than what they shared, the first of a group among them."""
    c = Grouped([(0, 4, 30)], [9] * 6, [100, 20, 3, 0, 700, 40], seed=1, poison=False)
    for r in (2, 0):
        c.ctx[r] = 100
        c.c.lens.copy_(dev(c.ctx))
        c.check(*c.run())


def test_requests_with_errors_are_left_out():
    n, own = [3, 4, 5, 2], [100, 20, 30, 5]
    c = Grouped([(0, 4, 20)], n, own, seed=4)
    c.c.lens[1] = -1
    c.check(*c.run(), error=(5, cache.DEVERR_LENGTH, 1), skip=(1,))
    c.c.lens[1] = c.ctx[1]
    held = c.c.held.clone()
    c.c.held[2] -= 1
    c.check(*c.run(), error=(5, cache.DEVERR_LENGTH, 2), skip=(2,))
    c.c.held.copy_(held)
    c.c.held[0] -= 1  # the first of the group: its shared pages are still held
    c.check(*c.run(), error=(5, cache.DEVERR_LENGTH, 0), skip=(0,))
    for bad in (3, -1, 10 ** 6):  # not even those, or no number of pages
        c.c.held[0] = bad
        c.check(*c.run(), error=(5, cache.DEVERR_LENGTH, 0), skip=(0,))
    c.c.held.copy_(held)
    c.c.lens[0] = -7
    c.check(*c.run(), error=(5, cache.DEVERR_LENGTH, 0), skip=(0,))


@pytest.mark.parametrize("n,own,group", [([9, 20, 9], [100, 10, 20], 4), ([100, 64, 2], [3000, 0, 5], 4)])
def test_bad_trees_are_left_out(n, own, group):
    for bad in (0, 1):
        c = Grouped([(0, 3, 20)], n, own, group=group, tree=True, seed=4, poison=False)
        c.parents[bad] = c.parents[bad].copy()
        c.parents[bad][3] = 5
        c.check(*c.run(), error=(5, binding.DEVERR_TREE, bad), skip=(bad,))
    c = Grouped([(0, 3, 20)], [9, 140, 9], own, tree=True, seed=4, poison=False)
    c.check(*c.run(), error=(5, binding.DEVERR_TREE, 1), skip=(1,))


def test_bad_pages_of_a_prefix_read_as_zeros():
    c = Grouped([(0, 3, 20)], [3, 4, 1], [30, 5, 0], heads=1, seed=4)
    c.c.page_table[0, 4] = -1
    c.kv[:, c.table[0, 4]] = 0
    c.check(*c.run(), error=(5, cache.DEVERR_PAGE, 0))


def test_bad_layout_writes_nothing():
    c = Grouped([(0, 2, 20)], [3, 4], [100, 200], seed=4)
    c.check(*c.run())  # a workspace that has seen a good call
    for cu in ([1, 3, 7], [0, 5, 4], [0, 3, 8]):
        good, c.cu = c.cu, np.array(cu, np.int32)
        out, lse = c.run()
        c.cu = good
        assert (out == 7).all() and (lse == 7).all()
        assert cache.last_error(c.c) == (5, binding.DEVERR_LAYOUT, -1)


def test_empty_calls():
    import torch
    c = Grouped([(0, 2, 3)], [0, 0], [5, 0], pad=4, seed=0)
    c.check(*c.run())
    q = torch.zeros((0, 8, 128), dtype=torch.bfloat16, device="cuda")
    assert cache.attention(c.c, 0, q, dev([0, 0, 0]), shared=dev(c.plan)).shape == q.shape
    assert cache.attention(c.c, 0, q, dev([0]), shared=dev(np.zeros((0, 4)))).shape == q.shape


@pytest.mark.parametrize("dtype,group,dim,tree,n", [("bf16", 4, 128, False, [9, 5, 1, 2]), ("f16", 4, 64, True, [60, 128, 20, 2]),
                                                    ("bf16", 4, 128, False, [700, 3, 64, 1])])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(dtype, group, dim, tree, n):
    """Of the step's own tokens, of a request's tokens behind the prefix, and of the prefix."""
    import torch
    ctx = [300, 5, 0, 127]
    c = Grouped([(0, 3, 11)], n, ctx, group=group, dim=dim, dtype=dtype, tree=tree, seed=dim + group)
    rng = np.random.default_rng(dim)
    seen = [oracle_cache.visible(m, c.ctx[r], c.parents[r] if tree else None) for r, m in enumerate(n)]
    spoilt = []
    for r, m in enumerate(n):
        for x in (np.inf, -np.inf, np.nan, np.inf):
            spoilt.append((r, c.ctx[r] + int(rng.integers(min(1, m - 1), m)), int(rng.integers(2)), int(rng.integers(dim)), x))
    spoilt.append((0, c.ctx[0] - 1, 0, 3, np.inf))

    def write(values):
        for r, t, h, e, x in values:
            c.kv[1][int(c.table[r, t // c.page]), t % c.page, h, e] = x
        c.c.v[0].copy_(c.kv[1])

    write([s[:4] + (0.0,) for s in spoilt])
    clean, clean_lse = c.run()
    c.check(clean, clean_lse)
    write(spoilt)
    out, lse = c.run()
    want = clean.float().cpu().numpy()
    for (r, t, h, e), x in {s[:4]: s[4] for s in spoilt}.items():
        rows = c.cu[r] + np.flatnonzero(seen[r][:, t])
        with np.errstate(invalid="ignore"):
            want[rows, h * group:(h + 1) * group, e] += np.float32(x)
    got = out.float().cpu().numpy()
    inf = ~np.isfinite(want)
    np.testing.assert_array_equal(got, want)
    assert inf.any() and torch.equal(lse, clean_lse)
    write([s[:4] + (0.0,) for s in spoilt] + [(1, 20, 1, 4, np.nan)])  # in the prefix: all of the group see it
    out, _ = c.run()
    want = clean.float().cpu().numpy()
    want[:c.cu[3], group:, 4] = np.nan
    np.testing.assert_array_equal(out.float().cpu().numpy(), want)


def test_strided_queries_and_outputs():
    import torch
    c = Grouped([(0, 3, 11)], [5, 1, 30], [200, 4, 60], heads=2, group=3, dim=64, seed=2)
    N, H, D = c.q.shape
    fused = torch.zeros((N, 3 * H, D), dtype=c.q.dtype, device="cuda")
    fused[:, :H] = c.q.cuda()
    by_head = torch.full((H, N, D), 7.0, dtype=c.q.dtype, device="cuda")
    c.check(*c.run(q=fused[:, :H], out=by_head.transpose(0, 1)))


def test_captured_call_follows_the_device_data():
    import torch
    c = Grouped([(0, 3, 11)], [4, 9, 1, 5], [300, 20, 500, 6], seed=6, poison=False)
    q, cu, plan = c.q.cuda(), dev(c.cu), dev(c.plan)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attention(c.c, 0, q, cu, out=out, lse=lse, shared=plan)
    apart = np.array([(r, r + 1, 0, 0) for r in range(4)], np.int32)
    for ctx, p in ((c.ctx, c.plan), ([180, 176, 400, 3], c.plan), (c.ctx, apart), ([200, 10, 300, 0], c.plan)):
        c.ctx = ctx
        c.c.lens.copy_(dev(ctx))
        plan.copy_(dev(p))
        graph.replay()
        c.check(out, lse)


def test_captures_of_the_same_stream_have_workspaces_of_their_own():
    import torch
    a = Grouped([(0, 3, 11)], [4, 9, 1], [300, 20, 500], seed=6, poison=False)
    q, cu, plan, s = a.q.cuda(), dev(a.cu), dev(a.plan), torch.cuda.Stream()
    want = cache.attention(a.c, 0, q, cu, shared=plan)
    torch.cuda.synchronize()
    kept = [w[-1] for w in a.c.workspaces.values()]
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(cache.attention(a.c, 0, q, cu, shared=plan))
    for w in kept:
        w.zero_()
    torch.cuda.synchronize()
    graphs[0].replay()
    with torch.cuda.stream(s):
        graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want) and not any(w.any() for w in kept)


def test_streams_threads_and_growing_calls():
    """One workspace of a stream serves plain and shared calls of all sizes."""
    import torch
    small = Grouped([(0, 3, 11)], [1, 2, 1], [30, 20, 5], seed=6, poison=False)
    n = [40, 90, 33]
    large = Grouped([(0, 3, 11)], n, [300, 20, 500], seed=6, poison=False)
    large.c = small.c
    both = []
    for c in (small, large):
        d = Grouped([(0, 3, 11)], c.n, [x - 176 for x in c.ctx], seed=6, poison=False)
        both.append((d, d.apart(), d.run()))
    c = both[1][0]
    q, cu, plan = c.q.cuda(), dev(c.cu), dev(c.plan)
    few = both[0][0]
    few_q, few_cu = c.q[:4].cuda(), dev(few.cu)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, s):
        for _ in range(3):
            a = cache.attention(c.c, 0, few_q, few_cu, stream=stream)
            b = cache.attention(c.c, 0, few_q, few_cu, shared=plan, stream=stream)
            d = cache.attention(c.c, 0, q, cu, shared=plan, stream=stream)
            e = cache.attention(c.c, 0, q, cu, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(d, both[1][2][0]) and torch.equal(e, both[1][1][0])
            assert (a.float() - b.float()).abs().max() < 0.05
    assert len(c.c.workspaces) == 2
    assert cache.last_error(c.c) == (0, 0, -1)


def test_explicit_workspaces():
    import torch
    c = Grouped([(0, 3, 11)], [4, 9, 1], [300, 20, 500], seed=6)
    size = cache.load().spec_attention_shared_workspace_size(c.c.ref, 8, 3, 14)
    c.check(*c.run(workspace=torch.full((size,), 255, dtype=torch.uint8, device="cuda")))
    with pytest.raises(binding.SpecRejectError):
        c.run(workspace=torch.zeros(size - 1, dtype=torch.uint8, device="cuda"))


def test_refusals():
    import torch
    c = Grouped([(0, 2, 11)], [4, 9], [30, 20], seed=6)
    for plan in (dev(c.plan[:1]), dev(c.plan).long(), dev(c.plan)[:, :3], dev(np.zeros((2, 8)))[:, :4]):
        with pytest.raises(TypeError):
            c.run(shared=plan)
    with pytest.raises(ValueError):
        c.run(shared=dev(c.plan).cpu())
    odd = torch.zeros(9, dtype=torch.int32, device="cuda")[1:].view(2, 4)
    with pytest.raises(binding.SpecRejectError):
        c.run(shared=odd)


# ---------------------------------------------------------------------------------------
# The plan
# ---------------------------------------------------------------------------------------


def planned(table, lens, held, page, least, B=None):
    import torch
    R, MP = table.shape
    k = torch.zeros((1, 4, page, 1, 8), dtype=torch.bfloat16, device="cuda")
    ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    c = cache.PagedCache(k, k.clone(), page_table=dev(table), lens=dev(lens), held=dev(held), ref_counts=ints(4),
                         free_pages=ints(4), num_free=ints(1))
    plan = cache.share(c, min_tokens=least, B=B)
    n = R if B is None else B
    want, bad = oracle_cache.share_plan(table[:n].tolist(), list(lens)[:n], list(held)[:n], page, least)
    np.testing.assert_array_equal(plan.cpu().numpy(), want)
    assert cache.last_error(c) == ((5, cache.DEVERR_LENGTH, bad[0]) if bad else (0, 0, -1))
    again = cache.share(c, min_tokens=least, B=B)
    assert torch.equal(again, plan)
    cache.last_error(c)
    return want


@pytest.mark.parametrize("R", [1, 2, 3, 31, 32, 33, 255, 256, 257, 511, 513, 1030])
@pytest.mark.parametrize("page,least", [(16, 0), (16, 100), (8, 1), (1, 3)])
def test_plans(R, page, least):
    rng = np.random.default_rng(R + page)
    for chance in (0.0, 0.1, 0.5, 1.0):  # of a new group
        table = rng.integers(0, 50, (R, 40)).astype(np.int32)
        for r in range(1, R):
            if rng.random() >= chance:
                keep = rng.integers(0, 41)
                table[r, :keep] = table[r - 1, :keep]
        lens = rng.integers(0, 40 * page + 1, R)
        planned(table, lens, np.full(R, 40), page, least)


def test_long_rows_and_a_part_of_the_batch():
    rng = np.random.default_rng(1)
    table = np.repeat(rng.integers(0, 10 ** 6, (1, 5000)), 9, 0).astype(np.int32)
    for r, col in ((2, 4999), (3, 0), (5, 1024), (6, 1023), (8, 3000)):
        table[r, col] += 1
    lens = np.full(9, 5000 * 16)
    want = planned(table, lens, np.full(9, 5000), 16, 256)
    assert want[:3, 2].tolist() == [4999 * 16] * 3 and want[3, 2] == 0
    planned(table, lens, np.full(9, 5000), 16, 256, B=4)
    planned(table, lens, np.full(9, 5000), 16, 256, B=0)
    planned(table, lens - np.arange(9) * 1111, np.full(9, 5000), 16, 2 ** 31 - 1)
    planned(table, lens - np.arange(9) * 1111, np.full(9, 5000), 16, 20000)


def test_requests_that_are_not_sound_are_apart():
    table = np.repeat(np.arange(10)[None], 8, 0).astype(np.int32)
    lens, held = np.full(8, 70), np.full(8, 10)
    lens[2], held[4], held[5], lens[7] = -1, 4, 11, 81
    want = planned(table, lens, held, 8, 0)
    assert want[:, :3].tolist() == [[0, 2, 64], [0, 2, 64], [2, 3, 0], [3, 4, 0], [4, 5, 0], [5, 6, 0], [6, 7, 0], [7, 8, 0]]


def test_plan_calls():
    import torch
    c = Grouped([(0, 3, 11), (3, 5, 40)], [1] * 6, [30, 20, 5, 0, 70, 16], seed=6)
    want = oracle_cache.share_plan(c.table.tolist(), c.ctx, c.c.held.tolist(), 16, 256)[0]
    assert want[:, 2].tolist() == [0, 0, 0, 640, 640, 0]  # 176 tokens are too few (as for the default)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    first = cache.share(c.c, stream=s)
    freed = torch.full((6, 4), 3, dtype=torch.int32, device="cuda")
    copy = torch.zeros_like(freed)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    copy.copy_(freed)
    del freed
    second = cache.share(c.c, stream=s)
    torch.cuda.synchronize()
    for plan in (first, second):
        np.testing.assert_array_equal(plan.cpu().numpy(), want)
    assert (copy == 3).all()
    out = torch.full((6, 4), 9, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.share(c.c, min_tokens=100, out=out)
    graph.replay()
    np.testing.assert_array_equal(out.cpu().numpy()[:, 2], [176, 176, 176, 640, 640, 0])
    c.c.lens[4] = 0
    graph.replay()
    np.testing.assert_array_equal(out.cpu().numpy()[:, 2], [176, 176, 176, 0, 0, 0])
    for kw in (dict(out=out[:3]), dict(out=out.long())):
        with pytest.raises(TypeError):
            cache.share(c.c, **kw)
    with pytest.raises(ValueError):
        cache.share(c.c, stream=types.SimpleNamespace(cuda_stream=0, device_index=1))
    for kw in (dict(B=7), dict(min_tokens=-1)):
        with pytest.raises(binding.SpecRejectError):
            cache.share(c.c, **kw)


# ---------------------------------------------------------------------------------------
# Together, as a serving loop uses them
# ---------------------------------------------------------------------------------------


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("window", [None, 40])
def test_samples_of_two_prompts(tree, window):
    """Prompts are cached with rotated keys, forked, and the branches go on for a few steps, chains of drafts or draft
    trees, over the shared prefix or a window.  Every attention is checked against rows rotated in 64 bits and rounded
    as the cache holds them."""
    import torch
    rng = np.random.default_rng(5 + tree)
    L, P, H, G, D, T = 2, 16, 2, 3, 64, 32
    c = cache.make_cache(L, 300, P, H, D, 9, 40)
    table = cache.rotation_table(640, T)
    angles = table.double().cpu().numpy()
    history = [[[] for _ in range(L)] for _ in range(9)]  # rows as the cache holds them
    gen = torch.Generator(device="cuda").manual_seed(3)

    def step(n, parents, plan, accepted):
        cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        N, dcu = int(cu[-1]), dev(cu)
        par = None if parents is None else dev(np.concatenate(parents))
        cache.reserve(c, dcu)
        starts = [len(history[r][0]) for r in range(len(n))]
        new = []
        for layer in range(L):
            q, k, v = (torch.randn((N, h, D), generator=gen, device="cuda").to(torch.bfloat16) for h in (H * G, H, H))
            qr = cache.append_rotated(c, layer, 2 * q, k, v, dcu, table, parent=par)
            kw = dict(shared=plan) if window is None else dict(window=window, sinks=5)
            out = cache.attention(c, layer, qr, dcu, parent=par, **kw)
            keys = c.k[layer].cpu()
            ids = c.page_table.cpu().numpy()
            for r, m in enumerate(n):
                a, b = cu[r], cu[r + 1]
                at = [(int(ids[r, (starts[r] + i) // P]), (starts[r] + i) % P) for i in range(m)]
                rows = [(keys[p, i].double().numpy(), v[a + j].double().cpu().numpy()) for j, (p, i) in enumerate(at)]
                new.append(rows)
                if m == 0:
                    continue
                depth = np.arange(m) if parents is None else oracle_cache.depths(parents[r])
                want = oracle_cache.rotate(k[a:b].double().cpu().numpy(), angles, starts[r] + depth, False)
                got = np.array([x[0] for x in rows])
                assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20).all()
                want_q = oracle_cache.rotate((2 * q[a:b]).double().cpu().numpy(), angles, starts[r] + depth, False)
                assert (np.abs(qr[a:b].double().cpu().numpy() - want_q) <= 2.0 ** -8 * np.abs(want_q) + 2.0 ** -19).all()
                tree_of = None if parents is None else parents[r]
                seen = oracle_cache.visible(m, starts[r], tree_of) if window is None else \
                    oracle_cache.visible_window(m, starts[r], window, 5, tree_of)
                for h in range(H):
                    past = history[r][layer] + rows
                    kk, vv = (np.array([x[i][h] for x in past]) for i in (0, 1))
                    hs = slice(h * G, (h + 1) * G)
                    o, _, A, S = oracle_cache.attention(qr[a:b, hs].double().cpu().numpy(), kk, vv, seen, D ** -0.5)
                    tol = 2.0 ** -8 * np.abs(o) + A * (2.0 ** -8 + 2 * (D + 8) * 2.0 ** -23 * S + 2.0 ** -13)[..., None]
                    assert (np.abs(out[a:b, hs].double().cpu().numpy() - o) <= tol).all()
        paths = accepted(n)
        acc = dev([len(p) - 1 for p in paths])
        if parents is None:
            cache.commit(c, dcu, acc)
        else:
            cache.commit(c, dcu, acc, parent=par, last_node=dev([p[-1] if p else 0 for p in paths]))
        for layer in range(L):
            for r, path in enumerate(paths):
                history[r][layer] += [new[layer * len(n) + r][i] for i in path]
        assert cache.last_error(c) == (0, 0, -1)
        assert c.lens.tolist() == [len(x[0]) for x in history]

    # requests 0 and 5 are the prompts, 1-4 and 6-8 their branches
    step([300, 0, 0, 0, 0, 77, 0, 0, 0], None, cache.share(c), lambda n: [list(range(m)) for m in n])
    cache.fork(c, dev([0, 0, 0, 0, 5, 5, 5]), dev([1, 2, 3, 4, 6, 7, 8]))
    for r in (1, 2, 3, 4, 6, 7, 8):
        history[r] = [list(x) for x in history[0 if r < 5 else 5]]
    plan = cache.share(c, min_tokens=64)
    assert plan[:, :3].tolist() == [[0, 5, 288]] * 5 + [[5, 9, 64]] * 4
    for _ in range(3):
        n = rng.integers(0, 7, 9)
        parents = None
        if tree:
            parents = [np.array([-1] * min(m, 1) + [int(rng.integers(0, i)) for i in range(1, m)], np.int32) for m in n]

        def accepted(n):
            paths = []
            for r, m in enumerate(n):
                if parents is None:
                    paths.append(list(range(int(rng.integers(0, m)) + 1 if m else 0)))
                    continue
                path, at = [], int(rng.integers(0, m)) if m else -1
                while at >= 0:
                    path.insert(0, at)
                    at = int(parents[r][at])
                paths.append(path)
            return paths

        step(n, parents, plan, accepted)
    assert cache.share(c, min_tokens=64)[:, :3].tolist() == plan[:, :3].tolist()
