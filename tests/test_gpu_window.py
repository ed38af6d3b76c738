"""GPU attention over the last positions and the first ones, against the 64-bit oracle, with the bound of
test_gpu_attention (its sums run over fewer keys)."""
import numpy as np
import pytest

from oracle import cache as oracle_cache
from speculative_decoding_rejection_spec_gb300 import binding, cache
from test_gpu_attention import Case, EDGES, built, dev  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu


class Windowed(Case):
    """A case whose keys that no row sees are not numbers, in pages that no row sees of no valid number."""

    def __init__(self, n, ctx, window, sinks, hide=True, **kw):
        super().__init__(n, ctx, **kw)
        self.window, self.sinks = window, sinks
        if hide:
            import torch
            self.hidden = self.table.copy()
            for r, m in enumerate(n):
                if m == 0:
                    continue
                seen = self.seen(r).any(0)
                for col in range(-(-len(seen) // self.page)):
                    here = seen[col * self.page:(col + 1) * self.page]
                    if not here.any():
                        self.hidden[r, col] = -5
                    rows = torch.from_numpy(np.flatnonzero(~here))
                    self.kv[0][self.table[r, col], rows] = float("nan")
                    self.kv[1][self.table[r, col], rows] = float("inf")
            self.write()
            self.c.page_table.copy_(dev(self.hidden))

    def write(self):
        self.c.k[self.layer], self.c.v[self.layer] = self.kv[0].cuda(), self.kv[1].cuda()

    def seen(self, r):
        return oracle_cache.visible_window(self.n[r], self.ctx[r], self.window, self.sinks,
                                           None if self.parents is None else self.parents[r])

    def run(self, **kw):
        return super().run(window=self.window, sinks=self.sinks, **kw)

    def check(self, out, lse, scale=None, error=(0, 0, -1), skip=()):
        assert cache.last_error(self.c) == error
        scale = self.dim ** -0.5 if scale is None else scale
        u = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -11
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for r, m in enumerate(self.n):
            a, b = self.cu[r], self.cu[r + 1]
            if r in skip:
                assert (out[a:b] == 7).all() and (lse[a:b] == 7).all()
                continue
            if m == 0:
                continue
            seen = self.seen(r)
            keys = np.flatnonzero(seen.any(0))
            seen, L = seen[:, keys], len(keys)
            pages, rows = self.table[r, keys // self.page], keys % self.page
            for h in range(self.heads):
                k, v = (self.kv[i][pages, rows, h].double().numpy() for i in (0, 1))
                hs = slice(h * self.group, (h + 1) * self.group)
                q = self.q[a:b, hs].double().numpy()
                o, z, A, S = oracle_cache.attention(q, k, v, seen, scale)
                es = (self.dim + 8) * 2.0 ** -23 * S
                tol = u * np.abs(o) + A * (u + 2 * es + 2 * L * 2.0 ** -23 + 2.0 ** -20)[..., None]
                if self.dtype == "f16":
                    tol = tol + L * 2.0 ** -25 * np.abs(v).max()
                diff = np.abs(out[a:b, hs] - o)
                assert (diff <= tol).all(), (r, h, float((diff - tol).max()), np.argwhere(~(diff <= tol))[:4])
                assert (np.abs(lse[a:b, hs] - z) <= es + L * 2.0 ** -23 + 2.0 ** -20 * (1 + np.abs(z))).all(), (r, h)
        assert (out[self.cu[-1]:] == 7).all() and (lse[self.cu[-1]:] == 7).all()  # padding rows


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("n", [1, 9, 33])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 1), (64, 0), (127, 4), (128, 0), (129, 130), (200, 16), (1000, 7)])
def test_contexts_around_the_tiles(dtype, dim, n, window, sinks):
    c = Windowed([n] * (len(EDGES) + 2), EDGES + [700, 1111], window, sinks, dim=dim, dtype=dtype, seed=n + window)
    c.check(*c.run())


@pytest.mark.parametrize("window", [1, 2, 100, 5000])
@pytest.mark.parametrize("sinks", [0, 1, 127, 128, 129, 300, 2 ** 31 - 1])
def test_windows_and_sinks(window, sinks):
    c = Windowed([1, 17, 3, 90], [900, 450, 10, 777], window, sinks, heads=1, group=2, page=8, dim=64, seed=sinks % 1000)
    c.check(*c.run())


@pytest.mark.parametrize("dim", [8, 40, 72, 96, 120])
def test_odd_head_dims(dim):
    c = Windowed([1, 5, 0, 17], [530, 3, 50, 260], 99, 3, dim=dim, heads=3, group=2, seed=dim)
    c.check(*c.run())


@pytest.mark.parametrize("heads,group", [(1, 1), (2, 3), (1, 7), (1, 71), (1, 128)])
def test_head_groups(heads, group):
    c = Windowed([1, 4, 0, 3], [400, 129, 5, 0], 150, 20, heads=heads, group=group, dim=64, seed=group)
    c.check(*c.run())


@pytest.mark.parametrize("page", [8, 16, 24, 40, 64, 128, 192, 1000])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "hpn"])
def test_page_sizes(page, layout):
    c = Windowed([3, 1, 40], [900, 427, 77], 130, 10, page=page, layout=layout, layers=2, layer=1, seed=page)
    c.check(*c.run())


@pytest.mark.parametrize("dtype,group,n", [("bf16", 4, [1, 31, 64, 65, 100, 0, 128, 2]), ("f16", 1, [128, 127, 20]),
                                           ("bf16", 7, [64, 40, 33, 128])])
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (60, 100), (300, 5)])
def test_trees(dtype, group, n, window, sinks):
    rng = np.random.default_rng(len(n))
    c = Windowed(n, rng.integers(0, 900, len(n)), window, sinks, group=group, dim=64, dtype=dtype, tree=True, seed=group)
    c.check(*c.run())


def test_deep_trees_whose_sinks_are_nodes():
    c = Windowed([128, 100, 60], [0, 3, 200], 10, 20, group=2, dim=64, tree=True, seed=1, hide=False)
    for r, m in enumerate(c.n):
        c.parents[r] = np.array([-1] + [max(0, i - 1 - i % 2) for i in range(1, m)], np.int32)
    c.check(*c.run())


def test_tree_that_is_a_chain_equals_the_chain():
    import torch
    a = Windowed([50, 7], [300, 100], 40, 6, seed=5)
    out, lse = a.run()
    a.parents = [np.arange(-1, 49, dtype=np.int32), np.arange(-1, 6, dtype=np.int32)]
    a.check(*a.run())
    b = Windowed([50, 7], [300, 100], 400, 6, seed=5)
    out, lse = b.run()
    b.parents = a.parents
    tree, tree_lse = b.run()
    assert torch.equal(out, tree) and torch.equal(lse, tree_lse)


@pytest.mark.parametrize("n,ctx,group", [([200], [0], 1), ([300], [1000], 4), ([64, 500, 1], [700, 13, 900], 2),
                                         ([129, 257], [0, 127], 5), ([1031], [100], 3)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 3), (128, 128), (333, 200)])
def test_prompt_chunks(n, ctx, group, window, sinks):
    c = Windowed(n, ctx, window, sinks, heads=2, group=group, page=32, seed=sum(n))
    c.check(*c.run())


@pytest.mark.parametrize("dim,group,dtype", [(72, 4, "bf16"), (96, 1, "f16"), (64, 128, "f16")])
def test_wide_blocks_of_odd_shapes(dim, group, dtype):
    n = [3 * 256 // group + 1, 130 // group + 1, 1]
    c = Windowed(n, [440, 0, 77], 100, 2, heads=2, group=group, dim=dim, page=24, dtype=dtype, pad=5, seed=dim)
    c.check(*c.run())


def test_many_row_blocks_per_share():
    rng = np.random.default_rng(8)
    n = np.where(rng.random(700) < 0.3, 0, rng.integers(1, 4, 700))
    n[::37] = 70
    ctx = rng.integers(0, 400, 700)
    ctx[::10] = rng.integers(0, 1500, 70)
    c = Windowed(n, ctx, 150, 4, heads=2, group=4, dim=64, page=16, dtype="f16", seed=12, hide=False, poison=False)
    c.check(*c.run())


@pytest.mark.parametrize("n,heads,ctx,window,sinks", [(1, 1, 9000, 4096, 4), (1, 4, 20011, 1000, 0), (6, 2, 22345, 9000, 500),
                                                      (33, 1, 7777, 7000, 200), (150, 1, 16000, 15000, 0)])
def test_long_contexts(n, heads, ctx, window, sinks):
    """Row blocks over many tiles, cut into the parts of several blocks, inside the sinks too."""
    c = Windowed([n], [ctx], window, sinks, heads=heads, page=64, seed=ctx, poison=False)
    c.check(*c.run())


def test_a_window_that_holds_all_is_plain_attention():
    """Nothing is left out: the same results, within the bound (the work is shared out otherwise), and the same bits
    whatever it is that holds all."""
    import torch
    for n, ctx, kw in (([1, 9, 300], [700, 129, 40], {}), ([64, 100], [300, 77], dict(tree=True, dtype="f16", dim=64))):
        c = Windowed(n, ctx, 2 ** 31 - 1, 0, seed=3, **kw)
        out, lse = c.run()
        c.check(out, lse)
        c.check(*Case.run(c))
        for c.window, c.sinks in ((1, 2 ** 31 - 1), (2 ** 40, 2 ** 40), (5000, 7)):
            again, again_lse = c.run()
            assert torch.equal(out, again) and torch.equal(lse, again_lse)


def test_a_window_of_one_is_the_own_value():
    import torch
    c = Windowed([5, 300], [40, 7], 1, 0, heads=2, group=3, seed=3)
    out, _ = c.run()
    for r, m in enumerate(c.n):
        for i in (0, m // 2, m - 1):
            t = c.ctx[r] + i
            v = c.kv[1][c.table[r, t // c.page], t % c.page].cuda()
            assert torch.equal(out[c.cu[r] + i], v.repeat_interleave(3, 0))


@pytest.mark.parametrize("dtype,group,dim,tree,n,ctx,window,sinks", [
    ("bf16", 4, 128, False, [9, 5, 1, 2], [300, 125, 64, 0], 6, 3), ("f16", 4, 64, True, [60, 128, 20, 2], [100, 0, 127, 1], 4, 2),
    ("bf16", 4, 128, False, [700, 3, 64], [0, 9000, 1000], 300, 130), ("bf16", 1, 128, True, [33], [9000], 50, 8),
    ("f16", 3, 80, False, [130, 400], [77, 5], 100, 0)])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(dtype, group, dim, tree, n, ctx, window, sinks):
    """Keys that slide out of the window between the rows of a step, and the step's own: the rows that do not see a
    value of inf or NaN are as they are with a zero there, bit for bit, the others become its sum with theirs."""
    import torch
    c = Windowed(n, ctx, window, sinks, group=group, dim=dim, dtype=dtype, tree=tree, seed=dim + group)
    rng = np.random.default_rng(len(n) + dim)
    seen = [c.seen(r) for r in range(len(n))]
    spoilt = {}
    for r, m in enumerate(n):
        some = np.flatnonzero(seen[r].any(0) & ~seen[r].all(0))
        for x in (np.inf, -np.inf, np.nan, np.inf, np.inf, np.nan, -np.inf):
            if len(some):
                spoilt[r, int(rng.choice(some)), int(rng.integers(2)), int(rng.integers(dim))] = x
    assert len(spoilt) > 4

    def write(which, values):
        for (r, t, h, e), x in values.items():
            c.kv[which][int(c.table[r, t // c.page]), t % c.page, h, e] = x
        c.write()

    write(1, {at: 0.0 for at in spoilt})
    clean, clean_lse = c.run()
    c.check(clean, clean_lse)
    write(1, spoilt)
    out, lse = c.run()
    want = clean.float().cpu().numpy()
    for (r, t, h, e), x in spoilt.items():
        rows = c.cu[r] + np.flatnonzero(seen[r][:, t])
        with np.errstate(invalid="ignore"):
            want[rows, h * group:(h + 1) * group, e] += np.float32(x)
    np.testing.assert_array_equal(out.float().cpu().numpy(), want)
    assert torch.equal(lse, clean_lse)
    assert cache.last_error(c.c) == (0, 0, -1)


def test_values_that_all_rows_see():
    """A value of inf inside every row's window, and one among the sinks, reach all of them."""
    c = Windowed([4, 200], [700, 900], 400, 5, heads=1, group=2, seed=3)
    for r, t in ((0, 600), (1, 2)):
        c.kv[1][int(c.table[r, t // c.page]), t % c.page, 0, 7] = float("inf")
    c.write()
    out, _ = c.run()
    out = out.float().cpu().numpy()
    assert np.isposinf(out[:, :, 7]).all()
    assert np.isfinite(np.delete(out, 7, 2)).all()


def test_bad_requests_are_left_out():
    c = Windowed([3, 4, 5, 2], [100, 200, 300, 50], 60, 2, seed=4)
    c.c.lens[1] = -1
    c.check(*c.run(), error=(5, cache.DEVERR_LENGTH, 1), skip=(1,))
    c.c.lens[1] = 200
    c.c.held[2] -= 1
    c.check(*c.run(), error=(5, cache.DEVERR_LENGTH, 2), skip=(2,))


def test_bad_trees_are_left_out():
    c = Windowed([9, 20, 9], [100, 10, 20], 30, 2, tree=True, seed=4)
    c.parents[1] = c.parents[1].copy()
    c.parents[1][3] = 5
    c.check(*c.run(), error=(5, binding.DEVERR_TREE, 1), skip=(1,))


def test_bad_pages_inside_the_window_are_reported():
    c = Windowed([3, 4], [100, 200], 60, 2, heads=1, seed=4)
    c.c.page_table[1, 11] = 2 ** 30
    c.run()
    assert cache.last_error(c.c) == (5, cache.DEVERR_PAGE, 1)


def test_bad_layout_writes_nothing():
    c = Windowed([3, 4], [100, 200], 60, 2, seed=4)
    for cu in ([1, 3, 7], [0, 5, 4], [0, 3, 8]):
        good, c.cu = c.cu, np.array(cu, np.int32)
        out, lse = c.run()
        c.cu = good
        assert (out == 7).all() and (lse == 7).all()
        assert cache.last_error(c.c) == (5, binding.DEVERR_LAYOUT, -1)


def test_captured_call_follows_the_device_data():
    import torch
    c = Windowed([4, 9, 1], [300, 20, 500], 100, 3, seed=6, hide=False, poison=False)
    q, cu = c.q.cuda(), dev(c.cu)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attention(c.c, 0, q, cu, out=out, lse=lse, window=100, sinks=3)
    for ctx in ([300, 20, 500], [3, 22, 128], [299, 0, 1]):
        c.ctx = ctx
        c.c.lens.copy_(dev(ctx))
        graph.replay()
        c.check(out, lse)


def test_streams_and_repeated_calls():
    import torch
    a = Windowed([4, 9, 1] * 8, [300, 20, 500] * 8, 90, 10, seed=6)
    b = Windowed([40, 1], [3000, 20], 1000, 4, seed=7, hide=False, poison=False)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    first = None
    for _ in range(4):
        results = []
        for s, c in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                results.append(c.run())
        torch.cuda.synchronize()
        for c, r in zip((a, b), results):
            c.check(*r)
        first = first or results
        assert all(torch.equal(x, y) for f, r in zip(first, results) for x, y in zip(f, r))
    out, lse = a.run(stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(out, first[0][0])


def test_refusals():
    c = Case([4], [30], seed=6)
    q, cu = c.q.cuda(), dev(c.cu)
    with pytest.raises(ValueError):
        cache.attention(c.c, 0, q, cu, sinks=4)
    with pytest.raises(ValueError):
        cache.attention(c.c, 0, q, cu, window=4, shared=cache.share(c.c))
    for kw in (dict(window=0), dict(window=-3), dict(window=-2 ** 40), dict(window=5, sinks=-1), dict(window=5, layer=1)):
        with pytest.raises(binding.SpecRejectError):
            cache.attention(c.c, kw.pop("layer", 0), q, cu, **kw)
