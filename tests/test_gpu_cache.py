"""GPU bookkeeping of the paged cache against the CPU oracle (exact: integers and copies)."""
import numpy as np
import pytest

from oracle import cache as oracle_cache
from speculative_decoding_rejection_spec_gb300 import binding, cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import torch
    import __graft_entry__ as G
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    G.build()
    cache.load()


def dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def cu_of(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


class Pair:
    """A cache on the GPU and its oracle, driven by the same calls."""

    def __init__(self, requests, max_pages, num_pages, page_size, layers=2, heads=2, dim=16, dtype="bf16", seed=0,
                 layout="nhd"):
        import torch
        dt = torch.bfloat16 if dtype == "bf16" else torch.float16
        gen = torch.Generator().manual_seed(seed)
        self.book = oracle_cache.Book(requests, max_pages, num_pages, page_size)
        kv = torch.randn((2, layers, num_pages, page_size, heads, dim), generator=gen).to(dt)
        self.k, self.v = kv[0].clone(), kv[1].clone()  # the oracle's rows
        c = cache.make_cache(layers, num_pages, page_size, heads, dim, requests, max_pages, dtype=dt)
        if layout == "hnd":  # pages of heads of tokens, keys and values side by side
            both = torch.empty((layers, num_pages, 2, heads, page_size, dim), dtype=dt, device="cuda")
            c = cache.PagedCache(both[:, :, 0].transpose(2, 3), both[:, :, 1].transpose(2, 3),
                                 page_table=c.page_table, lens=c.lens, held=c.held, ref_counts=c.ref_counts,
                                 free_pages=c.free_pages, num_free=c.num_free)
        c.k.copy_(kv[0])
        c.v.copy_(kv[1])
        self.c, self.gen = c, gen

    def reserve(self, n):
        for old, new, rows in self.book.reserve(n):
            for x in (self.k, self.v):
                x[:, new, :rows] = x[:, old, :rows]
        cache.reserve(self.c, dev(cu_of(n)))

    def append(self, n, pad=0):
        import torch
        N = int(sum(n))
        L, _, _, H, D = self.k.shape
        new = torch.randn((2, L, N + pad, H, D), generator=self.gen).to(self.k.dtype)
        cu = dev(cu_of(n))
        for layer in range(L):
            cache.append(self.c, layer, new[0, layer].cuda(), new[1, layer].cuda(), cu)
        t = 0
        for r, m in enumerate(n):
            for i in range(m):
                page, row = self.book.slot(r, int(self.book.lens[r]) + i)
                self.k[:, page, row], self.v[:, page, row] = new[0, :, t], new[1, :, t]
                t += 1
        return new

    def commit(self, n, accepted, parents=None, last=None, out_lens=None):
        before = self.book.lens.copy()
        moves = self.book.commit(n, accepted, parents, last)
        for r, a, b in moves:  # ascending levels
            (p0, i0), (p1, i1) = self.book.slot(r, a), self.book.slot(r, b)
            for x in (self.k, self.v):
                x[:, p1, i1] = x[:, p0, i0]
        kw = {}
        if parents is not None:
            kw = dict(parent=dev(np.concatenate(parents)), last_node=dev(last))
        cache.commit(self.c, dev(cu_of(n)), dev(accepted), out_lens=out_lens, **kw)
        if out_lens is not None:
            assert np.array_equal(out_lens.cpu().numpy(), self.book.lens)
            self.book.lens[:] = before

    def fork(self, src, dst):
        self.book.fork(src, dst)
        cache.fork(self.c, dev(src), dev(dst))

    def release(self, keep=None):
        self.book.release(keep, None if keep is None else len(keep))
        cache.release(self.c, None if keep is None else dev(keep))

    def check(self, error=(0, -1)):
        import torch
        status, bits, first = cache.last_error(self.c)
        assert (bits, first) == self.book.take_error() == error
        assert status == (5 if bits else 0)
        c, b = self.c, self.book
        assert int(c.num_free.item()) == b.num_free
        for got, want in ((c.page_table, b.table), (c.lens, b.lens), (c.held, b.held), (c.ref_counts, b.ref),
                          (c.free_pages, b.free)):
            assert np.array_equal(got.cpu().numpy(), want)
        assert torch.equal(c.k.cpu(), self.k) and torch.equal(c.v.cpu(), self.v)


def random_trees(rng, n):
    parents, last, acc = [], [], []
    for m in n:
        par = [-1] * min(m, 1) + [int(rng.integers(0, i)) for i in range(1, m)]
        at = int(rng.integers(0, m)) if m else 0
        depth, x = 0, at
        while m and par[x] >= 0:
            x, depth = par[x], depth + 1
        parents.append(np.array(par, np.int32))
        last.append(at)
        acc.append(depth if m else -1)
    return parents, np.array(last, np.int32), np.array(acc, np.int32)


@pytest.mark.parametrize("page_size,layout,dtype", [(16, "nhd", "bf16"), (8, "hnd", "f16"), (1, "nhd", "bf16"),
                                                    (5, "hnd", "bf16"), (64, "nhd", "f16")])
@pytest.mark.parametrize("seed", [0, 1])
def test_random_steps_match_the_oracle(page_size, layout, dtype, seed):
    """Many steps of everything together: chains and trees, forks, truncations, freed requests."""
    rng = np.random.default_rng(seed * 100 + page_size)
    R, top = 7, 120
    MP = -(-top // page_size)
    p = Pair(R, MP, 2 * R * MP, page_size, heads=3, dim=24, dtype=dtype, seed=seed, layout=layout)
    for step in range(12):
        n = rng.integers(0, 12, R)
        n = np.minimum(n, top - p.book.lens)
        p.reserve(n)
        p.append(n, pad=int(rng.integers(0, 3)))
        if step % 2:
            p.commit(n, [int(rng.integers(-1, m)) if m else 0 for m in n])
        else:
            parents, last, acc = random_trees(rng, n)
            p.commit(n, acc, parents, last)
        if step % 3 == 2:
            keep = np.where(rng.random(R) < 0.4, 0, rng.integers(0, top, R))
            p.release(keep)
        empty = np.nonzero(p.book.held == 0)[0]
        full = np.nonzero(p.book.lens > 0)[0]
        if len(empty) and len(full):
            p.fork(rng.choice(full, len(empty)), empty)
        if step % 4 == 3:
            p.release()
        p.check()
    p.release(np.zeros(R, np.int32))
    p.check()
    assert p.book.num_free == len(p.book.free)


def test_all_holders_of_a_page_write_it():
    """The last of the holders keeps the page; with one holder absent every writer copies."""
    p = Pair(5, 4, 24, 16)
    p.reserve([20, 0, 0, 0, 0])
    p.append([20, 0, 0, 0, 0])
    p.commit([20, 0, 0, 0, 0], [19, 0, 0, 0, 0])
    p.fork([0, 0, 0, 0], [4, 1, 3, 2])
    p.reserve([1, 1, 0, 1, 1])
    p.check()
    p.append([1, 1, 0, 1, 1])
    p.release([20, 20, 20, 20, 0])
    p.fork([2], [4])
    p.reserve([0, 0, 1, 0, 3])
    p.append([0, 0, 1, 0, 3])
    p.check()


def test_many_requests_and_pages():
    """More requests than the bookkeeping block has threads, long rows, forks from one source."""
    R, MP = 1500, 40
    p = Pair(R, MP, 20000, 8, layers=1, heads=1, dim=8)
    n = np.zeros(R, np.int64)
    n[:500] = np.arange(500) % 37
    p.reserve(n)
    p.append(n)
    p.commit(n, n - 1)
    p.check()
    p.fork([36] * 700 + [73] * 300, np.arange(500, 1500))
    p.reserve(np.ones(R, np.int64))
    p.check()
    p.append(np.ones(R, np.int64))
    p.release(np.where(np.arange(R) % 3 == 0, 0, 20))
    p.check()


def test_capacity_changes_nothing():
    p = Pair(4, 8, 6, 16)
    p.reserve([40, 0, 20, 0])  # 3 + 2 of 6 pages
    p.check()
    p.reserve([10, 16, 0, 17])  # 0 + 1 + 0 + 2
    p.check((cache.DEVERR_CAPACITY, 3))
    p.reserve([0, 16, 0, 0])
    p.check()
    p.reserve([0, 0, 0, 1])
    p.check((cache.DEVERR_CAPACITY, 3))


def test_bad_requests_are_skipped():
    p = Pair(4, 2, 12, 16)
    p.reserve([5, 33, 6, 0])  # more than two pages hold
    p.check((cache.DEVERR_LENGTH, 1))
    p.append([5, 0, 6, 0])
    p.commit([5, 0, 6, 0], [5, 0, 2, 0])  # five accepted drafts of four
    p.check((cache.DEVERR_LENGTH, 0))
    p.commit([5, 0, 0, 0], [-2, 0, 0, 0])
    p.check((cache.DEVERR_LENGTH, 0))
    p.release([0, -1, 3, 0])
    p.check((cache.DEVERR_LENGTH, 1))


def test_bad_forks_are_refused():
    p = Pair(6, 4, 20, 16)
    p.reserve([20, 9, 0, 0, 0, 0])
    p.append([20, 9, 0, 0, 0, 0])
    p.commit([20, 9, 0, 0, 0, 0], [19, 8, 0, 0, 0, 0])
    for src, dst, first in (([0, 0], [2, 2], 2), ([0], [0], 0), ([0], [1], 1), ([0, 9], [3, 4], 4), ([0], [-1], -1),
                            ([0, 5], [5, 2], 2)):
        p.fork(src, dst)
        p.check((cache.DEVERR_FORK, first))


def test_bad_trees_commit_nothing():
    p = Pair(3, 4, 20, 16)
    n = [6, 6, 6]
    p.reserve(n)
    p.append(n)
    good = np.array([-1, 0, 0, 1, 2, 2], np.int32)
    late = np.array([-1, 0, 4, 1, 2, 2], np.int32)  # a parent behind its child
    p.commit(n, [2, 2, 1], [good, late, good], [5, 4, 5])  # and a path longer than the count says
    p.check((oracle_cache.TREE, 1))
    assert p.book.lens.tolist() == [3, 0, 0]


def test_commit_into_other_lengths():
    import torch
    p = Pair(3, 4, 20, 16)
    n = [6, 0, 9]
    p.reserve(n)
    p.append(n)
    out = torch.full((3,), -5, dtype=torch.int32, device="cuda")
    p.commit(n, [2, 0, -1], out_lens=out)
    parents = [np.array([-1, 0, 0, 1, 2, 2], np.int32), np.zeros(0, np.int32), np.array([-1] + [0] * 8, np.int32)]
    p.commit(n, [2, 0, 1], parents, [5, 0, 7], out_lens=out)
    p.check()


def test_bad_layouts_do_nothing():
    """cu_new that starts elsewhere, decreases or passes the rows given."""
    import torch
    p = Pair(3, 4, 20, 16)
    rows = torch.ones((8, 2, 16), dtype=torch.bfloat16, device="cuda")
    par = dev([-1, 0, 0, 0, 0, 0, 0, 0])
    p.reserve([4, 4, 0])
    p.check()
    for cu in ([1, 2, 3, 4], [0, 5, 4, 6]):
        cache.reserve(p.c, dev(cu))
        p.book._error(oracle_cache.LAYOUT)
        p.check((oracle_cache.LAYOUT, -1))
    for cu in ([1, 2, 3, 4], [0, 5, 4, 6], [0, 4, 8, 9]):
        cache.append(p.c, 0, rows, rows, dev(cu))
        cache.commit(p.c, dev(cu), dev([0, 0, 0]), parent=par, last_node=dev([0, 0, 0]))
        p.book._error(oracle_cache.LAYOUT)
        p.check((oracle_cache.LAYOUT, -1))


def test_append_refuses_shared_and_missing_pages():
    """Rows go only to pages that their request alone holds."""
    import torch
    p = Pair(3, 4, 20, 16, layers=1)
    p.reserve([20, 0, 0])
    p.append([20, 0, 0])
    p.commit([20, 0, 0], [19, 0, 0])
    p.fork([0], [2])
    rows = torch.ones((30, 2, 16), dtype=torch.bfloat16, device="cuda")
    cache.append(p.c, 0, rows, rows, dev([0, 2, 4, 4]))  # a shared page; a request without pages
    p.book._error(oracle_cache.PAGE, 0)
    p.check((cache.DEVERR_PAGE, 0))
    cache.append(p.c, 0, rows, rows, dev([0, 0, 2, 2]))
    p.book._error(oracle_cache.PAGE, 1)
    p.check((cache.DEVERR_PAGE, 1))


def test_pages_released_twice_are_reported():
    p = Pair(2, 4, 8, 16)
    p.reserve([20, 20])
    table = p.book.table.copy()
    table[1, 1] = table[0, 1]  # a page in two tables that is counted once
    p.book.table[:] = table
    p.c.page_table.copy_(dev(table))
    cache.release(p.c, dev([0, 0]))
    status, bits, first = cache.last_error(p.c)
    assert (status, bits) == (5, cache.DEVERR_PAGE) and first in (0, 1)
    assert p.c.ref_counts.cpu().tolist() == [0, 0, 0, 0, 1, 0, 0, 0]
    assert int(p.c.num_free.item()) == 7 and sorted(p.c.free_pages.cpu().tolist()[:7]) == [0, 1, 2, 3, 5, 6, 7]


def test_strided_rows_and_wide_heads():
    """New rows as views of a fused projection; head rows above one warp's turn."""
    import torch
    for heads, dim in ((8, 128), (40, 64), (1, 1024), (5, 8)):
        c = cache.make_cache(2, 12, 16, heads, dim, 2, 6, dtype=torch.float16)
        n = [17, 30]
        cu = dev(cu_of(n))
        fused = torch.randn((47, 3 * heads, dim), device="cuda").half()
        k, v = fused[:, heads:2 * heads], fused[:, 2 * heads:].transpose(0, 1).contiguous().transpose(0, 1)
        cache.reserve(c, cu)
        cache.append(c, 1, k, v, cu)
        assert cache.last_error(c) == (0, 0, -1)
        table = c.page_table.cpu().numpy()
        t = 0
        for r, m in enumerate(n):
            for i in range(m):
                page = table[r, i // 16]
                assert torch.equal(c.k[1, page, i % 16], k[t]) and torch.equal(c.v[1, page, i % 16], v[t])
                t += 1
        assert not c.k[0].any()


def test_captured_step_follows_the_device_data():
    """A captured reserve, append, commit and release replays on whatever lengths are there."""
    import torch
    p = Pair(4, 8, 40, 8, layers=1)
    n = [3, 0, 9, 1]
    rows = [torch.zeros((13, 2, 16), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cu, acc = dev(cu_of(n)), dev([1, 0, 8, -1])

    def step():
        cache.reserve(p.c, cu)
        cache.append(p.c, 0, rows[0], rows[1], cu)
        cache.commit(p.c, cu, acc)
        cache.release(p.c)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(3):
        new = torch.randn((2, 13, 2, 16), generator=p.gen).to(torch.bfloat16)
        rows[0].copy_(new[0])
        rows[1].copy_(new[1])
        graph.replay()
        p.book.reserve(n)
        t = 0
        for r, m in enumerate(n):
            for j in range(m):
                page, row = p.book.slot(r, int(p.book.lens[r]) + j)
                p.k[0, page, row], p.v[0, page, row] = new[0, t], new[1, t]
                t += 1
        p.book.commit(n, [1, 0, 8, -1])
        p.book.release()
        p.check()


def test_binding_refusals():
    import torch
    c = cache.make_cache(1, 4, 16, 2, 64, 2, 2)
    cu = dev([0, 1, 2])
    rows = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (rows.half(), rows[:, :1], rows[:, :, :32], rows[0]):
        with pytest.raises(TypeError):
            cache.append(c, 0, bad, bad, cu)
    with pytest.raises(ValueError):
        cache.append(c, 0, rows, rows[:1], cu)
    with pytest.raises(TypeError):
        cache.reserve(c, cu.long())
    with pytest.raises(ValueError):
        cache.reserve(c, cu.cpu())
    with pytest.raises(ValueError):
        cache.commit(c, cu, dev([0, 0]), parent=dev([-1, -1]))
    with pytest.raises(binding.SpecRejectError):
        cache.append(c, 3, rows, rows, cu)
    with pytest.raises(ValueError):
        cache.PagedCache(c.k, c.v.transpose(2, 3).contiguous().transpose(2, 3), page_table=c.page_table, lens=c.lens,
                         held=c.held, ref_counts=c.ref_counts, free_pages=c.free_pages, num_free=c.num_free)


def test_offsets_past_32_bits():
    """The same steps in a cache of few pages and in the last pages of one of 5 GB of keys: bit for bit alike."""
    import torch
    heads, dim, page = 8, 128, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    caches = [cache.make_cache(2, pages, page, heads, dim, 4, 16) for pages in (48, 20000)]
    assert caches[1].k.numel() * 2 > 2 ** 32
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")

    def step(n, parent=None):
        cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
        N = sum(n)
        rows = [[torch.randn((N, h, dim), generator=gen, device="cuda").bfloat16() for h in (heads, heads, 2 * heads)]
                for _ in range(2)]
        outs = []
        for c in caches:
            cache.reserve(c, cu)
            for layer, (k, v, q) in enumerate(rows):
                cache.append(c, layer, k, v, cu)
                outs.append(cache.attention(c, layer, q, cu, parent=parent))
            assert cache.last_error(c) == (0, 0, -1)
        assert outs[0].isfinite().all() and torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
        return cu

    cu = step([300, 129, 65, 0])
    for c in caches:
        cache.commit(c, cu, ints(299, 128, 64, -1))
        cache.fork(c, ints(0), ints(3))
    parent = ints(*[-1, 0, 0, 1, 2, 4] * 4)
    cu = step([6] * 4, parent)  # requests 0 and 3 share their last page
    for c in caches:
        cache.commit(c, cu, ints(2, 3, 1, 0), parent=parent, last_node=ints(3, 5, 2, 0))
    step([1, 1, 1, 1])
    a, b = caches
    assert a.lens.tolist() == b.lens.tolist() == [303, 133, 67, 301]
    assert (torch.where(a.page_table >= 0, a.page_table + 20000 - 48, -1) == b.page_table).all()
