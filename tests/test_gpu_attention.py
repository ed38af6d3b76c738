"""GPU attention over the paged cache against the 64-bit oracle.

Error bound per output, u = eps / 2 of the type, A = sum p |v|, S = max scale * sum |q| |k|:
  p is rounded once (u each: u A), the output once (u |o|); fp32 sums of the products of a score
  (dim terms), of the weights and of the outputs (L terms) lose at most 2^-23 per term (the tensor
  cores may truncate), the scaled score and its exponential a few 2^-23 of their size:
  |o - exact| <= u |o| + A (u + 2 e_s + 2 L 2^-23 + 2^-20),  e_s = (dim + 8) 2^-23 S,
  |lse - exact| <= e_s + L 2^-23 + 2^-20 (1 + |lse|).
fp16 weights below its smallest normal are rounded to multiples of 2^-24: L 2^-25 max|v| more."""
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


class Case:
    """A cache with `ctx` committed tokens and `n` new ones per request, their rows in place."""

    def __init__(self, n, ctx, heads=2, group=4, dim=128, page=16, dtype="bf16", tree=False, layers=1, layer=0,
                 layout="nhd", pad=0, q_scale=2.0, seed=0, poison=True):
        import torch
        self.n, self.ctx, self.heads, self.group, self.dim, self.page = list(n), list(ctx), heads, group, dim, page
        self.layer, self.dtype, self.pad = layer, dtype, pad
        dt = torch.bfloat16 if dtype == "bf16" else torch.float16
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        R, L = len(n), [c + m for c, m in zip(ctx, n)]
        need = [-(-x // page) for x in L]
        MP, NP = max(max(need), 1) + 1, sum(need) + 3
        order = rng.permutation(NP)
        table = np.full((R, MP), 2 ** 30, np.int32)  # entries behind a request's pages are never used
        used = 0
        kv = torch.randn((2, NP, page, heads, dim), generator=gen).to(dt)
        if poison:  # what lies outside the requests' tokens
            kv_in = torch.zeros((NP, page), dtype=torch.bool)
        for r in range(R):
            table[r, :need[r]] = order[used:used + need[r]]
            used += need[r]
            if poison:
                for t in range(L[r]):
                    kv_in[table[r, t // page], t % page] = True
        if poison:
            kv[0][~kv_in] = float("nan")
            kv[1][~kv_in] = float("inf")
        self.kv, self.table = kv, table
        shape = (layers, NP, page, heads, dim) if layout == "nhd" else (layers, NP, heads, page, dim)
        k, v = (torch.zeros(shape, dtype=dt, device="cuda") for _ in range(2))
        if layout == "hnd":
            k, v = k.transpose(2, 3), v.transpose(2, 3)
        if layout == "hpn":
            k, v = (torch.zeros((layers, heads, NP, page, dim), dtype=dt, device="cuda").permute(0, 2, 3, 1, 4)
                    for _ in range(2))
        k[layer], v[layer] = kv[0].cuda(), kv[1].cuda()
        ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
        self.c = cache.PagedCache(k, v, page_table=dev(table), lens=dev(ctx), held=dev(need), ref_counts=ints(NP),
                                  free_pages=ints(NP), num_free=ints(1))
        N = sum(n)
        self.q = (q_scale * torch.randn((N + pad, heads * group, dim), generator=gen)).to(dt)
        self.cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.parents = None
        if tree:
            self.parents = [np.array([-1] * min(m, 1) + [int(rng.integers(max(0, i // 3 - 1), i)) for i in
                                                         range(1, m)], np.int32) for m in n]

    def run(self, **kw):
        import torch
        N, H = self.q.shape[:2]
        q = kw.pop("q", self.q.cuda())
        out = kw.pop("out", None)
        if out is None:
            out = torch.full(self.q.shape, 7.0, dtype=self.q.dtype, device="cuda")
        lse = torch.full((N, H), 7.0, device="cuda")
        parent = None
        if self.parents is not None:
            parent = dev(np.concatenate(self.parents + [np.zeros(self.pad, np.int32)]))
        cache.attention(self.c, self.layer, q, dev(self.cu), parent=parent, out=out, lse=lse, **kw)
        return out, lse

    def check(self, out, lse, scale=None, error=(0, 0, -1), skip=()):
        assert cache.last_error(self.c) == error
        scale = self.dim ** -0.5 if scale is None else scale
        u = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -11
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        worst = 0.0
        for r, m in enumerate(self.n):
            a, b = self.cu[r], self.cu[r + 1]
            if r in skip:
                assert (out[a:b] == 7).all() and (lse[a:b] == 7).all()
                continue
            if m == 0:
                continue
            L = self.ctx[r] + m
            pages = self.table[r, :-(-L // self.page)]
            seen = oracle_cache.visible(m, self.ctx[r], None if self.parents is None else self.parents[r])
            for h in range(self.heads):
                k, v = (self.kv[i][pages, :, h].reshape(-1, self.dim)[:L].double().numpy() for i in (0, 1))
                hs = slice(h * self.group, (h + 1) * self.group)
                q = self.q[a:b, hs].double().numpy()
                o, z, A, S = oracle_cache.attention(q, k, v, seen, scale)
                es = (self.dim + 8) * 2.0 ** -23 * S
                tol = u * np.abs(o) + A * (u + 2 * es + 2 * L * 2.0 ** -23 + 2.0 ** -20)[..., None]
                if self.dtype == "f16":
                    tol = tol + L * 2.0 ** -25 * np.abs(v).max()
                diff = np.abs(out[a:b, hs] - o)
                assert (diff <= tol).all(), (r, h, float((diff - tol).max()), np.argwhere(~(diff <= tol))[:4])
                assert (np.abs(lse[a:b, hs] - z) <= es + L * 2.0 ** -23 + 2.0 ** -20 * (1 + np.abs(z))).all()
                worst = max(worst, float((diff / tol).max()))
        assert (out[self.cu[-1]:] == 7).all() and (lse[self.cu[-1]:] == 7).all()  # padding rows
        return worst


EDGES = [0, 1, 7, 63, 64, 127, 128, 129, 255, 256, 300]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 9, 33])
def test_contexts_around_the_tiles(dtype, dim, n):
    c = Case([n] * len(EDGES), EDGES, dim=dim, dtype=dtype, seed=n + dim)
    c.check(*c.run())


@pytest.mark.parametrize("dim", [8, 16, 40, 72, 80, 96, 120])
def test_odd_head_dims(dim):
    c = Case([1, 5, 0, 17], [130, 3, 50, 260], dim=dim, heads=3, group=2, seed=dim)
    c.check(*c.run())


@pytest.mark.parametrize("heads,group", [(1, 1), (3, 1), (2, 3), (2, 5), (1, 7), (1, 16), (1, 71), (1, 128)])
def test_head_groups(heads, group):
    c = Case([1, 4, 0, 3], [200, 129, 5, 0], heads=heads, group=group, dim=64, seed=group)
    c.check(*c.run())


@pytest.mark.parametrize("page", [8, 16, 24, 32, 40, 64, 128, 192, 256, 1000])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_page_sizes(page, layout):
    c = Case([3, 1, 40], [500, 127, 77], page=page, layout=layout, layers=2, layer=1, seed=page)
    c.check(*c.run())


@pytest.mark.parametrize("dtype,group,n", [("bf16", 4, [1, 31, 64, 65, 100, 0, 128, 2]), ("f16", 1, [128, 127, 20]),
                                           ("bf16", 7, [64, 40, 33, 128])])
def test_trees(dtype, group, n):
    rng = np.random.default_rng(len(n))
    c = Case(n, rng.integers(0, 400, len(n)), group=group, dim=64, dtype=dtype, tree=True, seed=group)
    c.check(*c.run())


def test_tree_that_is_a_chain_equals_the_chain():
    import torch
    a = Case([50, 7], [300, 100], seed=5)
    out, lse = a.run()
    a.parents = [np.arange(-1, 49, dtype=np.int32), np.arange(-1, 6, dtype=np.int32)]
    tree, tree_lse = a.run()
    assert torch.equal(out, tree) and torch.equal(lse, tree_lse)


@pytest.mark.parametrize("n,ctx,group", [([200], [0], 1), ([300], [1000], 4), ([64, 500, 1], [700, 13, 900], 2),
                                         ([129, 257], [0, 127], 5), ([1031], [100], 3)])
def test_prompt_chunks(n, ctx, group):
    c = Case(n, ctx, heads=2, group=group, page=32, seed=sum(n))
    c.check(*c.run())


@pytest.mark.parametrize("dim,group,dtype", [(72, 4, "bf16"), (96, 1, "f16"), (40, 16, "bf16"), (128, 6, "f16"),
                                             (64, 128, "f16")])
@pytest.mark.parametrize("pad", [0, 5])
def test_wide_blocks_of_odd_shapes(dim, group, dtype, pad):
    """Row blocks of more than 128 rows, the last one ending with the tensor or before padding rows."""
    n = [3 * 256 // group + 1, 130 // group + 1, 1]
    c = Case(n, [140, 0, 77], heads=2, group=group, dim=dim, page=24, dtype=dtype, pad=pad, seed=dim)
    c.check(*c.run())


def test_many_row_blocks_per_share():
    """More row blocks than the device has SMs by far, narrow and wide ones of one tile to several: every
    share walks through a run of them, across requests without new tokens."""
    rng = np.random.default_rng(8)
    n = np.where(rng.random(1100) < 0.3, 0, rng.integers(1, 4, 1100))
    n[::37] = 70
    ctx = rng.integers(0, 200, 1100)
    ctx[::10] = rng.integers(0, 900, 110)
    c = Case(n, ctx, heads=2, group=4, dim=64, page=16, dtype="f16", seed=12, poison=False)
    c.check(*c.run())
    c = Case(n[:300], ctx[:300], heads=4, group=2, dim=128, page=32, seed=13, poison=False)
    c.check(*c.run())


@pytest.mark.parametrize("layout", ["hpn"])
def test_pages_inside_heads(layout):
    """A head's pages together: a page's stride is below a head's."""
    c = Case([3, 1, 40], [500, 127, 77], page=16, layout=layout, layers=2, layer=1, seed=3)
    c.check(*c.run())


@pytest.mark.parametrize("n,heads,ctx", [(1, 1, 9000), (1, 4, 20011), (6, 2, 12345), (33, 1, 7777)])
def test_long_contexts(n, heads, ctx):
    c = Case([n], [ctx], heads=heads, page=64, seed=ctx, poison=False)
    c.check(*c.run())


def test_ragged_batch():
    rng = np.random.default_rng(3)
    n, ctx = rng.integers(0, 10, 150), rng.integers(0, 700, 150)
    ctx[7], n[7] = 6000, 200
    c = Case(n, ctx, page=32, pad=11, seed=9)
    c.check(*c.run())


def test_large_scores():
    """Scores of hundreds: softmax rows that are nearly one-hot, maxima that move late."""
    for seed in range(3):
        c = Case([4, 12], [900, 333], q_scale=60.0, seed=seed)
        c.check(*c.run())


def test_maximum_rises_from_tile_to_tile():
    """Keys that grow along the context: every tile raises the running maximum by far."""
    import torch
    c = Case([3], [1500], heads=1, group=2, page=64, seed=1, poison=False)
    order = torch.from_numpy(c.table[0, :24].astype(np.int64))
    grow = torch.linspace(0, 6, 24 * 64).view(24, 64)
    base = torch.randn(128, generator=torch.Generator().manual_seed(4))
    for i in range(24):
        c.kv[0][order[i], :, 0] = (grow[i][:, None] * base[None, :]).to(c.kv.dtype)
    c.q[:, :] = (2 * base).to(c.q.dtype)
    c.c.k[0].copy_(c.kv[0].cuda())
    c.check(*c.run())


def test_strided_queries_and_outputs():
    import torch
    c = Case([5, 1, 30], [200, 4, 60], heads=2, group=3, dim=64, seed=2)
    N, H, D = c.q.shape
    fused = torch.zeros((N, 3 * H, D), dtype=c.q.dtype, device="cuda")
    fused[:, :H] = c.q.cuda()
    by_head = torch.full((H, N, D), 7.0, dtype=c.q.dtype, device="cuda")
    out, lse = c.run(q=fused[:, :H], out=by_head.transpose(0, 1))
    c.check(out, lse)


def test_scale_is_the_caller_s():
    c = Case([5], [300], seed=3)
    c.check(*c.run(scale=0.31), scale=0.31)


def test_repeated_calls_are_bit_identical():
    import torch
    c = Case([9] * 40, np.random.default_rng(0).integers(0, 3000, 40), page=32, seed=1, poison=False)
    out, lse = c.run()
    for _ in range(3):
        again, lse2 = c.run()
        assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_bad_requests_are_left_out():
    c = Case([3, 4, 5, 2], [100, 200, 300, 50], seed=4)
    c.c.lens[1] = -1
    out, lse = c.run()
    c.check(out, lse, error=(5, cache.DEVERR_LENGTH, 1), skip=(1,))
    c.c.lens[1] = 200
    c.c.lens[2] = 17 * 21  # more tokens than its columns hold
    out, lse = c.run()
    c.check(out, lse, error=(5, cache.DEVERR_LENGTH, 2), skip=(2,))


def test_bad_layout_writes_nothing():
    c = Case([3, 4], [100, 200], seed=4)
    for cu in ([1, 3, 7], [0, 5, 4], [0, 3, 8]):
        good, c.cu = c.cu, np.array(cu, np.int32)
        out, lse = c.run()
        c.cu = good
        assert (out == 7).all() and (lse == 7).all()
        assert cache.last_error(c.c) == (5, binding.DEVERR_LAYOUT, -1)


def test_bad_pages_read_as_zeros():
    c = Case([3, 4], [100, 200], heads=1, seed=4)
    for bad in (-1, len(c.kv[0]), 2 ** 30):
        table = c.table.copy()
        table[1, 2] = bad
        c.c.page_table.copy_(dev(table))
        page = c.table[1, 2]
        saved = c.kv[:, page].clone()
        c.kv[:, page] = 0  # what the oracle sees
        out, lse = c.run()
        c.check(out, lse, error=(5, cache.DEVERR_PAGE, 1))
        c.kv[:, page] = saved


def test_bad_trees_are_reported():
    c = Case([9, 140, 9], [100, 10, 20], tree=True, seed=4)
    out, lse = c.run()
    c.check(out, lse, error=(5, binding.DEVERR_TREE, 1), skip=(1,))  # more nodes than a tree may have
    c.parents[0] = c.parents[0].copy()
    c.parents[0][3] = 5
    out, lse = c.run()
    status, bits, first = cache.last_error(c.c)
    assert (status, bits, first) == (5, binding.DEVERR_TREE, 0)


def test_empty_calls():
    import torch
    c = Case([0, 0], [5, 0], seed=0)
    assert c.run()[0].shape == (0, 8, 128)
    c = Case([0, 0], [5, 0], pad=4, seed=0)
    c.check(*c.run())
    q = torch.zeros((0, 8, 128), dtype=torch.bfloat16, device="cuda")
    assert cache.attention(c.c, 0, q, dev([0])).shape == q.shape


def test_captured_call_follows_the_device_data():
    import torch
    c = Case([4, 9, 1], [300, 20, 500], seed=6, poison=False)
    q = c.q.cuda()
    cu = dev(c.cu)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attention(c.c, 0, q, cu, out=out, lse=lse)
    for ctx in ([300, 20, 500], [3, 22, 128], [299, 0, 1]):
        c.ctx = ctx
        c.c.lens.copy_(dev(ctx))
        graph.replay()
        c.check(out, lse)


def test_two_streams_at_once():
    import torch
    a = Case([4, 9, 1] * 8, [300, 20, 500] * 8, seed=6)
    b = Case([40, 1], [3000, 20], seed=7, poison=False)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        results = []
        for s, c in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                results.append(c.run())
        torch.cuda.synchronize()
        for c, r in zip((a, b), results):
            c.check(*r)


def test_explicit_stream():
    import torch
    c = Case([4, 9, 1], [300, 20, 500], seed=6)
    s = torch.cuda.Stream()
    q, cu = c.q.cuda(), dev(c.cu)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    cache.attention(c.c, 0, q, cu, out=out, lse=lse, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    c.check(out, lse)


def test_refusals():
    import torch
    c = Case([4], [30], seed=6)
    q, cu = c.q.cuda(), dev(c.cu)
    with pytest.raises(TypeError):
        cache.attention(c.c, 0, q.half(), cu)
    with pytest.raises(TypeError):
        cache.attention(c.c, 0, q[:, :, :64], cu)
    with pytest.raises(ValueError):
        cache.attention(c.c, 0, q.cpu(), cu)
    with pytest.raises(ValueError):
        cache.attention(c.c, 0, q, cu, out=torch.empty_like(q)[:2])
    with pytest.raises(TypeError):
        cache.attention(c.c, 0, q, cu, lse=torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda"))
    with pytest.raises(TypeError):
        cache.attention(c.c, 0, q, cu, parent=dev([-1, 0]))
    for kw in (dict(layer=1), dict(scale=0.0), dict(workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(binding.SpecRejectError):
            cache.attention(c.c, kw.pop("layer", 0), q, cu, **kw)
    with pytest.raises(binding.SpecRejectError):
        cache.attention(c.c, 0, q[:, :7], cu)


# ---------------------------------------------------------------------------------------
# The operators together, as a serving loop uses them
# ---------------------------------------------------------------------------------------


@pytest.mark.parametrize("tree", [False, True])
def test_serving_loop(tree):
    """A few steps of a toy two-layer model whose logits come from the attention's outputs: reserve,
    append and attend per layer, verify with the sampler or the tree verification, commit.  Every
    request's attention is checked against the rows that the accepted tokens should have left."""
    import torch
    rng = np.random.default_rng(11 + tree)
    L, P, H, G, D, B, V = 2, 16, 2, 2, 64, 5, 97
    c = cache.make_cache(L, 200, P, H, D, B + 2, 12)
    table = torch.randn((L, 3, V, H * G, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    head = torch.randn((H * G * D, V), generator=torch.Generator().manual_seed(2)).cuda()
    history = [[[] for _ in range(L)] for _ in range(B)]  # committed (k, v) rows
    tokens = rng.integers(0, V, B)
    for step in range(4):
        n = rng.integers(1, 7, B) if step else rng.integers(20, 40, B)
        if tree and step:
            parents = [np.array([-1] + [int(rng.integers(0, i)) for i in range(1, m)], np.int32) for m in n]
        else:
            parents = [np.arange(-1, m - 1, dtype=np.int32) for m in n]
        ids = rng.integers(0, V, n.sum())
        cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        ids[cu[:-1]] = tokens
        rows = table[:, :, torch.from_numpy(ids)].cuda()
        dcu, par = dev(cu), dev(np.concatenate(parents))
        cache.reserve(c, dcu)
        for layer in range(L):
            k, v = rows[layer, 0, :, :H], rows[layer, 1, :, :H]
            cache.append(c, layer, k, v, dcu)
            out = cache.attention(c, layer, rows[layer, 2], dcu, parent=par if tree else None)
            for r in range(B):
                a, b = cu[r], cu[r + 1]
                seen = oracle_cache.visible(n[r], len(history[r][layer]), parents[r])
                for h in range(H):
                    past = history[r][layer]
                    kk = np.array([x[0][h] for x in past] + list(k[a:b, h].double().cpu().numpy()))
                    vv = np.array([x[1][h] for x in past] + list(v[a:b, h].double().cpu().numpy()))
                    q = rows[layer, 2][a:b, h * G:(h + 1) * G].double().cpu().numpy()
                    o, _, A, S = oracle_cache.attention(q, kk, vv, seen, D ** -0.5)
                    es = (D + 8) * 2.0 ** -23 * S
                    tol = 2.0 ** -8 * np.abs(o) + A * (2.0 ** -8 + 2 * es + 2.0 ** -14)[..., None]
                    got = out[a:b, h * G:(h + 1) * G].double().cpu().numpy()
                    assert (np.abs(got - o) <= tol).all()
        logits = (out.float().reshape(len(ids), -1) @ head).to(torch.bfloat16)
        if tree:
            am = logits.float().argmax(1).cpu().numpy()
            for r in range(B):  # drafts that follow the model, so that paths go somewhere
                for i in range(1, n[r]):
                    if rng.random() < 0.6:
                        ids[cu[r] + i] = am[cu[r] + parents[r][i]]
            toks, acc, last, _ = binding.tree_verify_greedy(logits, par, dev(ids), dcu)
            cache.commit(c, dcu, acc, parent=par, last_node=last)
            last = last.cpu().numpy()
        else:
            cud = dev(cu - np.arange(B + 1))
            drafts = np.delete(ids, cu[:-1])
            toks, acc = binding.sample(logits, dev(drafts), cud, torch.rand((len(ids), 2), device="cuda"),
                                       torch.full((B,), 1.5, device="cuda"))
            cache.commit(c, dcu, acc)
        acc = acc.cpu().numpy()
        for r in range(B):
            path = list(range(acc[r] + 1))
            if tree:
                path, at = [], int(last[r])
                while at >= 0:
                    path.append(at)
                    at = int(parents[r][at])
                path.reverse()
                assert len(path) == acc[r] + 1
            for layer in range(L):
                for i in path:
                    history[r][layer].append((rows[layer, 0, cu[r] + i, :H].double().cpu().numpy(),
                                              rows[layer, 1, cu[r] + i, :H].double().cpu().numpy()))
        tokens = toks.cpu().numpy()[cu[:-1] + acc]
        cache.release(c)
        assert cache.last_error(c) == (0, 0, -1)
        assert c.lens.cpu().tolist()[:B] == [len(x[0]) for x in history]
        assert c.held.cpu().tolist()[:B] == [-(-len(x[0]) // P) for x in history]


@pytest.mark.parametrize("dtype,group,dim,tree,n,ctx", [
    ("bf16", 4, 128, False, [9, 5, 1, 2], [300, 125, 64, 0]), ("f16", 4, 64, True, [60, 128, 20, 2], [100, 0, 127, 1]),
    ("bf16", 4, 128, False, [700, 3, 64], [0, 20000, 1000]), ("bf16", 1, 128, True, [33], [9000]),
    ("f16", 3, 80, False, [130, 400], [77, 5]), ("f16", 7, 40, True, [64, 128], [4000, 3])])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(dtype, group, dim, tree, n, ctx):
    """A draft's value of inf or NaN leaves the rows that do not see it as they are with a zero there, bit for
    bit; the others become its sum with theirs.  A key of NaN makes the rows that see it NaN, and no others."""
    import torch
    c = Case(n, ctx, group=group, dim=dim, dtype=dtype, tree=tree, seed=dim + group)
    rng = np.random.default_rng(len(n) + dim)
    spoilt = []  # request, new token, kv head, element, value
    for r, m in enumerate(n):
        for x in (np.inf, -np.inf, np.nan, np.inf, np.inf):
            spoilt.append((r, int(rng.integers(min(1, m - 1), m)), int(rng.integers(2)), int(rng.integers(dim)), x))

    def place(r, j):
        t = ctx[r] + j
        return int(c.table[r, t // c.page]), t % c.page

    def write(which, values):
        for r, j, h, e, x in values:
            page, row = place(r, j)
            c.kv[which][page, row, h, e] = x
        (c.c.k, c.c.v)[which][0].copy_(c.kv[which])

    write(1, [s[:4] + (0.0,) for s in spoilt])
    clean, clean_lse = c.run()
    c.check(clean, clean_lse)
    for s in spoilt:  # (one element may be named twice)
        write(1, [s])
    out, lse = c.run()
    want = clean.float().cpu().numpy()
    seen = [oracle_cache.visible(m, ctx[r], c.parents[r] if tree else None) for r, m in enumerate(n)]
    last = {s[:4]: s[4] for s in spoilt}
    for (r, j, h, e), x in last.items():
        rows = c.cu[r] + np.flatnonzero(seen[r][:, ctx[r] + j])
        with np.errstate(invalid="ignore"):
            want[rows, h * group:(h + 1) * group, e] += np.float32(x)
    np.testing.assert_array_equal(out.float().cpu().numpy(), want)
    assert torch.equal(lse, clean_lse)

    write(1, [s[:4] + (0.0,) for s in spoilt])
    write(0, spoilt[2::5])
    out, lse = c.run()
    want, want_lse = clean.float().cpu().numpy(), clean_lse.cpu().numpy()
    for r, j, h, _, _ in spoilt[2::5]:
        rows = c.cu[r] + np.flatnonzero(seen[r][:, ctx[r] + j])
        want[rows, h * group:(h + 1) * group] = np.nan
        want_lse[rows, h * group:(h + 1) * group] = np.nan
    np.testing.assert_array_equal(out.float().cpu().numpy(), want)
    np.testing.assert_array_equal(lse.cpu().numpy(), want_lse)
    assert cache.last_error(c.c) == (0, 0, -1)


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64), ("bf16", 40)])
@pytest.mark.parametrize("n,group", [(70, 1), (9, 4), (33, 4), (1, 1), (250, 1)])
def test_row_blocks_cut_into_more_parts_than_a_warp_has_lanes(dtype, dim, n, group):
    """One row block over 120 tiles, behind another request's (its first part lies within a share)."""
    c = Case([1, n], [300, 15000], heads=1, group=group, dim=dim, page=64, dtype=dtype, seed=n + dim, poison=False)
    c.check(*c.run())
