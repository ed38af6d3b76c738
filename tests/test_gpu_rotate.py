"""GPU append with the rotation of positions against the 64-bit oracle.

Bound per turned element, u = eps / 2 of the type: a product, a fused product and sum in fp32, rounded to 16 bits once:
  |y - exact| <= u |y| + 2^-23 (|a c| + |b s|), and half of the smallest fp16, 2^-25, where numbers lose bits.
What does not turn, and the values, are copies."""
import numpy as np
import pytest

from oracle import cache as oracle_cache
from speculative_decoding_rejection_spec_gb300 import binding, cache
from test_gpu_attention import built, dev  # noqa: F401 (built: the module's fixture)
from test_gpu_cache_calls import BUSY

pytestmark = pytest.mark.gpu

DT = dict(bf16="bfloat16", f16="float16")


class Rows:
    """A cache whose pages hold each request's committed and new tokens, and a step's rows."""

    def __init__(self, n, ctx, heads=2, group=4, dim=128, turn=None, page=16, dtype="bf16", tree=False, interleaved=False,
                 layers=1, layer=0, positions=None, pad=0, seed=0, fused=False):
        import torch
        self.n, self.ctx, self.page, self.layer, self.pad, self.interleaved = list(n), list(ctx), page, layer, pad, interleaved
        self.dt = getattr(torch, DT[dtype])
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        need = [-(-(c + m) // page) for c, m in zip(ctx, n)]
        R, MP, NP = len(n), max(max(need), 1) + 1, sum(need) + 3
        order, used = rng.permutation(NP), 0
        self.table = np.full((R, MP), 2 ** 30, np.int32)
        ref = np.zeros(NP, np.int32)
        for r in range(R):
            self.table[r, :need[r]] = order[used:used + need[r]]
            ref[order[used:used + need[r]]] = 1
            used += need[r]
        self.k, self.v = (torch.randn((layers, NP, page, heads, dim), generator=gen).to(self.dt) for _ in range(2))
        ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.c = cache.PagedCache(self.k.cuda(), self.v.cuda(), page_table=dev(self.table), lens=dev(ctx),
                                  held=dev(need), ref_counts=dev(ref), free_pages=ints(NP), num_free=ints(1))
        N, H = sum(n) + pad, heads * group
        rows = torch.randn((N, H + 2 * heads, dim), generator=gen).to(self.dt)
        self.rows, self.heads = rows, (H, heads)
        at = rows.cuda()
        parts = (at[:, :H], at[:, H:H + heads], at[:, H + heads:])  # of one fused projection
        self.q, self.k_new, self.v_new = parts if fused else [x.contiguous() for x in parts]
        self.rotation = cache.rotation_table(positions or max(max(c + m for c, m in zip(ctx, n)), 1), turn or dim)
        self.cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.parents = None
        if tree:
            self.parents = [np.array([-1] * min(m, 1) + [int(rng.integers(max(0, i // 3 - 1), i)) for i in
                                                         range(1, m)], np.int32) for m in n]

    def run(self, **kw):
        import torch
        parent = None
        if self.parents is not None:
            parent = dev(np.concatenate(self.parents + [np.zeros(self.pad, np.int32)]))
        out = kw.pop("out", None)
        if out is None:
            out = torch.full(self.q.shape, 7.0, dtype=self.dt, device="cuda")
        return cache.append_rotated(self.c, self.layer, kw.pop("q", self.q), self.k_new, self.v_new, dev(self.cu),
                                    self.rotation, parent=parent, interleaved=self.interleaved, out=out, **kw)

    def check(self, out, error=(0, 0, -1), skip=()):
        import torch
        assert cache.last_error(self.c) == error
        H, h = self.heads
        u = 2.0 ** -8 if self.dt == torch.bfloat16 else 2.0 ** -11
        got_k, got_v = self.c.k.cpu(), self.c.v.cpu()
        k, v = self.k.clone(), self.v.clone()
        table = self.rotation.double().cpu().numpy()
        want_q = torch.full(self.q.shape, 7.0, dtype=torch.float64)
        turned, half = table.shape[1], table.shape[1] // 2
        for r, m in enumerate(self.n):
            if r in skip or m == 0:
                continue
            a, b = self.cu[r], self.cu[r + 1]
            new = np.arange(m) if self.parents is None else oracle_cache.depths(self.parents[r])
            x = self.rows[a:b, :H + h].double().numpy()
            y = oracle_cache.rotate(x, table, self.ctx[r] + new, self.interleaved)
            size = oracle_cache.rotate(np.abs(x), np.abs(table) * np.repeat([1, -1], half), self.ctx[r] + new,
                                       self.interleaved)  # |a c| + |b s| of the first of a pair
            other = oracle_cache.rotate(np.abs(x), np.abs(table), self.ctx[r] + new, self.interleaved)
            tol = u * np.abs(y) + 2.0 ** -23 * np.maximum(np.abs(size), np.abs(other)) + 2.0 ** -25
            tol[..., turned:] = 0
            place = [(int(self.table[r, (self.ctx[r] + i) // self.page]), (self.ctx[r] + i) % self.page)
                     for i in range(m)]
            p, i = (list(z) for z in zip(*place))
            mine = np.concatenate([out[a:b].double().cpu().numpy(), got_k[self.layer, p, i].double().numpy()], 1)
            assert (np.abs(mine - y) <= tol).all(), (r, np.abs(mine - y).max())
            k[self.layer, p, i] = got_k[self.layer, p, i]
            v[self.layer, p, i] = self.rows[a:b, H + h:]
            want_q[a:b] = out[a:b].double().cpu()
        assert torch.equal(got_k, k) and torch.equal(got_v, v)  # nothing else was written
        assert torch.equal(out.double().cpu(), want_q)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,turn", [(128, 128), (128, 64), (128, 16), (64, 64), (80, 80), (80, 32), (96, 96), (48, 16),
                                      (16, 16), (256, 256), (256, 32), (144, 112)])
def test_rotated_append(dtype, interleaved, dim, turn):
    r = Rows([1, 3, 0, 9, 40], [0, 15, 3, 200, 61], dim=dim, turn=turn, dtype=dtype, interleaved=interleaved, seed=dim)
    r.check(r.run())


@pytest.mark.parametrize("dim,turn", [(8, 8), (24, 8), (72, 24), (120, 120), (248, 40)])
def test_dimensions_of_neighbours_alone(dim, turn):
    r = Rows([1, 3, 7], [0, 15, 200], dim=dim, turn=turn, interleaved=True, seed=dim)
    r.check(r.run())


@pytest.mark.parametrize("heads,group", [(1, 1), (3, 1), (2, 3), (5, 7), (8, 4), (1, 71), (16, 1)])
def test_head_counts(heads, group):
    r = Rows([1, 4, 0, 3], [20, 12, 5, 0], heads=heads, group=group, dim=64, page=8, seed=group)
    r.check(r.run())


@pytest.mark.parametrize("interleaved", [False, True])
def test_trees_stand_at_their_depth(interleaved):
    n = [1, 31, 64, 65, 0, 128, 2, 100]
    r = Rows(n, [3, 0, 77, 500, 9, 16, 15, 31], heads=2, group=3, dim=64, tree=True, interleaved=interleaved, seed=3)
    r.check(r.run())
    deep = Rows([128, 5], [4, 0], dim=64, tree=True, seed=4)
    deep.parents[0] = np.arange(-1, 127, dtype=np.int32)  # a chain: as deep as a tree can be
    deep.check(deep.run())


def test_a_tree_that_is_a_chain_equals_the_chain():
    import torch
    a, b = (Rows([50, 7], [300, 100], dim=64, seed=5) for _ in range(2))
    b.parents = [np.arange(-1, 49, dtype=np.int32), np.arange(-1, 6, dtype=np.int32)]
    assert torch.equal(a.run(), b.run())
    assert torch.equal(a.c.k, b.c.k) and torch.equal(a.c.v, b.c.v)


def test_prompts_layers_and_padding():
    r = Rows([700, 1, 333], [10, 2000, 0], heads=4, group=2, dim=64, page=24, layers=3, layer=1, pad=9, seed=6)
    r.check(r.run())


def test_views_of_a_fused_projection_in_place():
    r = Rows([5, 1, 60], [200, 4, 60], heads=2, group=4, dim=128, fused=True, pad=3, seed=2)
    q = r.q
    before = q.clone()
    assert cache.append_rotated(r.c, 0, q, r.k_new, r.v_new, dev(r.cu), r.rotation, out=q) is q
    assert (q[66:] == before[66:]).all()
    q[66:] = 7
    r.check(q)


def test_a_table_with_longer_rows_and_a_table_of_one_row():
    import torch
    r = Rows([5, 1], [20, 4], dim=64, seed=2)
    wide = torch.full((25, 100), float("nan"), device="cuda")
    wide[:, :64] = r.rotation
    r.rotation = wide[:, :64]
    r.check(r.run())
    r = Rows([1, 1], [0, 0], dim=64, seed=2)
    assert r.rotation.shape[0] == 1
    r.check(r.run())


def test_keys_and_values_alone():
    import torch
    r = Rows([5, 1], [20, 4], seed=2)
    assert cache.append_rotated(r.c, 0, None, r.k_new, r.v_new, dev(r.cu), r.rotation) is None
    other = Rows([5, 1], [20, 4], seed=2)
    other.run()
    assert torch.equal(r.c.k, other.c.k) and torch.equal(r.c.v, other.c.v)


def test_far_positions():
    """Where the table's angles are large: position 99990 and on."""
    r = Rows([9], [99990], heads=1, group=1, dim=16, page=1000, seed=1)
    r.check(r.run())


def test_requests_with_errors_are_left_out():
    n, ctx = [3, 4, 5, 2], [10, 20, 30, 50]
    r = Rows(n, ctx, positions=52, seed=4)
    r.c.lens[1] = -1
    r.check(r.run(), error=(5, cache.DEVERR_LENGTH, 1), skip=(1,))
    r = Rows(n, ctx, positions=51, seed=4)  # the last request's end is not in the table
    r.check(r.run(), error=(5, cache.DEVERR_LENGTH, 3), skip=(3,))
    r = Rows(n, ctx, seed=4)
    r.c.ref_counts[int(r.table[2, 2])] = 2  # shared
    out = r.run()
    assert cache.last_error(r.c) == (5, cache.DEVERR_PAGE, 2)
    assert (out[9:12] == 7).all() and not (out[7:9] == 7).all(2).any()  # positions 30, 31 lie in column 1, 32 in 2
    r = Rows(n, ctx, seed=4)
    r.c.held[0] = 0
    r.check(r.run(), error=(5, cache.DEVERR_PAGE, 0), skip=(0,))
    for page in (-1, 10 ** 6):
        r = Rows(n, ctx, seed=4)
        r.c.page_table[3, 3] = page
        r.check(r.run(), error=(5, cache.DEVERR_PAGE, 3), skip=(3,))


@pytest.mark.parametrize("where,parent", [(0, 0), (1, 1), (1, -1), (5, 500), (8, 8)])
def test_malformed_trees_are_left_out(where, parent):
    r = Rows([9, 9, 4], [10, 20, 30], tree=True, seed=4)
    r.parents[1] = r.parents[1].copy()
    r.parents[1][where] = parent
    r.check(r.run(), error=(5, binding.DEVERR_TREE, 1), skip=(1,))


def test_a_tree_of_too_many_nodes():
    r = Rows([9, 129], [10, 20], tree=True, seed=4)
    r.check(r.run(), error=(5, binding.DEVERR_TREE, 1), skip=(1,))


def test_bad_layout_writes_nothing():
    r = Rows([3, 4], [100, 200], seed=4)
    for cu in ([1, 3, 7], [0, 5, 4], [0, 3, 8]):
        good, r.cu = r.cu, np.array(cu, np.int32)
        out = r.run()
        r.cu = good
        r.check(out, error=(5, binding.DEVERR_LAYOUT, -1), skip=(0, 1))


def test_empty_calls():
    import torch
    r = Rows([0, 0], [5, 0], pad=4, seed=0)
    r.check(r.run())
    none = torch.zeros((0, 8, 128), dtype=r.dt, device="cuda")
    kv = none[:, :2]
    assert cache.append_rotated(r.c, 0, none, kv, kv, dev([0]), r.rotation).shape == (0, 8, 128)


def test_captured_call_follows_the_device_data():
    import torch
    r = Rows([4, 9, 1], [30, 20, 50], positions=100, seed=6)
    cu, out = dev(r.cu), torch.full(r.q.shape, 7.0, dtype=r.dt, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append_rotated(r.c, 0, r.q, r.k_new, r.v_new, cu, r.rotation, out=out)
    for ctx in ([30, 20, 50], [33, 7, 63], [0, 0, 0]):
        r.ctx = ctx
        r.c.lens.copy_(dev(ctx))
        r.c.k.copy_(r.k)
        r.c.v.copy_(r.v)
        graph.replay()
        r.check(out)


def test_an_output_made_for_another_stream_is_that_stream_s_memory():
    import torch
    r = Rows([40, 90, 33], [300, 20, 500], seed=6)
    cu, s = dev(r.cu), torch.cuda.Stream()
    call = lambda **kw: cache.append_rotated(r.c, 0, r.q, r.k_new, r.v_new, cu, r.rotation, **kw)  # noqa: E731
    want = call()
    torch.cuda.synchronize()
    first = call(stream=s)
    freed = torch.full(r.q.shape, 3.0, dtype=r.dt, device="cuda")
    copy = torch.zeros_like(freed)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    copy.copy_(freed)
    del freed
    got = call(stream=s)
    torch.cuda.synchronize()
    assert (copy == 3).all() and torch.equal(first, want) and torch.equal(got, want)


def test_refusals():
    import types

    import torch
    r = Rows([4], [30], seed=6)
    cu = dev(r.cu)

    def call(q=r.q, k=r.k_new, v=r.v_new, rotation=r.rotation, layer=0, **kw):
        return cache.append_rotated(r.c, layer, q, k, v, cu, rotation, **kw)

    for kw in (dict(q=r.q.float()), dict(k=r.k_new.half()), dict(k=r.k_new[:, :1]), dict(v=r.v_new[:, :, :64]),
               dict(rotation=r.rotation.double()), dict(rotation=r.rotation[0]), dict(rotation=r.rotation.t()),
               dict(parent=dev([-1, 0])), dict(out=torch.zeros_like(r.q, dtype=torch.float32))):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(q=r.q[:2]), dict(v=r.v_new[:2]), dict(rotation=r.rotation.cpu()), dict(out=torch.zeros_like(r.q)[:2]),
               dict(q=None, out=r.q.clone()), dict(q=r.q.cpu()),
               dict(stream=types.SimpleNamespace(cuda_stream=0, device_index=1))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(layer=1), dict(rotation=r.rotation[:, :24]), dict(rotation=r.rotation[:, :0]),
               dict(rotation=torch.zeros((50, 136), device="cuda")), dict(rotation=r.rotation[:0])):
        with pytest.raises(binding.SpecRejectError):
            call(**kw)
    r.check(torch.full(r.q.shape, 7.0, dtype=r.dt, device="cuda"), skip=(0,))
