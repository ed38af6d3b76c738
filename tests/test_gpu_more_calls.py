"""Rotated append, windowed and shared attention where sizes are large, and calls at the same time."""
import threading

import numpy as np
import pytest

from oracle import cache as oracle_cache
from speculative_decoding_rejection_spec_gb300 import cache
from test_gpu_attention import Case, built, dev  # noqa: F401 (built: the module's fixture)
from test_gpu_shared import Grouped
from test_gpu_window import Windowed

pytestmark = pytest.mark.gpu


def test_offsets_past_32_bits():
    """The same steps in a cache of few pages and in the last pages of one of 5 GB of keys: bit for bit alike."""
    import torch
    heads, dim, page = 8, 128, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    caches = [cache.make_cache(2, pages, page, heads, dim, 4, 16) for pages in (48, 20000)]
    assert caches[1].k.numel() * 2 > 2 ** 32
    table = cache.rotation_table(1024, 96)

    def step(n, parent=None, plan=None):
        cu, N = dev(np.concatenate([[0], np.cumsum(n)])), sum(n)
        rows = [[torch.randn((N, h, dim), generator=gen, device="cuda").bfloat16() for h in (heads, heads, 2 * heads)]
                for _ in range(2)]
        outs = []
        for c in caches:
            cache.reserve(c, cu)
            for layer, (k, v, q) in enumerate(rows):
                q = cache.append_rotated(c, layer, q, k, v, cu, table, parent=parent)
                outs += [q, cache.attention(c, layer, q, cu, parent=parent, window=150, sinks=5),
                         cache.attention(c, layer, q, cu, parent=parent, shared=cache.share(c, min_tokens=64))]
            assert cache.last_error(c) == (0, 0, -1)
        half = len(outs) // 2
        assert all(x.isfinite().all() for x in outs)
        assert all(torch.equal(a, b) for a, b in zip(outs[:half], outs[half:]))
        return cu

    cu = step([300, 129, 65, 0])
    for c in caches:
        cache.commit(c, cu, dev([299, 128, 64, -1]))
        cache.release(c)
        cache.fork(c, dev([0]), dev([3]))
        assert cache.share(c, min_tokens=64)[3].tolist() == [3, 4, 0, 0]  # its neighbour is another
    step([6] * 4, dev([-1, 0, 0, 1, 2, 4] * 4))
    for c in caches:
        cache.release(c, dev([300, 0, 65, 300]))
        cache.fork(c, dev([0]), dev([1]))
        assert cache.share(c, min_tokens=64)[:2].tolist() == [[0, 2, 256, 0]] * 2
    step([3] * 4)


def test_batches_of_many_turns():
    """More requests than one look at the batch keeps, with and without groups."""
    rng = np.random.default_rng(4)
    B = 1300
    n = rng.integers(0, 3, B)
    ctx = rng.integers(0, 80, B)
    groups = [(a, a + 4, int(rng.integers(0, 12))) for a in range(0, B, 5)]
    c = Grouped(groups, n, ctx, heads=1, group=4, dim=64, page=16, dtype="f16", seed=1, poison=False)
    c.check(*c.run())
    c = Windowed(n, ctx + 60, 50, 3, heads=2, group=2, dim=64, page=16, seed=2, hide=False, poison=False)
    c.check(*c.run())


def test_one_long_prefix_under_many_requests():
    """Row blocks of the group cut over all blocks, and requests of no token of their own beside the step's."""
    c = Grouped([(0, 40, 500)], [1, 2] * 20, [0] * 40, heads=1, group=8, page=16, seed=3, poison=False)
    c.check(*c.run())


@pytest.mark.parametrize("kind", ["window", "shared"])
def test_host_threads_of_one_stream(kind):
    import torch
    n, ctx = [9] * 12, np.random.default_rng(0).integers(0, 1500, 12)
    if kind == "window":
        c, kw = Windowed(n, ctx, 300, 4, page=32, seed=1, hide=False, poison=False), dict(window=300, sinks=4)
    else:
        c = Grouped([(0, 8, 40)], n, ctx, page=32, seed=1, poison=False)
        kw = dict(shared=dev(c.plan))
    q, cu = c.q.cuda(), dev(c.cu)
    want = cache.attention(c.c, 0, q, cu, **kw)
    plain = cache.attention(c.c, 0, q, cu)
    results, others = [], []

    def work():
        torch.cuda.set_device(0)
        for _ in range(15):
            results.append(cache.attention(c.c, 0, q, cu, **kw))
            others.append(cache.attention(c.c, 0, q, cu))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert len(results) == 60 and all(torch.equal(x, want) for x in results)
    assert all(torch.equal(x, plain) for x in others)
    assert len(c.c.workspaces) == 1 and cache.last_error(c.c) == (0, 0, -1)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scores_that_grow_along_the_context(dtype):
    """Maxima that move in every tile, over a window and over a prefix (test_gpu_attention has them over a whole
    context): the two parts of a row are far apart in size."""
    import torch
    for make in (lambda: Windowed([3], [1500], 700, 9, heads=2, group=2, page=64, seed=1, dtype=dtype, hide=False, poison=False),
                 lambda: Grouped([(0, 2, 12)], [3, 5], [700, 0], heads=2, group=2, page=64, seed=1, dtype=dtype, poison=False)):
        c = make()
        base = torch.randn(128, generator=torch.Generator().manual_seed(4))
        for r in range(len(c.n)):
            L = c.ctx[r] + c.n[r]
            grow = torch.linspace(0, 3, -(-L // 64) * 64).view(-1, 64)
            for i in range(len(grow)):
                c.kv[0][int(c.table[r, i])] = (grow[i][:, None, None] * base).expand(64, 2, 128).to(c.kv.dtype)
        c.q[:, :] = (2 * base).to(c.q.dtype)
        c.c.k[0].copy_(c.kv[0].cuda())
        c.check(*c.run())


def test_small_weights_of_a_long_prefix_count():
    """One key of a request's own takes nearly all of the weight, each of 16384 shared ones e^-14 of it, 1.4% together:
    their sum comes out of another row block than the large weight.  The bound is test_gpu_attention_weights' (two parts,
    joined in fp32)."""
    import torch
    L, score = 16384, -14.0
    for dtype, u in (("bf16", 2.0 ** -8), ("f16", 2.0 ** -11)):
        c = Grouped([(0, 3, L // 64)], [1, 1, 1], [64, 64, 64], heads=1, group=1, dim=64, page=64, dtype=dtype, seed=2,
                    poison=False)
        c.kv.zero_()
        c.kv[0][..., 0] = -2000.0  # a request's own keys count for nothing
        for i in range(L // 64):
            c.kv[0][int(c.table[0, i]), :, 0, 0] = score
            c.kv[1][int(c.table[0, i])] = 1.0
        for r in range(3):
            c.kv[0][int(c.table[r, L // 64]), 5, 0, 0] = 0.0
        c.c.k[0].copy_(c.kv[0].cuda())
        c.c.v[0].copy_(c.kv[1].cuda())
        c.q.zero_()
        c.q[:, :, 0] = 1.0
        out, lse = c.run(scale=1.0)
        assert cache.last_error(c.c) == (0, 0, -1)
        p = L * np.exp(score)
        want = p / (1 + p)
        es = (64 + 8) * 2.0 ** -23 * -score
        tol = want * (2 * u + 2 * es + 2 * L * 2.0 ** -23 + 2.0 ** -20) + (L * 2.0 ** -32 if dtype == "f16" else 0)
        assert np.abs(out.double().cpu().numpy() - want).max() <= tol
        assert np.abs(lse.double().cpu().numpy() - np.log1p(p)).max() <= es + L * 2.0 ** -23 + 2.0 ** -20


@pytest.mark.parametrize("dim", [64, 80, 128])
@pytest.mark.parametrize("n,ctx", [([5, 1, 2], [200, 4, 60]), ([150, 40, 3], [100, 0, 500])])
def test_outputs_between_two_sectors(dim, n, ctx):
    """Outputs whose rows are 16-byte aligned and no more, whose tokens or heads are an odd number of 16 bytes apart, and
    what lies between them: written as others are, and not beside."""
    import torch
    plain = Case(n, ctx, heads=2, group=3, dim=dim, seed=2)
    window = Windowed(n, ctx, 90, 5, heads=2, group=3, dim=dim, seed=2)
    shared = Grouped([(0, 2, 6)], n, ctx, heads=2, group=3, dim=dim, seed=2)
    N, H, D = plain.q.shape
    for c in (plain, window, shared):
        want, want_lse = c.run()
        c.check(want, want_lse)
        for token, head, start in ((H * D, D, 8), (H * D + 8, D, 0), (H * (D + 8), D + 8, 0), (H * (D + 8) + 16, D + 8, 8)):
            memory = torch.full((start + N * token + 64,), 7.0, dtype=c.q.dtype, device="cuda")
            out = memory[start:].as_strided((N, H, D), (token, head, 1))
            out, lse = c.run(out=out)
            assert torch.equal(out, want) and torch.equal(lse, want_lse)
            out.fill_(7.0)
            assert (memory == 7).all()
