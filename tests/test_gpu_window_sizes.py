"""GPU attention over a window behind very long contexts (its pages stand in the table many times over): the work goes
by what the rows see, and so does what is refused.  The bound is test_gpu_attention's."""
import numpy as np
import pytest

from oracle import cache as oracle_cache
from speculative_decoding_rejection_spec_gb300 import cache
from test_gpu_attention import built, dev  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu

PAGE, COLUMNS, GROUP, DIM = 4096, 2 ** 17, 128, 64
END = PAGE * COLUMNS  # 2^29 positions


class Far:
    """A request whose n new tokens end at the last position of its pages, of which there are eight."""

    def __init__(self, n):
        import torch
        gen, rng = torch.Generator().manual_seed(n), np.random.default_rng(n)
        self.n, self.len = n, END - n
        self.kv = torch.randn((2, 8, PAGE, 1, DIM), generator=gen).bfloat16()
        self.table = rng.integers(0, 8, (1, COLUMNS)).astype(np.int32)
        at = self.kv.cuda()
        ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.c = cache.PagedCache(at[0][None], at[1][None], page_table=dev(self.table), lens=dev([self.len]),
                                  held=dev([COLUMNS]), ref_counts=ints(8), free_pages=ints(8), num_free=ints(1))
        self.q = (2 * torch.randn((n, GROUP, DIM), generator=gen)).bfloat16()

    def run(self, parent=None, **kw):
        import torch
        out = torch.full(self.q.shape, 7.0, dtype=self.q.dtype, device="cuda")
        cache.attention(self.c, 0, self.q.cuda(), dev([0, self.n]), parent=None if parent is None else dev(parent), out=out,
                        **kw)
        return out.double().cpu().numpy()


@pytest.mark.parametrize("tree", [False, True])
def test_a_window_at_the_end_of_a_long_context(tree):
    c, window, sinks = Far(66), 500, 10
    parent = [-1] + [i // 2 for i in range(65)] if tree else None
    out = c.run(parent, window=window, sinks=sinks)
    assert cache.last_error(c.c) == (0, 0, -1)
    # the sinks and the last 600 committed positions: no row sees one between them
    place = np.concatenate([np.arange(sinks), np.arange(c.len - 600, END)])
    seen = oracle_cache.visible_window(c.n, sinks + 600, window, sinks, parent)
    k, v = (c.kv[i][c.table[0, place // PAGE], place % PAGE, 0].double().numpy() for i in (0, 1))
    want, _, A, S = oracle_cache.attention(c.q.double().numpy(), k, v, seen, DIM ** -0.5)
    u, L = 2.0 ** -8, len(place)
    tol = u * np.abs(want) + A * (u + 2 * (DIM + 8) * 2.0 ** -23 * S + 2 * L * 2.0 ** -23 + 2.0 ** -20)[..., None]
    assert (np.abs(out - want) <= tol).all()


@pytest.mark.parametrize("n,kw", [(1100, {}), (300, dict(window=END))])
def test_work_past_counting_is_refused(n, kw):
    """550 row blocks over 2^22 tiles, 150 over as many of a window that holds all."""
    c = Far(n)
    assert (c.run(**kw) == 7).all()
    assert cache.last_error(c.c) == (5, cache.DEVERR_LENGTH, 0)
