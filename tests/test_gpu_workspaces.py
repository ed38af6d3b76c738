"""Workspaces that a cache keeps for attention: enough for every later call on their stream, whatever came first."""
import itertools

import pytest

from speculative_decoding_rejection_spec_gb300 import binding, cache
from test_gpu_attention import built, dev  # noqa: F401 (built: the module's fixture)
from test_gpu_shared import Grouped

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("order", list(itertools.permutations(["plain 0", "plain 1", "window 1", "shared 0", "shared 1"], 4)))
def test_calls_of_few_rows_in_any_order(order):
    """One query row per kv head: the smallest workspace of a plain call is smaller than that of an empty shared one."""
    import torch
    c = cache.make_cache(1, 8, 16, 8, 128, 4, 2)
    plan = cache.share(c)
    for what in order:
        kind, n = what.split()
        n = int(n)
        cu = dev([0] + [n] * 4)
        cache.reserve(c, cu)
        q = torch.ones((n, 8, 128), dtype=torch.bfloat16, device="cuda")
        kw = dict(plain={}, window=dict(window=3), shared=dict(shared=plan))[kind]
        out = cache.attention(c, 0, q, cu, **kw)
        assert out.shape == (n, 8, 128) and (out == 0).all()
    assert cache.last_error(c) == (0, 0, -1)


def test_a_shared_call_of_no_request():
    import torch
    c = cache.make_cache(1, 8, 16, 8, 128, 4, 2)
    none, cu = torch.zeros((0, 8, 128), dtype=torch.bfloat16, device="cuda"), dev([0])
    cache.attention(c, 0, none, cu)
    cache.attention(c, 0, none, cu, shared=cache.share(c, B=0))


def test_sizes_of_workspaces_that_are_given():
    """A user's own workspace, of the size asked for: enough for its kind of call, and one byte less is not."""
    import torch
    c = Grouped([(0, 3, 11)], [4, 9, 1], [300, 20, 500], seed=6)
    for shared, kw in ((True, {}), (False, dict(shared=None)), (False, dict(shared=None, window=10 ** 6))):
        size = cache.attention_workspace_size(c.c, 8, 3, 14, shared=shared)
        c.check(*c.run(workspace=torch.full((size,), 255, dtype=torch.uint8, device="cuda"), **kw))
        with pytest.raises(binding.SpecRejectError):
            c.run(workspace=torch.zeros(size - 1, dtype=torch.uint8, device="cuda"), **kw)
    with pytest.raises(ValueError):
        cache.attention_workspace_size(c.c, 9, 3, 14, shared=True)
    assert cache.attention_workspace_size(cache.make_cache(1, 2, 16, 8, 128, 1, 2), 32, 1, 16384, shared=True) < 600e6
