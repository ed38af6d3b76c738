"""GPU append with the rotation where a warp has more than one pass over a token's heads: from some 1200 tokens on a
token has two warps, from some 2400 on one; and few tokens of many heads.  The bound is test_gpu_rotate's."""
import numpy as np
import pytest

from test_gpu_attention import built  # noqa: F401 (the module's fixture)
from test_gpu_rotate import Rows

pytestmark = pytest.mark.gpu

MANY = [1500, 1, 0, 700, 600]  # 2801 tokens and padding: a warp each
SOME = [900, 1, 0, 410, 200]   # 1511: two


@pytest.mark.parametrize("n", [MANY, SOME])
@pytest.mark.parametrize("heads,group,dim,turn,interleaved,dtype", [
    (8, 4, 128, 128, False, "bf16"), (8, 4, 128, 64, True, "f16"), (5, 3, 80, 32, False, "f16"),
    (5, 2, 256, 256, True, "bf16"), (6, 2, 256, 128, False, "bf16"), (9, 1, 48, 16, False, "bf16"),
    (4, 7, 64, 64, True, "bf16")])
def test_chunks(n, heads, group, dim, turn, interleaved, dtype):
    r = Rows(n, [10, 2000, 3, 500, 0], heads=heads, group=group, dim=dim, turn=turn, interleaved=interleaved, dtype=dtype,
             page=24, pad=9, seed=dim)
    r.check(r.run())


@pytest.mark.parametrize("batch", [24, 50])
@pytest.mark.parametrize("interleaved", [False, True])
def test_trees(batch, interleaved):
    rng = np.random.default_rng(batch)
    n = rng.integers(1, 129, batch)
    r = Rows(n, rng.integers(0, 300, batch), heads=7, group=4, dim=128, turn=96, tree=True, interleaved=interleaved, pad=5,
             seed=batch)
    r.check(r.run())


def test_in_place():
    """Queries turned where they are, as views of one projection."""
    r = Rows(MANY, [10, 2000, 3, 500, 0], heads=4, group=5, dim=128, fused=True, pad=3, seed=2)
    r.q[sum(MANY):] = 7
    r.check(r.run(out=r.q))


@pytest.mark.parametrize("heads,group,dim,turn,interleaved", [
    (24, 1, 256, 256, True), (24, 2, 256, 64, False), (70, 1, 128, 128, False), (40, 3, 64, 64, True)])
@pytest.mark.parametrize("n", [[1], [1, 9, 0, 30], [200, 150]])
def test_few_tokens_of_many_heads(heads, group, dim, turn, interleaved, n):
    r = Rows(n, [20, 3, 7, 0][:len(n)], heads=heads, group=group, dim=dim, turn=turn, interleaved=interleaved, seed=heads)
    r.check(r.run())
