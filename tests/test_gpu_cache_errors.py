"""Requests with bad data: nothing of theirs is written, and the others are as if they were alone."""
import pytest

from speculative_decoding_rejection_spec_gb300 import binding
from test_gpu_attention import Case, built  # noqa: F401 (built: the module's fixture)

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
