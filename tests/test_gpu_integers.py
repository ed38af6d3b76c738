"""Integers that do not fit 32 bits are refused, not taken for their low bits."""
import pytest

from speculative_decoding_rejection_spec_gb300 import binding, cache
from test_gpu_attention import Case, built, dev  # noqa: F401 (built: the module's fixture)
from test_gpu_rotate import Rows

pytestmark = pytest.mark.gpu
WRAPPED = [2 ** 32, -2 ** 32, 2 ** 33 + 1]


@pytest.mark.parametrize("layer", WRAPPED)
def test_layers(layer):
    import torch
    r = Rows([4], [30], layers=2, seed=6)
    cu = dev(r.cu)
    for call in (lambda: cache.append_rotated(r.c, layer, r.q, r.k_new, r.v_new, cu, r.rotation),
                 lambda: cache.append(r.c, layer, r.k_new, r.v_new, cu)):
        with pytest.raises(binding.SpecRejectError):
            call()
    r.check(torch.full(r.q.shape, 7.0, dtype=r.dt, device="cuda"), skip=(0,))
    c = Case([4], [30], layers=2)
    for kw in (dict(), dict(window=5), dict(shared=torch.zeros((1, 4), dtype=torch.int32, device="cuda"))):
        out = torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device="cuda")
        with pytest.raises(binding.SpecRejectError):
            cache.attention(c.c, layer, c.q.cuda(), dev(c.cu), out=out, **kw)
        assert (out == 7).all()


def test_requests_of_a_plan():
    c = Case([1, 1], [30, 20]).c
    for B in (2 ** 32, 2 ** 32 + 2, -2 ** 32 + 1, 3, -1):
        with pytest.raises(binding.SpecRejectError):
            cache.share(c, B=B)
    assert cache.share(c, B=1).tolist() == [[0, 1, 0, 0]]


def test_workspace_sizes():
    c = Case([1, 1], [30, 20]).c
    for heads, B in ((2 ** 32 + 8, 2), (8, 2 ** 32 + 2)):
        with pytest.raises(ValueError):
            cache.attention_workspace_size(c, heads, B, 4)
