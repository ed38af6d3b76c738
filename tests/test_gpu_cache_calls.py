"""How the cache's calls treat streams, host threads, captures and the memory that they allocate."""
import pytest

from speculative_decoding_rejection_spec_gb300 import cache
from test_gpu_attention import Case, built, dev  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu

BUSY = 200_000_000  # cycles, about a tenth of a second


def test_an_output_made_for_another_stream_is_that_stream_s_memory():
    """Work queued on the current stream still reads a tensor that was freed there when the call on another
    stream makes its output: the output is other memory."""
    import torch
    c = Case([40, 90, 33], [300, 20, 500], seed=6)
    q, cu, s = c.q.cuda(), dev(c.cu), torch.cuda.Stream()
    want = cache.attention(c.c, 0, q, cu)
    torch.cuda.synchronize()
    first = cache.attention(c.c, 0, q, cu, stream=s)
    freed = torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda")
    copy = torch.zeros_like(freed)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    copy.copy_(freed)
    del freed
    got = cache.attention(c.c, 0, q, cu, stream=s)
    torch.cuda.synchronize()
    assert (copy == 3).all()
    assert torch.equal(first, want) and torch.equal(got, want)


def test_an_output_made_for_another_stream_lives_until_the_current_one_has_read_it():
    import torch
    c = Case([40, 90, 33], [300, 20, 500], seed=6)
    q, cu, s = c.q.cuda(), dev(c.cu), torch.cuda.Stream()
    want = cache.attention(c.c, 0, q, cu)
    copy, half = torch.zeros_like(want), q * 0.5
    torch.cuda.synchronize()
    got = cache.attention(c.c, 0, q, cu, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(BUSY)
    copy.copy_(got)
    del got
    other = cache.attention(c.c, 0, half, cu, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and not torch.equal(other, want)
