"""How the cache's calls treat streams, host threads, captures and the memory that they allocate."""
import threading
import types

import numpy as np
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


def small_cache(stream=None, pages=256):
    return cache.make_cache(2, pages, 16, 8, 128, 4, 16, stream=stream)


def test_a_cache_made_on_a_stream_is_ready_there():
    """The current stream is busy; the cache's own goes on at once."""
    import torch
    s = torch.cuda.Stream()
    rows = torch.randn((50, 8, 128), device="cuda").bfloat16()
    cu = dev([0, 20, 50, 50, 50])
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    c = small_cache(s)
    cache.reserve(c, cu, stream=s)
    cache.append(c, 1, rows, -rows, cu, stream=s)
    assert cache.last_error(c, stream=s) == (0, 0, -1)
    torch.cuda.synchronize()
    assert cache.last_error(c) == (0, 0, -1)
    table = c.page_table.tolist()
    for r, (a, b) in enumerate(((0, 20), (20, 50))):
        for t in range(b - a):
            at = table[r][t // 16], t % 16
            assert torch.equal(c.k[1][at], rows[a + t]) and torch.equal(c.v[1][at], -rows[a + t])
    assert not c.k[0].any() and not c.v[0].any()
    assert c.held.tolist() == [2, 2, 0, 0] and c.num_free.tolist() == [252]


def test_a_cache_made_on_a_stream_is_that_stream_s_memory():
    """A cache that is dropped while its stream still writes to it does not go to the current stream."""
    import torch
    s = torch.cuda.Stream()
    rows = torch.ones((50, 8, 128), device="cuda").bfloat16()
    cu = dev([0, 20, 50, 50, 50])
    torch.cuda.synchronize()
    c = small_cache(s)
    size = 2 * c.k.numel()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    cache.reserve(c, cu, stream=s)
    cache.append(c, 1, rows, rows, cu, stream=s)
    del c
    mine = torch.full((size,), 2.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    assert (mine == 2).all()


def test_host_threads_of_one_stream_share_its_workspace():
    """Threads that come and go leave nothing behind, and calls of several at once are right."""
    import torch
    c = Case([9] * 12, np.random.default_rng(0).integers(0, 3000, 12), page=32, seed=1, poison=False)
    q, cu = c.q.cuda(), dev(c.cu)
    want = cache.attention(c.c, 0, q, cu)
    results, threads = [], []

    def work():
        torch.cuda.set_device(0)
        results.extend([cache.attention(c.c, 0, q, cu) for _ in range(20)])

    for _ in range(2):
        threads = [threading.Thread(target=work) for _ in range(5)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    torch.cuda.synchronize()
    assert len(results) == 200 and all(torch.equal(x, want) for x in results)
    assert len(c.c.workspaces) == 1


def test_workspaces_of_few_streams_are_kept():
    import torch
    c = Case([9] * 12, np.random.default_rng(0).integers(0, 3000, 12), page=32, seed=1, poison=False)
    q, cu = c.q.cuda(), dev(c.cu)
    want = cache.attention(c.c, 0, q, cu)
    streams = [torch.cuda.Stream() for _ in range(20)]
    torch.cuda.synchronize()
    results = [cache.attention(c.c, 0, q, cu, stream=s) for s in streams * 3]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in results)
    assert 0 < len(c.c.workspaces) <= cache.KEPT_WORKSPACES


def test_a_capture_on_the_given_stream_has_a_workspace_of_its_own():
    """Only ``stream=`` is capturing, not the current stream: the graph does not touch the kept workspace."""
    import torch
    c = Case([9, 3], [5000, 700], page=32, seed=1, poison=False)
    q, cu, s = c.q.cuda(), dev(c.cu), torch.cuda.Stream()
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    want = cache.attention(c.c, 0, q, cu, stream=s)
    torch.cuda.synchronize()
    kept = [w[-1] for w in c.c.workspaces.values()]
    assert kept and all(w.any() for w in kept)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        graph.capture_begin(capture_error_mode="relaxed")
    cache.attention(c.c, 0, q, cu, out=out, stream=s)
    with torch.cuda.stream(s):
        graph.capture_end()
    for w in kept:
        w.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert not any(w.any() for w in kept)


def test_streams_of_other_devices_are_refused():
    c = Case([9, 3], [50, 7], seed=1)
    cu = dev(c.cu)
    other = types.SimpleNamespace(cuda_stream=0, device_index=1)
    with pytest.raises(ValueError):
        cache.attention(c.c, 0, c.q.cuda(), cu, stream=other)
    with pytest.raises(ValueError):
        cache.reserve(c.c, cu, stream=other)
    with pytest.raises(ValueError):
        cache.last_error(c.c, stream=other)
    with pytest.raises(ValueError):
        small_cache(other)
    c.check(*c.run())


def test_the_current_stream_stays_current():
    """Behind a call on another stream, behind a refused one too."""
    import torch
    c = Case([9, 3], [50, 7], seed=1)
    q, cu, s, mine = c.q.cuda(), dev(c.cu), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(mine):
        cache.attention(c.c, 0, q, cu, stream=s)
        assert torch.cuda.current_stream() == mine
        with pytest.raises(TypeError):
            cache.attention(c.c, 0, q.half(), cu, stream=s)
        assert torch.cuda.current_stream() == mine
    torch.cuda.synchronize()


def test_a_captured_call_on_the_given_stream_makes_its_output_there():
    """The output of a call that only ``stream=`` captures lies in the graph's memory and follows the replays."""
    import torch
    c = Case([9, 3], [5000, 700], page=32, seed=1, poison=False)
    q, cu, s = c.q.cuda(), dev(c.cu), torch.cuda.Stream()
    want = cache.attention(c.c, 0, q, cu)
    half = cache.attention(c.c, 0, q * 0.5, cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        graph.capture_begin(capture_error_mode="relaxed")
    out = cache.attention(c.c, 0, q, cu, stream=s)
    with torch.cuda.stream(s):
        graph.capture_end()
    keep = [torch.zeros_like(out) for _ in range(4)]  # what the current stream hands out is other memory
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and not any(x.any() for x in keep)
    q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, half)
