"""Small softmax weights next to a large one, over contexts that no other block shares."""
import numpy as np
import pytest

from speculative_decoding_rejection_spec_gb300 import cache
from test_gpu_attention import Case, built, dev  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n", [1, 150])
def test_small_weights_of_a_long_context_count(dtype, n):
    """One key takes nearly all of the weight, each of 65535 others e^-16.266 = 1.448 * 2^-24 of it, 0.56% together.
    A weight is rounded once, by half a step u of its type; fp16 holds it as 2^7 or more times its ratio to the
    largest, 1.448 * 2^-17, which is below its smallest normal: half of 2^-24 there, 2^-32 of the largest."""
    import torch
    L, score = 65536, -1041 / 64  # exact in both types
    R = 400 if n == 1 else 8  # more rows than blocks: most are whole in one
    c = Case([n], [L - n], heads=1, group=1, dim=64, page=64, dtype=dtype, seed=2, poison=False)
    c.kv.zero_()
    c.kv[0][..., 0] = score
    c.kv[1][...] = 1.0
    first = int(c.table[0, 0])
    c.kv[0][first, 0, 0, 0] = 0.0
    c.kv[1][first, 0] = 0.0
    many = cache.PagedCache(c.kv[:1].cuda(), c.kv[1:].cuda(), page_table=dev(np.repeat(c.table, R, 0)),
                            lens=dev([L - n] * R), held=dev([L // 64] * R), ref_counts=c.c.ref_counts,
                            free_pages=c.c.free_pages, num_free=c.c.num_free)  # every request reads the same pages
    q = torch.zeros((R * n, 1, 64), dtype=c.q.dtype, device="cuda")
    q[:, :, 0] = 1.0
    lse = torch.zeros((R * n, 1), device="cuda")
    out = cache.attention(many, 0, q, dev(np.arange(R + 1) * n), scale=1.0, lse=lse).double().cpu().numpy()
    assert cache.last_error(many) == (0, 0, -1)
    p = np.exp(score)
    keys = np.tile(np.arange(L - n, L), R)  # others that each row sees
    want = (keys * p / (1 + keys * p))[:, None, None]
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    # scores, exponentials and sums in fp32 as in test_gpu_attention
    es = (64 + 8) * 2.0 ** -23 * -score
    tol = want * (2 * u + 2 * es + 2 * L * 2.0 ** -23 + 2.0 ** -20) + (L * 2.0 ** -32 if dtype == "f16" else 0)
    assert (np.abs(out - want) <= tol).all(), (np.abs(out - want).max(), tol.min(), want.min())
    z = np.log1p(keys * p)[:, None]
    assert (np.abs(lse.double().cpu().numpy() - z) <= es + L * 2.0 ** -23 + 2.0 ** -20).all()


def shared(c, requests, **kw):
    """Attention of `requests` requests of the case's one, over the same pages: more rows than the device has
    blocks, so that most rows are whole in one."""
    import torch
    pages = int(c.c.held[0])
    many = cache.PagedCache(c.kv[:1].cuda(), c.kv[1:].cuda(), page_table=dev(np.repeat(c.table, requests, 0)),
                            lens=dev(c.ctx * requests), held=dev([pages] * requests), ref_counts=c.c.ref_counts,
                            free_pages=c.c.free_pages, num_free=c.c.num_free)
    n = c.n[0]
    q = c.q.cuda().repeat(requests, 1, 1)
    lse = torch.zeros(q.shape[:2], device="cuda")
    out = cache.attention(many, 0, q, dev(np.arange(requests + 1) * n), lse=lse, **kw)
    assert cache.last_error(many) == (0, 0, -1)
    return out, lse


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("base", [1024, 1536, 2560, 4096, 5120, 7168, 12288])
@pytest.mark.parametrize("step", [1, 2, 4, 8])
def test_scores_whose_steps_are_whole_exponents(dtype, base, step):
    """Scores of 2^23 to 2^27, whose steps in fp32 are 1 to 8: sums, differences and the limits that they are held
    against round to those, and no weight may leave its type's range.  Outputs are averages of the values."""
    import torch
    L = 4096
    c = Case([1], [L - 1], heads=1, group=4, dim=64, page=64, dtype=dtype, seed=3, poison=False)
    rows = torch.zeros((L // 64, 64, 64))
    rows[..., 0] = float(base)
    rows[..., 1] = (torch.arange(L) // 128 * step).float().view(L // 64, 64)  # every tile's maximum rises a little
    pages = torch.from_numpy(c.table[0, :L // 64].astype(np.int64))
    c.kv.zero_()
    c.kv[0][pages, :, 0] = rows.to(c.kv.dtype)
    c.kv[1][...] = 1 + torch.rand(c.kv[1].shape, generator=torch.Generator().manual_seed(base)).to(c.kv.dtype)
    c.q.zero_()
    c.q[:, :, 0] = 8192.0
    c.q[:, :, 1] = torch.arange(4) + 1.0
    out, lse = shared(c, 400, scale=1.0)
    # a weight and its rounded one differ by half a step u, so do the output and its rounded one; sums in fp32
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    off = 2 * u + 2 * L * 2.0 ** -23
    out = out.double().cpu().numpy()
    assert (out >= 1 - 2 * off).all() and (out <= 2 + 4 * off).all(), (out.min(), out.max())
    assert lse.isfinite().all()


@pytest.mark.parametrize("dtype,q,k", [("f16", 8192, 14000), ("f16", 8192, 20000), ("f16", -8192, 18000),
                                       ("f16", 4096, 43000), ("bf16", 2 ** 12, 3 * 2 ** 15), ("bf16", 2 ** 14, 5 * 2 ** 14),
                                       ("bf16", -2 ** 14, 5 * 2 ** 13)])
def test_scores_whose_steps_are_many_exponents(dtype, q, k):
    """Scores up to the largest that the header names, 2^28 (fp16) and 2^31 (bf16) over log2 e: their steps are 16
    and 128 exponents.  Keys of one score share the weight, whatever it is."""
    import torch
    L = 1536
    c = Case([1], [L - 1], heads=1, group=4, dim=64, page=64, dtype=dtype, seed=3, poison=False)
    scale = torch.ones(L)
    scale[L // 3:2 * L // 3] = 0.75 if q > 0 else 1.25  # the lower scores, behind the first: weights of zero
    pages = torch.from_numpy(c.table[0, :L // 64].astype(np.int64))
    c.kv.zero_()
    c.kv[0][pages, :, 0, 0] = (k * scale).view(L // 64, 64).to(c.kv.dtype)
    v = torch.randn((L, 64), generator=torch.Generator().manual_seed(7)).to(c.kv.dtype)
    c.kv[1][pages, :, 0] = v.view(L // 64, 64, 64)
    c.q.zero_()
    c.q[:, :, 0] = float(q)
    out, lse = shared(c, 400, scale=1.0)
    top = v[scale == 1].double()
    want, mass = top.mean(0).numpy(), top.abs().mean(0).numpy()
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    tol = u * np.abs(want) + mass * (u + 2 * L * 2.0 ** -23 + 2.0 ** -20)
    out = out.double().cpu().numpy()
    assert (np.abs(out - want) <= tol).all(), np.abs(out - want).max()
    score = float(c.q[0, 0, 0]) * float((k * scale[:1]).to(c.kv.dtype)[0])
    assert (np.abs(lse.double().cpu().numpy() - score) <= 2.0 ** -21 * abs(score)).all()
