"""Runs append or rotated append, compiled for the host, on memory that ends where the calls may read no further; a
read behind it ends this process.  reads.py LIBRARY ENTRY, with the sizes as JSON."""
import ctypes
import json
import mmap
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.dirname(os.path.abspath(__file__)))))
from oracle import cache as oracle_cache  # noqa: E402
from speculative_decoding_rejection_spec_gb300.cache import BF16, Rotation, SpecCache  # noqa: E402

libc = ctypes.CDLL(None, use_errno=True)
libc.mprotect.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
keep = []


def edge(a):
    """A copy of an array that ends with readable memory."""
    size = -(-max(a.nbytes, 1) // mmap.PAGESIZE) * mmap.PAGESIZE
    m = mmap.mmap(-1, size + mmap.PAGESIZE)
    start = ctypes.addressof(ctypes.c_char.from_buffer(m))
    assert libc.mprotect(start + size, mmap.PAGESIZE, 0) == 0
    b = np.frombuffer(m, a.dtype, a.size, size - a.nbytes).reshape(a.shape)
    b[...] = a
    keep.append(m)
    return b


def bf16(x):
    """float64 to bfloat16, as uint16: to the nearest, ties to even."""
    y = np.asarray(x, np.float32).view(np.uint32)
    return ((y + 0x7fff + (y >> 16 & 1)) >> 16).astype(np.uint16)


def number(x):
    return (x.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def main(library, entry, n, ctx, held, pad=0, heads=2, group=2, dim=64, turn=64, page=16, columns=4, tree=False,
         interleaved=False, seed=0, error=(0, 2 ** 31 - 1)):
    lib, rng = ctypes.CDLL(library), np.random.default_rng(seed)
    R, rows, N, H = len(n), sum(n), sum(n) + pad, heads * group
    used, table = 0, np.full((R, columns), 2 ** 30, np.int32)
    order = rng.permutation(sum(held) + 2).astype(np.int32)
    for r in range(R):
        table[r, :held[r]] = order[used:used + held[r]]
        used += held[r]
    cells = edge(table.reshape(-1)[:(R - 1) * columns + held[-1]])  # the last request's columns end the memory
    k, v = (edge(np.full((len(order), page, heads, dim), 0x7fc0, np.uint16)) for _ in range(2))
    x = bf16(rng.standard_normal((rows, H + 2 * heads, dim)))
    q, k_new, v_new = edge(x[:, :H]), edge(x[:, H:H + heads]), edge(x[:, H + heads:])  # rows of padding: none
    out = edge(np.full((rows, H, dim), 0x7fc0, np.uint16))
    cu = edge(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))
    lens, holds = edge(np.array(ctx, np.int32)), edge(np.array(held, np.int32))
    ones, word = edge(np.ones(len(order), np.int32)), edge(np.array([0, 2 ** 31 - 1], np.int32))
    scratch = edge(np.zeros(1 << 16, np.uint8))
    parents = [np.array([-1] * min(m, 1) + [int(rng.integers(max(0, i // 2 - 1), i)) for i in range(1, m)], np.int32)
               for m in n]
    parent = edge(np.concatenate(parents)) if tree else None
    angle = np.arange(max(c + m for c, m in zip(ctx, n)))[:, None] * 0.1 ** np.arange(turn // 2)
    turns = edge(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32))
    at = lambda a: None if a is None else a.ctypes.data  # noqa: E731
    c = SpecCache(k=at(k), v=at(v), dtype=BF16, num_layers=1, num_pages=len(order), page_size=page, num_kv_heads=heads,
                  head_dim=dim, layer_stride=0, page_stride=page * heads * dim, token_stride=heads * dim, head_stride=dim,
                  page_table=at(cells), table_stride=columns, num_requests=R, max_pages=columns, lens=at(lens),
                  held=at(holds), ref_counts=at(ones), free_pages=at(ones), num_free=at(ones), error=at(word),
                  scratch=at(scratch))
    i64, i32, ptr = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
    kv = [ptr(at(k_new)), i64(heads * dim), i64(dim), ptr(at(v_new)), i64(heads * dim), i64(dim)]
    if entry == "append":
        status = lib.spec_cache_append(ctypes.byref(c), 0, *kv, ptr(at(cu)), i32(R), i64(N), None)
    else:
        rotation = Rotation(table=at(turns), row_stride=turn, positions=len(turns), dim=turn, neighbours=int(interleaved))
        status = lib.spec_cache_append_rotated(
            ctypes.byref(c), 0, *kv, ptr(at(q)), i64(H * dim), i64(dim), i32(H), ptr(at(out)), i64(H * dim), i64(dim),
            ptr(at(cu)), i32(R), i64(N), ptr(at(parent)), ctypes.byref(rotation), None)
    assert status == 0 and word.tolist() == list(error), (status, word)
    # rows in their places, turned: a product, a fused product and sum, a rounding
    want_k, want_v, want_q = (np.full(a.shape, np.nan) for a in (k, v, out))
    for r, m in enumerate(n):
        new = oracle_cache.depths(parents[r]) if tree else np.arange(m)
        a = x[cu[r]:cu[r + 1]]
        y = number(a[:, :H + heads])
        if entry != "append":
            y = oracle_cache.rotate(y, turns.astype(np.float64), ctx[r] + new, interleaved)
        for i in range(m):
            column, token = divmod(ctx[r] + i, page)
            if column < held[r]:
                want_k[table[r, column], token] = y[i, H:]
                want_v[table[r, column], token] = number(a[i, H + heads:])
                want_q[cu[r] + i] = y[i, :H]
    for got, want, u in ((k, want_k, 2.0 ** -8), (v, want_v, 0.0), (out, want_q, 2.0 ** -8)):
        if got is out and entry == "append":
            continue
        got, there = number(got), np.isfinite(want)
        assert np.isnan(got[~there]).all()
        assert (np.abs(got[there] - want[there]) <= u * (np.abs(want[there]) + 2.0 ** -12)).all()


if __name__ == "__main__":
    main(sys.argv[1], sys.argv[2], **json.loads(sys.argv[3]))
