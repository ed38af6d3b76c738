"""Rotated append, windowed and shared attention and the plan of shared prefixes without a GPU: the host's argument
checks, workspace sizes, and their oracles on hand-made cases."""
import ctypes
import os
import re

import numpy as np
import pytest

from oracle import cache as oracle_cache
from speculative_decoding_rejection_spec_gb300 import cache
from test_cache_cpu import BAD_STRUCTS, FAKE, ROOT, lib, struct  # noqa: F401 (lib: the fixture)

P, ODD = ctypes.c_void_p(FAKE), ctypes.c_void_p(FAKE + 8)


def rotation(**kw):
    f = dict(table=FAKE, row_stride=64, positions=100, dim=64, neighbours=0)
    f.update(kw)
    return cache.Rotation(**f)


def rotated(lib, s, layer=0, k=P, kt=128, kh=64, v=P, vt=128, vh=64, q=P, qt=256, qh=64, heads=4, out=P, ot=256, oh=64,
            cu=P, B=1, N=4, parent=None, turn=None):
    turn = rotation() if turn is None else turn
    return lib.spec_cache_append_rotated(ctypes.byref(s), layer, k, kt, kh, v, vt, vh, q, qt, qh, heads, out, ot, oh, cu,
                                         B, N, parent, None if turn == "none" else ctypes.byref(turn), None)


def window(lib, s, q=P, heads=4, cu=P, B=1, N=4, parent=None, scale=1.0, window=16, sinks=0, out=P, ws=P, size=1 << 40,
           layer=0):
    return lib.spec_attention_window(ctypes.byref(s), layer, q, 256, 64, heads, cu, B, N, parent, scale, window, sinks,
                                     out, 256, 64, None, ws, size, None)


def shared(lib, s, q=P, heads=4, cu=P, B=1, N=4, parent=None, scale=1.0, plan=P, out=P, ws=P, size=1 << 40, layer=0):
    return lib.spec_attention_shared(ctypes.byref(s), layer, q, 256, 64, heads, cu, B, N, parent, scale, plan, out, 256,
                                     64, None, ws, size, None)


@pytest.mark.parametrize("kw,status", BAD_STRUCTS)
def test_every_entry_checks_the_cache(lib, kw, status):  # noqa: F811
    s = struct(**kw)
    assert rotated(lib, s) == status
    assert window(lib, s) == status
    assert shared(lib, s) == status
    assert lib.spec_cache_share(ctypes.byref(s), 1, 16, P, None) == status
    assert lib.spec_attention_shared_workspace_size(ctypes.byref(s), 4, 1, 4) == 0


def test_rotated_append_argument_checks(lib):  # noqa: F811
    s = struct()
    for kw in (dict(layer=2), dict(layer=-1), dict(k=None), dict(v=None), dict(q=None), dict(out=None), dict(k=ODD),
               dict(v=ODD), dict(q=ODD), dict(out=ODD), dict(kt=0), dict(kt=100), dict(vh=4), dict(qt=-256),
               dict(qh=60), dict(ot=4), dict(oh=0), dict(cu=None), dict(cu=ctypes.c_void_p(FAKE + 2)), dict(B=4),
               dict(B=-1), dict(N=-1), dict(heads=-1), dict(parent=ctypes.c_void_p(FAKE + 2)), dict(turn="none")):
        assert rotated(lib, s, **kw) == 1, kw
    for kw in (dict(table=None), dict(table=FAKE + 8), dict(positions=0), dict(dim=0), dict(dim=66), dict(dim=33),
               dict(row_stride=60), dict(row_stride=66), dict(dim=-16)):
        assert rotated(lib, s, turn=rotation(**kw)) == 1, kw
    assert rotated(lib, s, turn=rotation(dim=24)) == 2
    assert rotated(lib, s, turn=rotation(dim=20, neighbours=1)) == 2
    assert rotated(lib, s, N=2 ** 31) == 2
    wide = dict(head_dim=264, token_stride=528, head_stride=264, page_stride=16 * 528, layer_stride=160 * 528)
    assert rotated(lib, struct(**wide), kt=528, kh=264, vt=528, vh=264, qt=1056, qh=264, ot=1056, oh=264) == 2


def test_window_argument_checks(lib):  # noqa: F811
    s = struct()
    for kw in (dict(window=0), dict(window=-1), dict(sinks=-1), dict(layer=2), dict(q=None), dict(out=None), dict(q=ODD),
               dict(cu=None), dict(B=4), dict(N=-1), dict(heads=3), dict(scale=0.0), dict(scale=float("nan")),
               dict(ws=None), dict(parent=ctypes.c_void_p(FAKE + 2))):
        assert window(lib, s, **kw) == 1, kw
    assert window(lib, s, size=16) == 3
    assert window(lib, struct(page_size=12, page_stride=12 * 128)) == 2
    assert window(lib, s, N=2 ** 29) == 2


def test_shared_argument_checks(lib):  # noqa: F811
    s = struct()
    for kw in (dict(plan=None), dict(plan=ODD), dict(layer=-1), dict(q=None), dict(out=ODD), dict(cu=None), dict(B=4),
               dict(N=-1), dict(heads=5), dict(scale=-1.0), dict(ws=None)):
        assert shared(lib, s, **kw) == 1, kw
    size = lib.spec_attention_shared_workspace_size(ctypes.byref(s), 4, 1, 4)
    plain = lib.spec_attention_workspace_size(ctypes.byref(s), 4, 1, 4)
    assert size > plain > 0
    assert shared(lib, s, size=size - 1) == 3 and shared(lib, s, size=plain) == 3
    # sums of every row twice: 64 elements, maximum and weight
    grown = lib.spec_attention_shared_workspace_size(ctypes.byref(s), 4, 3, 4004)
    assert grown - size >= 2 * 4000 * 4 * (64 * 4 + 8)


def test_share_argument_checks(lib):  # noqa: F811
    s = ctypes.byref(struct())
    for B, least, out in ((4, 16, P), (-1, 16, P), (1, -1, P), (1, 16, None), (1, 16, ODD)):
        assert lib.spec_cache_share(s, B, least, out, None) == 1


def test_constant_matches_the_header():
    src = open(os.path.join(ROOT, "include", "spec_cache.h")).read()
    assert int(re.search(r"#define SPEC_ROTATION_MAX_HEAD_DIM (\d+)", src).group(1)) == cache.ROTATION_MAX_HEAD_DIM


def test_integers_out_of_range_are_not_wrapped():
    assert cache._clamped(2 ** 32 + 5) == 2 ** 31 - 1 and cache._clamped(-2 ** 32) == -1 and cache._clamped(7) == 7


def test_rotation_table_by_hand():
    t = cache.rotation_table(5000, 8, base=100.0, device="cpu").double().numpy()
    assert t.shape == (5000, 8)
    for p in (0, 1, 4999):
        for i in range(4):
            a = p * 100.0 ** (-2 * i / 8)
            assert abs(t[p, i] - np.cos(a)) <= 2.0 ** -24 and abs(t[p, 4 + i] - np.sin(a)) <= 2.0 ** -24


def test_rotation_oracle_by_hand():
    """Quarter turns: (a, b) becomes (-b, a)."""
    table = np.array([[1, 1, 0, 0], [0, 0, 1, 1]])
    x = np.array([[[1.0, 2, 3, 4, 5, 6]]])
    np.testing.assert_array_equal(oracle_cache.rotate(x, table, [0], False), x)
    np.testing.assert_array_equal(oracle_cache.rotate(x, table, [1], False), [[[-3, -4, 1, 2, 5, 6]]])
    np.testing.assert_array_equal(oracle_cache.rotate(x, table, [1], True), [[[-2, 1, -4, 3, 5, 6]]])
    # what the rotation is for: scores depend on distances alone
    t = cache.rotation_table(60, 6, device="cpu").double().numpy()
    rng = np.random.default_rng(0)
    a, b = rng.standard_normal((2, 1, 1, 6))
    dots = [float((oracle_cache.rotate(a, t, [p + 9], False) * oracle_cache.rotate(b, t, [p], False)).sum())
            for p in (0, 20, 50)]
    assert np.allclose(dots, dots[0], atol=1e-6)


def test_window_oracle_by_hand():
    seen = oracle_cache.visible_window(2, 5, 3, 1)
    np.testing.assert_array_equal(seen.astype(int), [[1, 0, 0, 1, 1, 1, 0], [1, 0, 0, 0, 1, 1, 1]])
    # a root with two children and a grandchild of the second: depths 0 1 1 2
    seen = oracle_cache.visible_window(4, 3, 2, 0, [-1, 0, 0, 2])
    np.testing.assert_array_equal(seen.astype(int), [[0, 0, 1, 1, 0, 0, 0], [0, 0, 0, 1, 1, 0, 0],
                                                     [0, 0, 0, 1, 0, 1, 0], [0, 0, 0, 0, 0, 1, 1]])
    assert oracle_cache.visible_window(3, 9, 100, 0).sum() == 10 + 11 + 12
    assert oracle_cache.visible_window(3, 2, 1, 4)[:, :4].tolist() == [[True, True, True, False]] + [[True] * 4] * 2


def test_share_oracle_by_hand():
    table = [[5, 6, 7, 8], [5, 6, 9, 1], [5, 6, 9, 2], [4, 6, 9, 2], [4, 6, 9, 2]]
    plan, bad = oracle_cache.share_plan(table, [32, 30, 31, 32, 8], [4] * 5, 8, 8)
    assert bad == []
    assert plan.tolist() == [[0, 3, 16, 0]] * 3 + [[3, 5, 8, 0]] * 2
    plan, bad = oracle_cache.share_plan(table, [32, 30, 31, 32, 33], [4] * 5, 8, 17)
    assert bad == [4]
    assert plan.tolist() == [[0, 1, 0, 0], [1, 3, 24, 0], [1, 3, 24, 0], [3, 4, 0, 0], [4, 5, 0, 0]]
