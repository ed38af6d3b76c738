"""The paged key/value cache around the verify step (``include/spec_cache.h``), over torch tensors.

Argument marshalling only, as in ``binding``: every operation runs in the library's CUDA kernels,
asynchronously on a stream of the cache's device: the current one, or ``stream=``, which then has to be
behind the work that makes the tensors given, and they have to live until it has run.  Errors the host can
see raise; errors in device data are collected in the cache's error word (``last_error``).

One step of a serving loop:

    cache.reserve(c, cu_new)
    for layer in range(layers):
        cache.append(c, layer, k_new, v_new, cu_new)
        out = cache.attention(c, layer, q, cu_new, parent=parent)   # parent: draft trees
    tokens, accepted = binding.sample(logits, ...)                  # or binding.tree_verify_greedy
    cache.commit(c, cu_new, accepted)                               # trees: parent=, last_node=

In place of ``append``, ``append_rotated`` turns keys and queries by their positions on the way; attention over the
last positions alone takes ``window=`` and ``sinks=``, and requests that share a prefix (forked ones) have it read
once for all with ``shared=cache.share(c)``.

``cu_new`` is a device int32 [B + 1]; row ``cu_new[r] + i`` of a step's tensors is new token i of
request r.  Chains of k_r drafts are k_r + 1 new tokens: ``cu_new = cu_num_draft + arange(B + 1)``.
"""
from __future__ import annotations

import contextlib
import ctypes
import threading
from dataclasses import dataclass, field

import torch

from .binding import SpecRejectError, load as _load_library

F16, BF16 = 2, 1
MAX_TREE = 128
ATTENTION_MAX_HEAD_DIM = 128
ROTATION_MAX_HEAD_DIM = 256
KEPT_WORKSPACES = 8  # of attention, per cache: those of the streams first seen last
DEVERR_PAGE, DEVERR_CAPACITY, DEVERR_LENGTH, DEVERR_FORK = 32, 64, 128, 256

EXPORTED = [
    "spec_cache_scratch_size", "spec_cache_init", "spec_cache_error", "spec_cache_reserve", "spec_cache_append",
    "spec_cache_commit", "spec_cache_fork", "spec_cache_release", "spec_attention_workspace_size", "spec_attention",
    "spec_cache_append_rotated", "spec_attention_window", "spec_cache_share", "spec_attention_shared_workspace_size",
    "spec_attention_shared",
]

_P, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class SpecCache(ctypes.Structure):
    """spec_cache."""
    _fields_ = [("k", _P), ("v", _P), ("dtype", _i32), ("num_layers", _i32), ("num_pages", _i32),
                ("page_size", _i32), ("num_kv_heads", _i32), ("head_dim", _i32), ("layer_stride", _i64),
                ("page_stride", _i64), ("token_stride", _i64), ("head_stride", _i64), ("page_table", _P),
                ("table_stride", _i64), ("num_requests", _i32), ("max_pages", _i32), ("lens", _P), ("held", _P),
                ("ref_counts", _P), ("free_pages", _P), ("num_free", _P), ("error", _P), ("scratch", _P)]


class Rotation(ctypes.Structure):
    """spec_rotation."""
    _fields_ = [("table", _P), ("row_stride", _i64), ("positions", _i32), ("dim", _i32), ("neighbours", _i32)]


_lib = None


def load():
    global _lib
    if _lib is not None:
        return _lib
    lib = _load_library()
    C = ctypes.POINTER(SpecCache)
    for name, result, args in (
            ("spec_cache_scratch_size", _sz, [_i32, _i32]),
            ("spec_cache_init", ctypes.c_int, [C, _P]),
            ("spec_cache_error", ctypes.c_int, [C, _P, _P, _P]),
            ("spec_cache_reserve", ctypes.c_int, [C, _P, _i32, _P]),
            ("spec_cache_append", ctypes.c_int, [C, _i32, _P, _i64, _i64, _P, _i64, _i64, _P, _i32, _i64, _P]),
            ("spec_cache_commit", ctypes.c_int, [C, _P, _i32, _i64, _P, _P, _P, _P, _P]),
            ("spec_cache_fork", ctypes.c_int, [C, _P, _P, _i32, _P]),
            ("spec_cache_release", ctypes.c_int, [C, _P, _i32, _P]),
            ("spec_attention_workspace_size", _sz, [C, _i32, _i32, _i64]),
            ("spec_attention", ctypes.c_int, [C, _i32, _P, _i64, _i64, _i32, _P, _i32, _i64, _P, ctypes.c_float, _P,
                                              _i64, _i64, _P, _P, _sz, _P]),
            ("spec_cache_append_rotated", ctypes.c_int, [C, _i32, _P, _i64, _i64, _P, _i64, _i64, _P, _i64, _i64, _i32,
                                                         _P, _i64, _i64, _P, _i32, _i64, _P,
                                                         ctypes.POINTER(Rotation), _P]),
            ("spec_attention_window", ctypes.c_int, [C, _i32, _P, _i64, _i64, _i32, _P, _i32, _i64, _P, ctypes.c_float,
                                                     _i32, _i32, _P, _i64, _i64, _P, _P, _sz, _P]),
            ("spec_cache_share", ctypes.c_int, [C, _i32, _i32, _P, _P]),
            ("spec_attention_shared_workspace_size", _sz, [C, _i32, _i32, _i64]),
            ("spec_attention_shared", ctypes.c_int, [C, _i32, _P, _i64, _i64, _i32, _P, _i32, _i64, _P, ctypes.c_float,
                                                     _P, _P, _i64, _i64, _P, _P, _sz, _P])):
        f = getattr(lib, name)
        f.restype, f.argtypes = result, args
    _lib = lib
    return lib


@dataclass
class PagedCache:
    """A cache over the caller's tensors.

    k, v [layers, pages, page_size, kv_heads, head_dim] (bfloat16 or float16, the same strides, unit
    stride inside; views of one tensor are fine); page_table [requests, max_pages], lens and held
    [requests], ref_counts and free_pages [pages], num_free [1]: int32, as spec_cache.h describes
    them.  ``make_cache`` makes an empty one.  The tensors stay those given: write into them.
    """
    k: object
    v: object
    page_table: object
    lens: object
    held: object
    ref_counts: object
    free_pages: object
    num_free: object
    error: object = None
    scratch: object = None
    struct: SpecCache = field(default=None, repr=False)

    def __post_init__(self):
        k, v, dev = self.k, self.v, self.k.device
        if dev.type != "cuda":
            raise ValueError("a cache lives on a CUDA device")
        if k.dtype not in (torch.bfloat16, torch.float16) or v.dtype != k.dtype:
            raise TypeError("keys and values must both be bfloat16 or both float16")
        if k.dim() != 5 or k.shape != v.shape or k.stride(4) != 1 or v.stride(4) != 1:
            raise ValueError("keys and values must be [layers, pages, page_size, kv_heads, head_dim] alike, with "
                             "unit stride along head_dim")
        if v.device != dev:
            raise ValueError("keys and values must be on one device")
        if any(k.stride(i) != v.stride(i) for i in range(4) if k.shape[i] > 1):
            raise ValueError("keys and values must have the same strides")
        L, NP, P, H, D = (int(x) for x in k.shape)
        R, MP = (int(x) for x in self.page_table.shape)
        for name, shape in (("page_table", (R, MP)), ("lens", (R,)), ("held", (R,)), ("ref_counts", (NP,)),
                            ("free_pages", (NP,)), ("num_free", (1,))):
            _int32(getattr(self, name), shape, name, dev, contiguous=name != "page_table")
        if MP > 1 and self.page_table.stride(1) != 1:
            raise ValueError("page_table must have unit stride along its columns")
        size = load().spec_cache_scratch_size(R, NP)
        if size == 0:
            raise ValueError("a cache needs at least one request and one page")
        if self.scratch is None:
            self.scratch = torch.zeros(size, dtype=torch.uint8, device=dev)
        if self.error is None:
            self.error = torch.tensor([0, 2 ** 31 - 1], dtype=torch.int32, device=dev)
        _int32(self.error, (2,), "error", dev)
        if self.scratch.numel() < size or self.scratch.device != dev:
            raise ValueError(f"scratch must hold {size} bytes on {dev}")
        stride = [k.stride(i) if k.shape[i] > 1 else 0 for i in range(4)]
        self.struct = SpecCache(
            k=k.data_ptr(), v=v.data_ptr(), dtype=_code(k), num_layers=L, num_pages=NP, page_size=P, num_kv_heads=H,
            head_dim=D, layer_stride=stride[0], page_stride=stride[1], token_stride=stride[2], head_stride=stride[3],
            page_table=self.page_table.data_ptr(), table_stride=self.page_table.stride(0) if R > 1 else MP,
            num_requests=R, max_pages=MP, lens=self.lens.data_ptr(), held=self.held.data_ptr(),
            ref_counts=self.ref_counts.data_ptr(), free_pages=self.free_pages.data_ptr(),
            num_free=self.num_free.data_ptr(), error=self.error.data_ptr(), scratch=self.scratch.data_ptr())
        # what every call needs, looked up once: the tensors of a cache do not change
        self.ref, self.device, self.index = ctypes.byref(self.struct), dev, dev.index
        self.dtype, self.heads, self.dim = k.dtype, H, D
        # attention's, by stream: (rows, workspace); the lock is held from the look to the launches, as a call's
        # two kernels and their workspace belong together whichever host threads call
        self.workspaces, self.lock = {}, threading.RLock()


def _code(t) -> int:
    return BF16 if t.dtype == torch.bfloat16 else F16


def _int32(t, shape, name, device, contiguous=True):
    if t.dtype is not torch.int32 or t.shape != shape or (contiguous and not t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")


def _clamped(x):
    """An integer as the library takes it (ctypes would keep its low 32 bits): what lies outside of int32 is as good as
    its ends, or refused as they are."""
    return max(-1, min(x, 2 ** 31 - 1))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _of_device(stream, index):
    """Refuses a stream of another device than the cache's: a launch there would fail in the driver."""
    if stream.device_index != index:
        raise ValueError(f"stream must be one of cuda:{index}")


def _call(c, name, stream, *args):
    """Calls a library function on the cache's device and a stream (the device's current one, by its raw
    handle, unless one is given)."""
    index = c.index
    if stream is not None:
        _of_device(stream, index)
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return _call(c, name, stream, *args)
    status = getattr(_lib, name)(c.ref, *args, torch._C._cuda_getCurrentRawStream(index) if stream is None
                                 else stream.cuda_stream)
    if status != 0:
        raise SpecRejectError(status, name)


def make_cache(num_layers: int, num_pages: int, page_size: int, num_kv_heads: int, head_dim: int, num_requests: int,
               max_pages: int, dtype=None, device="cuda", stream=None) -> PagedCache:
    """An empty cache: every page free.  Keys and values are zero.  With ``stream`` it is made there and its
    tensors are memory of that stream: calls on it may follow at once, other streams wait for it."""
    dev = torch.device(device)
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    if stream is not None:
        _of_device(stream, dev.index)
        with torch.cuda.stream(stream):
            return make_cache(num_layers, num_pages, page_size, num_kv_heads, head_dim, num_requests, max_pages, dtype,
                              dev)
    ints = lambda *shape: torch.empty(shape, dtype=torch.int32, device=dev)  # noqa: E731
    kv = torch.zeros((2, num_layers, num_pages, page_size, num_kv_heads, head_dim),
                     dtype=torch.bfloat16 if dtype is None else dtype, device=dev)
    c = PagedCache(kv[0], kv[1], page_table=ints(num_requests, max_pages), lens=ints(num_requests),
                   held=ints(num_requests), ref_counts=ints(num_pages), free_pages=ints(num_pages), num_free=ints(1))
    _call(c, "spec_cache_init", None)
    return c


def last_error(c: PagedCache, stream=None):
    """(status, error_bits, first_bad_request) since the last call, and clears them (synchronises)."""
    if stream is not None:
        _of_device(stream, c.index)
    bits, first = ctypes.c_int32(0), ctypes.c_int32(0)
    with torch.cuda.device(c.device):
        s = torch.cuda.current_stream() if stream is None else stream
        st = load().spec_cache_error(c.ref, s.cuda_stream, ctypes.byref(bits), ctypes.byref(first))
    if st not in (0, 5, 6):
        raise SpecRejectError(st, "spec_cache_error")
    return int(st), int(bits.value), int(first.value)


def _cu(c, cu_new) -> int:
    shape = cu_new.shape
    if len(shape) != 1 or shape[0] < 1:
        raise TypeError("cu_new must be a 1-D int32 tensor of B + 1 entries")
    _int32(cu_new, shape, "cu_new", c.device)
    return shape[0] - 1


def _rows(c, t, heads, name):
    """Checks a [N, heads, head_dim] tensor; returns its token and head strides."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not c.dtype or len(shape) != 3 or (heads is not None and shape[1] != heads) or \
            shape[2] != c.dim or (stride[2] != 1 and t.numel()):
        raise TypeError(f"{name} must be a {c.dtype} tensor [N, heads, {c.dim}] with unit stride inside")
    if t.device != c.device:
        raise ValueError(f"{name} must be on {c.device}")
    return stride[0], stride[1]


def reserve(c: PagedCache, cu_new, stream=None):
    """Pages for the new tokens of every request (spec_cache_reserve)."""
    B = _cu(c, cu_new)
    _call(c, "spec_cache_reserve", stream, cu_new.data_ptr(), B)


def append(c: PagedCache, layer: int, k_new, v_new, cu_new, stream=None):
    """Writes the new tokens' keys and values [N, kv_heads, head_dim] of one layer (spec_cache_append)."""
    B = _cu(c, cu_new)
    kt, kh = _rows(c, k_new, c.heads, "k_new")
    vt, vh = _rows(c, v_new, c.heads, "v_new")
    N = k_new.shape[0]
    if v_new.shape[0] != N:
        raise ValueError("k_new and v_new must have the same rows")
    _call(c, "spec_cache_append", stream, _clamped(layer), k_new.data_ptr(), kt, kh, v_new.data_ptr(), vt, vh,
          cu_new.data_ptr(), B, N)


def rotation_table(positions: int, dim: int, base: float = 10000.0, device="cuda"):
    """The table of ``append_rotated`` for positions 0 .. positions - 1: pair i turns by p * base ** (-2 i / dim)
    radians at position p.  float32 [positions, dim], cosines before sines, computed in 64 bits.  Scaled or otherwise
    spaced rotations are tables of the caller's making."""
    half = dim // 2
    speed = base ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * speed
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def append_rotated(c: PagedCache, layer: int, q, k_new, v_new, cu_new, rotation, parent=None, interleaved=False,
                   out=None, stream=None):
    """``append`` with the keys turned by their positions on the way; returns the queries q [N, q_heads, head_dim] of
    the same tokens, turned alike (spec_cache_append_rotated).

    ``rotation`` (float32 [positions, dim], ``rotation_table``) holds dim / 2 cosines and as many sines per position;
    it turns the first ``dim`` elements of each head, pairs of elements i and dim / 2 + i, or of neighbours with
    ``interleaved``.  Chains stand at positions lens + i, with ``parent`` (int32 [N]) the nodes of draft trees at
    lens + depth.  ``out`` may be q itself; rows of requests with errors, and behind ``cu_new[B]``, are left as they
    were in it.  ``q`` may be None.  A result made for a call on another ``stream`` is memory of that stream, kept for
    the current one.
    """
    if torch._C._cuda_getDevice() != c.index:
        with torch.cuda.device(c.index):
            return append_rotated(c, layer, q, k_new, v_new, cu_new, rotation, parent, interleaved, out, stream)
    if stream is not None:
        return _on_stream(c, stream, out is None and q is not None, append_rotated, c, layer, q, k_new, v_new, cu_new,
                          rotation, parent, interleaved, out)
    B = _cu(c, cu_new)
    kt, kh = _rows(c, k_new, c.heads, "k_new")
    vt, vh = _rows(c, v_new, c.heads, "v_new")
    N = k_new.shape[0]
    if v_new.shape[0] != N or (q is not None and q.shape[0] != N):
        raise ValueError("q, k_new and v_new must have the same rows")
    shape, stride = rotation.shape, rotation.stride()
    if rotation.dtype is not torch.float32 or len(shape) != 2 or (stride[1] != 1 and rotation.numel()):
        raise TypeError("rotation must be a float32 tensor [positions, dim] with unit stride inside")
    if rotation.device != c.device:
        raise ValueError(f"rotation must be on {c.device}")
    if parent is not None:
        _int32(parent, (N,), "parent", c.device)
    H = qt = qh = ot = oh = 0
    if q is not None:
        qt, qh = _rows(c, q, None, "q")
        H = q.shape[1]
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
            ot, oh = H * c.dim, c.dim
        elif out.shape != q.shape:
            raise ValueError("out must have the shape of q")
        else:
            ot, oh = _rows(c, out, H, "out")
    elif out is not None:
        raise ValueError("out needs q")
    turn = Rotation(rotation.data_ptr(), stride[0], _clamped(shape[0]), _clamped(shape[1]), 1 if interleaved else 0)
    _call(c, "spec_cache_append_rotated", None, _clamped(layer), k_new.data_ptr(), kt, kh, v_new.data_ptr(), vt, vh,
          _ptr(q), qt, qh, H, _ptr(out), ot, oh, cu_new.data_ptr(), B, N, _ptr(parent), ctypes.byref(turn))
    return out


def share(c: PagedCache, min_tokens: int = 512, B: int | None = None, out=None, stream=None):
    """Which of the requests 0 .. B-1 (None: all) share the pages of a prefix of ``min_tokens`` tokens or more with
    their neighbours (spec_cache_share): int32 [B, 4], per request the first of its group, the end, the tokens that the
    group shares, 0.  The plan of ``attention(shared=...)`` for all layers and steps in which the requests keep these
    pages; ordered like the calls that change the cache.

    A prefix read once saves its bytes and costs a join of every row.  Single tokens of eight or more requests gain from
    64 shared tokens on, pairs of requests and steps of nine tokens from about 1000 (64 requests, 8 kv heads of 128, own
    context 200: 512 tokens under groups of eight 47.6 -> 39.2 us, under pairs 50 -> 53, nine tokens each 52 -> 59; 4096
    tokens 148 -> 54, 177 -> 110, 157 -> 93).  The default is for single tokens.  A group shares what its shortest link
    does (prefixes inside prefixes: give a ``min_tokens`` above the common one), and reads apart once its first request
    was released, until the next plan."""
    if torch._C._cuda_getDevice() != c.index:
        with torch.cuda.device(c.index):
            return share(c, min_tokens, B, out, stream)
    if stream is not None:
        return _on_stream(c, stream, out is None, share, c, min_tokens, B, out)
    if B is None:
        B = c.lens.shape[0]
    if out is None:  # (of more requests than there are, the library refuses it)
        out = torch.empty((max(min(B, c.lens.shape[0]), 0), 4), dtype=torch.int32, device=c.device)
    else:
        _int32(out, (B, 4), "out", c.device)
    _call(c, "spec_cache_share", None, _clamped(B), _clamped(min_tokens), out.data_ptr())
    return out


def commit(c: PagedCache, cu_new, num_accepted, parent=None, last_node=None, out_lens=None, stream=None):
    """Advances lengths by num_accepted + 1; with a tree (``parent`` and ``last_node``) moves the
    accepted path's rows together (spec_cache_commit)."""
    B = _cu(c, cu_new)
    _int32(num_accepted, (B,), "num_accepted", c.device)
    if (parent is None) != (last_node is None):
        raise ValueError("a tree needs both parent and last_node")
    N = 2 ** 31 - 1
    if parent is not None:
        N = int(parent.shape[0])
        _int32(parent, (N,), "parent", c.device)
        _int32(last_node, (B,), "last_node", c.device)
    if out_lens is not None:
        _int32(out_lens, (B,) if out_lens is not c.lens else c.lens.shape, "out_lens", c.device)
    _call(c, "spec_cache_commit", stream, cu_new.data_ptr(), B, N, num_accepted.data_ptr(), _ptr(parent),
          _ptr(last_node), _ptr(out_lens))


def fork(c: PagedCache, src, dst, stream=None):
    """Makes requests ``dst`` share the committed tokens of requests ``src`` (spec_cache_fork)."""
    F = int(src.shape[0])
    _int32(src, (F,), "src", c.device)
    _int32(dst, (F,), "dst", c.device)
    _call(c, "spec_cache_fork", stream, src.data_ptr(), dst.data_ptr(), F)


def release(c: PagedCache, keep_lens=None, stream=None):
    """Truncates requests 0 .. B-1 to ``keep_lens`` (int32 [B]; None: every request, committed tokens
    kept) and gives back the pages behind (spec_cache_release)."""
    B = int(c.lens.shape[0])
    if keep_lens is not None:
        B = int(keep_lens.shape[0])
        _int32(keep_lens, (B,), "keep_lens", c.device)
    _call(c, "spec_cache_release", stream, _ptr(keep_lens), B)


def attention_workspace_size(c: PagedCache, num_q_heads: int, B: int, N: int, shared: bool = False) -> int:
    """Bytes of a ``workspace`` for calls of ``attention`` on N rows, of those with ``shared`` or of the others.  (Shared
    ones keep two sums per row and query head: 2 (4 dim + 16) bytes with dim 64 or 128, 553 MB of 16384 tokens with 32
    heads of 128; the others 42 MB at most.)"""
    name = "spec_attention_shared_workspace_size" if shared else "spec_attention_workspace_size"
    n = getattr(load(), name)(c.ref, _clamped(int(num_q_heads)), _clamped(int(B)), int(N))
    if n == 0:
        raise ValueError(f"invalid or unsupported sizes for {name}")
    return int(n)


def _on_stream(c, stream, made, function, *args):
    """A call with ``stream`` current: what it allocates is memory of the stream that writes it (the current one's may
    have been freed with work queued there that still uses it), and of its graph under capture.  ``made``: the result
    is new, and the stream that was current will read it."""
    if torch._C._cuda_getDevice() != c.index:
        with torch.cuda.device(c.index):
            return _on_stream(c, stream, made, function, *args)
    _of_device(stream, c.index)
    before = dict(zip(("stream_id", "device_index", "device_type"), torch._C._cuda_getCurrentStream(c.index)))
    torch.cuda.set_stream(stream)
    try:
        result = function(*args)
    finally:
        torch._C._cuda_setStream(**before)
    if made:
        result.record_stream(torch.cuda.Stream(**before))
    return result


def _workspace(c, H, B, N, shared, handle):
    """A workspace for one call on the current stream (of the cache's device, the current one; its raw handle): that
    of the stream, kept with the cache (its calls run one after the other), for KEPT_WORKSPACES streams; under
    capture a new one from the graph's memory, as graphs may run at the same time.  The caller holds the
    cache's lock until it has launched the call."""
    rows = min(256, N * (H // c.heads))  # its size grows with these, for shared prefixes with all rows as well: their
    all_rows = N * H if shared else -1   # layout has more parts even where there are none
    kept = None if torch._C._cuda_isCurrentStreamCapturing() else c.workspaces.get(handle, _none_kept)
    if kept is not None and kept[0] >= rows and kept[1] >= all_rows:
        return kept[2]
    if kept is not None:
        rows, all_rows = max(rows, kept[0]), max(all_rows, kept[1])
    size = (_lib.spec_attention_shared_workspace_size if shared else _lib.spec_attention_workspace_size)(c.ref, H, B, N)
    if size and kept is not None:
        size = max(size, 0 if kept[2] is None else kept[2].numel())
    workspace = torch.empty(size, dtype=torch.uint8, device=c.device)
    if size and kept is not None:
        c.workspaces.pop(handle, None)
        while len(c.workspaces) >= KEPT_WORKSPACES:  # (memory of its own stream: what runs there goes on)
            del c.workspaces[next(iter(c.workspaces))]
        c.workspaces[handle] = (rows, all_rows, workspace)
    return workspace


_none_kept = (-1, -1, None)  # rows of a softmax group's partial sums, rows in all, the workspace
_no_lock = contextlib.nullcontext()


def attention(c: PagedCache, layer: int, q, cu_new, parent=None, scale=None, out=None, lse=None, workspace=None,
              stream=None, window=None, sinks=0, shared=None):
    """Attention of the new tokens q [N, q_heads, head_dim] over the cache (spec_attention); returns
    out, like q.

    ``parent`` (int32 [N]) makes the new tokens draft trees, otherwise they are chains; ``scale``
    defaults to head_dim ** -0.5; ``out`` may be given (one made for a call on another ``stream`` is
    memory of that stream, kept for the current one); ``lse`` (float32 [N, q_heads], given) receives
    the log of each row's softmax sum; ``workspace`` (uint8, ``attention_workspace_size``) may be given, calls that
    can run at the same time and calls of several host threads need one each (without one, the cache keeps one per
    stream, for KEPT_WORKSPACES streams, and a captured graph has its own).  Rows behind
    ``cu_new[B]`` are left as they were in ``out``.

    ``window`` (>= 1): a row sees the last ``window`` positions, its own among them, and the first ``sinks`` ones
    (spec_attention_window; positions of a tree's nodes are by depth).  ``shared`` (int32 [B, 4], ``share``): requests
    whose prefix lies in the same pages have it read once for all (spec_attention_shared); for steps in which requests
    have about as many new tokens each (one chunk of 2048 tokens among 127 single ones takes longer with a plan than
    without, 882 us against 340 behind 2048 shared tokens).  Not both: what lies behind a window is read by few requests,
    if any.
    """
    if torch._C._cuda_getDevice() != c.index:
        with torch.cuda.device(c.index):
            return attention(c, layer, q, cu_new, parent, scale, out, lse, workspace, stream, window, sinks, shared)
    if stream is not None:
        return _on_stream(c, stream, out is None, attention, c, layer, q, cu_new, parent, scale, out, lse, workspace,
                          None, window, sinks, shared)
    B = _cu(c, cu_new)
    qt, qh = _rows(c, q, None, "q")
    N, H, _ = q.shape
    if parent is not None:
        _int32(parent, (N,), "parent", c.device)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
        ot, oh = H * c.dim, c.dim
    elif out.shape != q.shape:
        raise ValueError("out must have the shape of q")
    else:
        ot, oh = _rows(c, out, H, "out")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (N, H) or not lse.is_contiguous() or
                            lse.device != c.device):
        raise TypeError(f"lse must be a contiguous float32 tensor of shape {(N, H)} on {c.device}")
    if workspace is not None and (workspace.dtype is not torch.uint8 or workspace.device != c.device or
                                  not workspace.is_contiguous()):
        raise TypeError(f"workspace must be a contiguous uint8 tensor on {c.device}")
    given = (c.dim ** -0.5 if scale is None else scale,)
    if window is not None:
        if shared is not None:
            raise ValueError("attention takes a window or a plan of shared prefixes, not both")
        function = _lib.spec_attention_window
        given += (_clamped(window), _clamped(sinks))
    elif sinks:
        raise ValueError("sinks need a window")
    elif shared is not None:
        _int32(shared, (B, 4), "shared", c.device)
        function = _lib.spec_attention_shared
        given += (shared.data_ptr(),)
    else:
        function = _lib.spec_attention
    handle = torch._C._cuda_getCurrentRawStream(c.index)
    with c.lock if workspace is None else _no_lock:
        if workspace is None:
            workspace = _workspace(c, H, B, N, shared is not None, handle)
        status = function(c.ref, _clamped(layer), q.data_ptr(), qt, qh, H, cu_new.data_ptr(), B, N, _ptr(parent), *given,
                          out.data_ptr(), ot, oh, _ptr(lse), workspace.data_ptr(), workspace.numel(), handle)
    if status != 0:
        raise SpecRejectError(status, function.__name__)
    return out
