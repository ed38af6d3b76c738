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
KEPT_WORKSPACES = 8  # of attention, per cache: those of the streams first seen last
DEVERR_PAGE, DEVERR_CAPACITY, DEVERR_LENGTH, DEVERR_FORK = 32, 64, 128, 256

EXPORTED = [
    "spec_cache_scratch_size", "spec_cache_init", "spec_cache_error", "spec_cache_reserve", "spec_cache_append",
    "spec_cache_commit", "spec_cache_fork", "spec_cache_release", "spec_attention_workspace_size", "spec_attention",
]

_P, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class SpecCache(ctypes.Structure):
    """spec_cache."""
    _fields_ = [("k", _P), ("v", _P), ("dtype", _i32), ("num_layers", _i32), ("num_pages", _i32),
                ("page_size", _i32), ("num_kv_heads", _i32), ("head_dim", _i32), ("layer_stride", _i64),
                ("page_stride", _i64), ("token_stride", _i64), ("head_stride", _i64), ("page_table", _P),
                ("table_stride", _i64), ("num_requests", _i32), ("max_pages", _i32), ("lens", _P), ("held", _P),
                ("ref_counts", _P), ("free_pages", _P), ("num_free", _P), ("error", _P), ("scratch", _P)]


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
                                              _i64, _i64, _P, _P, _sz, _P])):
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
    _call(c, "spec_cache_append", stream, layer, k_new.data_ptr(), kt, kh, v_new.data_ptr(), vt, vh,
          cu_new.data_ptr(), B, N)


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


def attention_workspace_size(c: PagedCache, num_q_heads: int, B: int, N: int) -> int:
    n = load().spec_attention_workspace_size(c.ref, int(num_q_heads), int(B), int(N))
    if n == 0:
        raise ValueError("invalid or unsupported sizes for spec_attention_workspace_size")
    return int(n)


def _workspace(c, H, B, N):
    """A workspace for one call on the current stream (of the cache's device, the current one): that of the
    stream, kept with the cache (its calls run one after the other), for KEPT_WORKSPACES streams; under
    capture a new one from the graph's memory, as graphs may run at the same time.  The caller holds the
    cache's lock until it has launched the call."""
    rows = min(256, N * (H // c.heads))  # its size grows with these
    handle = torch._C._cuda_getCurrentRawStream(c.index)
    capturing = torch._C._cuda_isCurrentStreamCapturing()
    kept = None if capturing else c.workspaces.get(handle)
    if kept is not None and kept[0] >= rows:
        return kept[1]
    size = _lib.spec_attention_workspace_size(c.ref, H, B, N)
    workspace = torch.empty(size, dtype=torch.uint8, device=c.device)
    if size and not capturing:
        c.workspaces.pop(handle, None)
        while len(c.workspaces) >= KEPT_WORKSPACES:  # (memory of its own stream: what runs there goes on)
            del c.workspaces[next(iter(c.workspaces))]
        c.workspaces[handle] = (rows, workspace)
    return workspace


_no_lock = contextlib.nullcontext()


def attention(c: PagedCache, layer: int, q, cu_new, parent=None, scale=None, out=None, lse=None, workspace=None,
              stream=None):
    """Attention of the new tokens q [N, q_heads, head_dim] over the cache (spec_attention); returns
    out, like q.

    ``parent`` (int32 [N]) makes the new tokens draft trees, otherwise they are chains; ``scale``
    defaults to head_dim ** -0.5; ``out`` may be given (one made for a call on another ``stream`` is
    memory of that stream, kept for the current one); ``lse`` (float32 [N, q_heads], given) receives
    the log of each row's softmax sum; ``workspace`` (uint8) may be given, calls that can run at the
    same time and calls of several host threads need one each (without one, the cache keeps one per
    stream, for KEPT_WORKSPACES streams, and a captured graph has its own).  Rows behind
    ``cu_new[B]`` are left as they were in ``out``.
    """
    if torch._C._cuda_getDevice() != c.index:
        with torch.cuda.device(c.index):
            return attention(c, layer, q, cu_new, parent, scale, out, lse, workspace, stream)
    if stream is not None:
        # all of the call on that stream: what it allocates is memory of the stream that writes it (the current
        # one's may have been freed with work queued there that still uses it), and of its graph under capture
        _of_device(stream, c.index)
        before = dict(zip(("stream_id", "device_index", "device_type"), torch._C._cuda_getCurrentStream(c.index)))
        torch.cuda.set_stream(stream)
        try:
            result = attention(c, layer, q, cu_new, parent, scale, out, lse, workspace)
        finally:
            torch._C._cuda_setStream(**before)
        if out is None:
            result.record_stream(torch.cuda.Stream(**before))  # which will read it
        return result
    B = _cu(c, cu_new)
    qt, qh = _rows(c, q, None, "q")
    N, H, _ = q.shape
    if parent is not None:
        _int32(parent, (N,), "parent", c.device)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
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
    with c.lock if workspace is None else _no_lock:
        if workspace is None:
            workspace = _workspace(c, H, B, N)
        _call(c, "spec_attention", None, layer, q.data_ptr(), qt, qh, H, cu_new.data_ptr(), B, N, _ptr(parent),
              c.dim ** -0.5 if scale is None else scale, out.data_ptr(), ot, oh, _ptr(lse), workspace.data_ptr(),
              workspace.numel())
    return out
