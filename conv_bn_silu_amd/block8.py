"""The 8-bit operators of a served transformer block: a linear layer in 8-bit
integers, a paged key/value cache that quantises what it is given, and attention
of each sequence's newest tokens over it (C ABI in ``include/cbs_block8.h``).

As in ``binding``, this module only marshals arguments: every step runs in the
HIP kernels, on the current stream, and PyTorch supplies memory (outputs and
workspaces come from its allocator) and streams.  Forward only: the operators
are for serving and refuse inputs that require gradients.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import CbsError, ERR_INVALID_ARG, Library, OK, default_library, lib

DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2, torch.int8: 3}
ACTIVATIONS = {None: 0, "silu": 1}

# Every function include/cbs_block8.h declares.
EXPORTS = ["cbs_int8_linear", "cbs_int8_linear_workspace", "cbs_cache_write", "cbs_cache_read", "cbs_paged_attention",
           "cbs_paged_attention_workspace"]


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


def _declare():
    vp, i, l, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    cache = ctypes.POINTER(_Cache)
    lib.cbs_int8_linear.argtypes = [vp, vp, l, vp, vp, vp, vp, l, l, l, i, i, vp, l, vp]
    lib.cbs_int8_linear_workspace.argtypes = [l, l, l]
    lib.cbs_cache_write.argtypes = [vp, cache, vp, l, l, vp, l, l, vp, l, i, vp]
    lib.cbs_cache_read.argtypes = [vp, cache, vp, l, vp, vp, i, vp]
    lib.cbs_paged_attention.argtypes = [vp, vp, l, l, cache, vp, l, l, vp, vp, l, l, i, i, f, vp, i, vp, l, vp]
    lib.cbs_paged_attention_workspace.argtypes = [vp, l, l, i, i, i, i, l]
    for name in EXPORTS:
        getattr(lib, name).restype = l if name.endswith("_workspace") else i


_declare()


def _device_tensor(t, what, dtypes, device=None):
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise TypeError(f"{what} must be a tensor of type {' or '.join(str(d) for d in dtypes)}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{what} is on another device")
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{what} requires a gradient: these operators are forward only")


def _contiguous(t, shape, what):
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous, of shape {shape}")


def _output(out, shape, dtype, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _device_tensor(out, "out", (dtype,), device)
    _contiguous(out, tuple(shape), "out")
    return out


def _workspace(nbytes, device):
    return torch.empty(nbytes, dtype=torch.int8, device=device) if nbytes > 0 else None


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device):
    return torch.cuda.current_stream(device).cuda_stream


_VALUES = (torch.float32, torch.bfloat16, torch.float16)


def int8_linear(x, w, w_scale, bias=None, activation=None, out=None, library: Library | None = None):
    """y = act(x @ w.T) in 8-bit integers: the rows of x are quantised with one
    scale a row, multiplied by w exactly, and scaled back.

    x: [..., K] float32, bfloat16 or float16 (rows K apart or further, each
    contiguous); w: int8 [N, K]; w_scale: float32 [N] (w * w_scale is the weight);
    bias: float32 [N] or None; activation: None or "silu".  Returns [..., N] of
    x's type.
    """
    _device_tensor(x, "x", _VALUES)
    dev = x.device
    _device_tensor(w, "w", (torch.int8,), dev)
    _device_tensor(w_scale, "w_scale", (torch.float32,), dev)
    if x.dim() < 1 or w.dim() != 2 or x.shape[-1] != w.shape[1]:
        raise ValueError("x must be [..., K] and w [N, K]")
    if activation not in ACTIVATIONS:
        raise ValueError("activation must be None or 'silu'")
    N, K = w.shape
    _contiguous(w, (N, K), "w")
    _contiguous(w_scale, (N,), "w_scale")
    if bias is not None:
        _device_tensor(bias, "bias", (torch.float32,), dev)
        _contiguous(bias, (N,), "bias")
    x2 = x if x.dim() == 2 else x.reshape(-1, K)
    if K > 1 and x2.stride(1) != 1 or (x2.shape[0] > 1 and x2.stride(0) < K):
        x2 = x2.contiguous()
    M = x2.shape[0]
    y = _output(out, (*x.shape[:-1], N), x.dtype, dev)
    need = lib.cbs_int8_linear_workspace(M, N, K)
    ws = _workspace(need, dev)
    lib_ = library or default_library()
    lib_._check(lib.cbs_int8_linear(lib_.handle, x2.data_ptr(), x2.stride(0) if M > 1 else K, w.data_ptr(),
                                    w_scale.data_ptr(), _ptr(bias), y.data_ptr(), M, N, K, DTYPES[x.dtype],
                                    ACTIVATIONS[activation], _ptr(ws), need, _stream(dev)), "cbs_int8_linear")
    return y


class PagedCache:
    """A paged key/value cache over the caller's tensors.

    k, v: contiguous [pages, heads, page_size, dim], int8 (with k_scale, v_scale:
    float32 [pages, heads, page_size]) or float32, bfloat16, float16 (without).
    A token's slot is page * page_size + offset.
    """

    def __init__(self, k, v, k_scale=None, v_scale=None):
        _device_tensor(k, "k", tuple(DTYPES))
        _device_tensor(v, "v", (k.dtype,), k.device)
        if k.dim() != 4:
            raise ValueError("k must be [pages, heads, page_size, dim]")
        shape = tuple(k.shape)
        _contiguous(k, shape, "k")
        _contiguous(v, shape, "v")
        if k.dtype == torch.int8:
            for t, what in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                _device_tensor(t, what, (torch.float32,), k.device)
                _contiguous(t, shape[:3], what)
        elif k_scale is not None or v_scale is not None:
            raise ValueError("only an int8 cache has scales")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.heads, self.page_size, self.dim = shape
        self._record = _Cache(k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale), *shape, DTYPES[k.dtype])
        self._ref = ctypes.byref(self._record)

    @classmethod
    def empty(cls, pages, heads, page_size, dim, dtype=torch.int8, device="cuda"):
        """A cache of zeros."""
        k, v = (torch.zeros(pages, heads, page_size, dim, dtype=dtype, device=device) for _ in range(2))
        if dtype != torch.int8:
            return cls(k, v)
        return cls(k, v, *(torch.zeros(pages, heads, page_size, device=device) for _ in range(2)))


def _slots(cache, slots, tokens=None):
    _device_tensor(slots, "slots", (torch.int32,), cache.k.device)
    if slots.dim() != 1 or not slots.is_contiguous() or (tokens is not None and slots.shape[0] != tokens):
        raise ValueError("slots must be contiguous, one for each token")


def cache_write(cache: PagedCache, k, v, slots, library: Library | None = None):
    """Write tokens into the cache, quantising them (one scale for each token and
    head) where it is int8.

    k, v: [tokens, heads, dim] float32, bfloat16 or float16, dim contiguous;
    slots: int32 [tokens]; a token whose slot is outside the cache is skipped.
    """
    dev = cache.k.device
    _device_tensor(k, "k", _VALUES, dev)
    _device_tensor(v, "v", (k.dtype,), dev)
    want = (k.shape[0], cache.heads, cache.dim) if k.dim() == 3 else None
    for t, what in ((k, "k"), (v, "v")):
        if tuple(t.shape) != want or (cache.dim > 1 and t.stride(2) != 1):
            raise ValueError(f"{what} must be [tokens, {cache.heads}, {cache.dim}] with dim contiguous")
    tokens = k.shape[0]
    _slots(cache, slots, tokens)
    lib_ = library or default_library()
    lib_._check(lib.cbs_cache_write(lib_.handle, cache._ref, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(),
                                    v.stride(0), v.stride(1), slots.data_ptr(), tokens, DTYPES[k.dtype],
                                    _stream(dev)), "cbs_cache_write")


def cache_read(cache: PagedCache, slots, dtype=torch.bfloat16, library: Library | None = None):
    """Read tokens back as (k, v), each [tokens, heads, dim] of `dtype`; a slot
    outside the cache reads as zeros."""
    _slots(cache, slots)
    if dtype not in _VALUES:
        raise TypeError("dtype must be float32, bfloat16 or float16")
    dev = cache.k.device
    shape = (slots.shape[0], cache.heads, cache.dim)
    k, v = torch.empty(shape, dtype=dtype, device=dev), torch.empty(shape, dtype=dtype, device=dev)
    lib_ = library or default_library()
    lib_._check(lib.cbs_cache_read(lib_.handle, cache._ref, slots.data_ptr(), shape[0], k.data_ptr(), v.data_ptr(),
                                   DTYPES[dtype], _stream(dev)), "cbs_cache_read")
    return k, v


def paged_attention(q, cache: PagedCache, table, starts, lens, window: int = 0, scale: float | None = None, out=None,
                    library: Library | None = None):
    """Causal attention of each sequence's newest tokens over its cache.

    q: [tokens, heads, dim] bfloat16 or float16, dim contiguous, the sequences'
    new tokens one after the other; heads a multiple of the cache's.
    table: int32 [batch, width], each sequence's pages in order; starts: int32
    [batch + 1], where each sequence's rows of q begin; lens: int32 [batch], tokens
    of each sequence in the cache, the new ones included (write them first).
    window: 0, or how many latest keys (its own included) a token sees.
    scale: of the scores, 1 / sqrt(dim) by default.

    Returns [tokens, heads, dim] of q's type; a token that sees no key gets zeros.
    Nothing is read back to the host.
    """
    _device_tensor(q, "q", (torch.bfloat16, torch.float16))
    dev = q.device
    if cache.k.device != dev:
        raise ValueError("the cache is on another device")
    if cache.k.dtype not in (torch.int8, q.dtype):
        raise TypeError("the cache must be int8 or of q's type")
    if q.dim() != 3 or q.shape[2] != cache.dim or q.shape[1] % cache.heads or q.shape[1] == 0 or q.stride(2) != 1:
        raise ValueError(f"q must be [tokens, a multiple of {cache.heads}, {cache.dim}] with dim contiguous")
    for t, what in ((table, "table"), (starts, "starts"), (lens, "lens")):
        _device_tensor(t, what, (torch.int32,), dev)
    if table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("table must be [batch, width] with contiguous rows")
    batch, width = table.shape
    _contiguous(starts, (batch + 1,), "starts")
    _contiguous(lens, (batch,), "lens")
    if window < 0:
        raise ValueError("window must not be negative")
    tokens, heads, dim = q.shape
    y = _output(out, (tokens, heads, dim), q.dtype, dev)
    lib_ = library or default_library()
    need = lib.cbs_paged_attention_workspace(lib_.handle, batch, tokens, heads, cache.heads, dim, cache.page_size,
                                             width)
    ws = _workspace(need, dev)
    lib_._check(lib.cbs_paged_attention(lib_.handle, q.data_ptr(), q.stride(0), q.stride(1), cache._ref,
                                        table.data_ptr(), table.stride(0) if batch > 1 else width, width,
                                        starts.data_ptr(), lens.data_ptr(), batch, tokens, heads, int(window),
                                        dim ** -0.5 if scale is None else float(scale), y.data_ptr(),
                                        DTYPES[q.dtype], _ptr(ws), need, _stream(dev)), "cbs_paged_attention")
    return y
