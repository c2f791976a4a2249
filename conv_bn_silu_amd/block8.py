"""The 8-bit operators of a served transformer block: a linear layer in 8-bit
integers, a paged key/value cache that quantises what it is given, and attention
of each sequence's newest tokens over it (C ABI in ``include/cbs_block8.h``).

Every step runs in the HIP kernels, on the current stream, and PyTorch supplies
memory (outputs and workspaces come from its allocator) and streams.  The
arguments are marshalled natively (``csrc/py_block8.cpp``, built into
``_block8.so``): a call costs the host little more than its launches.  Forward
only: the operators are for serving and refuse inputs that require gradients or carry tangents.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .binding import CbsError, Library, default_library, lib

try:
    from . import _block8
except ImportError as e:
    raise ImportError("_block8.so is not built, or not for this PyTorch; run __graft_entry__.build() or "
                      "python conv_bn_silu_amd/build.py") from e

ACTIVATIONS = {None: 0, "silu": 1}

# Every function include/cbs_block8.h declares.
EXPORTS = ["cbs_int8_linear", "cbs_int8_linear_workspace", "cbs_int8_linear_rows", "cbs_int8_linear_rows_workspace",
           "cbs_rows8_bytes", "cbs_cache_write", "cbs_cache_read", "cbs_paged_attention", "cbs_paged_attention_workspace"]


def _declare():
    """The C ABI's types, for calls of it through ``binding.lib``."""
    vp, i, l, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    cache = vp
    lib.cbs_int8_linear.argtypes = [vp, vp, l, vp, vp, vp, vp, l, l, l, i, i, vp, l, vp]
    lib.cbs_int8_linear_workspace.argtypes = [l, l, l]
    lib.cbs_int8_linear_rows.argtypes = [vp, vp, vp, vp, vp, vp, l, l, l, i, i, vp, l, vp]
    lib.cbs_int8_linear_rows_workspace.argtypes = [l, l, l]
    lib.cbs_rows8_bytes.argtypes = [l, l]
    lib.cbs_cache_write.argtypes = [vp, cache, vp, l, l, vp, l, l, vp, l, i, vp]
    lib.cbs_cache_read.argtypes = [vp, cache, vp, l, vp, vp, i, vp]
    lib.cbs_paged_attention.argtypes = [vp, vp, l, l, cache, vp, l, l, vp, vp, l, l, i, i, f, vp, i, vp, l, vp]
    lib.cbs_paged_attention_workspace.argtypes = [vp, l, l, i, i, i, i, l]
    for name in EXPORTS:
        getattr(lib, name).restype = l if name.endswith(("_workspace", "_bytes")) else i


_declare()


def _handle(library):
    """The handle's address; None where there is none to be had: the arguments are
    judged first, and `_checked` then says why."""
    try:
        handle = (library or default_library()).handle
    except CbsError:
        return None
    return handle.value if handle else None


def _checked(got, library, what):
    """A native call's result, or its status raised."""
    if type(got) is int:
        (library or default_library())._check(got, what)
    return got


class Rows8:
    """Rows in 8 bits, [..., K]: codes in [-127, 127], each row with a scale, as the linear layer makes
    them of its input and ``add_rms_norm`` gives them.  They lie as the layer's matrix kernels read them, in
    one int8 tensor (`buffer`; the layout is in include/cbs_block8.h).  shape: a tuple, [..., K].  dtype: of what they were made of, and
    of the layer's output.
    """

    def __init__(self, buffer, shape, dtype):
        self.buffer, self.shape, self.dtype = buffer, shape, dtype

    def _split(self):
        r, blocks = (math.prod(self.shape[:-1]) + 15) // 16 * 16, (self.shape[-1] + 127) // 128 * 2
        return self.buffer[:4 * r].view(torch.float32), self.buffer[4 * r:].view(blocks, r, 64)

    @property
    def scale(self):
        """float32 [...], in the buffer."""
        lead = self.shape[:-1]
        return self._split()[0][:math.prod(lead)].view(lead)

    @property
    def codes(self):
        """int8 [..., K], a copy."""
        rows = self._split()[1].transpose(0, 1).flatten(1)
        return rows[:math.prod(self.shape[:-1]), :self.shape[-1]].reshape(self.shape)

    def dequantize(self, dtype=None):
        """codes * scale, a copy of `dtype` (that of what they were made of by default)."""
        return (self.codes.float() * self.scale[..., None]).to(dtype or self.dtype)


def int8_linear(x, w, w_scale, bias=None, activation=None, out=None, library: Library | None = None):
    """y = act(x @ w.T) in 8-bit integers: the rows of x are quantised with one
    scale a row, multiplied by w exactly, and scaled back.

    x: [..., K] float32, bfloat16 or float16 (rows K apart or further, each
    contiguous, else they are copied); w: int8 [N, K]; w_scale: float32 [N]
    (w * w_scale is the weight); bias: float32 [N] or None; activation: None or
    "silu".  Returns [..., N] of x's type.  x may be ``Rows8``, quantised already.
    """
    if type(x) is Rows8:
        return _checked(_block8.int8_linear_rows(_handle(library), x.buffer, x.shape, x.dtype, w, w_scale, bias,
                                                 ACTIVATIONS.get(activation, -1), out), library, "cbs_int8_linear_rows")
    return _checked(_block8.int8_linear(_handle(library), x, w, w_scale, bias, ACTIVATIONS.get(activation, -1), out),
                    library, "cbs_int8_linear")


class PagedCache:
    """A paged key/value cache over the caller's tensors.

    k, v: contiguous [pages, heads, page_size, dim], int8 (with k_scale, v_scale:
    float32 [pages, heads, page_size]) or float32, bfloat16, float16 (without).
    A token's slot is page * page_size + offset.  The tensors' contents may be changed
    at will; other tensors take a PagedCache of their own.
    """

    def __init__(self, k, v, k_scale=None, v_scale=None):
        self._record = _block8.cache(k, v, k_scale, v_scale)
        self._tensors = k, v, k_scale, v_scale
        self.pages, self.heads, self.page_size, self.dim = k.shape

    # what the kernels are given is the record's, so these cannot be set
    k, v, k_scale, v_scale = (property(lambda self, i=i: self._tensors[i]) for i in range(4))

    @classmethod
    def empty(cls, pages, heads, page_size, dim, dtype=torch.int8, device="cuda"):
        """A cache of zeros."""
        k, v = (torch.zeros(pages, heads, page_size, dim, dtype=dtype, device=device) for _ in range(2))
        if dtype != torch.int8:
            return cls(k, v)
        return cls(k, v, *(torch.zeros(pages, heads, page_size, device=device) for _ in range(2)))


def cache_write(cache: PagedCache, k, v, slots, library: Library | None = None):
    """Write tokens into the cache, quantising them (one scale for each token and
    head) where it is int8.

    k, v: [tokens, heads, dim] float32, bfloat16 or float16, dim contiguous;
    slots: int32 [tokens]; a token whose slot is outside the cache is skipped, and
    no two may name one slot (what that holds afterwards is undefined).
    """
    _checked(_block8.cache_write(_handle(library), cache._record, k, v, slots), library, "cbs_cache_write")


def cache_read(cache: PagedCache, slots, dtype=torch.bfloat16, library: Library | None = None):
    """Read tokens back as (k, v), each [tokens, heads, dim] of `dtype`; a slot
    outside the cache reads as zeros."""
    return _checked(_block8.cache_read(_handle(library), cache._record, slots, dtype), library, "cbs_cache_read")


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
    return _checked(_block8.paged_attention(_handle(library), q, cache._record, table, starts, lens, window, scale, out),
                    library, "cbs_paged_attention")
