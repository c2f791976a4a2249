"""What a served transformer block's step does between its linear layers, its paged
cache and its attention (C ABI in ``include/cbs_step.h``): the residual's addition with
the root-mean-square norm, rotary positions, and the cache's pages by the sequences'
lengths.

As in ``block8``, every step runs in the HIP kernels, on the current stream; PyTorch
supplies memory and streams (and copies inputs whose rows the kernels cannot read in place); nothing is read back to the host, so that a whole step
can be captured in a graph.  Forward only: inputs that require gradients or carry tangents are refused.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .binding import Library, lib
from .block8 import PagedCache, Rows8, _block8, _checked, _handle

# Every function include/cbs_step.h declares.
EXPORTS = ["cbs_add_rms_norm", "cbs_rotary_apply", "cbs_rotary_cache_write", "cbs_grow_pages", "cbs_grow_pages_workspace",
           "cbs_release_pages", "cbs_release_pages_workspace"]


def _declare():
    """The C ABI's types, for calls of it through ``binding.lib``."""
    vp, i, l, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    lib.cbs_add_rms_norm.argtypes = [vp, vp, l, vp, l, i, vp, i, f, vp, l, vp, i, l, l, i, vp]
    lib.cbs_rotary_apply.argtypes = [vp, vp, vp, l, l, vp, l, i, i, i, vp, l, l, vp]
    lib.cbs_rotary_cache_write.argtypes = [vp, vp, vp, vp, l, l, vp, l, l, vp, l, l, vp, vp, l, i, i, vp, l, l, vp]
    lib.cbs_grow_pages.argtypes = [vp, vp, vp, l, l, vp, vp, l, l, vp, vp, vp, vp, l, vp]
    lib.cbs_grow_pages_workspace.argtypes = [l, l]
    lib.cbs_release_pages.argtypes = [vp, vp, vp, l, l, vp, vp, l, vp, l, vp]
    lib.cbs_release_pages_workspace.argtypes = [l, l]
    for name in EXPORTS:
        getattr(lib, name).restype = l if name.endswith("_workspace") else i


_declare()


def add_rms_norm(x, weight=None, residual=None, eps: float = 1e-6, int8: bool = False, out=None, sum_out=None,
                 library: Library | None = None):
    """y = h * weight / sqrt(mean(h^2) + eps) over the last axis, with h = x + residual.

    x: [..., K] float32, bfloat16 or float16; weight: [K] of x's type or float32, or None
    for ones; residual: of x's shape, of x's type or float32, or None (then h is x).  x and the residual are read in
    place where they are rows one distance apart, each contiguous (a slice of a wider matrix's columns, say); other
    layouts, as some heads of a [tokens, heads, dim] tensor, are copied by PyTorch first.
    int8: give y as ``Rows8`` for ``int8_linear`` (quantised without a rounding to x's type in between).

    Returns y, of x's type; with a residual (y, h), h of the residual's type.  sum_out may be the
    (contiguous) residual itself, which is then updated in its place.
    """
    got = _checked(_block8.add_rms_norm(_handle(library), x, weight, residual, eps, int8, out, sum_out), library,
                   "cbs_add_rms_norm")
    if not int8:
        return got
    y, h = got if residual is not None else (got, None)
    y = Rows8(y, x.shape, x.dtype)
    return y if residual is None else (y, h)


def rotary_frequencies(dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       context: int = 0, low: float = 1.0, high: float = 32.0, device="cuda"):
    """Frequencies of the pairs of `dim` rotated dims, base^(-2i / dim), in radians per position
    (float64: in float32 they would be off by 2^-25 of a far position).

    For contexts `factor` times as long as the `context` tokens that a model was trained on:

    * "positions": all frequencies divided by the factor;
    * "base": the base enlarged by factor^(dim / (dim - 2)), which leaves the fastest pair as it is and divides
      the slowest by the factor;
    * "turns": a pair that turns `high` times or more within the context stays, one that turns `low` times
      or less is divided by the factor, and between the two the frequency goes linearly with
      the number of turns;
    * "pairs": the same with the share going linearly with the pair's number, between the pairs that turn `high`
      and `low` times: their numbers rounded outwards, the first 0 or more, the second dim - 1 or less.  The second
      may lie past the last pair, dim / 2 - 1, which then keeps a share of its frequency.
    """
    if dim < 2 or dim % 2 or not base > 1 or not factor >= 1:
        raise ValueError("dim must be even and positive, base above 1, factor 1 or more")
    if scaling == "base":
        if dim < 4:
            raise ValueError("a base can be enlarged for 4 dims or more")
        base = base * factor ** (dim / (dim - 2))
    i = torch.arange(dim // 2, dtype=torch.float64)
    f = torch.as_tensor(base, dtype=torch.float64) ** (-2 * i / dim)
    if scaling == "positions":
        f = f / factor
    elif scaling in ("turns", "pairs"):
        if context < 1 or not 0 < low < high:
            raise ValueError("context must be the tokens trained on, and 0 < low < high")
        if scaling == "turns":
            share = ((context * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)  # of what stays
        else:
            def pair(turns):
                return dim * math.log(context / (2 * math.pi * turns)) / (2 * math.log(base))
            first, last = max(0, math.floor(pair(high))), min(dim - 1, math.ceil(pair(low)))
            share = 1 - ((i - first) / max(last - first, 1e-3)).clamp(0, 1)
        f = f * (share + (1 - share) / factor)
    elif scaling not in (None, "base"):
        raise ValueError("scaling must be None, 'positions', 'base', 'turns' or 'pairs'")
    return f.to(device)


def rotary(x, positions, frequencies, interleaved: bool = False, magnitude: float = 1.0, out=None,
           library: Library | None = None):
    """Heads turned by their tokens' positions: pair i becomes magnitude * (a cos t - b sin t, b cos t + a sin t)
    with t = position * frequencies[i].

    x: [tokens, heads, dim] float32, bfloat16 or float16, dim (up to 512) contiguous, heads up to 65536; positions: int32
    [tokens]; frequencies: float64 [pairs], 2 * pairs up to dim; pair i is (i, i + pairs), or
    (2i, 2i + 1) where `interleaved`; the dims past 2 * pairs stay as they are.  Queries and keys that lie side by
    side in a projection's output are turned in one call.

    Returns [tokens, heads, dim] of x's type: a new tensor, or `out`, which may be x itself.
    """
    return _checked(_block8.rotary(_handle(library), x, positions, frequencies, interleaved, magnitude, out), library,
                    "cbs_rotary_apply")


def rotary_cache_write(cache: PagedCache, q, k, v, positions, slots, frequencies, interleaved: bool = False,
                       magnitude: float = 1.0, out=None, library: Library | None = None):
    """Queries turned, and keys turned on their way into the cache, with the values: ``rotary`` of q
    and k and ``cache_write`` in one pass over them.

    q: [tokens, heads, dim], k, v: [tokens, cache heads, dim] float32, bfloat16 or float16, dim
    contiguous (parts of one projection's output, say); positions, slots: int32 [tokens]; a token whose
    slot is outside the cache is not written (its queries are turned), and no two may name one slot.
    An int8 cache quantises the turned keys as they are in float32.

    Returns the turned queries: a new tensor, or `out`, which may be q itself.
    """
    return _checked(_block8.rotary_cache_write(_handle(library), cache._record, q, k, v, positions, slots, frequencies,
                                               interleaved, magnitude, out), library, "cbs_rotary_cache_write")


class PagePool:
    """The pages of a cache that no sequence has, on the device.

    free: int32 [pages], a stack of page numbers, of which the first counts[0] are there; counts: int32 [3], besides
    what the last ``grow_pages`` reported.  The tensors' contents may be changed at will; other
    tensors take a PagePool of their own.  Calls on one pool follow each other (in one stream, or by events).
    """

    def __init__(self, free, counts, page_size):
        self._record = _block8.pool(free, counts, page_size)
        self._tensors = free, counts
        self.pages, self.page_size = free.shape[0], page_size

    # what the kernels are given is the record's, so these cannot be set
    free, counts = (property(lambda self, i=i: self._tensors[i]) for i in range(2))

    @classmethod
    def full(cls, pages, page_size, device="cuda"):
        """A pool of all pages of a cache; page 0 is taken first."""
        return cls(torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device),
                   torch.tensor([pages, 0, 0], dtype=torch.int32, device=device), page_size)

    def report(self):
        """(free pages, pages that the last growth lacked, sequences that it left); waits for the device."""
        return tuple(self.counts.tolist())


def grow_pages(pool: PagePool, table, lens, more, tokens: int, library: Library | None = None):
    """Room in the cache for more[b] new tokens of each sequence.

    table: int32 [batch, width], each sequence's pages in order; lens: int32 [batch], its tokens; both are
    updated.  more: int32 [batch]; tokens: the batch's rows (the new tokens' number or more: the rest is padding).

    Returns (starts, slots, positions): int32 [batch + 1], where each sequence's new tokens begin in the
    batch, and int32 [tokens], the new tokens' slots in the cache and their positions; what ``rotary_cache_write`` and
    ``paged_attention`` take.  They lie in one allocation: who keeps one of them for long keeps the memory of all
    three, and clones it instead.  Sequences grow in order as long as there are pages; the first that lacks
    some, and all after it, are left as they are, as is one that would pass its row of the table or whose tokens pass
    `tokens`.  Tokens without a place (and padding) have slot -1 and position 0.  ``pool.report()`` says how it went.

    ``paged_attention`` goes by lens and does not look at slots: it takes the rows of a sequence that was left for its
    last old tokens, so that its output there stands for no token.  Where a step may be short of pages, use rows with
    ``slots >= 0`` only (``masked_fill_`` by ``slots < 0`` does it without the host), and bring the other tokens again.
    """
    return _checked(_block8.grow_pages(_handle(library), pool._record, table, lens, more, tokens), library, "cbs_grow_pages")


def release_pages(pool: PagePool, table, lens, keep, library: Library | None = None):
    """Sequences keep their first keep[b] tokens (0 where they have ended, fewer where drafts were rejected);
    the other pages go back to the pool, their entries of the table become -1, and lens is updated.  Entries that name
    no page of the pool (-1 where a page has been given back before, say) give nothing back.

    What ``grow_pages`` took and is given back at once lies in the pool as it did before.
    """
    _checked(_block8.release_pages(_handle(library), pool._record, table, lens, keep), library, "cbs_release_pages")
