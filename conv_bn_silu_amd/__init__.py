"""MI355X-native fused conv2d + folded BatchNorm + SiLU.

The operator runs in hand-written HIP kernels for gfx950 behind a C ABI
(``include/conv_bn_silu.h``, built into ``libconv_bn_silu.so`` next to this
file).  ``binding`` is a thin ctypes layer over that ABI; PyTorch supplies
device memory and streams only.  The binding is imported lazily so that the
input generator (``synth``) can be used without the shared library.

``block8`` holds the 8-bit operators of a served transformer block
(``include/cbs_block8.h``): a linear layer in 8-bit integers, a paged key/value
cache that quantises what it is given, and attention over it.  ``step`` holds
what a step does between those (``include/cbs_step.h``): the residual's addition with the
root-mean-square norm, rotary positions, the cache's pages by the sequences' lengths.
"""
from __future__ import annotations

import importlib

_BLOCK8 = ("int8_linear", "Rows8", "PagedCache", "cache_write", "cache_read", "paged_attention")
_STEP = ("add_rms_norm", "rotary", "rotary_cache_write", "rotary_frequencies", "PagePool", "grow_pages", "release_pages")

__all__ = ["conv_bn_silu", "conv_bn_silu_unfused", "fold_bn", *_BLOCK8, *_STEP, "binding", "block8", "step", "synth"]


def __getattr__(name):
    if name in ("binding", "block8", "step", "synth"):
        value = importlib.import_module(f"{__name__}.{name}")
    elif name in ("conv_bn_silu", "conv_bn_silu_unfused", "fold_bn", "Library"):
        value = getattr(importlib.import_module(f"{__name__}.binding"), name)
    elif name in _BLOCK8:
        value = getattr(importlib.import_module(f"{__name__}.block8"), name)
    elif name in _STEP:
        value = getattr(importlib.import_module(f"{__name__}.step"), name)
    else:
        raise AttributeError(name)
    globals()[name] = value  # found once: looking it up here again took 7 us an import
    return value
