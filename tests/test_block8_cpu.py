"""The 8-bit block operators without a GPU: the library exports what the header
declares, and refuses what it does not serve before any kernel."""
import ctypes
import os
import re

import pytest
import torch

from conv_bn_silu_amd import binding as B
from conv_bn_silu_amd import block8
import block8_oracle as O

pytestmark = pytest.mark.cpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_header_and_binding_agree():
    text = open(os.path.join(ROOT, "include", "cbs_block8.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    assert sorted(set(re.findall(r"\b(cbs_\w+)\s*\(", text))) == sorted(block8.EXPORTS)
    for name in block8.EXPORTS:
        assert hasattr(B.lib, name)


def test_package_exports():
    import conv_bn_silu_amd as pkg
    for name in ("int8_linear", "PagedCache", "cache_write", "cache_read", "paged_attention"):
        assert getattr(pkg, name) is getattr(block8, name)


def test_bad_handles_come_first():
    null = [None] * 2
    assert B.lib.cbs_int8_linear(None, None, 1, None, None, None, None, 1, 1, 1, 0, 0, None, 0, None) == B.ERR_BAD_HANDLE
    fake = ctypes.c_void_p(0xdeadbeef)
    assert B.lib.cbs_cache_write(fake, None, None, 1, 1, None, 1, 1, None, 1, 0, None) == B.ERR_BAD_HANDLE
    assert B.lib.cbs_cache_read(fake, None, None, 1, *null, 0, None) == B.ERR_BAD_HANDLE
    assert B.lib.cbs_paged_attention(fake, None, 1, 1, None, None, 1, 1, None, None, 1, 1, 1, 0, 1.0, None, 1, None, 0,
                                     None) == B.ERR_BAD_HANDLE
    assert B.lib.cbs_paged_attention_workspace(None, 1, 1, 1, 1, 64, 16, 1) == -1


def test_linear_workspace():
    ws = B.lib.cbs_int8_linear_workspace
    assert ws(0, 8, 8) == 0 and ws(5, 8, 8) > 0
    for bad in ((-1, 8, 8), (1, 0, 8), (1, 8, 0), (1, 8, 131073), (2 ** 24 + 1, 8, 8)):
        assert ws(*bad) == -1


def cpu_cache():
    return torch.zeros(4, 2, 16, 64, dtype=torch.int8)


def test_binding_refuses_host_tensors_and_types():
    x, w, s = torch.zeros(2, 8), torch.zeros(3, 8, dtype=torch.int8), torch.zeros(3)
    with pytest.raises(ValueError):
        block8.int8_linear(x, w, s)
    with pytest.raises(TypeError):
        block8.int8_linear(x.double(), w, s)
    with pytest.raises(TypeError):
        block8.int8_linear(None, w, s)
    with pytest.raises(ValueError):
        block8.PagedCache(cpu_cache(), cpu_cache(), torch.zeros(4, 2, 16), torch.zeros(4, 2, 16))
    with pytest.raises(TypeError):
        block8.PagedCache(cpu_cache().to(torch.int16), cpu_cache())


def test_oracle_quantizes_by_the_definition():
    """Hand-checked: 254 / 127 = 2; halves go to even codes."""
    codes, s = O.quantize(torch.tensor([[254.0, 3.0, 5.0, -1.0, -3.0, 0.9]]))
    assert s.tolist() == [2.0] and codes.tolist() == [[127.0, 2.0, 2.0, 0.0, -2.0, 0.0]]
    codes, s = O.quantize(torch.zeros(1, 4))
    assert s.tolist() == [2.0 ** -126] and codes.tolist() == [[0.0] * 4]


def test_oracle_attention_against_a_library_softmax():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(n, 2, 16, generator=g) for n in (3, 9, 9))
    pages = torch.zeros(3, 2, 4, 16, dtype=O.F64), torch.zeros(3, 2, 4, 16, dtype=O.F64)
    table = torch.tensor([[2, 0, 1]])
    for t, src in zip(pages, (k, v)):
        for j in range(9):
            t[table[0, j // 4], :, j % 4] = src[j].double()
    out, _, mine = O.attention(q, *pages, table, [0, 3], [9], 0, 0.25, 0.0)
    mask = torch.arange(9)[None] <= torch.arange(6, 9)[:, None]
    z = torch.einsum("ihd,jhd->hij", q.double(), k.double()) * 0.25
    want = torch.einsum("hij,jhd->ihd", torch.softmax(z.masked_fill(~mask, float("-inf")), -1), v.double())
    assert bool(mine.all()) and torch.allclose(out, want, rtol=1e-12, atol=1e-12)
