"""A step's other operators without a GPU: the header, refusals, the oracle, the frequencies."""
import ctypes
import math
import os
import re

import pytest
import torch
from torch.autograd import forward_ad

from conv_bn_silu_amd import binding as B
from conv_bn_silu_amd import block8, step
import step_oracle as S

pytestmark = pytest.mark.cpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F64 = torch.float64


def test_header_and_binding_agree():
    text = open(os.path.join(ROOT, "include", "cbs_step.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    assert sorted(set(re.findall(r"\b(cbs_\w+)\s*\(", text))) == sorted(step.EXPORTS)
    for name in step.EXPORTS:
        assert hasattr(B.lib, name)


def test_package_exports():
    import conv_bn_silu_amd as pkg
    for name in pkg._STEP:
        assert getattr(pkg, name) is getattr(step, name)
    assert pkg.Rows8 is block8.Rows8


def test_bad_handles_come_first():
    fake, null = ctypes.c_void_p(0xdeadbeef), None
    assert B.lib.cbs_add_rms_norm(null, null, 1, null, 1, 0, null, 0, 1e-6, null, 1, null, 0, 1, 1, 0, null) == B.ERR_BAD_HANDLE
    assert B.lib.cbs_rotary_apply(fake, null, null, 1, 1, null, 1, 1, 2, 0, null, 1, 1, null) == B.ERR_BAD_HANDLE
    assert B.lib.cbs_rotary_cache_write(fake, null, null, null, 1, 1, null, 1, 1, null, 1, 1, null, null, 1, 1, 0, null, 1, 1,
                                        null) == B.ERR_BAD_HANDLE
    assert B.lib.cbs_grow_pages(null, null, null, 1, 1, null, null, 1, 1, null, null, null, null, 0, null) == B.ERR_BAD_HANDLE
    assert B.lib.cbs_release_pages(fake, null, null, 1, 1, null, null, 1, null, 0, null) == B.ERR_BAD_HANDLE
    assert B.lib.cbs_int8_linear_rows(null, null, null, null, null, null, 1, 1, 1, 0, 0, null, 0, null) == B.ERR_BAD_HANDLE


def test_sizes():
    rows, grow, release = B.lib.cbs_rows8_bytes, B.lib.cbs_grow_pages_workspace, B.lib.cbs_release_pages_workspace
    # scales of 16 rows, codes of 16 rows by 128
    assert rows(0, 5) == 0 and rows(1, 1) == 16 * (4 + 128) and rows(17, 129) == 32 * (4 + 256)
    for bad in ((-1, 8), (1, 0), (1, 131073), (2 ** 24 + 1, 8)):
        assert rows(*bad) == -1
    for bad in ((-1, 8, 8), (1, 0, 8), (1, 8, 131073)):
        assert B.lib.cbs_int8_linear_rows_workspace(*bad) == -1
    assert B.lib.cbs_int8_linear_rows_workspace(8192, 8192, 8192) == 0
    assert grow(0, 0) == 0 and grow(1, 1 << 30) >= 0 and grow(65536, 0) > 0
    assert grow(-1, 0) == grow(0, -1) == grow(65537, 0) == grow(0, (1 << 30) + 1) == -1
    assert release(0, 0) == 0 and release(65536, 1) > 0 and release(1, 2 ** 31 - 1) > 0
    assert release(-1, 0) == release(0, -1) == release(65537, 1) == release(1, 2 ** 31) == -1


def test_binding_refuses_host_tensors_and_types():
    x = torch.zeros(2, 3, 8)
    i32 = torch.zeros(2, dtype=torch.int32)
    f = torch.zeros(4, dtype=F64)
    for call in (lambda: step.add_rms_norm(x), lambda: step.rotary(x, i32, f),
                 lambda: step.PagePool(i32, torch.zeros(3, dtype=torch.int32), 16),
                 lambda: step.PagePool.full(4, 16, device="cpu"),
                 lambda: block8.int8_linear(block8.Rows8(torch.zeros(0, dtype=torch.int8), (0, 4), torch.float32),
                                            torch.zeros(3, 4, dtype=torch.int8), torch.zeros(3))):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    for call in (lambda: step.add_rms_norm(x.double()), lambda: step.add_rms_norm(None), lambda: step.rotary(x.int(), i32, f),
                 lambda: step.PagePool(i32.long(), i32, 16)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(AttributeError):
        object.__new__(step.PagePool).free = i32


def test_gradients_and_tangents_are_refused():
    x = torch.zeros(2, 8)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(ValueError, match="tangent"):
            step.add_rms_norm(dual)
        with pytest.raises(ValueError, match="tangent"):
            step.rotary(dual.view(2, 1, 8), None, None)
    with pytest.raises(ValueError, match="gradient"):
        step.add_rms_norm(x.requires_grad_())


def test_rows8_layout():
    """A buffer laid out by hand reads back."""
    M, K, R, Kp = 5, 130, 16, 256
    codes = torch.randint(-127, 128, (M, K), dtype=torch.int8)
    buffer = torch.full((R * 4 + R * Kp,), 77, dtype=torch.int8)
    scale = torch.rand(M) + 0.5
    buffer[:R * 4].view(torch.float32)[:M] = scale
    for m in range(M):
        for k in range(Kp):
            buffer[R * 4 + ((k // 64) * R + m) * 64 + k % 64] = codes[m, k] if k < K else 0
    rows = block8.Rows8(buffer, (5, 130), torch.bfloat16)
    assert buffer.numel() == B.lib.cbs_rows8_bytes(M, K)
    assert torch.equal(rows.codes, codes) and torch.equal(rows.scale, scale)
    assert torch.equal(rows.dequantize(torch.float32), codes.float() * scale[:, None])
    assert rows.dequantize().dtype == torch.bfloat16
    wide = block8.Rows8(buffer, (1, 5, 130), torch.bfloat16)
    assert wide.codes.shape == (1, 5, 130) and wide.scale.shape == (1, 5)


def test_frequencies():
    plain = step.rotary_frequencies(8, 10000.0, device="cpu")
    assert plain.dtype == F64 and torch.allclose(plain, torch.tensor([1, 0.1, 0.01, 0.001], dtype=F64), rtol=1e-15)
    assert torch.allclose(step.rotary_frequencies(8, scaling="positions", factor=4.0, device="cpu"), plain / 4, rtol=1e-15)
    based = step.rotary_frequencies(8, scaling="base", factor=4.0, device="cpu")
    assert float(based[0]) == 1 and math.isclose(float(based[-1]), float(plain[-1]) / 4, rel_tol=1e-12)
    # 1000 tokens: 159 turns of the fastest pair, 15.9, 1.59 and 0.159
    turns = step.rotary_frequencies(8, scaling="turns", factor=4.0, context=1000, low=1.0, high=4.0, device="cpu")
    assert torch.equal(turns[:2], plain[:2]) and math.isclose(float(turns[3]), float(plain[3]) / 4, rel_tol=1e-12)
    share = (1000 * 0.01 / (2 * math.pi) - 1) / 3
    assert math.isclose(float(turns[2]), 0.01 * (share + (1 - share) / 4), rel_tol=1e-12)
    # pair numbers: 4 turns at 8 log(1000 / 8 pi) / (2 log 10000) = 1.60, 1 turn at 2.20: from pair 1 to pair 3
    pairs = step.rotary_frequencies(8, scaling="pairs", factor=4.0, context=1000, low=1.0, high=4.0, device="cpu")
    assert torch.equal(pairs[:2], plain[:2]) and math.isclose(float(pairs[3]), float(plain[3]) / 4, rel_tol=1e-12)
    assert math.isclose(float(pairs[2]), 0.01 * (0.5 + 0.5 / 4), rel_tol=1e-12)
    for bad in (dict(dim=7), dict(dim=0), dict(base=1.0), dict(factor=0.5), dict(scaling="x"), dict(scaling="turns"),
                dict(dim=2, scaling="base"), dict(scaling="pairs", context=100, low=4.0, high=1.0)):
        with pytest.raises(ValueError):
            step.rotary_frequencies(**{**dict(dim=8, device="cpu"), **bad})


@pytest.mark.parametrize("dim,context", [(8, 131072), (64, 131072), (128, 65536), (128, 131072), (128, 4096), (64, 300)])
def test_frequencies_by_pairs_past_the_last_pair(dim, context):
    """The share of each pair by the rule, one at a time; in long contexts the pair that turns `low` times is not there, and
    the slowest keeps a share."""
    low, high, factor, base = 1.0, 32.0, 4.0, 10000.0
    got = step.rotary_frequencies(dim, base, "pairs", factor, context, low, high, device="cpu")

    def number(turns):  # where base^(-2 i / dim) * context is that many whole turns
        return math.log(context / (2 * math.pi * turns)) / math.log(base) * dim / 2

    first, last = max(0, math.floor(number(high))), math.ceil(number(low))
    assert last < dim
    for i in range(dim // 2):
        f = base ** (-2 * i / dim)
        share = min(1.0, max(0.0, (last - i) / (last - first)))
        assert math.isclose(float(got[i]), f * share + f / factor * (1 - share), rel_tol=1e-12), i
    slowest = base ** (2 / dim - 1)
    if context * slowest > 2 * math.pi * low:
        assert last > dim // 2 - 1 and float(got[-1]) > 1.05 * slowest / factor


def test_oracle_norm_and_rotation():
    """Hand-checked: rows of 3 and 4; quarter turns."""
    y, _, h = S.norm(torch.tensor([[1.0, 5.0]]), torch.tensor([2.0, 1.0]), torch.tensor([[2.0, -1.0]]), 0.0)
    assert h.tolist() == [[3.0, 4.0]] and torch.allclose(y, torch.tensor([[6.0, 4.0]], dtype=F64) / math.sqrt(12.5), rtol=1e-15)
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    f = torch.tensor([math.pi / 2, math.pi], dtype=F64)
    half, _ = S.rotate(x, torch.tensor([1]), f, False, 1.0)
    assert torch.allclose(half, torch.tensor([[[-3.0, -2.0, 1.0, -4.0, 9.0]]], dtype=F64), atol=1e-15)
    near, _ = S.rotate(x, torch.tensor([-1]), f, True, 2.0)
    assert torch.allclose(near, torch.tensor([[[4.0, -2.0, -6.0, -8.0, 9.0]]], dtype=F64), atol=1e-14)


def test_oracle_pages():
    """Hand-checked: two sequences of 3 and 0 tokens, pages of 2."""
    s = S.Pages([7, 5, 6, 9, 1, 0, 0, 0, 0, 0], 5, 2, [[3, 2, -1, -1], [-1, -1, -1, -1]], [3, 0])
    starts, slots, positions = s.grow([2, 3], 6)
    # 3 + 2 tokens: the last of page 2, then page 1; three of the other: pages 9 and 6
    assert starts == [0, 2, 5] and slots == [5, 2, 18, 19, 12, -1] and positions == [3, 4, 0, 1, 2, 0]
    assert s.table == [[3, 2, 1, -1], [9, 6, -1, -1]] and s.lens == [5, 3] and s.counts() == [2, 0, 0]
    s.release([3, 0])
    assert s.below[:5] == [7, 5, 6, 9, 1] and s.counts() == [5, 0, 0] and s.lens == [3, 0]
    starts, slots, positions = s.grow([9, 11], 12)  # the first would pass its row, the second the batch
    assert starts == [0, 9, 12] and slots == [-1] * 12 and s.counts() == [5, 0, 2]
    s.table[1].append(-1)
    starts, slots, positions = s.grow([4, 9], 13)  # two pages for the first, then three of five
    assert slots == [5, 2, 3, 18, *[-1] * 9] and s.counts() == [3, 2, 1] and s.lens == [7, 0]
