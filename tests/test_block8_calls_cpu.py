"""What the 8-bit block operators' Python classes promise, without a GPU."""
import pytest
import torch
from torch.autograd import forward_ad

from conv_bn_silu_amd import block8

pytestmark = pytest.mark.cpu


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale"])
def test_a_caches_tensors_cannot_be_replaced(name):
    """The kernels go on using the tensors that the cache was made of."""
    cache = object.__new__(block8.PagedCache)
    with pytest.raises(AttributeError):
        setattr(cache, name, None)


def test_tangents_are_refused():
    """A tangent would be dropped in silence, as a gradient would."""
    x, w, s = torch.zeros(2, 8), torch.zeros(3, 8, dtype=torch.int8), torch.zeros(3)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(ValueError, match="tangent"):
            block8.int8_linear(dual, w, s)
        with pytest.raises(ValueError, match="tangent"):
            block8.PagedCache(dual.view(1, 1, 2, 8), x.view(1, 1, 2, 8))
        with pytest.raises(ValueError, match="device tensor"):  # a tangent that no one asks for
            with forward_ad._set_fwd_grad_enabled(False):
                block8.int8_linear(dual, w, s)
    with pytest.raises(ValueError, match="gradient"):
        block8.int8_linear(x.requires_grad_(), w, s)
