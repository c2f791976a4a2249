"""What the 8-bit block operators' Python classes promise, without a GPU."""
import pytest

from conv_bn_silu_amd import block8

pytestmark = pytest.mark.cpu


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale"])
def test_a_caches_tensors_cannot_be_replaced(name):
    """The kernels go on using the tensors that the cache was made of."""
    cache = object.__new__(block8.PagedCache)
    with pytest.raises(AttributeError):
        setattr(cache, name, None)
