"""The serving operators' binding, without a GPU."""

import pytest

import nvfp4_quantized_matmul_amd as nv


@pytest.mark.parametrize("name", ["k", "v", "k_scales", "v_scales", "pages", "heads", "page", "dim", "device", "index"])
def test_a_cache_cannot_be_renamed(name):
    """The kernels go by the addresses and sizes that a cache was made with: an
    assigned tensor would be checked in their place, and not used."""
    cache = object.__new__(nv.KVCache)      # without tensors, which have to be on a GPU
    with pytest.raises(AttributeError):
        setattr(cache, name, 0)
    with pytest.raises(AttributeError):
        delattr(cache, name)
