"""The binding's cache object (CPU)."""

import pytest

sv = pytest.importorskip("adaptive_draft_verification_amd",
                         reason="libspecverify.so not built (python adaptive_draft_verification_amd/build.py)")


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale", "device", "n_kv_heads",
                                  "head_dim", "page_size"])
def test_cache_fields_cannot_be_exchanged(name):
    """The library's struct holds the addresses taken at the start: a new tensor would not be
    the one that is read."""
    cache = object.__new__(sv.PagedCache)
    with pytest.raises(AttributeError):
        setattr(cache, name, None)
