"""Serving operators, edges that need no GPU."""
import pytest

torch = pytest.importorskip("torch")


def test_a_cache_does_not_change_its_tensors(i8l):
    """The library holds a cache's pointers: assigning or deleting a tensor would leave it
    with memory that may be freed."""
    c = i8l.KVCache.__new__(i8l.KVCache)
    for name in ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail", "heads",
                 "page_size", "head_dim", "dtype", "device", "n_pages", "n_slots"):
        with pytest.raises(AttributeError):
            setattr(c, name, torch.zeros(1))
        with pytest.raises(AttributeError):
            delattr(c, name)
