"""Serving operators, edges that need no GPU."""
import ctypes

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


def test_partial_results_are_aligned(i8l):
    """Attention's workspace holds (maximum, sum) of every row and split, filled up to 16
    bytes, then their outputs, which are written 16 bytes at a time."""
    from test_serving_abi import cache_struct

    for heads, n, max_len, splits in ((1, 1, 700, 3), (5, 3, 700, 3), (1, 1, 500, 2)):
        for D in (16, 64, 256):
            c = cache_struct(heads=heads, head_dim=D)
            count = n * heads * splits
            need = i8l.lib().i8l_attention_workspace_bytes(ctypes.byref(c), n, heads, 1, max_len, 0)
            assert need == 4 * ((2 * count + 3) // 4 * 4 + count * D)


def test_tensors_that_require_a_gradient_are_refused(i8l):
    """No result without a gradient where one is expected; under no_grad() the call goes on
    (here to the next refusal, of tensors that are not on a GPU)."""
    X, W = torch.zeros((2, 64)).half(), torch.zeros(64).half()
    G = torch.zeros((2, 64)).half().requires_grad_()
    f = torch.ones(2, requires_grad=True)
    kv = torch.zeros((1, 1, 16)).half().requires_grad_()
    refused = [lambda: i8l.rmsnorm_quant(G, W), lambda: i8l.rmsnorm_quant(X, W, residual=G),
               lambda: i8l.rmsnorm_quant(X, torch.nn.Parameter(W)),
               lambda: i8l.linear_codes(X, f, X, W), lambda: i8l.linear_codes(X, W, X, f),
               lambda: i8l.linear_codes(X, W, X, W, bias=G), lambda: i8l.cache_write(None, kv, X, X, X),
               lambda: i8l.cache_write(None, X, kv, X, X),
               lambda: i8l.cache_attention(kv, None, X, X),
               lambda: i8l.cache_attention(X, None, X, X, alibi=f)]
    for call in refused:
        with pytest.raises(RuntimeError, match="no gradients"):
            call()
    with torch.no_grad():
        for call in refused:
            with pytest.raises((TypeError, ValueError)):
                call()
