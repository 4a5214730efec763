"""Refusals of the calls for positions that need no GPU."""
import pytest

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("name", ["dq", "q", "dk", "k", "q_weight", "k_weight"])
def test_backward_refuses_what_requires_a_gradient(i8l, name):
    """The gradient has no gradient of its own: a tensor that requires one would end the graph
    unnoticed.  Under no_grad the call goes on (here to the check for a GPU)."""
    x = torch.zeros((2, 4, 64), dtype=torch.float16)
    w = torch.ones(64, dtype=torch.float16)
    a = dict(dq=x, q=x, dk=x, k=x, q_weight=w, k_weight=w)
    a[name] = a[name].clone().requires_grad_()
    pos = torch.zeros(2, dtype=torch.int32)
    dq = a.pop("dq")
    with pytest.raises(RuntimeError, match="gradient"):
        i8l.rotate_heads_backward(dq, pos, **a)
    with torch.no_grad(), pytest.raises(ValueError, match="on a GPU"):
        i8l.rotate_heads_backward(dq, pos, **a)
