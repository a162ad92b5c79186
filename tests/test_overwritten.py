"""Buffers that a call writes again: autograd learns of it."""
import pytest

import align_moe_route_amd as amr

torch = pytest.importorskip("torch")


def test_saved_tensor_is_not_read_again():
    a, b, x = torch.ones(3), torch.ones(2), torch.ones(3, requires_grad=True)
    y = (x * a).sum()
    amr._overwritten(b)
    y.backward(retain_graph=True)
    with torch.no_grad():
        amr._overwritten(a, b)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_tensors_of_inference_mode():
    with torch.inference_mode():
        t = torch.zeros(2)
        amr._overwritten(t)
    amr._overwritten(t)
