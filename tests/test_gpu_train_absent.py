"""route_sort_train's backward pass where neither the weights nor the loss got a
gradient: it is entered, and gives the logits none."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
amr = pytest.importorskip("align_moe_route_amd")


class Cut(torch.autograd.Function):
    """A consumer whose backward pass has nothing for its inputs."""

    @staticmethod
    def forward(ctx, weights, loss):
        return weights.sum() + loss.sum()

    @staticmethod
    def backward(ctx, grad):
        return None, None


def test_both_gradients_absent(monkeypatch):
    x = torch.randn(20, 32, device="cuda", requires_grad=True)
    out, bal = amr.route_sort_train(x, torch.zeros(32, device="cuda"), 4, 1, 1, 16, balance_coef=0.1)
    entered = []
    out.weights.grad_fn.register_prehook(lambda grads: entered.append(len(grads)))

    def none(*args, **kw):
        raise AssertionError("a gradient of nothing was computed")

    monkeypatch.setattr(amr, "router_backward", none)
    Cut.apply(out.weights, bal.loss).backward()
    assert len(entered) == 1
    assert x.grad is None
