"""The 4-bit values of tensors that require a gradient."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
amr = pytest.importorskip("align_moe_route_amd")


def test_values_do_not_drop_a_gradient():
    x = torch.randn(6, 40, device="cuda")
    leaf, v = x.clone().requires_grad_(), torch.full_like(x, 7.0)
    for bad in (lambda: amr.mxfp4_quantize(leaf, values=v), lambda: amr.mxfp4_quantize(leaf * 2, values=v),
                lambda: amr.mxfp4_quantize(x, values=v.clone().requires_grad_())):
        with pytest.raises(ValueError, match="gradient"):
            bad()
    assert bool((v == 7.0).all())  # nothing was launched
    q = amr.mxfp4_quantize(leaf)  # codes are whole numbers: nothing to lose
    with torch.no_grad():
        q2 = amr.mxfp4_quantize(leaf, values=v)
    assert torch.equal(q.codes, q2.codes) and torch.equal(q.scales, q2.scales)
    w = torch.full_like(x, 7.0)
    amr.mxfp4_quantize(leaf.detach(), values=w)
    assert torch.equal(v, w)
    y = leaf + (w - leaf.detach())  # the documented form: the gradient passes the rounding by
    # two roundings, of w - x and of the sum
    assert bool(((y.detach() - w).abs() <= 2.0 ** -23 * (x.abs() + w.abs())).all())
    (y * 3).sum().backward()
    assert bool((leaf.grad == 3).all())
