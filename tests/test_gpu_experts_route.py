"""experts_train with a route that does not belong to its weights: refused where that is
known, NaN for the tokens that it concerns where it is not; and with buffers that a later
route is written into before the backward pass."""
import numpy as np
import pytest
import torch

import align_moe_route_amd as amr
from experts_cases import Routed, ids_of, normal

pytestmark = pytest.mark.gpu
H, I, block = 40, 24, 32


def weights(E):
    return normal((E, 2 * I, H), torch.bfloat16, 2, H ** -0.5), normal((E, H, I), torch.bfloat16, 3, I ** -0.5)


@pytest.mark.parametrize("M", [1, 50])
def test_route_of_more_experts(M):
    E, k = 16, 4
    x, logits, bias = normal((M, H), torch.bfloat16, 1), normal((M, E), torch.float32, 4), torch.zeros(E, device="cuda")
    hidden = normal((M, H), torch.bfloat16, 5)
    routes = [amr.route_sort(logits, bias, k, 4, 2, block), amr.route_sort_train(logits, bias, k, 4, 2, block)[0],
              amr.route_sort_static(logits, bias, k, 4, 2, block),
              amr.gate_route_sort(hidden, normal((E, H), torch.bfloat16, 6), bias, k, 4, 2, block)[1]]
    routes.append(amr.route_sort(logits, bias, k, 4, 2, block, out=amr.RouteSortOutput(*(t.clone() for t in routes[0]))))
    for route in routes:
        assert (route.experts, route.block) == (E, block)
        amr.experts_train(x, *weights(E), route, block)
        with pytest.raises(ValueError):
            amr.experts_train(x, *weights(E // 2), route, block)
        with pytest.raises(ValueError):
            amr.experts_train(x, *weights(E), route, block // 2)
    local = amr.route_sort(logits, bias, k, 4, 2, block, local=(3, 6))
    amr.experts_train(x, *weights(6), local, block)
    with pytest.raises(ValueError):
        amr.experts_train(x, *weights(5), local, block)


def test_route_of_no_tensors():
    x, v = normal((4, H), torch.bfloat16, 1), torch.ones(4, 2, device="cuda")
    for bad in (None, 7, torch.zeros(4), torch.zeros(999, dtype=torch.int32)):
        with pytest.raises(ValueError):
            amr.experts_train(x, *weights(3), amr.RouteSortOutput(None, v, bad, bad, bad), block)


@pytest.mark.parametrize("M,E,held", [(3, 12, 7), (40, 9, 6)])
def test_route_made_by_hand(M, E, held):
    """Weights of the first experts only: the others' tokens are NaN, with their gradients."""
    k = 2
    ids = ids_of(M, E, k, 1)
    ids[0] = 0, 1
    ids[1] = 0, E - 1
    r = Routed(ids, E, block)
    w = weights(E)
    v, dout = torch.rand(M, k, device="cuda"), normal((M, H), torch.bfloat16, 7)

    def run(*w):
        leaves = [t.clone().requires_grad_() for t in (normal((M, H), torch.bfloat16, 4), *w, v)]
        out = amr.experts_train(*leaves[:3], amr.RouteSortOutput(r.ids, leaves[3], *r.meta), block)
        out.backward(dout)
        return [out, *(t.grad for t in leaves)]
    out, dx, d_up, d_down, dv = run(*(t[:held].contiguous() for t in w))
    want = run(*w)
    gone = torch.from_numpy((ids >= held)).cuda()
    token = gone.any(1)
    assert out[token].isnan().all() and dx[token].isnan().all() and dv[gone].isnan().all()
    assert torch.equal(out[~token], want[0][~token]) and torch.equal(dx[~token], want[1][~token])
    assert torch.equal(dv[~gone], want[4][~gone])
    assert torch.equal(d_up, want[2][:held]) and torch.equal(d_down, want[3][:held])
    assert np.array_equal(token.cpu().numpy(), (ids >= held).any(1)) and 0 < int(token.sum()) < M


@pytest.mark.parametrize("M", [2, 30])
def test_longer_buffers(M):
    """Metadata in buffers that are longer than these sizes need, and than any could."""
    E, k = 5, 2
    r = Routed(ids_of(M, E, k, 1), E, block)
    longer = [torch.cat([r.meta[0], torch.full((700,), 3, dtype=torch.int32, device="cuda")]),
              torch.cat([r.meta[1], torch.full((9,), 77, dtype=torch.int32, device="cuda")]), r.meta[2]]
    w, v, dout = weights(E), torch.rand(M, k, device="cuda"), normal((M, H), torch.bfloat16, 7)

    def run(meta):
        leaves = [t.clone().requires_grad_() for t in (normal((M, H), torch.bfloat16, 4), *w, v)]
        out = amr.experts_train(*leaves[:3], amr.RouteSortOutput(r.ids, leaves[3], *meta), block)
        out.backward(dout)
        return [out, *(t.grad for t in leaves)]
    for a, b in zip(run(longer), run(r.meta)):
        assert a.isfinite().all() and torch.equal(a, b)


@pytest.mark.parametrize("which", ["route", "static", "gate", "sort"])
def test_route_written_over_before_the_backward_pass(which):
    """The backward pass of the first layer would read the second one's metadata."""
    M, E, k = 20, 16, 4
    x, bias = normal((M, H), torch.bfloat16, 1).requires_grad_(), torch.zeros(E, device="cuda")
    logits = [normal((M, E), torch.float32, 4 + i) for i in range(2)]
    gate = [normal((E, H), torch.bfloat16, 6 + i) for i in range(2)]
    ids = [torch.from_numpy(ids_of(M, E, k, 8 + i)).cuda() for i in range(2)]

    def layer(i, buf):
        if which == "route":
            return amr.route_sort(logits[i], bias, k, 4, 2, block, out=buf)
        if which == "static":
            return amr.route_sort_static(logits[i], bias, k, 4, 2, block, out=buf)
        if which == "gate":
            return amr.gate_route_sort(x.detach(), gate[i], bias, k, 4, 2, block, out=buf)[1]
        meta = amr.sort_from_ids(ids[i], E, block, out=buf and amr.SortOutput(*buf[2:]))
        return amr.RouteSortOutput(ids[i], torch.full((M, k), 0.25, device="cuda"), *meta)
    first = layer(0, None)
    out = amr.experts_train(x, *weights(E), first, block)
    layer(1, None)  # another call in buffers of its own takes nothing away
    out.sum().backward(retain_graph=True)
    layer(1, first)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()
    out = amr.experts_train(x, *weights(E), first, block)  # of what the buffers hold now
    out.sum().backward()
