"""balance_loss on logits that require a gradient."""
import numpy as np
import pytest

from oracle import balance as ob
from test_gpu_balance import DT, gpu, make

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
amr = pytest.importorskip("align_moe_route_amd")


def buffers(B, E):
    i32 = dict(dtype=torch.int32, device="cuda")
    return amr.BalanceOutput(torch.empty(1, device="cuda"), torch.empty(B, E, **i32), torch.empty(B + 1, **i32),
                             torch.empty(B, E, device="cuda"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,E,k,B,masked", [(1, 8, 2, 1, 0), (333, 61, 7, 5, 0.2), (700, 500, 8, 1, 0), (90, 1500, 4, 3, 0.3)])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("other_stream", [False, True])
def test_loss_carries_its_gradient(M, E, k, B, masked, dtype, given, other_stream):
    x, ids, off, mask = make(M, E, k, B, masked, dtype, M + E)
    coef, up = 0.3, 1.7
    leaf = x.cuda().requires_grad_()
    args = dict(seq_offsets=gpu(off), mask=gpu(mask))
    gi = gpu(ids)
    plain = amr.balance_loss(x.cuda(), gi, coef, **args)
    assert plain.loss.grad_fn is None
    out = buffers(B, E) if given else None
    stream = torch.cuda.Stream() if other_stream else None
    torch.cuda.synchronize()
    bal = amr.balance_loss(leaf, gi, coef, out=out, stream=stream, **args)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(plain, bal))
    assert bal.loss.requires_grad and not bal.shares.requires_grad
    if given:
        assert out.loss.grad_fn is None and out.loss.data_ptr() == bal.loss.data_ptr()
        for t in out[1:]:  # the next step writes them before this one's backward pass
            t.fill_(3)
    task = (leaf.float() ** 2).sum() * 0.5
    (task + up * bal.loss.sum()).backward()
    x64 = x.double().numpy()
    counts = ob.balance(x64, ids, coef, off, mask)[1]
    ref, size = ob.backward(x64, ids, float(np.float32(coef)), float(np.float32(up)), None, counts, off, mask)
    half = 2.0 ** -8 if dtype == "bf16" else ob.U
    err = ob.grad_bound(np.abs(x64).max(), E) * size + ob.FLUSH
    # the two terms are rounded to the logits' type each, and so is their sum
    tol = err + half * (np.abs(ref) + err) + half * np.abs(x64) + half * 1.01 * (np.abs(ref) + np.abs(x64) + err)
    assert (np.abs(leaf.grad.double().cpu().numpy() - (ref + x64)) <= tol).all()


def test_where_there_is_nothing_to_train():
    x, ids, _, _ = make(40, 30, 3, 1, 0, "f32", 1)
    leaf = x.cuda().requires_grad_()
    with torch.no_grad():
        bal = amr.balance_loss(leaf, gpu(ids))
    assert not bal.loss.requires_grad
    bal = amr.balance_loss(leaf, gpu(ids))
    bal.loss.mul_(2.0)  # a tensor as any other
    bal.loss.sum().backward()
    want = amr.router_backward(x.cuda(), gpu(ids), balance=amr.balance_loss(x.cuda(), gpu(ids)),
                               grad_loss=torch.full((1,), 2.0, device="cuda"))
    assert torch.equal(leaf.grad, want)


def test_training_step_captured_with_the_calls_themselves():
    """The form that a captured step takes, on logits that a model has made."""
    M, E, k = 200, 64, 4
    x, ids, _, _ = make(M, E, k, 1, 0, "f32", 2)
    gx, gi = x.cuda(), gpu(ids)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    leaf = gx.clone().requires_grad_()
    out, grad = buffers(1, E), torch.empty_like(gx)
    with torch.cuda.stream(s):
        amr.balance_loss(gx, gi, 0.1, out=out)  # the stream's workspace
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            bal = amr.balance_loss(leaf, gi, 0.1, out=out)
            amr.router_backward(leaf, gi, balance=bal, coef=0.1, out=grad)
    for i in range(4):
        with torch.no_grad():
            leaf.copy_(torch.randn(M, E, device="cuda"))
        graph.replay()
        want = amr.balance_loss(leaf.detach(), gi, 0.1)
        wgrad = amr.router_backward(leaf.detach(), gi, balance=want, coef=0.1)
        torch.cuda.synchronize()
        assert all(torch.equal(p.detach(), q) for p, q in zip(bal, want)) and torch.equal(grad, wgrad)
