"""route_sort_train under autograd, and the example that trains a router over
4-bit experts."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import balance as ob

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
amr = pytest.importorskip("align_moe_route_amd")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("use", ["both", "weights", "loss", "none"])
def test_gradients_reach_the_logits(dtype, use):
    rng = np.random.default_rng(1)
    M, E, k, coef = 60, 48, 6, 0.2
    x = torch.from_numpy(rng.standard_normal((M, E))).to(dtype)
    off = np.array([0, 7, 7, 41, 60], np.int32)
    mask = rng.random(M) >= 0.2
    gw = rng.standard_normal((M, k)).astype(np.float32)
    leaf = x.cuda().requires_grad_()
    scale = torch.ones(E, device="cuda", dtype=dtype)
    out, bal = amr.route_sort_train(leaf * scale, torch.zeros(E, device="cuda"), k, 4, 2, 16, balance_coef=coef,
                                    seq_offsets=torch.from_numpy(off).cuda(), mask=torch.from_numpy(mask).cuda())
    plain = amr.route_sort(x.cuda(), torch.zeros(E, device="cuda"), k, 4, 2, 16)
    npp = int(plain.num_post_pad)
    assert torch.equal(out.ids, plain.ids) and torch.equal(out.weights, plain.weights)
    assert torch.equal(out.sorted_ids[:npp], plain.sorted_ids[:npp])
    if use == "none":
        (leaf.sum() * 2).backward()
        assert bool((leaf.grad == 2).all())
        return
    total = 0.0
    if use != "loss":
        total = total + (out.weights * torch.from_numpy(gw).cuda()).sum()
    if use != "weights":
        total = total + 1.5 * bal.loss.sum()
    total.backward()
    x64, ids = x.double().numpy(), out.ids.cpu().numpy()
    loss, counts, _, _ = ob.balance(x64, ids, coef, off, mask)
    ref, size = ob.backward(x64, ids, float(np.float32(coef)), 1.5, gw if use != "loss" else None,
                            counts if use != "weights" else None, off, mask)
    err = ob.grad_bound(np.abs(x64).max(), E) * size + ob.FLUSH
    half = 2.0 ** -8 if dtype == torch.bfloat16 else ob.U
    got = leaf.grad.double().cpu().numpy()
    assert (np.abs(got - ref) <= err + half * (np.abs(ref) + err)).all()
    assert abs(float(bal.loss.detach()) - loss) <= 1e-4 * abs(loss)


def test_example_trains():
    spec = importlib.util.spec_from_file_location("finetune_router", os.path.join(ROOT, "examples", "finetune_router.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    history = ex.run(steps=60, report=None)
    first, last = np.mean([d for d, _ in history[:4]]), np.mean([d for d, _ in history[-4:]])
    assert np.isfinite(history).all() and last < 0.8 * first


def test_experts_match_dense_products():
    """Both grouped products of the example against dense ones on the decoded weights."""
    from oracle import mxfp4 as om
    spec = importlib.util.spec_from_file_location("finetune_router", os.path.join(ROOT, "examples", "finetune_router.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    g = torch.Generator(device="cuda").manual_seed(3)
    M, E, k, hidden, inner, block = 40, 6, 2, 160, 64, 32
    experts = ex.FrozenExperts(E, hidden, inner, g)
    x = torch.randn(M, hidden, device="cuda", generator=g).bfloat16()
    route = amr.route_sort(torch.randn(M, E, device="cuda", generator=g), torch.zeros(E, device="cuda"), k, 1, 1, block)
    out = experts(x, route, k, block).double().cpu().numpy()
    w1 = om.decode(experts.w1.codes.cpu().numpy(), experts.w1.scales.cpu().numpy())
    w2 = om.decode(experts.w2.codes.cpu().numpy(), experts.w2.scales.cpu().numpy())
    xq = om.quantize(x.double().cpu().numpy())
    xv = om.decode(xq[0], xq[1])
    ids = route.ids.cpu().numpy()
    for t in range(M):
        for j in range(k):
            h = torch.from_numpy(xv[t] @ w1[ids[t, j]].T)
            b = h.bfloat16().float()
            act = (torch.nn.functional.silu(b[:inner].bfloat16()) * b[inner:].bfloat16()).double().numpy()
            q = om.quantize(act[None])
            want = om.decode(q[0], q[1])[0] @ w2[ids[t, j]].T
            # a BF16 rounding of h or of the activation that falls the other way moves a
            # value by 2^-7 and may move its 4-bit level by one step (a third at most)
            size = np.abs(om.decode(q[0], q[1])[0]) @ np.abs(w2[ids[t, j]]).T
            assert (np.abs(out[t, j] - want) <= 0.1 * size + 1e-6).all()
