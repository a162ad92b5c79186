"""Rows at the border of what the router's gradient and the trained weights are
defined for: NaN beside -infinity, and logits so low that FP32 scores vanish."""
import numpy as np
import pytest

from oracle import balance as ob
from test_gpu_balance import DT, check_backward, gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
amr = pytest.importorskip("align_moe_route_amd")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,k", [(64, 1), (64, 2), (64, 16), (64, 20), (700, 4), (700, 30), (2000, 3)])
def test_nan_pick_reaches_every_pick_of_its_row(E, k, dtype):
    """The weights share their sum, so one NaN logit makes each of them NaN, also
    where the other picks have the score zero."""
    rng = np.random.default_rng(E + k)
    x = torch.from_numpy(rng.standard_normal((7, E))).to(DT[dtype])
    ids = np.stack([np.sort(rng.choice(E, k, replace=False)) for _ in range(7)]).astype(np.int32)
    nan, inf = float("nan"), float("inf")
    for t, other in ((0, -inf), (1, nan), (2, None), (3, -1000.0), (4, inf)):
        if other is not None:
            x[t, ids[t]] = other
        x[t, ids[t, k // 2]] = nan
    x[5, ids[5]] = -inf  # no NaN: every weight zero
    check_backward(x, ids, None, None, balance=False)


def far_rows(M, E, dtype, rng):
    """Ordinary rows and, six of them at a time, rows whose scores are subnormal or
    zero in FP32, in every way that padding or a diverging router makes them."""
    x = torch.from_numpy(rng.standard_normal((M, E))).to(DT[dtype])
    low, inf = torch.finfo(DT[dtype]).min, float("inf")
    kind = torch.arange(M) % 12
    x[kind == 1] = low
    x[kind == 2] = -inf
    x[kind == 3] -= 1000
    x[kind == 4] -= 95
    x[kind == 5] -= 100
    x[kind == 6] = -inf
    x[kind == 6, 0] = -3000
    x[kind == 7] -= 84  # about the border
    x[kind == 8, : E // 2] = low  # a row that is not far: finite picks remain
    return x


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("M,E,k,n_group,topk_group", [(60, 48, 6, 4, 2), (601, 896, 16, 8, 4), (48, 64, 20, 1, 1),
                                                      (90, 512, 33, 1, 1), (36, 4096, 2, 8, 4)])
def test_trained_weights_of_far_rows(M, E, k, n_group, topk_group, dtype, masked):
    rng = np.random.default_rng(M + E)
    x = far_rows(M, E, dtype, rng)
    mask = rng.random(M) >= 0.3 if masked else None
    gw = rng.standard_normal((M, k)).astype(np.float32)
    bias = torch.zeros(E, device="cuda")
    leaf = x.cuda().requires_grad_()
    out, bal = amr.route_sort_train(leaf, bias, k, n_group, topk_group, 16, balance_coef=0.2, mask=gpu(mask))
    got, ids = out.weights.detach().double().cpu().numpy(), out.ids.cpu().numpy()
    x64 = x.double().numpy()
    want = ob.weights(x64, ids)
    assert np.isfinite(got).all() and bool(torch.isfinite(bal.loss.detach()).all())
    xk = np.take_along_axis(x64, ids.astype(np.int64), 1)
    top = xk.max(axis=1, keepdims=True)
    # far rows: a difference of logits d, exact where the weight is a normal number, then
    # an exponential (score_bound of d) and a sum of k of them; a weight below 2^-126 may
    # be zero.  Others: a rounding of each score (half a step, 2^-150 at least beside a sum
    # of exp(-87) or more), and the route's 2^-22.
    with np.errstate(invalid="ignore"):
        d = np.where(np.isneginf(top), 0.0, np.minimum(top - xk, 100.0))
    far = 2 * ob.score_bound(d) * want + (k + 2) * ob.U * want + 2.0 ** -126
    near = (2.0 ** -22 + 2 * ob.U) * want + (k + 1) * 2.0 ** -24
    assert (np.abs(got - want) <= np.where(top < -87, far, near)).all()
    plain = amr.route_sort(x.cuda(), bias, k, n_group, topk_group, 16)
    assert torch.equal(out.ids, plain.ids)
    keep = torch.from_numpy(top[:, 0] >= -87).cuda()
    assert bool(keep.any()) and bool((~keep).any())
    assert torch.equal(out.weights[keep], plain.weights[keep])  # the route's own, bit for bit
    # the gradient is that of these weights
    (out.weights * gpu(gw)).sum().backward()
    ref, size = ob.backward(x64, ids, 1.0, 1.0, gw, None, None, mask)
    err = ob.grad_bound(200.0, E) * size + ob.FLUSH
    half = 2.0 ** -8 if dtype == "bf16" else ob.U
    assert (np.abs(leaf.grad.double().cpu().numpy() - ref) <= err + half * (np.abs(ref) + err)).all()


def test_far_weights_in_many_tokens_and_dropped_picks():
    """More tokens than the launch's workgroups hold at once; picks outside [0, E)
    weigh nothing; a NaN reaches its whole row."""
    M, E, k = 70001, 24, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, E, device="cuda", generator=g) - 200.0
    x[1::3] += 200.0
    x[6, :] = float("nan")
    ids = torch.randint(-1, E + 1, (M, k), dtype=torch.int32, device="cuda", generator=g)
    ids[3] = E
    ids[6] = torch.arange(k)
    w = torch.full((M, k), 7.0, device="cuda")
    assert amr.lib().moe_route_far_weights(x.data_ptr(), 0, ids.data_ptr(), M, E, k, w.data_ptr(),
                                           torch.cuda.current_stream().cuda_stream) == amr.MRS_OK
    got, ids, x64 = w.double().cpu().numpy(), ids.cpu().numpy(), x.double().cpu().numpy()
    want = ob.weights(x64, ids)
    near = (np.take_along_axis(x64, np.clip(ids, 0, E - 1).astype(np.int64), 1) >= -87) & (ids >= 0) & (ids < E)
    near = near.any(axis=1)
    assert (got[near] == 7.0).all()
    assert np.isnan(got[6]).all()
    far = ~near
    far[6] = False
    assert far.sum() > 40000 and (got[3] == 0).all()
    assert (np.abs(got - want)[far] <= (2 * ob.score_bound(20.0) + (k + 2) * ob.U) * want[far]).all()
