"""Experts' operators on subnormal values, infinities in rows of any sizes, the weights'
gradient of an expert with many rows by its large tiles, gradients that are broadcast.

Tolerances as in the other tests of these calls: half a step of the output's type, and
C / 16 + 16 FP32 roundings of 2^-23 of a sum's magnitudes."""
import numpy as np
import pytest
import torch

import align_moe_route_amd as amr
from experts_cases import HALF, Routed, check, f64, ids_of, normal
from oracle import experts as orc

pytestmark = pytest.mark.gpu


def steps(C):
    return C / 16 + 16


def subnormal(shape, t, seed):
    """Whole multiples, up to 60, of the type's smallest value."""
    g = torch.Generator().manual_seed(seed)
    least = 2.0 ** -24 if t == torch.float16 else 2.0 ** -133
    return (torch.randint(-60, 61, shape, generator=g).double() * least).to(t).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("K,N", [(200, 72), (203, 77)])
def test_subnormal_operands(K, N, dtype):
    """One operand below the type's normal range, the other large: the sums are normal."""
    t = HALF[dtype]
    large = 4.0 if t == torch.float16 else 2.0 ** 60
    M, E, k, block = 40, 4, 2, 32
    r = Routed(ids_of(M, E, k, 5), E, block)
    args = (r.sid, r.eob, r.npp, M, k, block)
    f32 = torch.float32
    x, w = subnormal((M, K), t, 6), normal((E, N, K), t, 7) * large
    y = amr.grouped_gemm(x, w, *r.meta, k, block, out_dtype=f32)
    check(y[:r.npp], *orc.product(f64(x), f64(w), *args, True), steps(K), f32)
    assert f64(y[:r.npp][torch.from_numpy(r.live).cuda()]).all()
    dy = subnormal((r.cap, N), t, 8)
    dx = amr.grouped_gemm_dx(dy, w, *r.meta, M, k, block, out_dtype=f32)
    check(dx[:r.npp], *orc.product_dx(f64(dy), f64(w), *args), steps(N), f32)
    x, w = normal((M, K), t, 9) * large, subnormal((E, N, K), t, 10)
    y = amr.grouped_gemm(x, w, *r.meta, k, block, out_dtype=f32)
    check(y[:r.npp], *orc.product(f64(x), f64(w), *args, True), steps(K), f32)
    dw = amr.grouped_gemm_dw(dy, x, E, *r.meta, k, block, out_dtype=f32)
    check(dw, *orc.product_dw(f64(dy), f64(x), E, *args, True), steps(r.npp), f32)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_subnormal_mix_and_activation(dtype):
    t = HALF[dtype]
    M, E, k, N = 40, 4, 2, 40
    r = Routed(ids_of(M, E, k, 5), E, 32)
    rows = amr.slot_rows(r.meta[0], r.meta[2], M, k)
    y, v = subnormal((r.cap, N), t, 1), torch.rand(M, k, generator=torch.Generator().manual_seed(2)).cuda() + 1
    want, mag = orc.combine(f64(y), rows.cpu().numpy(), f64(v))
    check(amr.combine(y, rows, v), want, mag, k + 2, t)
    dout = subnormal((M, N), t, 3)
    dy = amr.combine_backward(dout, rows, r.meta[0], r.meta[2], weights=v)
    want = orc.combine_backward(f64(dout), rows.cpu().numpy(), f64(v), None, r.cap)[0]
    check(dy[:r.npp], want[:r.npp], np.abs(want[:r.npp]), 1, t)
    a = torch.cat([subnormal((30, N), t, 4), normal((30, N), t, 5)], dim=1)  # silu(g) = g / 2 and a little
    want = orc.swiglu(f64(a))
    check(amr.swiglu(a), want, np.abs(want), 12, t)


@pytest.mark.parametrize("K,N", [(72, 136), (67, 129), (67, 136), (72, 129), (5, 9), (3, 300)])
def test_nan_and_infinity_stay_in_their_rows(K, N):
    """Through either path: a row's end, where chunks are moved or overlap, holds them."""
    M, E, k, block = 20, 3, 2, 32
    r = Routed(ids_of(M, E, k, 10), E, block)
    token = np.where(r.live, r.sid[:r.npp] // k, -1)
    x, w = normal((M, K), torch.bfloat16, 11), normal((E, N, K), torch.bfloat16, 12)
    x[4, 0], x[9, K - 1] = float("nan"), float("inf")
    y = f64(amr.grouped_gemm(x, w, *r.meta, k, block))[:r.npp]
    assert np.isnan(y[token == 4]).all() and np.isinf(y[token == 9]).all()
    assert np.isfinite(y[(token != 4) & (token != 9)]).all()
    x, dy = normal((M, K), torch.bfloat16, 13), normal((r.cap, N), torch.bfloat16, 14)
    i, j = (int(at) for at in np.flatnonzero(r.live)[[3, -2]])
    dy[i, N - 1], dy[j, 0] = float("inf"), float("nan")
    dx = f64(amr.grouped_gemm_dx(dy, w, *r.meta, M, k, block))[:r.npp]
    other = np.ones(r.npp, dtype=bool)
    other[[i, j]] = False
    assert np.isinf(dx[i]).all() and np.isnan(dx[j]).all() and np.isfinite(dx[other]).all()
    dw = f64(amr.grouped_gemm_dw(dy, x, E, *r.meta, k, block))
    e, f = r.eob[i // block], r.eob[j // block]
    assert np.isinf(dw[e, N - 1]).all() and np.isnan(dw[f, 0]).all()
    dw[e, N - 1], dw[f, 0] = 0, 0
    assert np.isfinite(dw).all()


@pytest.mark.parametrize("rows", [4097, 4500, 8200])
def test_many_rows_by_large_tiles(rows):
    """128 tiles of 256 x 256 and more, an expert whose rows are not all looked up at once.
    Small integers: every sum is exact."""
    E, K, N, block = 8, 1024, 1024, 128
    ids = np.zeros((rows, 1), dtype=np.int32)
    ids[::97, 0] = 1 + np.arange(len(ids[::97])) % (E - 1)
    r = Routed(ids, E, block)
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-2, 3, (rows, K), generator=g).to(torch.bfloat16).cuda()
    dy = torch.randint(-2, 3, (r.cap, N), generator=g).to(torch.bfloat16).cuda()
    by_row = torch.randint(-2, 3, (r.cap, K), generator=g).to(torch.bfloat16).cuda()
    dw = amr.grouped_gemm_dw(dy, x, E, *r.meta, 1, block, out_dtype=torch.float32)
    ds = amr.grouped_gemm_dw(dy, by_row, E, *r.meta, 1, block, tokens=rows, out_dtype=torch.float32)
    expert = np.where(r.live, r.eob[np.arange(r.npp) // block], -1)
    assert (expert == 0).sum() > 4000
    for e in range(E):
        at = torch.from_numpy(np.flatnonzero(expert == e)).cuda()
        token = torch.from_numpy(r.sid[:r.npp][expert == e]).cuda().long()
        d = dy[at].double().t().contiguous()
        assert torch.equal(dw[e].double(), d @ x[token].double())
        assert torch.equal(ds[e].double(), d @ by_row[at].double())


def test_broadcast_gradient_adds_up():
    """A gradient of ones that is one value in memory gives what a whole tensor of ones gives,
    and is added to what the leaves hold."""
    M, E, k, H, I, block = 30, 4, 2, 72, 40, 32
    r = Routed(ids_of(M, E, k, 3, 0.2), E, block)
    parts = [normal((M, H), torch.bfloat16, 1), normal((E, 2 * I, H), torch.bfloat16, 2, H ** -0.5),
             normal((E, H, I), torch.bfloat16, 4, I ** -0.5), torch.rand(M, k, device="cuda") + 0.1]

    def layer(leaves):
        return amr.experts_train(*leaves[:3], amr.RouteSortOutput(r.ids, leaves[3], *r.meta), block)
    whole = [p.clone().requires_grad_() for p in parts]
    layer(whole).backward(torch.ones(M, H, dtype=torch.bfloat16, device="cuda"))
    leaves = [p.clone().requires_grad_() for p in parts]
    held = [torch.full_like(p, 2.0) for p in parts]
    for leaf, h in zip(leaves, held):
        leaf.grad = h.clone()
    layer(leaves).sum().backward()
    for leaf, h, w in zip(leaves, held, whole):
        assert w.grad.any() and torch.equal(leaf.grad, h + w.grad)
    out = layer(leaves)
    leaves[0].grad = None
    out.backward(torch.ones(1, 1, dtype=torch.bfloat16, device="cuda").expand(M, H))
    assert torch.equal(leaves[0].grad, whole[0].grad)
