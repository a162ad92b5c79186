"""The gated activation, slot_rows and the mix of the outputs on the GPU against the
float64 oracle.

Tolerances, beside half a step of the output's type: the sigmoid's exponential is off
by at most (|g| + 4) 2^-23, its sum and quotient by 2^-23 each; a product adds 2^-24.  The
gate's gradient is a difference of terms of at most (1 + |g|) |dh u| sigmoid(g).  A sum
of k products has 2 k roundings of 2^-24 of its magnitudes; a dot product over N has a
chain of N / 64 + 6 sums a lane, each of a product: 2 (N / 64 + 14) roundings."""
import numpy as np
import pytest
import torch

import align_moe_route_amd as amr
from experts_cases import HALF, STEP, Routed, check, f64, ids_of, normal
from oracle import experts as orc

pytestmark = pytest.mark.gpu


def near(got, want, slack, dtype):
    rel, tiny = STEP[dtype]
    err = np.abs(f64(got) - want)
    bound = rel * (np.abs(want) + slack) + slack + tiny
    assert (err <= bound).all(), float(np.max(err / bound))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,I,used", [(1, 1, None), (3, 7, 3), (5, 8, 0), (64, 384, 40), (200, 1001, 199), (33, 16, 99),
                                         (2, 20000, None), (1000, 9, 1000)])
def test_swiglu(rows, I, used, dtype):
    t = HALF[dtype]
    a, dh = normal((rows, 2 * I), t, 1, 3.0), normal((rows, I), t, 2)
    a[0, 0] = -60000.0 if dtype == "f16" else -1e30
    npp = None if used is None else torch.full((1,), used, dtype=torch.int32, device="cuda")
    n = rows if used is None else min(used, rows)
    h = torch.full((rows, I), 7.0, dtype=t, device="cuda")
    assert amr.swiglu(a, npp, out=h) is h
    A, D = f64(a)[:n], f64(dh)[:n]
    g, u = A[:, :I], A[:, I:]
    with np.errstate(over="ignore"):
        s = orc.sigmoid(g)
        grow = (np.minimum(np.abs(g), 200.0) + 8) * 2.0 ** -23
        near(h[:n], orc.swiglu(A), np.abs(g * s * u) * grow, t)
        assert (h[n:] == 7.0).all()
        da = torch.full((rows, 2 * I), 7.0, dtype=t, device="cuda")
        amr.swiglu_backward(a, dh, npp, out=da)
        want = orc.swiglu_backward(A, D)
    grow = np.concatenate([np.abs(D * u) * s * (1 + np.abs(g)) * grow, np.abs(D * g) * s * grow], axis=1)
    near(da[:n], want, grow, t)
    assert (da[n:] == 7.0).all()
    keep = a.clone()
    amr.swiglu_backward(a, dh, npp, out=a)  # in place
    assert torch.equal(a[:n], da[:n]) and torch.equal(a[n:], keep[n:])


def test_swiglu_against_differences():
    a = torch.randn(6, 10, dtype=torch.float64, generator=torch.Generator().manual_seed(3))
    dh = torch.randn(6, 5, dtype=torch.float64, generator=torch.Generator().manual_seed(4))
    a, dh = a.half().cuda(), dh.half().cuda()
    da = f64(amr.swiglu_backward(a, dh))
    A, D = f64(a), f64(dh)
    for i in np.ndindex(A.shape):
        up, down = A.copy(), A.copy()
        up[i] += 1e-5
        down[i] -= 1e-5
        want = ((orc.swiglu(up) - orc.swiglu(down)) * D).sum() / 2e-5
        assert abs(da[i] - want) < 2e-3 * max(1.0, abs(want))


# M, E, k, N, block, dropped
SHAPES = [(1, 4, 1, 8, 16, 0.0), (1, 8, 8, 512, 16, 0.0), (5, 3, 2, 1, 16, 0.3), (40, 6, 3, 67, 48, 0.2),
          (33, 70, 64, 24, 16, 0.1), (130, 5, 2, 1040, 64, 0.0), (9, 12, 9, 3583, 16, 0.1), (64, 4, 1, 520, 128, 0.5)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_combine(shape, weighted, dtype):
    M, E, k, N, block, dropped = shape
    t = HALF[dtype]
    r = Routed(ids_of(M, E, k, 5, dropped), E, block)
    rows = amr.slot_rows(r.meta[0], r.meta[2], M, k)
    want_rows = orc.slot_rows(r.sid, r.npp, M, k)
    assert np.array_equal(rows.cpu().numpy(), want_rows)
    y = normal((r.cap, N), t, 6)
    y[r.npp:] = float("nan")
    y[:r.npp][torch.from_numpy(~r.live).cuda()] = float("nan")
    v = torch.rand(M, k, generator=torch.Generator().manual_seed(7)).cuda() if weighted else None
    Y, V = f64(y), None if v is None else f64(v)
    want, mag = orc.combine(Y, want_rows, V)
    for odt in (t, torch.float32):
        check(amr.combine(y, rows, v, out_dtype=odt), want, mag, k + 2, odt)
    dout = normal((M, N), t, 8)
    dy = torch.full((r.cap, N), 7.0, dtype=t, device="cuda")
    got = amr.combine_backward(dout, rows, r.meta[0], r.meta[2], weights=v, y=y, out=dy)
    want, want_v, mag = orc.combine_backward(f64(dout), want_rows, V, Y, r.cap)
    assert got[0] is dy
    check(dy[:r.npp], want[:r.npp], np.abs(want[:r.npp]), 1, t)
    assert (dy[r.npp:] == 7.0).all() and not f64(dy[:r.npp])[~r.live].any()
    check(got[1], want_v, mag, N / 64 + 14, torch.float32)
    only = amr.combine_backward(dout, rows, r.meta[0], r.meta[2], weights=v)
    assert torch.equal(only[:r.npp], dy[:r.npp])


@pytest.mark.parametrize("M,E,k,block", [(1024, 16, 8, 16), (1025, 16, 8, 16), (2000, 40, 1, 400), (2000, 30, 1, 512)])
def test_slot_rows_sizes(M, E, k, block):
    """Both sides of the border between one launch and two, by slots and by rows."""
    ids = ids_of(M, E, k, 9, 0.2)
    r = Routed(ids, E, block)
    out = torch.full((M, k), 5, dtype=torch.int32, device="cuda")
    assert amr.slot_rows(r.meta[0], r.meta[2], M, k, out=out) is out
    assert np.array_equal(out.cpu().numpy(), orc.slot_rows(r.sid, r.npp, M, k))


def test_combine_in_slot_order():
    y = normal((15, 33), torch.bfloat16, 1)
    v = torch.rand(5, 3, device="cuda")
    want, mag = orc.combine(f64(y), np.arange(15, dtype=np.int32).reshape(5, 3), f64(v))
    check(amr.combine(y, 3, v), want, mag, 5, torch.bfloat16)


def test_rows_outside_add_nothing():
    y = normal((4, 20), torch.float16, 1)
    rows = torch.tensor([[0, 4], [-5, 3], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device="cuda")
    got = amr.combine(y, rows)
    assert torch.equal(got[0], y[0]) and torch.equal(got[1], y[3]) and not got[2].any()


def test_no_tokens():
    i32 = torch.int32
    sid, npp = torch.zeros(1, dtype=i32, device="cuda"), torch.zeros(1, dtype=i32, device="cuda")
    rows = amr.slot_rows(sid, npp, 0, 2)
    assert rows.shape == (0, 2)
    assert amr.combine(torch.zeros(1, 8, device="cuda").half(), rows).shape == (0, 8)
    assert amr.swiglu(torch.zeros(0, 8, device="cuda").half()).shape == (0, 4)
