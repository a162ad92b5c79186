"""Offsets past 32 bits: weights, rows and codes of more than 4 GiB.  The float64
answers are taken at a few rows; tolerances as in the other tests of these calls."""
import numpy as np
import pytest
import torch

import align_moe_route_amd as amr
from experts_cases import STEP, Routed, f64, ids_of, normal
from oracle import int4 as oi4

pytestmark = pytest.mark.gpu


def near(got, want, mag, steps, dtype):
    rel, tiny = STEP[dtype]
    slack = steps * 2.0 ** -23 * mag
    assert (np.abs(f64(got) - want) <= rel * (np.abs(want) + slack) + slack + tiny).all()


def test_weights_and_their_gradient():
    """E N K = 2.4e9 values: the last experts lie past 4 GiB in w and in dw."""
    M, E, k, K, N, block = 40, 900, 2, 3584, 768, 16
    ids = ids_of(M, E, k, 1)
    ids[:, 1] = np.arange(M) % 3 + E - 3  # routes to the last three
    ids[:, 0] = np.minimum(ids[:, 0], E - 4)
    r = Routed(ids, E, block)
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    w[-3:] = normal((3, N, K), torch.bfloat16, 2, K ** -0.5)
    x, dy = normal((M, K), torch.bfloat16, 3), normal((r.cap, N), torch.bfloat16, 4)
    y = amr.grouped_gemm(x, w, *r.meta, k, block)
    dx = amr.grouped_gemm_dx(dy, w, *r.meta, M, k, block)
    dw = amr.grouped_gemm_dw(dy, x, E, *r.meta, k, block)
    s, xs, ds = r.sid[:r.npp], f64(x), f64(dy)
    for e in range(E - 3, E):
        at = np.flatnonzero(r.live & (r.eob[np.arange(r.npp) // block] == e))
        assert len(at)
        m, xe = f64(w[e]), xs[s[at] // k]
        near(y[at], xe @ m.T, np.abs(xe) @ np.abs(m.T), K / 16 + 16, torch.bfloat16)
        near(dx[at], ds[at] @ m, np.abs(ds[at]) @ np.abs(m), N / 16 + 16, torch.bfloat16)
        near(dw[e], ds[at].T @ xe, np.abs(ds[at]).T @ np.abs(xe), 17, torch.bfloat16)


def test_rows():
    """140000 rows of 16384 columns: y, dy, the activation and the mix past 4 GiB."""
    M, E, k, K, N, block = 140000, 2, 1, 8, 16384, 128
    ids = (np.arange(M) % 2)[:, None].astype(np.int32)
    r = Routed(ids, E, block)
    x, w = normal((M, K), torch.float16, 1), normal((E, N, K), torch.float16, 2)
    y = amr.grouped_gemm(x, w, *r.meta, k, block)
    at = np.flatnonzero(r.live)[[0, -400, -1]]
    token, e = r.sid[at], r.eob[at // block]
    xs, ws = f64(x[torch.from_numpy(token).cuda().long()]), f64(w)
    want = np.stack([ws[e[i]] @ xs[i] for i in range(3)])
    mag = np.stack([np.abs(ws[e[i]]) @ np.abs(xs[i]) for i in range(3)])
    near(y[at], want, mag, 17, torch.float16)
    dx = amr.grouped_gemm_dx(y, w, *r.meta, M, k, block)
    Y = f64(y[at])
    near(dx[at], np.stack([Y[i] @ ws[e[i]] for i in range(3)]), np.stack([np.abs(Y[i]) @ np.abs(ws[e[i]]) for i in range(3)]),
         N / 16 + 16, torch.float16)
    rows = amr.slot_rows(r.meta[0], r.meta[2], M, k)
    v = torch.full((M, k), 2.0, device="cuda")
    out = amr.combine(y, rows, v)
    assert torch.equal(out[token], 2 * y[at])
    dy, dv = amr.combine_backward(out, rows, r.meta[0], r.meta[2], weights=v, y=y)
    assert torch.equal(dy[at], 2 * out[token])
    near(dv[token, 0], (f64(out[token]) * Y).sum(1), np.abs(f64(out[token]) * Y).sum(1), N / 64 + 14, torch.float32)
    h = amr.swiglu(y, r.meta[2])
    g, u = Y[:, :N // 2], Y[:, N // 2:]
    near(h[at], g / (1 + np.exp(-g)) * u, np.abs(g / (1 + np.exp(-g)) * u), 40, torch.float16)
    del dx, out, dy, h


def test_int4_codes():
    """Codes and scales of the last experts past 4 GiB and 2 GiB."""
    E, N, K, group = 4096, 1024, 2176, 32
    codes = torch.full((E, N, K // 2), 0x88, dtype=torch.uint8, device="cuda")
    scales = torch.ones(E, N, K // group, dtype=torch.bfloat16, device="cuda")
    tail = amr.int4_quantize(normal((2, N, K), torch.bfloat16, 1, K ** -0.5), group)
    codes[-2:], scales[-2:] = tail.codes, tail.scales
    x = normal((2, K), torch.bfloat16, 2)
    ids = torch.tensor([[E - 1, 0], [E - 2, 5]], dtype=torch.int32, device="cuda")
    y = amr.int4_matvec(x, amr.Int4(codes, scales), ids)
    assert not y[:, 1].any()
    w = oi4.values(tail.codes.cpu().numpy(), f64(tail.scales))
    for t, e in ((0, 1), (1, 0)):
        want = w[e] @ f64(x[t])
        size = np.repeat(f64(tail.scales[e]), group, axis=-1) @ np.abs(f64(x[t]))
        near(y[t, 0], want, size, 34 * 55 + 10, torch.bfloat16)
