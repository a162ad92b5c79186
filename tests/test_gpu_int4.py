"""4-bit weights with group scales on the GPU against the float64 oracle.

Codes and scales are exact.  Products, beside half a step of the output's type: a
chunk of 32 columns is a chain of 32 pair products whose partial sums are bounded by
55 |scale| sum |x| (codes enter as 16 + c <= 31, and 24 sum x is taken off), then a chain
of K / 2048 + 8 chunk sums (K k / 2048 for sums over picks)."""
import numpy as np
import pytest
import torch

import align_moe_route_amd as amr
from experts_cases import HALF, STEP, f64, ids_of, normal
from oracle import int4 as orc

pytestmark = pytest.mark.gpu
NAME = {torch.bfloat16: "bf16", torch.float16: "f16"}


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 31), (5, 128), (4, 1001), (70, 260), (2, 5000)])
def test_quantize(rows, K, dtype, kind, group):
    w = normal((rows, K + 3), dtype, 1, 0.02)[:, :K]  # rows of a wider buffer
    if K > 3:
        w[0, 3] = 0.0
    if rows > 2:
        w[1], w[2, K // 2] = 0.0, float("inf")
        w[2, 0] = float("nan")
    if rows > 3:
        w[3] *= 1e-6 if dtype == torch.float16 else 1e-36  # subnormal values and scales
    q = amr.int4_quantize(w, group, scale_dtype=HALF[kind])
    codes, scales = orc.quantize(w.float().cpu().numpy(), group, kind)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert np.array_equal(f64(q.scales), scales.astype(np.float64), equal_nan=True)


def test_quantize_ties_and_large():
    w = torch.zeros(2, 128, device="cuda")
    w[0, :6] = torch.tensor([7.0, 0.5, 1.5, 2.5, -0.5, -6.5])
    w[1, :2] = torch.tensor([3e38, 1.0])
    for kind in ("bf16", "f16"):
        q = amr.int4_quantize(w, 128, scale_dtype=HALF[kind])
        codes, scales = orc.quantize(w.cpu().numpy(), 128, kind)
        assert np.array_equal(q.codes.cpu().numpy(), codes)
        assert np.array_equal(f64(q.scales), scales.astype(np.float64), equal_nan=True)


def product(M, E, k, K, N, group, dtype, per_slot, dropped, seed=1):
    t = HALF[dtype]
    ids = ids_of(M, E, k, seed, dropped)
    q = amr.int4_quantize(normal((E, N, K), t, seed + 1, K ** -0.5), group)
    x = normal((M, k, K) if per_slot else (M, K), t, seed + 2)
    w = orc.values(q.codes.cpu().numpy(), f64(q.scales))
    scale = np.repeat(f64(q.scales), group, axis=-1)
    return torch.from_numpy(ids).cuda(), q, x, orc.matvec(f64(x), w, ids), orc.matvec(np.abs(f64(x)), scale, ids)


def near(got, want, slack, dtype):
    rel, tiny = STEP[dtype]
    err = np.abs(f64(got) - want)
    bound = rel * (np.abs(want) + slack) + slack + tiny
    assert (err <= bound).all(), float(np.max(err / bound))


# M, E, k, K, N, group, dropped
SHAPES = [(1, 4, 1, 1, 1, 32, 0.0), (1, 4, 2, 31, 6, 32, 0.0), (2, 3, 2, 128, 16, 64, 0.0), (3, 5, 4, 257, 50, 128, 0.2),
          (1, 16, 8, 384, 200, 32, 0.0), (4, 6, 3, 1001, 34, 64, 0.1), (1, 8, 4, 2048, 64, 128, 0.0),
          (2, 4, 2, 2500, 66, 32, 0.0), (9, 3, 2, 3584, 24, 128, 0.0), (1, 2, 2, 7168, 10, 64, 0.0), (1, 70, 64, 130, 8, 32, 0.1)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_matvec(shape, per_slot, dtype):
    M, E, k, K, N, group, dropped = shape
    t = HALF[dtype]
    ids, q, x, p, size = product(M, E, k, K, N, group, dtype, per_slot, dropped)
    slack = (34 * 55 + K / 2048 + 8) * 2.0 ** -23 * size
    near(amr.int4_matvec(x, q, ids), p, slack, t)
    v = torch.rand(M, k, generator=torch.Generator().manual_seed(3)).cuda()
    V = f64(v)[:, :, None]
    near(amr.int4_matvec(x, q, ids, weights=v), (p * V).sum(1), ((slack + (k + 4) * 2.0 ** -23 * size * 8) * V).sum(1), t)
    if N % 2 == 0:
        h = N // 2
        g, u, sg, su = p[..., :h], p[..., h:], slack[..., :h], slack[..., h:]
        # |d silu| <= 1.1, and the sigmoid's own roundings
        grow = np.abs(orc.silu_gate(p)) * (np.abs(g) + 8) * 2.0 ** -23
        near(amr.int4_matvec(x, q, ids, gated=True), orc.silu_gate(p),
             1.1 * sg * (np.abs(u) + su) + np.abs(g) * su + grow, t)


@pytest.mark.parametrize("K", [96, 5, 8, 33])
def test_dropped_rows_are_not_read(K):
    M, E, k, N = 3, 4, 3, 20
    ids, q, x, p, size = product(M, E, k, K, N, 32, "bf16", True, 0.0)
    ids[0, 1], ids[2, 2] = -1, E
    x[0, 1], x[2, 2] = float("nan"), float("inf")
    y = f64(amr.int4_matvec(x, q, ids))
    p[0, 1], p[2, 2] = 0.0, 0.0
    assert not y[0, 1].any() and not y[2, 2].any() and np.abs(y - p).max() < 0.05
    assert np.isfinite(f64(amr.int4_matvec(x, q, ids, gated=True))).all()
    v = torch.rand(M, k, device="cuda")
    assert np.abs(f64(amr.int4_matvec(x, q, ids, weights=v)) - (p * f64(v)[:, :, None]).sum(1)).max() < 0.05


def test_nan_scale_reaches_its_row_only():
    ids, q, x, p, _ = product(2, 3, 2, 256, 12, 64, "f16", False, 0.0)
    q.scales[0, 5, 1] = float("nan")
    y = f64(amr.int4_matvec(x, q, ids))
    hit = (ids.cpu().numpy() == 0)[:, :, None] & (np.arange(12) == 5)
    assert np.isnan(y[hit]).all() and np.isfinite(y[~hit]).all()


def test_same_expert_twice_and_out():
    ids, q, x, p, size = product(2, 3, 2, 160, 18, 32, "bf16", False, 0.0)
    ids[:] = 1
    out = torch.full((2, 2, 18), 9.0, dtype=torch.bfloat16, device="cuda")
    assert amr.int4_matvec(x, q, ids, out=out) is out
    assert torch.equal(out[:, 0], out[:, 1])
