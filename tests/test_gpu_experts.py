"""Products grouped by expert and their gradients on the GPU against the float64
oracle.

Tolerance: half a step of the output's type, plus the roundings of FP32 sums.  A sum
over C values is a chain of matrix instructions of 16 or 32 products each, at most 16
roundings inside one and one to the next: C / 16 + 16 of them, each at most 2^-23 of
the sum of magnitudes."""
import numpy as np
import pytest
import torch

import align_moe_route_amd as amr
from experts_cases import HALF, Routed, check, f64, ids_of, normal
from oracle import experts as orc

pytestmark = pytest.mark.gpu

# M, E, k, K, N, block, dropped
SHAPES = [
    (1, 4, 1, 8, 8, 16, 0.0),          # one token, one route
    (1, 8, 8, 64, 128, 32, 0.0),
    (5, 3, 2, 1, 1, 16, 0.0),          # single columns
    (7, 4, 3, 7, 5, 16, 0.2),
    (33, 6, 2, 63, 65, 48, 0.1),       # odd widths, blocks of 16-row tiles
    (40, 5, 5, 64, 64, 32, 0.0),
    (70, 3, 2, 200, 72, 64, 0.0),
    (130, 2, 1, 136, 264, 128, 0.0),   # more than a tile of every size
    (300, 4, 2, 520, 257, 128, 0.1),
    (260, 2, 2, 72, 520, 256, 0.0),
    (64, 12, 4, 1001, 395, 64, 0.1),
    (9, 4, 2, 8, 2048, 16, 0.0),
    (150, 1, 1, 640, 384, 128, 0.0),   # one expert
    (40, 3, 2, 5, 300, 32, 0.1),       # rows of fewer than eight values on one side
    (40, 3, 2, 300, 3, 64, 0.0),
    (200, 2, 1, 9, 15, 128, 0.0),      # just above eight
]


def steps(C):
    return C / 16 + 16


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("by_tokens", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_products(shape, by_tokens, f32, dtype):
    M, E, k, K, N, block, dropped = shape
    r = Routed(ids_of(M, E, k, 1, dropped), E, block)
    t = HALF[dtype]
    odt = torch.float32 if f32 else t
    x = normal((M if by_tokens else r.cap, K), t, 2)
    w = normal((E, N, K), t, 3, K ** -0.5)
    dy = normal((r.cap, N), t, 4, 0.25)
    tokens = None if by_tokens else M
    args = (r.sid, r.eob, r.npp, M, k, block)
    xs, ws, ds = f64(x), f64(w), f64(dy)

    y = torch.full((r.cap, N), 7.0, dtype=odt, device="cuda")
    assert amr.grouped_gemm(x, w, *r.meta, k, block, tokens=tokens, out=y) is y
    want, mag = orc.product(xs, ws, *args, by_tokens)
    check(y[:r.npp], want, mag, steps(K), odt)
    assert (y[r.npp:] == 7.0).all() and not f64(y[:r.npp])[~r.live].any()

    dx = amr.grouped_gemm_dx(dy, w, *r.meta, M, k, block, out_dtype=odt)
    want, mag = orc.product_dx(ds, ws, *args)
    check(dx[:r.npp], want, mag, steps(N), odt)
    assert not f64(dx[:r.npp])[~r.live].any()

    dw = amr.grouped_gemm_dw(dy, x, E, *r.meta, k, block, tokens=tokens, out_dtype=odt)
    want, mag = orc.product_dw(ds, xs, E, *args, by_tokens)
    rows = int(np.bincount(r.eob[:r.npp // block], minlength=E).max()) * block if r.npp else 0
    check(dw, want, mag, steps(rows), odt)
    assert torch.equal(dw, amr.grouped_gemm_dw(dy, x, E, *r.meta, k, block, tokens=tokens, out_dtype=odt))


@pytest.mark.parametrize("K,N", [(200, 72), (1096, 520), (203, 77), (64, 1040), (771, 9)])
@pytest.mark.parametrize("tile", [16, 32, 64, 128, 16 | amr.MRS_TILE_NARROW, 32 | amr.MRS_TILE_NARROW,
                                  64 | amr.MRS_TILE_NARROW])
def test_tiles(tile, K, N):
    """Every tile size, with rows of whole chunks and of others, short and long sums, tiles
    whose waves have no row with a slot, and both kinds of x rows."""
    M, E, k, block = 330, 5, 2, 128
    r = Routed(ids_of(M, E, k, 21, 0.1), E, block)
    args = (r.sid, r.eob, r.npp, M, k, block)
    for t, odt in ((torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32)):
        x, w = normal((M, K), t, 22), normal((E, N, K), t, 23, K ** -0.5)
        xr, dy = normal((r.cap, K), t, 24), normal((r.cap, N), t, 25)
        y = amr.grouped_gemm(x, w, *r.meta, k, block, out_dtype=odt, tile=tile)
        check(y[:r.npp], *orc.product(f64(x), f64(w), *args, True), steps(K), odt)
        y = amr.grouped_gemm(xr, w, *r.meta, k, block, tokens=M, out_dtype=odt, tile=tile)
        check(y[:r.npp], *orc.product(f64(xr), f64(w), *args, False), steps(K), odt)
        dx = amr.grouped_gemm_dx(dy, w, *r.meta, M, k, block, out_dtype=odt, tile=tile)
        check(dx[:r.npp], *orc.product_dx(f64(dy), f64(w), *args), steps(N), odt)


@pytest.mark.parametrize("K,N,rows", [(520, 776, 5000), (203, 301, 4500)])
def test_many_rows_of_an_expert(K, N, rows):
    """Sums over more rows than are kept at a time, beside an expert of few."""
    ids = np.zeros((rows, 1), dtype=np.int32)
    ids[::600] = 1
    r = Routed(ids, 2, 64)
    x, dy = normal((rows, K), torch.bfloat16, 26), normal((r.cap, N), torch.bfloat16, 27)
    s = r.sid[:r.npp]
    xs, ds = f64(x), f64(dy)
    for out in (torch.bfloat16, torch.float32):
        dw = amr.grouped_gemm_dw(dy, x, 2, *r.meta, 1, 64, out_dtype=out)
        for e in range(2):
            at = np.flatnonzero(r.live & (r.eob[np.arange(r.npp) // 64] == e))
            check(dw[e], ds[at].T @ xs[s[at]], np.abs(ds[at]).T @ np.abs(xs[s[at]]), steps(len(at)), out)


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("wide", [False, True])
def test_padding_rows_hold_nothing(block, wide):
    """NaN in padding rows, past num_post_pad, in unrouted tokens and in the weights of
    experts without a route reaches nothing."""
    M, E, k, K, N = 37, 6, 2, 72 if wide else 67, 136 if wide else 129
    ids = ids_of(M, E, k, 5, 0.2, only=4)
    ids[3] = -1
    r = Routed(ids, E, block)
    x, w = normal((M, K), torch.bfloat16, 6), normal((E, N, K), torch.bfloat16, 7, K ** -0.5)
    dy = normal((r.cap, N), torch.bfloat16, 8)
    used = np.zeros(E, dtype=bool)
    used[ids[ids >= 0]] = True
    xs, ws, ds = f64(x), f64(w), f64(dy)
    x[3] = float("nan")
    w[torch.from_numpy(~used).cuda()] = float("nan")
    pad = torch.ones(r.cap, dtype=torch.bool)
    pad[:r.npp] = torch.from_numpy(~r.live)
    dy[pad.cuda()] = float("nan")
    args = (r.sid, r.eob, r.npp, M, k, block)
    y = amr.grouped_gemm(x, w, *r.meta, k, block)
    check(y[:r.npp], *orc.product(xs, ws, *args, True), steps(K), torch.bfloat16)
    dx = amr.grouped_gemm_dx(dy, w, *r.meta, M, k, block)
    check(dx[:r.npp], *orc.product_dx(ds, ws, *args), steps(N), torch.bfloat16)
    dw = amr.grouped_gemm_dw(dy, x, E, *r.meta, k, block)
    check(dw, *orc.product_dw(ds, xs, E, *args, True), steps(r.npp), torch.bfloat16)
    assert not f64(dw)[~used].any()
    xr = normal((r.cap, K), torch.bfloat16, 9)
    xrs = f64(xr)
    xr[pad.cuda()] = float("nan")
    y = amr.grouped_gemm(xr, w, *r.meta, k, block, tokens=M)
    check(y[:r.npp], *orc.product(xrs, ws, *args, False), steps(K), torch.bfloat16)
    dw = amr.grouped_gemm_dw(dy, xr, E, *r.meta, k, block, tokens=M)
    check(dw, *orc.product_dw(ds, xrs, E, *args, False), steps(r.npp), torch.bfloat16)


def test_nan_and_infinity_stay_in_their_rows():
    M, E, k, K, N, block = 20, 3, 2, 72, 136, 32
    r = Routed(ids_of(M, E, k, 10), E, block)
    x, w = normal((M, K), torch.bfloat16, 11), normal((E, N, K), torch.bfloat16, 12)
    x[4, 5], x[9, 71] = float("nan"), float("inf")
    y = f64(amr.grouped_gemm(x, w, *r.meta, k, block))[:r.npp]
    token = np.where(r.live, r.sid[:r.npp] // k, -1)
    assert np.isnan(y[token == 4]).all() and np.isinf(y[token == 9]).all()
    assert np.isfinite(y[(token != 4) & (token != 9)]).all()


@pytest.mark.parametrize("dropped", [0.0, 1.0])
def test_no_routes(dropped):
    M = 0 if dropped == 0.0 else 5
    E, k, K, N, block = 4, 2, 24, 40, 16
    r = Routed(np.full((M, k), -1, dtype=np.int32), E, block)
    assert r.npp == 0
    x, w = normal((M, K), torch.float16, 1), normal((E, N, K), torch.float16, 2)
    y = amr.grouped_gemm(x, w, *r.meta, k, block, out=torch.full((max(r.cap, 1), N), 3.0, device="cuda").half())
    assert (y == 3.0).all()
    dy = normal((max(r.cap, 1), N), torch.float16, 3)
    dw = amr.grouped_gemm_dw(dy, x, E, *r.meta, k, block)
    assert dw.shape == (E, N, K) and not dw.any()


def test_any_alignment():
    """Matrices that begin at any element's address."""
    M, E, k, K, N, block = 50, 4, 2, 128, 72, 64
    r = Routed(ids_of(M, E, k, 13), E, block)
    args = (r.sid, r.eob, r.npp, M, k, block)

    def shifted(t):
        buf = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:] = t.reshape(-1)
        return buf[1:].view(t.shape)
    x, w, dy = (shifted(normal(s, torch.float16, i)) for i, s in enumerate([(M, K), (E, N, K), (r.cap, N)]))
    y = amr.grouped_gemm(x, w, *r.meta, k, block, out=shifted(torch.zeros(r.cap, N, device="cuda").half()))
    check(y[:r.npp], *orc.product(f64(x), f64(w), *args, True), steps(K), torch.float16)
    dx = amr.grouped_gemm_dx(dy, w, *r.meta, M, k, block, out=shifted(torch.zeros(r.cap, K, device="cuda").half()))
    check(dx[:r.npp], *orc.product_dx(f64(dy), f64(w), *args), steps(N), torch.float16)
    dw = amr.grouped_gemm_dw(dy, x, E, *r.meta, k, block, out=shifted(torch.zeros(E, N, K, device="cuda")))
    check(dw, *orc.product_dw(f64(dy), f64(x), E, *args, True), steps(r.npp), torch.float32)
