"""4-bit rows and their grouped product on the GPU against the float64 oracle
(oracle/mxfp4.py)."""
import numpy as np
import pytest

from oracle import mxfp4 as om
from oracle import route_sort as orc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
amr = pytest.importorskip("align_moe_route_amd")

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def check_rows(x, x64):
    """Codes, scales and values of x equal the oracle's, bit for bit."""
    v = torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda")
    q = amr.mxfp4_quantize(x, values=v)
    codes, scales, values = om.quantize(x64.reshape(-1, x64.shape[-1]))
    assert np.array_equal(q.scales.cpu().numpy().reshape(scales.shape), scales)
    assert np.array_equal(q.codes.cpu().numpy().reshape(codes.shape), codes)
    got = v.double().cpu().numpy().reshape(values.shape)
    assert np.array_equal(got, values, equal_nan=True)
    ok = ~np.isnan(values)
    assert np.array_equal(np.signbit(got)[ok], np.signbit(values)[ok])
    q2 = amr.mxfp4_quantize(x)  # without the values
    assert torch.equal(q2.codes, q.codes) and torch.equal(q2.scales, q.scales)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,K,extra", [(1, 1, 0), (3, 31, 0), (5, 32, 0), (2, 33, 7), (7, 128, 8), (4, 129, 0),
                                          (33, 1000, 24), (1, 3584, 0), (257, 640, 0), (19, 1001, 3)])
def test_quantize(dtype, rows, K, extra):
    print(f"[gpu] mxfp4 quantize {dtype} rows={rows} K={K} extra={extra}", flush=True)
    rng = np.random.default_rng(rows * 1000 + K)
    x = rng.standard_normal((rows, K + extra)) * np.exp(2 * rng.standard_normal((1, K + extra)))
    x[rng.random(x.shape) < 0.05] = 0.0
    t = torch.from_numpy(x).to(DT[dtype]).cuda()[:, :K]
    check_rows(t, t.double().cpu().numpy())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantize_ties_and_neighbours(dtype):
    """Every rounding boundary, the values beside it, and each sign, at scales
    from the smallest to the largest of the type."""
    eps = torch.finfo(DT[dtype]).eps
    base = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.5, 0.5, 1, 1.5, 2, 3, 4, 6])
    v = np.concatenate([base, base * (1 - eps), base * (1 + eps)])
    v = np.concatenate([v, -v, np.zeros(6)])  # 96 values, three blocks
    v[31::32] = 4.0  # fixes each block's scale at one
    lo, hi = {"f32": (-140, 124), "bf16": (-130, 124), "f16": (-22, 13)}[dtype]
    rows = np.stack([np.ldexp(v, e) for e in range(lo, hi + 1)])
    with np.errstate(over="ignore"):
        t = torch.from_numpy(rows).to(DT[dtype]).cuda()
    assert bool(torch.isfinite(t).all())
    check_rows(t, t.double().cpu().numpy())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantize_not_finite(dtype):
    x = torch.randn(6, 96, generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    x[0, 5], x[1, 40], x[2, 95], x[3, 0] = float("nan"), float("inf"), float("-inf"), torch.finfo(DT[dtype]).max
    x[4, :32] = 0
    x[5, :32] = -0.0
    check_rows(x.cuda(), x.double().numpy())


def test_quantize_leading_dimensions_streams_and_nothing():
    x = torch.randn(3, 4, 72, device="cuda")
    check_rows(x, x.double().cpu().numpy())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        check_rows(x, x.double().cpu().numpy())
    q = amr.mxfp4_quantize(torch.empty(0, 64, device="cuda"))
    assert q.codes.shape == (0, 64) and q.scales.shape == (0, 4)


# ------------------------------------------------------------------- product

def routed(rng, M, E, k, block, drop=0.0, skew=0.0):
    p = 1.0 / np.arange(1, E + 1) ** skew
    ids = np.stack([np.sort(rng.choice(E, k, replace=False, p=p / p.sum())) for _ in range(M)]).astype(np.int32)
    ids[rng.random(ids.shape) < drop] = -1
    out = amr.sort_from_ids(torch.from_numpy(ids).cuda(), E, block)
    npp = int(out.num_post_pad.item())
    return out, npp


def random_rows(rng, shape, K):
    """Packed rows of random codes and scale bytes near one; the columns past K are zero."""
    Kp = om.padded(K)
    codes = rng.integers(0, 256, shape + (Kp // 2,), dtype=np.uint8)
    scales = rng.integers(124, 131, shape + (Kp // 32,), dtype=np.uint8)
    nib = np.arange(Kp // 2)[None] * 2
    codes = np.where(nib + 1 < K, codes, np.where(nib < K, codes & 15, 0)).astype(np.uint8)
    return codes, scales


def to_gpu(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


POISON = -12345.0


def run_product(rng, M, E, k, K, N, block, dtype, in_order, drop=0.0, skew=0.0, edit=None):
    meta, npp = routed(rng, M, E, k, block, drop, skew)
    rows = amr.max_rows(M, E, k, block)
    xc, xs = random_rows(rng, (rows if in_order else M,), K)
    wc, ws = random_rows(rng, (E, N), K)
    if edit:
        edit(xc, xs, wc, ws)
    gxc, gxs, gwc, gws = to_gpu(xc, xs, wc, ws)
    y = torch.full((rows, N), POISON, dtype=dtype, device="cuda")
    amr.grouped_gemm_mxfp4(amr.MXFP4(gxc, gxs), amr.MXFP4(gwc, gws), meta.sorted_ids, meta.expert_of_block,
                           meta.num_post_pad, k, block, tokens=M if in_order else None, out=y)
    torch.cuda.synchronize()
    sid, eob = meta.sorted_ids.cpu().numpy(), meta.expert_of_block.cpu().numpy()
    ref, ab = om.product(xc, xs, wc, ws, sid, eob, npp, M, k, block, in_order)
    got = y.double().cpu().numpy()
    assert (got[npp:] == float(torch.tensor(POISON, dtype=dtype))).all(), "rows past num_post_pad were written"
    pad = ~((sid[:npp] >= 0) & (sid[:npp] < M * k))
    assert (got[:npp][pad] == 0).all(), "padding rows are zeros"
    return got[:npp], ref, ab


SHAPES = [  # M, E, k, K, N, block, drop, skew; the kernel is chosen by the sizes
    (1, 8, 2, 128, 16, 16, 0, 0),
    (1, 32, 16, 3584, 768, 32, 0, 0),
    (3, 8, 8, 256, 17, 16, 0, 0),
    (5, 4, 1, 100, 1, 16, 0, 0),
    (64, 40, 4, 384, 96, 48, 0, 0),
    (200, 8, 4, 640, 130, 32, 0, 0),
    (300, 8, 4, 512, 256, 64, 0, 0),
    (700, 8, 4, 896, 300, 128, 0, 0.5),
    (1000, 4, 2, 1152, 520, 256, 0.3, 1.0),
    (257, 3, 2, 128, 64, 128, 0, 0),
    (129, 2, 1, 384, 257, 64, 0.9, 0),
    (400, 5, 3, 33, 31, 96, 0, 0),
    (90, 6, 2, 2000, 70, 32, 1.0, 0),   # every route dropped
    (611, 1, 1, 256, 48, 128, 0, 0),
    (400, 3, 1, 2200, 72, 128, 0, 0),   # long rows, to the few-rows kernel as well
    (150, 3, 1, 4500, 40, 64, 0, 0),
    (70, 2, 1, 6200, 264, 32, 0, 0.5),
    (9, 3, 1, 9000, 33, 48, 0, 0),
    # many experts with few rows: whole strips of weights, tiles of 16 and 64 rows
    # most of which are padding
    (70, 200, 2, 256, 40, 16, 0.1, 0),
    (70, 200, 2, 384, 264, 48, 0, 0),
    (90, 220, 3, 128, 24, 64, 0.5, 0),
    (60, 250, 4, 300, 270, 128, 0.2, 0.5),
    (100, 130, 2, 640, 300, 256, 0, 0),
    (2, 60, 20, 700, 80, 16, 0, 0),
    (2, 90, 40, 520, 200, 32, 0, 0),    # 32-column tiles of the few-rows kernel
]


@pytest.mark.parametrize("in_order", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,E,k,K,N,block,drop,skew", SHAPES)
def test_product(M, E, k, K, N, block, drop, skew, dtype, in_order):
    print(f"[gpu] mxfp4 product M={M} E={E} k={k} K={K} N={N} block={block} {dtype} {in_order}", flush=True)
    rng = np.random.default_rng(M + K + N)
    got, ref, ab = run_product(rng, M, E, k, K, N, block, DT[dtype], in_order, drop, skew)
    assert (np.abs(got - ref) <= om.tolerance(ref, ab, om.padded(K), dtype == "bf16")).all()


@pytest.mark.parametrize("M,E,k,block", [(2, 8, 4, 16), (300, 4, 2, 64), (900, 8, 4, 128), (100, 4, 2, 32)])
def test_product_exact_sums(M, E, k, block):
    """Scales of one: every partial sum is a multiple of 1/4 below 2^22, exact in FP32."""
    def ones(xc, xs, wc, ws):
        xs[:], ws[:] = 127, 127
    rng = np.random.default_rng(M)
    got, ref, _ = run_product(rng, M, E, k, 640, 77, block, torch.float32, False, edit=ones)
    assert np.array_equal(got, ref)


@pytest.mark.parametrize("M,E,k,block", [(2, 8, 4, 16), (300, 4, 2, 64), (900, 8, 4, 128)])
def test_product_nan_blocks(M, E, k, block):
    """A NaN block reaches its token's or its output's results and nothing else."""
    def edit(xc, xs, wc, ws):
        xs[0, 1] = 255      # also the row that padding rows could read
        ws[1, 2, 0] = 255
    rng = np.random.default_rng(M)
    got, ref, ab = run_product(rng, M, E, k, 256, 40, block, torch.float32, False, edit=edit)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    assert (np.abs(got - ref)[ok] <= om.tolerance(ref, ab, 256, False)[ok]).all()


@pytest.mark.parametrize("M,block", [(4, 16), (300, 64), (900, 128)])
def test_product_scale_range(M, block):
    """Scales far apart: sums follow the larger; a result past FP32's range is infinite."""
    def edit(xc, xs, wc, ws):
        xs[:] = np.random.default_rng(1).integers(60, 190, xs.shape)
        ws[:] = np.random.default_rng(2).integers(60, 190, ws.shape)
    rng = np.random.default_rng(M)
    got, ref, ab = run_product(rng, M, 4, 2, 512, 48, block, torch.float32, False, edit=edit)
    past = np.abs(ref) > np.finfo(np.float32).max
    assert np.array_equal(got[past], np.copysign(np.inf, ref[past]))
    assert (np.abs(got - ref)[~past] <= om.tolerance(ref, ab, 512, False)[~past]).all()


def test_product_foreign_experts_and_no_tokens():
    """Blocks of an expert outside [0, E) are not written; no token, no launch."""
    rng = np.random.default_rng(3)
    meta, npp = routed(rng, 100, 6, 2, 32)
    xc, xs = random_rows(rng, (100,), 128)
    wc, ws = random_rows(rng, (6, 20), 128)
    x, w = amr.MXFP4(*to_gpu(xc, xs)), amr.MXFP4(*to_gpu(wc, ws))
    eob = meta.expert_of_block.clone()
    eob[0], eob[1] = 6, -1
    y = torch.full((amr.max_rows(100, 6, 2, 32), 20), POISON, device="cuda")
    amr.grouped_gemm_mxfp4(x, w, meta.sorted_ids, eob, meta.num_post_pad, 2, 32, out=y)
    assert bool((y[:64] == POISON).all()) and bool((y[64:npp] != POISON).all())
    none = amr.MXFP4(torch.empty(0, 64, dtype=torch.uint8, device="cuda"),
                     torch.empty(0, 4, dtype=torch.uint8, device="cuda"))
    i32 = dict(dtype=torch.int32, device="cuda")
    out = amr.grouped_gemm_mxfp4(none, w, torch.zeros(1, **i32), torch.zeros(1, **i32), torch.zeros(1, **i32), 2, 32)
    assert out.shape == (1, 20)


def test_quantize_and_product_replayed_from_a_graph():
    """Captured once, replayed with new inputs: equal to the eager calls."""
    rng = np.random.default_rng(5)
    meta, npp = routed(rng, 96, 8, 2, 32)
    x = torch.randn(96, 300, device="cuda").bfloat16()
    w = amr.mxfp4_quantize(torch.randn(8, 40, 300, device="cuda"))
    q = amr.mxfp4_quantize(x)
    y = torch.zeros(amr.max_rows(96, 8, 2, 32), 40, device="cuda")
    args = (w, meta.sorted_ids, meta.expert_of_block, meta.num_post_pad, 2, 32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            amr.mxfp4_quantize(x, out=q)
            amr.grouped_gemm_mxfp4(q, *args, out=y)
    for i in range(4):
        x.copy_(torch.randn(96, 300, device="cuda") * (i + 1))
        graph.replay()
        want = amr.grouped_gemm_mxfp4(amr.mxfp4_quantize(x), *args, out=torch.zeros_like(y))
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_offsets_past_32_bits():
    """Rows and weights whose byte offsets pass 2^32: the last rows, the last experts."""
    K, rows = 65536, 70000
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, K, generator=torch.Generator(device="cuda").manual_seed(0), device="cuda").bfloat16()
    q = amr.mxfp4_quantize(x)
    codes, scales, _ = om.quantize(x[-3:].double().cpu().numpy())
    assert np.array_equal(q.codes[-3:].cpu().numpy(), codes) and np.array_equal(q.scales[-3:].cpu().numpy(), scales)
    assert not bool(q.codes[:-3].any())
    del x, q
    E, N, K, M, k = 3000, 256, 16384, 40, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    wc = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    ws = torch.randint(124, 131, (E, N, K // 32), dtype=torch.uint8, device="cuda", generator=g)
    rng = np.random.default_rng(2)
    xc, xs = random_rows(rng, (M,), K)
    for block in (16, 64):  # both by the few-rows kernel
        ids = np.stack([np.sort(rng.choice(np.arange(E - (20 if block == 16 else 4), E), k, replace=False))
                        for _ in range(M)]).astype(np.int32)
        out = amr.sort_from_ids(torch.from_numpy(ids).cuda(), E, block)
        y = amr.grouped_gemm_mxfp4(amr.MXFP4(*to_gpu(xc, xs)), amr.MXFP4(wc, ws), out.sorted_ids, out.expert_of_block,
                                   out.num_post_pad, k, block, out_dtype=torch.float32)
        npp = int(out.num_post_pad.item())
        lo = E - 20
        ref, ab = om.product(xc, xs, wc[lo:].cpu().numpy(), ws[lo:].cpu().numpy(), out.sorted_ids.cpu().numpy(),
                             out.expert_of_block.cpu().numpy() - lo, npp, M, k, block)
        assert (np.abs(y[:npp].double().cpu().numpy() - ref) <= om.tolerance(ref, ab, K, False)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [16, 32])
def test_weights_larger_than_the_caches(block, dtype):
    """More than 256 MB of weights: an expert's only row tile reads them past the
    L2, experts with several share them; both, side by side."""
    E, N, K, M, k, used = 300, 260, 7900, 150, 2, 16
    print(f"[gpu] mxfp4 product of large weights block={block} {dtype}", flush=True)
    Kp = (K + 127) // 128 * 128
    g = torch.Generator(device="cuda").manual_seed(3)
    wc = torch.randint(0, 256, (E, N, Kp // 2), dtype=torch.uint8, device="cuda", generator=g)
    wc[:, :, K // 2:] = 0
    ws = torch.randint(124, 131, (E, N, Kp // 32), dtype=torch.uint8, device="cuda", generator=g)
    assert wc.numel() > 256 << 20
    rng = np.random.default_rng(block)
    xc, xs = random_rows(rng, (M,), K)
    p = 0.8 ** np.arange(used)
    ids = np.stack([np.sort(rng.choice(np.arange(E - used, E), k, replace=False, p=p / p.sum()))
                    for _ in range(M)]).astype(np.int32)
    tiles = (np.bincount(ids.ravel(), minlength=E)[-used:] + block - 1) // block
    assert (tiles == 1).any() and (tiles > 1).any()
    out = amr.sort_from_ids(torch.from_numpy(ids).cuda(), E, block)
    y = amr.grouped_gemm_mxfp4(amr.MXFP4(*to_gpu(xc, xs)), amr.MXFP4(wc, ws), out.sorted_ids, out.expert_of_block,
                               out.num_post_pad, k, block,
                               out_dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    npp, lo = int(out.num_post_pad.item()), E - used
    ref, ab = om.product(xc, xs, wc[lo:].cpu().numpy(), ws[lo:].cpu().numpy(), out.sorted_ids.cpu().numpy(),
                         out.expert_of_block.cpu().numpy() - lo, npp, M, k, block)
    assert (np.abs(y[:npp].double().cpu().numpy() - ref) <= om.tolerance(ref, ab, K, dtype == "bf16")).all()
