"""Each kernel of the grouped 4-bit product, named by the test and not left to the
choice by sizes, at the places where its tiles, steps and stages end."""
import functools

import numpy as np
import pytest

from oracle import mxfp4 as om
from test_gpu_mxfp4 import DT, POISON, random_rows, routed, run_product, to_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
amr = pytest.importorskip("align_moe_route_amd")

KERNELS = {"rows16": (amr.PRODUCT_ROWS_16, 16), "rows32": (amr.PRODUCT_ROWS_32, 16),
           "tile16": (amr.PRODUCT_TILE_16, 16), "tile32": (amr.PRODUCT_TILE_32, 32),
           "tile64": (amr.PRODUCT_TILE_64, 64), "tile128": (amr.PRODUCT_TILE_128, 128)}


@pytest.fixture(params=list(KERNELS))
def kernel(request, monkeypatch):
    """The name of a kernel, which every product of the test then takes."""
    number, _ = KERNELS[request.param]
    monkeypatch.setattr(amr, "grouped_gemm_mxfp4", functools.partial(amr.grouped_gemm_mxfp4, kernel=number))
    print(f"[gpu] mxfp4 product by {request.param}", flush=True)
    return request.param


def check(got, ref, ab, Kp, bf16):
    assert (np.abs(got - ref) <= om.tolerance(ref, ab, Kp, bf16)).all()


SHAPES = [  # M, E, k, K, N, block, drop, skew; blocks that every kernel's rows divide
    (1, 8, 2, 128, 16, 128, 0, 0),       # one step, half of it
    (3, 8, 8, 256, 17, 128, 0, 0),       # one whole step
    (5, 4, 1, 100, 1, 256, 0, 0),
    (300, 3, 1, 2200, 72, 128, 0, 0),    # nine steps of 256: the scales are staged twice
    (130, 2, 1, 2100, 264, 256, 0, 0),   # the second stage is half a step; a second column tile of 8
    (150, 3, 1, 4500, 40, 128, 0, 0),    # 18 steps, three stages
    (60, 3, 1, 9000, 33, 384, 0, 0),     # 35 steps and a half, stores of single values
    (700, 8, 4, 896, 300, 128, 0, 0.5),
    (1000, 4, 2, 1152, 520, 256, 0.3, 1.0),
    (400, 5, 3, 33, 31, 384, 0, 0),
    (90, 6, 2, 2000, 70, 128, 1.0, 0),   # every route dropped
    (257, 3, 2, 640, 256, 128, 0, 0),
]


@pytest.mark.parametrize("in_order", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,E,k,K,N,block,drop,skew", SHAPES)
def test_shapes(kernel, M, E, k, K, N, block, drop, skew, dtype, in_order):
    rng = np.random.default_rng(M + K + N)
    got, ref, ab = run_product(rng, M, E, k, K, N, block, DT[dtype], in_order, drop, skew)
    check(got, ref, ab, om.padded(K), dtype == "bf16")


@pytest.mark.parametrize("factor", [1, 3])
def test_blocks_of_its_own_rows(kernel, factor):
    """The smallest block that the kernel takes, and an odd multiple of it."""
    block = KERNELS[kernel][1] * factor
    rng = np.random.default_rng(block)
    got, ref, ab = run_product(rng, 250, 7, 3, 1100, 100, block, torch.float32, False, 0.1, 0.5)
    check(got, ref, ab, om.padded(1100), False)


@pytest.mark.parametrize("block", [128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_last_tile_of_an_expert(kernel, block, dtype):
    """Experts whose rows end at, before and after each 16 and 32 of a tile of 128;
    an expert without any."""
    counts = [1, 15, 16, 17, 31, 32, 33, 0, 63, 64, 65, 95, 96, 97, 127, 128, 129, 160, 255, 256, 257]
    ids = np.repeat(np.arange(len(counts), dtype=np.int32), counts)
    rng = np.random.default_rng(block)
    rng.shuffle(ids)
    M, E, N, K = len(ids), len(counts), 68, 700
    meta = amr.sort_from_ids(torch.from_numpy(ids[:, None].copy()).cuda(), E, block)
    npp = int(meta.num_post_pad)
    xc, xs = random_rows(rng, (M,), K)
    wc, ws = random_rows(rng, (E, N), K)
    y = torch.full((amr.max_rows(M, E, 1, block), N), POISON, dtype=DT[dtype], device="cuda")
    amr.grouped_gemm_mxfp4(amr.MXFP4(*to_gpu(xc, xs)), amr.MXFP4(*to_gpu(wc, ws)), *meta, 1, block, out=y)
    sid = meta.sorted_ids.cpu().numpy()
    ref, ab = om.product(xc, xs, wc, ws, sid, meta.expert_of_block.cpu().numpy(), npp, M, 1, block)
    got = y.double().cpu().numpy()
    assert (got[npp:] == float(torch.tensor(POISON, dtype=DT[dtype]))).all()
    assert (got[:npp][sid[:npp] >= M] == 0).all()
    check(got[:npp], ref, ab, om.padded(K), dtype == "bf16")


def test_exact_sums(kernel):
    """Scales of one: every partial sum is a multiple of 1/4 below 2^22, exact in FP32."""
    def ones(xc, xs, wc, ws):
        xs[:], ws[:] = 127, 127
    rng = np.random.default_rng(4)
    got, ref, _ = run_product(rng, 500, 5, 2, 4224, 77, 128, torch.float32, False, edit=ones)
    assert np.array_equal(got, ref)


@pytest.mark.parametrize("K", [256, 2176, 4480])
@pytest.mark.parametrize("N", [40, 41])
def test_nan_blocks(kernel, K, N):
    """A NaN block, in the first and the last 32 columns, reaches its token's or its
    output's results and nothing else."""
    def edit(xc, xs, wc, ws):
        xs[0, 0] = 255      # also the row that padding rows could read
        xs[7, -1] = 255
        xs[9, -3] = 255     # in the half of a last step that is there
        ws[1, 2, 0] = 255
        ws[2, N - 1, -1] = 255
    rng = np.random.default_rng(K)
    got, ref, ab = run_product(rng, 300, 4, 2, K, N, 128, torch.float32, False, edit=edit)
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.isnan(ref).any()
    ok = ~np.isnan(ref)
    assert (np.abs(got - ref)[ok] <= om.tolerance(ref, ab, K, False)[ok]).all()


def test_scale_range(kernel):
    """Scales far apart: sums follow the larger; a result past FP32's range is infinite."""
    def edit(xc, xs, wc, ws):
        xs[:] = np.random.default_rng(1).integers(60, 190, xs.shape)
        ws[:] = np.random.default_rng(2).integers(60, 190, ws.shape)
    rng = np.random.default_rng(6)
    got, ref, ab = run_product(rng, 400, 4, 2, 512, 48, 128, torch.float32, False, edit=edit)
    past = np.abs(ref) > np.finfo(np.float32).max
    assert np.array_equal(got[past], np.copysign(np.inf, ref[past]))
    assert (np.abs(got - ref)[~past] <= om.tolerance(ref, ab, 512, False)[~past]).all()


@pytest.mark.parametrize("M,E", [(9000, 3), (20000, 2), (40000, 12), (140000, 3)])
def test_many_row_tiles(kernel, M, E):
    """Enough row tiles for runs of 2 to 16 of them on an XCD, in whole blocks and not."""
    rng = np.random.default_rng(M)
    got, ref, ab = run_product(rng, M, E, 1, 128, 7, 128, torch.float32, False)
    check(got, ref, ab, 128, False)


def test_foreign_experts(kernel):
    """Blocks of an expert outside [0, E) are not written."""
    rng = np.random.default_rng(3)
    meta, npp = routed(rng, 300, 6, 2, 128)
    xc, xs = random_rows(rng, (300,), 128)
    wc, ws = random_rows(rng, (6, 20), 128)
    eob = meta.expert_of_block.clone()
    eob[0], eob[1] = 6, -1
    y = torch.full((amr.max_rows(300, 6, 2, 128), 20), POISON, device="cuda")
    amr.grouped_gemm_mxfp4(amr.MXFP4(*to_gpu(xc, xs)), amr.MXFP4(*to_gpu(wc, ws)), meta.sorted_ids, eob,
                           meta.num_post_pad, 2, 128, out=y)
    assert bool((y[:256] == POISON).all()) and bool((y[256:npp] != POISON).all()) and bool((y[npp:] == POISON).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights_past_4_gib(kernel, dtype):
    """The last experts of weights whose byte offsets pass 2^32, which no cache holds:
    experts of one row tile and of several, side by side."""
    E, N, K, M, block, used = 2200, 260, 16384 - 128, 700, 128, 9
    g = torch.Generator(device="cuda").manual_seed(1)
    wc = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    ws = torch.randint(124, 131, (E, N, K // 32), dtype=torch.uint8, device="cuda", generator=g)
    assert wc.numel() > 1 << 32
    rng = np.random.default_rng(2)
    xc, xs = random_rows(rng, (M,), K)
    p = 0.6 ** np.arange(used)
    ids = rng.choice(np.arange(E - used, E), (M, 1), p=p / p.sum()).astype(np.int32)
    meta = amr.sort_from_ids(torch.from_numpy(ids).cuda(), E, block)
    y = amr.grouped_gemm_mxfp4(amr.MXFP4(*to_gpu(xc, xs)), amr.MXFP4(wc, ws), *meta, 1, block, out_dtype=DT[dtype])
    npp, lo = int(meta.num_post_pad), E - used
    ref, ab = om.product(xc, xs, wc[lo:].cpu().numpy(), ws[lo:].cpu().numpy(), meta.sorted_ids.cpu().numpy(),
                         meta.expert_of_block.cpu().numpy() - lo, npp, M, 1, block)
    check(y[:npp].double().cpu().numpy(), ref, ab, K, dtype == "bf16")
