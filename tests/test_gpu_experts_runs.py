"""Products whose row tiles go to the XCDs in runs of other lengths than an expert's tiles
would choose: one expert, few experts, blocks of many tiles.  Inputs are small integers:
every sum is exact."""
import numpy as np
import pytest
import torch

import align_moe_route_amd as amr
from experts_cases import Routed, ids_of

pytestmark = pytest.mark.gpu


def whole(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-1, 2, shape, generator=g).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("M,E,k,K,N,block", [
    (512, 1, 1, 72, 600, 128), (512, 1, 1, 67, 301, 128), (300, 8, 2, 136, 264, 128), (256, 4, 2, 200, 136, 64),
    (512, 8, 2, 64, 1536, 128), (256, 8, 2, 72, 136, 1024), (64, 16, 2, 67, 129, 2048), (64, 64, 1, 40, 264, 4096),
    (200, 4, 2, 64, 1024, 128), (1000, 2, 1, 40, 72, 64), (40, 20, 1, 24, 40, 1 << 14), (128, 1, 1, 64, 64, 16)])
def test_products(M, E, k, K, N, block):
    r = Routed(ids_of(M, E, k, 3, 0.05), E, block)
    x, w, dy = whole((M, K), 1), whole((E, N, K), 2), whole((r.cap, N), 3)
    live = np.flatnonzero(r.live)
    expert = r.eob[live // block]
    y = torch.full((r.cap, N), 7.0, device="cuda")
    dx = torch.full((r.cap, K), 7.0, device="cuda")
    amr.grouped_gemm(x, w, *r.meta, k, block, out_dtype=torch.float32, out=y)
    amr.grouped_gemm_dx(dy, w, *r.meta, M, k, block, out_dtype=torch.float32, out=dx)
    pad = torch.from_numpy(~r.live).cuda()
    assert not y[:r.npp][pad].any() and not dx[:r.npp][pad].any()
    assert (y[r.npp:] == 7.0).all() and (dx[r.npp:] == 7.0).all()
    for e in range(E):
        at = torch.from_numpy(live[expert == e]).cuda()
        token = torch.from_numpy(r.sid[live[expert == e]] // k).long().cuda()
        assert torch.equal(y[at].double(), x[token].double() @ w[e].double().t())
        assert torch.equal(dx[at].double(), dy[at].double() @ w[e].double())
