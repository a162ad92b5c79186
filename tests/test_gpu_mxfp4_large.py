"""Quantisation of more rows than one launch has threads for."""
import numpy as np
import pytest

from oracle import mxfp4 as om

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
amr = pytest.importorskip("align_moe_route_amd")


@pytest.mark.parametrize("rows,K,stride,values", [
    ((1 << 28) + 1000, 1, 1, True),   # 2^32 groups of eight columns and more: three launches
    (65540, 262144, 262144, False),   # 2^31 groups and four rows: two launches
    ((1 << 27) + 77, 3, 5, True),     # two launches, rows of another stride
])
def test_more_rows_than_a_launch(rows, K, stride, values):
    print(f"[gpu] mxfp4 quantize rows={rows} K={K} stride={stride}", flush=True)
    x = torch.zeros(rows, stride, dtype=torch.bfloat16, device="cuda")
    most = (1 << 31) // ((K + 127) // 128 * 16)  # rows of a launch
    at = sorted({r + d for r in range(0, rows, most) for d in (-2, -1, 0, 1)} | {rows - 1, rows - 2, rows // 3})
    at = torch.tensor([r for r in at if 0 <= r < rows], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(rows % 1000)
    x[at] = torch.randn(at.numel(), stride, device="cuda", generator=g).bfloat16()
    v = torch.full((rows, K), 7.0, dtype=torch.bfloat16, device="cuda") if values else None
    q = amr.mxfp4_quantize(x[:, :K], values=v)
    codes, scales, want = om.quantize(x[at][:, :K].double().cpu().numpy())
    assert np.array_equal(q.codes[at].cpu().numpy(), codes) and np.array_equal(q.scales[at].cpu().numpy(), scales)
    if values:
        assert np.array_equal(v[at].double().cpu().numpy(), want)
        v[at] = 0
        assert not bool(v.any())
    q.codes[at] = 0  # every other row is zeros
    q.scales[at] = 0
    assert not bool(q.codes.view(torch.int64).any()) and not bool(q.scales.view(torch.int32).any())
