"""Refusals of moe_grouped_gemm_mxfp4_ex's kernel argument; no call here reaches
a launch."""
import pytest

import align_moe_route_amd as amr

P = 0x10000  # aligned fake device address: never dereferenced, validation fails first


def product(kernel, M=4, k=2, E=8, K=128, N=16, block=16, xc=P):
    return amr.lib().moe_grouped_gemm_mxfp4_ex(xc, P, P, P, P, P, P, M, k, E, K, N, block, 0, 1, P, None, kernel)


@pytest.mark.parametrize("kernel,block,code", [
    (-1, 128, -1), (7, 128, -1), (amr.PRODUCT_TILE_32, 16, -1), (amr.PRODUCT_TILE_32, 48, -1),
    (amr.PRODUCT_TILE_64, 96, -1), (amr.PRODUCT_TILE_128, 64, -1), (amr.PRODUCT_TILE_128, 192, -1),
])
def test_kernels_that_do_not_fit(kernel, block, code):
    assert product(kernel, block=block) == code


@pytest.mark.parametrize("kernel", range(7))
def test_other_refusals_come_with_every_kernel(kernel):
    assert product(kernel, block=128, xc=None) == -2
    assert product(kernel, block=128, xc=P + 8) == -3
    assert product(kernel, block=128, K=64) == -1
    assert product(kernel, block=128, M=0) == 0
    assert product(kernel, block=128, M=1 << 22, N=1 << 28) == -5  # more tiles than a launch holds
