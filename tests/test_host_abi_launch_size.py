"""Products of more tiles than a launch has threads for are refused; no call here
reaches a launch."""
import pytest

import align_moe_route_amd as amr

P = 0x10000  # aligned fake device address: never dereferenced, validation fails first


@pytest.mark.parametrize("M,k,E,N,block", [
    (1 << 22, 8, 8, 2048, 16),      # 2^21 row tiles of 16, 8 column tiles: 2^24 workgroups of 256 threads
    (1 << 24, 8, 8, 8192, 128),     # 2^20 row tiles of 128, 32 column tiles
    (1 << 28, 1, 4096, 1, 16),      # 2^24 row tiles
    (1000, 2, 4096, 1 << 24, 256),  # few rows, many column tiles
])
@pytest.mark.parametrize("x_rows", [amr.MRS_X_TOKENS, amr.MRS_X_SORTED])
def test_product_of_too_many_tiles(M, k, E, N, block, x_rows):
    assert amr.max_rows(M, E, k, block) > 0
    assert amr.lib().moe_grouped_gemm_mxfp4(P, P, P, P, P, P, P, M, k, E, 128, N, block, x_rows, amr.MRS_DTYPE_BF16, P,
                                            None) == amr.MRS_ERR_OVERFLOW
