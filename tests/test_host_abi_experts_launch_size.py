"""The experts' calls at sizes that would take 2^32 threads in a launch are refused, from
the sizes on that the header names; no call here reaches a launch."""
import pytest

import align_moe_route_amd as amr

P = 0x10000  # aligned fake device address: never dereferenced, validation fails first


@pytest.mark.parametrize("M,k,E,K,N,block", [
    (1 << 16, 1, 1, 8, 1 << 20, 16),      # 4096 row tiles of 16, 4096 column tiles of 256
    (1 << 20, 4, 1, 8, 1 << 20, 128),     # 2^15 row tiles of 128
    (1 << 28, 1, 1, 8, 64, 16),           # 2^24 row tiles, one column tile
])
def test_products(M, k, E, K, N, block):
    L = amr.lib()
    assert amr.max_rows(M, E, k, block) * -(-N // 256) >= 1 << 27
    assert L.moe_grouped_gemm(P, P, 1, P, P, P, M, k, E, K, N, block, 0, 1, P, None) == amr.MRS_ERR_OVERFLOW
    assert L.moe_grouped_gemm_dx(P, P, 1, P, P, P, M, k, E, N, K, block, 1, P, None) == amr.MRS_ERR_OVERFLOW


@pytest.mark.parametrize("E,N,K", [(4096, 8191, 8193), (1, 1 << 20, 1 << 20), (4096, 1 << 20, 128)])
def test_weights_gradient(E, N, K):
    assert E * -(-N // 128) * -(-K // 128) >= 1 << 22
    assert amr.lib().moe_grouped_gemm_dw(P, P, 1, P, P, P, 4, 2, E, K, N, 16, 0, 1, P, None) == amr.MRS_ERR_OVERFLOW


@pytest.mark.parametrize("M,N", [(1 << 26, 1), (1 << 15, 1 << 20), ((1 << 25), 513)])
def test_combine(M, N):
    assert M * -(-N // 512) > (1 << 26) - 4
    assert amr.lib().moe_combine(P, 1, P, P, 64, M, 1, N, 1, P, None) == amr.MRS_ERR_OVERFLOW


@pytest.mark.parametrize("M,k,capacity", [(1 << 26, 1, 0), (1 << 20, 64, 64), ((1 << 26) - 2, 1, 256), (1 << 25, 1, (1 << 31) - 1)])
def test_combine_backward(M, k, capacity):
    assert M * k + capacity / 64 > (1 << 26) - 12
    assert amr.lib().moe_combine_backward(P, P, 1, P, P, P, P, capacity, M, k, 8, P, P, None) == amr.MRS_ERR_OVERFLOW


@pytest.mark.parametrize("M,k,capacity", [((1 << 31) - 256, 1, 64), (4, 2, (1 << 31) - 256)])
def test_slot_rows(M, k, capacity):
    assert amr.lib().moe_slot_rows(P, P, capacity, M, k, P, None) == amr.MRS_ERR_OVERFLOW


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_int4_matvec(mode):
    M, k, N = (1 << 23, 1, 64) if mode == 2 else (1 << 20, 64, 512)
    assert M * k * -(-N // 32) >= 1 << 24
    assert amr.lib().moe_int4_matvec(P, 1, P, P, P, P if mode == 2 else None, M, k, 8, 4096, N, 32, 0, mode, P,
                                     None) == amr.MRS_ERR_OVERFLOW


def test_int4_quantize():
    assert amr.lib().moe_int4_quantize(P, 0, (1 << 34) + 1, 128, 128, 32, 1, P, P, None) == amr.MRS_ERR_OVERFLOW
