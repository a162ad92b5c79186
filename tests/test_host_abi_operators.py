"""Refusals of the 4-bit and balance entry points, through the C ABI and the
binding; no call here reaches a launch."""
import pytest

import align_moe_route_amd as amr

torch = pytest.importorskip("torch")
P = 0x10000  # aligned fake device address: never dereferenced, validation fails first


def quant(x=P, dtype=0, rows=4, K=64, stride=64, codes=P, scales=P, values=None):
    return amr.lib().moe_mxfp4_quantize(x, dtype, rows, K, stride, codes, scales, values, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -1), (dict(K=0), -1), (dict(K=262145, stride=262145), -1), (dict(stride=63), -1),
    (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(x=None), -2), (dict(codes=None), -2), (dict(scales=None), -2),
    (dict(x=P + 2), -3), (dict(x=P + 1, dtype=1), -3), (dict(codes=P + 2), -3), (dict(values=P + 2), -3),
    (dict(rows=1 << 40), -5), (dict(rows=0, x=None), 0),
])
def test_quantize_codes(kw, code):
    assert quant(**kw) == code


def product(xc=P, xs=P, wc=P, ws=P, sid=P, eob=P, npp=P, M=4, k=2, E=8, K=128, N=16, block=16, x_rows=0, dt=1, y=P):
    return amr.lib().moe_grouped_gemm_mxfp4(xc, xs, wc, ws, sid, eob, npp, M, k, E, K, N, block, x_rows, dt, y, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), -1), (dict(k=0), -1), (dict(k=65), -1), (dict(E=0), -1), (dict(E=4097), -1), (dict(K=0), -1),
    (dict(K=64), -1), (dict(K=200), -1), (dict(N=0), -1), (dict(block=8), -1), (dict(block=24), -1),
    (dict(x_rows=2), -1), (dict(x_rows=-1), -1), (dict(dt=2), -1), (dict(M=2 ** 30, k=64), -5),
    (dict(M=1 << 20, N=2 ** 30), -5),
    (dict(xc=P + 8), -3), (dict(wc=P + 4), -3), (dict(xs=P + 2), -3), (dict(ws=P + 1), -3), (dict(y=P + 2), -3),
    (dict(sid=P + 2), -3), (dict(eob=P + 2), -3), (dict(npp=P + 2), -3), (dict(M=0), 0),
] + [({n: None}, -2) for n in ("xc", "xs", "wc", "ws", "sid", "eob", "npp", "y")])
def test_product_codes(kw, code):
    assert product(**kw) == code


def balance(logits=P, dt=0, ids=P, off=None, mask=None, M=4, E=8, k=2, B=1, loss=P, counts=P, tokens=P, shares=P,
            ws=P, nbytes=1 << 30):
    return amr.lib().moe_balance_loss(logits, dt, ids, off, mask, M, E, k, B, 1.0, loss, counts, tokens, shares, ws,
                                      nbytes, None)


SIZES = [(dict(M=-1), -1), (dict(E=0), -1), (dict(E=4097), -1), (dict(k=0), -1), (dict(k=65), -1), (dict(B=0), -1),
         (dict(B=2), -1), (dict(B=65536, off=P), -1), (dict(dt=2), -1), (dict(logits=None), -2), (dict(ids=None), -2),
         (dict(logits=P + 2), -3), (dict(logits=P + 1, dt=1), -3), (dict(ids=P + 2), -3), (dict(off=P + 2), -3),
         (dict(M=(1 << 30) + 1, k=1), -5), (dict(M=1 << 28, k=8), -5)]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(loss=None), -2), (dict(counts=None), -2), (dict(tokens=None), -2), (dict(shares=None), -2),
    (dict(loss=P + 2), -3), (dict(ws=None), -4), (dict(nbytes=64), -4), (dict(ws=P + 8), -3),
])
def test_balance_codes(kw, code):
    assert balance(**kw) == code


def backward(logits=P, dt=0, ids=P, gw=P, counts=P, tokens=P, gl=P, off=None, mask=None, M=4, E=8, k=2, B=1, out=P):
    return amr.lib().moe_router_backward(logits, dt, ids, gw, counts, tokens, gl, off, mask, M, E, k, B, 1.0, out, None)


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(out=None), -2), (dict(tokens=None), -2), (dict(gw=P + 2), -3), (dict(out=P + 2), -3), (dict(gl=P + 1), -3),
    (dict(M=0), 0),
])
def test_backward_codes(kw, code):
    assert backward(**kw) == code


def test_balance_workspace():
    assert amr.balance_workspace_bytes(0, 896, 16) > 0
    assert amr.balance_workspace_bytes(131072, 4096, 16) < 64 << 20
    for bad in ((-1, 8, 2, 1), (1, 0, 1, 1), (1, 5000, 1, 1), (1, 8, 65, 1), (1, 8, 2, 0)):
        with pytest.raises(ValueError):
            amr.balance_workspace_bytes(*bad)


def test_binding_refuses_host_tensors_and_wrong_types():
    x, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: amr.mxfp4_quantize(x), lambda: amr.balance_loss(x, ids), lambda: amr.router_backward(x, ids),
                 lambda: amr.grouped_gemm_mxfp4(amr.MXFP4(x, x), amr.MXFP4(x, x), ids, ids, ids, 2, 16),
                 lambda: amr.grouped_gemm_mxfp4((x, x), amr.MXFP4(x, x), ids, ids, ids, 2, 16)):
        with pytest.raises(ValueError):
            call()
