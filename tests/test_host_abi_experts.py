"""Refusals of the experts' entry points, through the C ABI; no call here reaches a
launch."""
import pytest

import align_moe_route_amd as amr

torch = pytest.importorskip("torch")
P = 0x10000  # aligned fake device address: never dereferenced, validation fails first


def product(a=P, b=P, dt=1, sid=P, eob=P, npp=P, M=4, k=2, E=8, K=40, N=24, block=16, rows=0, odt=1, out=P, which=""):
    L = amr.lib()
    if which == "_dx":
        return L.moe_grouped_gemm_dx(a, b, dt, sid, eob, npp, M, k, E, K, N, block, odt, out, None)
    return getattr(L, "moe_grouped_gemm" + which)(a, b, dt, sid, eob, npp, M, k, E, K, N, block, rows, odt, out, None)


@pytest.mark.parametrize("which", ["", "_dx", "_dw"])
@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), -1), (dict(k=0), -1), (dict(k=65), -1), (dict(E=0), -1), (dict(E=4097), -1), (dict(K=0), -1),
    (dict(K=(1 << 20) + 1), -1), (dict(N=0), -1), (dict(N=(1 << 20) + 1), -1), (dict(block=8), -1), (dict(block=24), -1),
    (dict(dt=0), -1), (dict(dt=3), -1), (dict(odt=2), -1), (dict(dt=2, odt=1), -1), (dict(M=2 ** 30, k=64), -5),
    (dict(a=P + 1), -3), (dict(b=P + 1), -3), (dict(out=P + 1), -3), (dict(out=P + 2, odt=0), -3),
    (dict(sid=P + 2), -3), (dict(eob=P + 2), -3), (dict(npp=P + 2), -3),
] + [({n: None}, -2) for n in ("a", "b", "sid", "eob", "npp", "out")])
def test_product_codes(kw, code, which):
    assert product(which=which, **kw) == code


@pytest.mark.parametrize("tile,code", [(8, -1), (48, -1), (256, -1), (128, -1), (-16, -1), (32, 0)])
def test_tile_codes(tile, code):
    """64 divides neither by 48 nor by 128; no token, so no launch."""
    L = amr.lib()
    assert L.moe_grouped_gemm_ex(P, P, 1, P, P, P, 0, 2, 8, 40, 24, 64, 0, 1, P, None, tile) == code
    assert L.moe_grouped_gemm_dx_ex(P, P, 1, P, P, P, 0, 2, 8, 40, 24, 64, 1, P, None, tile) == code


def test_no_tokens_need_no_launch():
    assert product(M=0) == 0 and product(M=0, which="_dx") == 0
    assert product(rows=2) == -1 and product(rows=2, which="_dw") == -1
    assert product(M=0, which="_dw", out=None) == -2  # dw is written even so


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -1), (dict(I=0), -1), (dict(I=262145), -1), (dict(dt=0), -1), (dict(rows=1 << 31), -1),
    (dict(rows=(1 << 31) - 1, I=9), -5), (dict(a=None), -2), (dict(out=None), -2), (dict(a=P + 1), -3),
    (dict(out=P + 1), -3), (dict(npp=P + 2), -3), (dict(rows=0, a=None), 0),
])
def test_swiglu_codes(kw, code, grad):
    c = dict(a=P, dh=P, dt=1, npp=None, rows=4, I=8, out=P)
    c.update(kw)
    L = amr.lib()
    rc = (L.moe_swiglu_backward(c["a"], c["dh"], c["dt"], c["npp"], c["rows"], c["I"], c["out"], None) if grad else
          L.moe_swiglu(c["a"], c["dt"], c["npp"], c["rows"], c["I"], c["out"], None))
    assert rc == code


@pytest.mark.parametrize("kw,code", [
    (dict(cap=-1), -1), (dict(M=-1), -1), (dict(k=0), -1), (dict(k=65), -1), (dict(cap=2 ** 31), -5),
    (dict(M=2 ** 26, k=64), -5), (dict(M=0, sid=None), 0), (dict(sid=None), -2), (dict(npp=None), -2),
    (dict(rows=None), -2), (dict(sid=P + 2), -3), (dict(npp=P + 2), -3), (dict(rows=P + 2), -3),
])
def test_slot_rows_codes(kw, code):
    c = dict(sid=P, npp=P, cap=64, M=4, k=2, rows=P)
    c.update(kw)
    assert amr.lib().moe_slot_rows(c["sid"], c["npp"], c["cap"], c["M"], c["k"], c["rows"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(cap=-1), -1), (dict(M=-1), -1), (dict(k=0), -1), (dict(k=65), -1), (dict(N=0), -1), (dict(N=1 << 21), -1),
    (dict(dt=0), -1), (dict(odt=2), -1), (dict(cap=2 ** 31), -5), (dict(M=2 ** 26, k=64), -5), (dict(M=2 ** 24, k=1, N=1 << 20), -5),
    (dict(M=0, y=None), 0), (dict(y=None), -2), (dict(out=None), -2), (dict(y=P + 1), -3), (dict(rows=P + 2), -3),
    (dict(v=P + 2), -3), (dict(out=P + 1), -3), (dict(out=P + 2, odt=0), -3),
])
def test_combine_codes(kw, code):
    c = dict(y=P, dt=1, rows=P, v=P, cap=64, M=4, k=2, N=8, odt=1, out=P)
    c.update(kw)
    assert amr.lib().moe_combine(c["y"], c["dt"], c["rows"], c["v"], c["cap"], c["M"], c["k"], c["N"], c["odt"], c["out"],
                                 None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(cap=-1), -1), (dict(M=-1), -1), (dict(k=0), -1), (dict(k=65), -1), (dict(N=0), -1), (dict(dt=0), -1),
    (dict(y=None), -1), (dict(dv=None), -1), (dict(cap=2 ** 31), -5), (dict(M=2 ** 26, k=64), -5), (dict(M=0, dout=None), 0),
    (dict(dout=None), -2), (dict(rows=None), -2), (dict(sid=None), -2), (dict(npp=None), -2), (dict(dy=None), -2),
    (dict(dout=P + 1), -3), (dict(y=P + 1), -3), (dict(rows=P + 2), -3), (dict(sid=P + 2), -3), (dict(npp=P + 2), -3),
    (dict(v=P + 2), -3), (dict(dy=P + 1), -3), (dict(dv=P + 2), -3),
])
def test_combine_backward_codes(kw, code):
    c = dict(dout=P, y=P, dt=1, rows=P, sid=P, npp=P, v=P, cap=64, M=4, k=2, N=8, dy=P, dv=P)
    c.update(kw)
    assert amr.lib().moe_combine_backward(c["dout"], c["y"], c["dt"], c["rows"], c["sid"], c["npp"], c["v"], c["cap"],
                                          c["M"], c["k"], c["N"], c["dy"], c["dv"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -1), (dict(K=0), -1), (dict(K=262145, stride=262145), -1), (dict(stride=63), -1), (dict(group=16), -1),
    (dict(group=96), -1), (dict(dt=3), -1), (dict(sdt=0), -1), (dict(rows=1 << 40), -5), (dict(rows=0, w=None), 0),
    (dict(w=None), -2), (dict(codes=None), -2), (dict(scales=None), -2), (dict(w=P + 2), -3), (dict(w=P + 1, dt=1), -3),
    (dict(codes=P + 2), -3), (dict(scales=P + 1), -3),
])
def test_int4_quantize_codes(kw, code):
    c = dict(w=P, dt=0, rows=4, K=64, stride=64, group=64, sdt=1, codes=P, scales=P)
    c.update(kw)
    assert amr.lib().moe_int4_quantize(c["w"], c["dt"], c["rows"], c["K"], c["stride"], c["group"], c["sdt"], c["codes"],
                                       c["scales"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), -1), (dict(k=0), -1), (dict(k=65), -1), (dict(E=0), -1), (dict(E=4097), -1), (dict(K=0), -1),
    (dict(K=262145), -1), (dict(N=0), -1), (dict(N=(1 << 20) + 1), -1), (dict(group=48), -1), (dict(dt=0), -1),
    (dict(mode=3), -1), (dict(mode=-1), -1), (dict(mode=1, N=7), -1), (dict(mode=2), -1), (dict(v=P), -1),
    (dict(M=0, x=None), 0), (dict(M=2 ** 25, k=64), -5), (dict(x=None), -2), (dict(codes=None), -2),
    (dict(scales=None), -2), (dict(ids=None), -2), (dict(y=None), -2), (dict(x=P + 1), -3), (dict(codes=P + 8), -3),
    (dict(scales=P + 1), -3), (dict(ids=P + 2), -3), (dict(mode=2, v=P + 2), -3), (dict(y=P + 1), -3),
])
def test_int4_matvec_codes(kw, code):
    c = dict(x=P, dt=1, codes=P, scales=P, ids=P, v=None, M=2, k=2, E=8, K=64, N=16, group=32, slot=0, mode=0, y=P)
    c.update(kw)
    assert amr.lib().moe_int4_matvec(c["x"], c["dt"], c["codes"], c["scales"], c["ids"], c["v"], c["M"], c["k"], c["E"],
                                     c["K"], c["N"], c["group"], c["slot"], c["mode"], c["y"], None) == code


def test_empty_tensors_have_no_address():
    """Without a token the weights of a sum, and their gradient, are empty."""
    L = amr.lib()
    assert L.moe_combine_backward(None, P, 1, None, P, P, None, 64, 0, 2, 8, P, None, None) == 0
    assert L.moe_int4_matvec(None, 1, P, P, None, None, 0, 2, 8, 64, 16, 32, 0, 2, None, None) == 0


@pytest.mark.parametrize("tile,code", [(amr.MRS_TILE_NARROW, -1), (amr.MRS_TILE_NARROW | 128, -1),
                                       (amr.MRS_TILE_NARROW | 64, 0), (amr.MRS_TILE_NARROW * 2 | 64, -1)])
def test_narrow_tile_codes(tile, code):
    L = amr.lib()
    assert L.moe_grouped_gemm_ex(P, P, 1, P, P, P, 0, 2, 8, 40, 24, 128, 0, 1, P, None, tile) == code
    assert L.moe_grouped_gemm_dx_ex(P, P, 1, P, P, P, 0, 2, 8, 40, 24, 128, 1, P, None, tile) == code
