"""The experts' entry points on another stream than the current one, on two streams
at once, with another current device, and their refusals of tensors."""
import contextlib

import pytest
import torch

import align_moe_route_amd as amr
from experts_cases import Routed, ids_of, normal

pytestmark = pytest.mark.gpu
PAUSE = 20_000_000  # cycles of a busy stream, about 10 ms

M, E, k, H, I, block = 96, 6, 2, 128, 40, 32


def parts():
    r = Routed(ids_of(M, E, k, 1), E, block)
    t = torch.bfloat16
    return dict(x=normal((M, H), t, 1), w1=normal((E, 2 * I, H), t, 2, 0.1), w2=normal((E, H, I), t, 3, 0.1),
                v=torch.rand(M, k, device="cuda"), dout=normal((M, H), t, 4), sid=r.meta[0], eob=r.meta[1], npp=r.meta[2],
                ids=r.ids), r.npp


def calls(p, npp, stream, fresh):
    """Every entry point, on `stream`; `fresh` gives the tensor that a call is handed."""
    def f(name):
        return fresh(p[name])
    meta = lambda: (f("sid"), f("eob"), f("npp"))  # noqa: E731
    a = amr.grouped_gemm(f("x"), f("w1"), *meta(), k, block, stream=stream)
    h = amr.swiglu(a, f("npp"), stream=stream)
    y = amr.grouped_gemm(h, f("w2"), *meta(), k, block, tokens=M, stream=stream)
    rows = amr.slot_rows(f("sid"), f("npp"), M, k, stream=stream)
    out = amr.combine(y, rows, f("v"), stream=stream)
    dy, dv = amr.combine_backward(f("dout"), rows, f("sid"), f("npp"), weights=f("v"), y=y, stream=stream)
    dw2 = amr.grouped_gemm_dw(dy, h, E, *meta(), k, block, tokens=M, stream=stream)
    dh = amr.grouped_gemm_dx(dy, f("w2"), *meta(), M, k, block, stream=stream)
    da = amr.swiglu_backward(a, dh, f("npp"), stream=stream)
    q1 = amr.int4_quantize(f("w1"), 32, stream=stream)
    q2 = amr.int4_quantize(f("w2"), 64, stream=stream)
    g = amr.int4_matvec(f("x"), q1, f("ids"), gated=True, stream=stream)
    s = amr.int4_matvec(g, q2, f("ids"), weights=f("v"), stream=stream)
    return [a[:npp], h[:npp], y[:npp], rows, out, dy[:npp], dv, dw2, dh[:npp], da[:npp], *q1, *q2, g, s]


def test_held_until_their_stream_has_passed():
    """Temporaries dropped at once, before the call's stream has started, and memory of
    the current stream given anew: neither reaches the results."""
    p, npp = parts()
    want = calls(p, npp, None, lambda t: t)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(PAUSE)

    def fresh(t):
        c = t.clone()
        torch.cuda.current_stream().synchronize()
        return c
    got = calls(p, npp, s, fresh)
    kept = [torch.full_like(t, 1) for t in (*p.values(), *got) for _ in range(3)]
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i
    del kept


def test_two_streams_at_once():
    p, npp = parts()
    want = calls(p, npp, None, lambda t: t)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append([calls(p, npp, None, lambda t: t) for _ in range(3)])
    torch.cuda.synchronize()
    for one in got:
        for again in one:
            assert all(torch.equal(a, b) for a, b in zip(again, want))


def test_current_device(monkeypatch):
    """With another device current, the tensors' becomes it for the call."""
    p, npp = parts()
    want = calls(p, npp, None, lambda t: t)
    entered = []

    @contextlib.contextmanager
    def device(d):
        entered.append(d)
        yield
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: p["x"].device.index + 1)
    got = calls(p, npp, None, lambda t: t)
    monkeypatch.undo()
    assert len(entered) == 13 and set(entered) == {p["x"].device}
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    p, npp = parts()
    meta = (p["sid"], p["eob"], p["npp"])
    x, w1 = p["x"], p["w1"]
    y = torch.zeros(amr.max_rows(M, E, k, block), 2 * I, device="cuda").bfloat16()
    dims = torch.zeros(M, k, 130, device="cuda")
    rows = amr.slot_rows(p["sid"], p["npp"], M, k)
    q = amr.int4_quantize(w1, 64)
    for i, call in enumerate((
            lambda: amr.grouped_gemm(x.cpu(), w1, *meta, k, block),
            lambda: amr.grouped_gemm(x, w1.half(), *meta, k, block),
            lambda: amr.grouped_gemm(x.t(), w1, *meta, k, block),
            lambda: amr.grouped_gemm(x[:, :64].contiguous(), w1, *meta, k, block),
            lambda: amr.grouped_gemm(x, w1, *meta, k, block, tokens=M),            # too few sorted rows
            lambda: amr.grouped_gemm(x, w1, p["sid"][:8], *meta[1:], k, block),    # metadata of other sizes
            lambda: amr.grouped_gemm(x, w1, meta[0].long(), *meta[1:], k, block),
            lambda: amr.grouped_gemm(x, w1, *meta, k, block, out=y[:, :3].contiguous()),
            lambda: amr.grouped_gemm(x, w1, *meta, k, block, out=y.float(), out_dtype=torch.bfloat16),
            lambda: amr.grouped_gemm(x.clone().requires_grad_(), w1, *meta, k, block),
            lambda: amr.grouped_gemm_dx(y[:9], w1, *meta, M, k, block),
            lambda: amr.grouped_gemm_dx(y, p["w2"], *meta, M, k, block),
            lambda: amr.grouped_gemm_dw(y, x.half(), E, *meta, k, block),
            lambda: amr.grouped_gemm_dw(y, x, E, *meta, k, block, out=y),
            lambda: amr.swiglu(y[:, :5].contiguous()),
            lambda: amr.swiglu(y, torch.zeros(1, device="cuda")),
            lambda: amr.swiglu_backward(y, y),
            lambda: amr.swiglu(y.clone().requires_grad_()),
            lambda: amr.slot_rows(p["sid"], p["npp"], -1, k),
            lambda: amr.slot_rows(p["sid"].cpu(), p["npp"], M, k),
            lambda: amr.combine(y, rows, p["v"][:5]),
            lambda: amr.combine(y, rows.long()),
            lambda: amr.combine(y[:7], 2),
            lambda: amr.combine(y, rows, p["v"].clone().requires_grad_()),
            lambda: amr.combine_backward(p["dout"], rows[:3], p["sid"], p["npp"]),
            lambda: amr.combine_backward(p["dout"], rows, p["sid"][:3], p["npp"], y=torch.zeros(
                y.shape[0], H, device="cuda").bfloat16()),
            lambda: amr.combine_backward(p["dout"], rows, p["sid"], p["npp"], y=y[:, :9].contiguous()),
            lambda: amr.experts_train(x, w1, p["w2"].half(), amr.RouteSortOutput(p["ids"], p["v"], *meta), block),
            lambda: amr.experts_train(x, w1[:, :70].contiguous(), p["w2"], amr.RouteSortOutput(p["ids"], p["v"], *meta),
                                      block),
            lambda: amr.int4_quantize(w1, 48),
            lambda: amr.int4_quantize(w1.transpose(0, 2)),
            lambda: amr.int4_matvec(x, (q.codes, q.scales), p["ids"]),
            lambda: amr.int4_matvec(x, amr.Int4(q.codes, q.scales.half()), p["ids"]),
            lambda: amr.int4_matvec(x, amr.Int4(q.codes[:, :, :32], q.scales), p["ids"]),
            lambda: amr.int4_matvec(x[:, :5].contiguous(), amr.Int4(q.codes[:, :, :0], q.scales), p["ids"]),
            lambda: amr.int4_matvec(dims.bfloat16(), q, p["ids"]),
            lambda: amr.int4_matvec(x, q, p["ids"].long()),
            lambda: amr.int4_matvec(x, q, p["ids"][:4]),
            lambda: amr.int4_matvec(x, q, p["ids"], gated=True, weights=p["v"]),
            lambda: amr.int4_matvec(x, q, p["ids"], weights=p["v"].double()),
            lambda: amr.int4_matvec(x.clone().requires_grad_(), q, p["ids"]),
            lambda: amr.int4_matvec(x, q, p["ids"], out=y))):
        with pytest.raises(ValueError):
            call()
            print("refusal", i, "is missing")
    for call in (lambda: amr.grouped_gemm(x.float(), w1.float(), *meta, k, block),
                 lambda: amr.grouped_gemm(x, w1, *meta, k, block, out_dtype=torch.float16),
                 lambda: amr.swiglu(y.float()), lambda: amr.combine(y.float(), rows),
                 lambda: amr.combine(y, rows, out_dtype=torch.float64), lambda: amr.int4_quantize(w1.double()),
                 lambda: amr.int4_matvec(x.float(), q, p["ids"])):
        with pytest.raises((NotImplementedError, amr.RouteSortError)):
            call()
    with pytest.raises(amr.RouteSortError):
        amr.grouped_gemm(x, w1, *meta, k, block, tile=64)
