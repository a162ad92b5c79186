"""experts_train: the whole layer under autograd against a float64 chain, alone and
behind route_sort_train; decode with int4 experts behind the router.

Tolerance: every stage rounds its result to 16 bits (u = half a step, relative) and
its FP32 sums (steps of 2^-23 of the magnitudes); the chain below carries the bound of
each value's error through the maps that use it, with |silu'| <= 1.1, |silu''| <= 0.5,
and 5 % for the products of two errors."""
import numpy as np
import pytest
import torch

import align_moe_route_amd as amr
from experts_cases import HALF, STEP, Routed, f64, ids_of, normal
from oracle import experts as orc
from oracle import int4 as oi4

pytestmark = pytest.mark.gpu
A = np.abs


class Chain:
    """The layer slot by slot in float64, each value with a bound of the GPU's error."""

    def __init__(self, x, w1, w2, v, ids, dout, u):
        M, k = ids.shape
        E, two, H = w1.shape
        I = two // 2
        self.out, self.dx = np.zeros((M, H)), np.zeros((M, H))
        self.dw1, self.dw2, self.dv = np.zeros_like(w1), np.zeros_like(w2), np.zeros((M, k))
        b = self.bound = {n: np.zeros_like(getattr(self, n)) for n in ("out", "dx", "dw1", "dw2", "dv")}
        r = lambda n: (n / 16 + 16) * 2.0 ** -23  # roundings of an FP32 sum of n products
        mag = {n: np.zeros_like(b[n]) for n in b}
        for t in range(M):
            for j in range(k):
                e = ids[t, j]
                if e < 0:
                    continue
                a = w1[e] @ x[t]
                da_ = u * A(a) + r(H) * (A(w1[e]) @ A(x[t]))
                g, up = a[:I], a[I:]
                dg_, du_ = da_[:I], da_[I:]
                s = orc.sigmoid(g)
                silu, d1 = g * s, s + g * s * (1 - s)
                h = silu * up
                fast = (A(g) + 8) * 2.0 ** -23
                dh_ = 1.1 * dg_ * (A(up) + du_) + A(silu) * du_ + (u + fast) * A(h)
                y = w2[e] @ h
                dy_ = A(w2[e]) @ dh_ + u * A(y) + r(I) * (A(w2[e]) @ A(h))
                self.out[t] += v[t, j] * y
                b["out"][t] += v[t, j] * dy_
                mag["out"][t] += A(v[t, j] * y)
                self.dv[t, j] = dout[t] @ y
                b["dv"][t, j] = A(dout[t]) @ dy_ + r(H) * (A(dout[t]) @ A(y))
                gy = v[t, j] * dout[t]
                gy_ = u * A(gy)
                gh = gy @ w2[e]
                gh_ = gy_ @ A(w2[e]) + u * A(gh) + r(H) * (A(gy) @ A(w2[e]))
                self.dw2[e] += np.outer(gy, h)
                b["dw2"][e] += np.outer(gy_, A(h)) + np.outer(A(gy), dh_)
                mag["dw2"][e] += np.outer(A(gy), A(h))
                gg, gu = gh * up * d1, gh * silu
                gg_ = gh_ * A(up) * 1.1 + A(gh) * du_ * 1.1 + A(gh * up) * 0.5 * dg_ + u * A(gg) + \
                    A(gh * up) * s * (1 + A(g)) * fast
                gu_ = gh_ * A(silu) + A(gh) * 1.1 * dg_ + (u + fast) * A(gu)
                ga, ga_ = np.concatenate([gg, gu]), np.concatenate([gg_, gu_])
                self.dw1[e] += np.outer(ga, x[t])
                b["dw1"][e] += np.outer(ga_, A(x[t]))
                mag["dw1"][e] += np.outer(A(ga), A(x[t]))
                gx = ga @ w1[e]
                self.dx[t] += gx
                b["dx"][t] += ga_ @ A(w1[e]) + u * A(gx) + r(two) * (A(ga) @ A(w1[e]))
                mag["dx"][t] += A(gx)
        for n in ("out", "dw1", "dw2", "dx"):
            b[n] = 1.05 * (b[n] + r(M) * mag[n] + u * A(getattr(self, n))) + 1e-7

    def check(self, **got):
        for n, t in got.items():
            err = A(f64(t).reshape(getattr(self, n).shape) - getattr(self, n))
            bad = err > self.bound[n]
            assert not bad.any(), (n, float(np.max(err / (self.bound[n] + 1e-300))))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,E,k,H,I,block,dropped", [(1, 4, 2, 16, 8, 16, 0.0), (30, 4, 2, 72, 40, 32, 0.2),
                                                     (40, 3, 2, 67, 33, 16, 0.0), (70, 2, 1, 136, 72, 128, 0.0)])
def test_layer(M, E, k, H, I, block, dropped, dtype):
    t = HALF[dtype]
    r = Routed(ids_of(M, E, k, 3, dropped), E, block)
    x, w1, w2 = normal((M, H), t, 1), normal((E, 2 * I, H), t, 2, H ** -0.5), normal((E, H, I), t, 4, I ** -0.5)
    v = torch.rand(M, k, generator=torch.Generator().manual_seed(5)).cuda() + 0.1
    dout = normal((M, H), t, 6)
    for leaf in (x, w1, w2, v):
        leaf.requires_grad_()
    route = amr.RouteSortOutput(r.ids, v, *r.meta)
    out = amr.experts_train(x, w1, w2, route, block)
    out.backward(dout)
    c = Chain(f64(x), f64(w1), f64(w2), f64(v), r.ids.cpu().numpy(), f64(dout), STEP[t][0])
    c.check(out=out, dx=x.grad, dw1=w1.grad, dw2=w2.grad, dv=v.grad)
    # a second pass, whose gradient is an expanded one, adds up
    before = x.grad.clone()
    amr.experts_train(x, w1, w2, route, block).sum().backward()
    assert not torch.equal(before, x.grad) and x.grad.isfinite().all()


@pytest.mark.parametrize("need", [(1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1), (0, 0, 0, 0)])
def test_some_gradients_only(need):
    M, E, k, H, I, block = 20, 3, 2, 24, 16, 16
    r = Routed(ids_of(M, E, k, 3), E, block)
    parts = [normal((M, H), torch.bfloat16, 1), normal((E, 2 * I, H), torch.bfloat16, 2),
             normal((E, H, I), torch.bfloat16, 4), torch.rand(M, k, device="cuda")]

    def run(flags):
        leaves = [p.clone().requires_grad_(bool(f)) for p, f in zip(parts, flags)]
        out = amr.experts_train(*leaves[:3], amr.RouteSortOutput(r.ids, leaves[3], *r.meta), block)
        if any(flags):
            out.float().square().sum().backward()
        return out, [p.grad for p in leaves]
    out, grads = run(need)
    want_out, want = run((1, 1, 1, 1))
    assert torch.equal(out, want_out) and out.requires_grad == any(need)
    for g, w, f in zip(grads, want, need):
        assert (g is None) == (not f) and (not f or torch.equal(g, w))


def test_behind_the_router():
    """Gradients pass route.weights to the logits; the route is route_sort's."""
    M, E, k, H, I, block = 48, 16, 4, 64, 32, 16
    x, w1, w2 = normal((M, H), torch.bfloat16, 1), normal((E, 2 * I, H), torch.bfloat16, 2, H ** -0.5), \
        normal((E, H, I), torch.bfloat16, 3, I ** -0.5)
    logits, dout = normal((M, E), torch.float32, 4).requires_grad_(), normal((M, H), torch.bfloat16, 5)
    bias = torch.zeros(E, device="cuda")
    route, _ = amr.route_sort_train(logits, bias, k, 4, 2, block)
    amr.experts_train(x, w1, w2, route, block).backward(dout)
    plain = amr.route_sort(logits.detach(), bias, k, 4, 2, block)
    c = Chain(f64(x), f64(w1), f64(w2), f64(plain.weights), plain.ids.cpu().numpy(), f64(dout), STEP[torch.bfloat16][0])
    s = 1.0 / (1.0 + np.exp(-f64(logits)))
    ids = plain.ids.cpu().numpy()
    want, bound = np.zeros((M, E)), np.zeros((M, E))
    for t in range(M):
        st = s[t, ids[t]]
        T, d = st.sum(), st * (1 - st)
        want[t, ids[t]] = (c.dv[t] - c.dv[t] @ st / T) / T * d
        bound[t, ids[t]] = (c.bound["dv"][t] + c.bound["dv"][t] @ st / T) / T * d + 1e-6
    assert (A(f64(logits.grad) - want) <= bound).all()


def test_entry_points_make_the_same():
    """The calls that a captured step makes itself give what autograd gives, on every
    replay beside eager work."""
    M, E, k, H, I, block = 64, 6, 2, 128, 64, 32
    r = Routed(ids_of(M, E, k, 7), E, block)
    x, w1, w2 = normal((M, H), torch.bfloat16, 1), normal((E, 2 * I, H), torch.bfloat16, 2, H ** -0.5), \
        normal((E, H, I), torch.bfloat16, 3, I ** -0.5)
    v, dout = torch.rand(M, k, device="cuda"), normal((M, H), torch.bfloat16, 5)

    def step():
        a = amr.grouped_gemm(x, w1, *r.meta, k, block)
        h = amr.swiglu(a, r.meta[2])
        y = amr.grouped_gemm(h, w2, *r.meta, k, block, tokens=M)
        rows = amr.slot_rows(r.meta[0], r.meta[2], M, k)
        out = amr.combine(y, rows, v)
        dy, dv = amr.combine_backward(dout, rows, r.meta[0], r.meta[2], weights=v, y=y)
        dw2 = amr.grouped_gemm_dw(dy, h, E, *r.meta, k, block, tokens=M)
        da = amr.swiglu_backward(a, amr.grouped_gemm_dx(dy, w2, *r.meta, M, k, block), r.meta[2])
        dw1 = amr.grouped_gemm_dw(da, x, E, *r.meta, k, block)
        dx = amr.combine(amr.grouped_gemm_dx(da, w1, *r.meta, M, k, block), rows)
        return out, dx, dw1, dw2, dv

    def auto():
        leaves = [p.clone().requires_grad_() for p in (x, w1, w2, v)]
        out = amr.experts_train(*leaves[:3], amr.RouteSortOutput(r.ids, leaves[3], *r.meta), block)
        out.backward(dout)
        return out, *(p.grad for p in leaves)
    for got, want in zip(step(), auto()):
        assert torch.equal(got, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in (11, 12, 13):  # new inputs in the same memory; eager work between the replays
        x.copy_(normal((M, H), torch.bfloat16, seed))
        want = auto()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(held, want):
            assert torch.equal(got, w)


@pytest.mark.parametrize("M", [1, 3])
def test_decode_with_int4_experts(M):
    """Router, gated first product, second product and mix, from the router's ids."""
    E, k, H, I = 64, 4, 256, 96
    hidden = normal((M, H), torch.bfloat16, 1)
    w_gate = normal((E, H), torch.bfloat16, 2, H ** -0.5)
    up = amr.int4_quantize(normal((E, 2 * I, H), torch.bfloat16, 3, H ** -0.5), 64)
    down = amr.int4_quantize(normal((E, H, I), torch.bfloat16, 4, I ** -0.5), 32)
    _, route = amr.gate_route_sort(hidden, w_gate, torch.zeros(E, device="cuda"), k, 8, 4, 16)
    h = amr.int4_matvec(hidden, up, route.ids, gated=True)
    out = amr.int4_matvec(h, down, route.ids, weights=route.weights)
    ids, v = route.ids.cpu().numpy(), f64(route.weights)
    wu, wd = (oi4.values(q.codes.cpu().numpy(), f64(q.scales)) for q in (up, down))
    p = oi4.matvec(f64(hidden), wu, ids)
    want_h = oi4.silu_gate(p)
    u = STEP[torch.bfloat16][0]
    mag = oi4.matvec(A(f64(hidden)), A(wu), ids)
    # a chunk's partial sums are bounded by 55 |scale| sum |x| <= 55 / 7 of the group's largest product, far
    # below u; 2^-16 of the magnitudes covers them and the sigmoid
    eh = u * A(want_h) + 2.0 ** -16 * (1.1 * mag[..., :I] * A(p[..., I:]) + A(p[..., :I]) * mag[..., I:] + A(want_h)) * 8
    assert (A(f64(h) - want_h) <= eh).all()
    want = (oi4.matvec(want_h, wd, ids) * v[:, :, None]).sum(1)
    eo = (oi4.matvec(eh, A(wd), ids) * v[:, :, None]).sum(1) + u * A(want) + \
        2.0 ** -13 * (oi4.matvec(A(want_h), A(wd), ids) * v[:, :, None]).sum(1)
    assert (A(f64(out) - want) <= 1.05 * eo).all()
