"""The experts' operators at the ends of their ranges and as parts of other calls: the
longest rows, the most experts and picks, batches without a token or with dropped tokens
that hold NaN, one expert-parallel rank's metadata, a replayed graph of a decode step.

Inputs are small integers where sums are compared: every product and partial sum is an
integer below 2^24, so FP32 holds it and the results are exact before their rounding."""
import numpy as np
import pytest
import torch

import align_moe_route_amd as amr
from experts_cases import Routed, f64, ids_of, normal

pytestmark = pytest.mark.gpu


def whole(shape, seed, most=2, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("K,N", [(1 << 20, 1), (1 << 20, 9), (1, 1 << 20), ((1 << 20) - 3, 16), (8, (1 << 20) - 8)])
def test_longest_rows(K, N):
    M, E, k, block = 3, 2, 1, 16
    r = Routed(ids_of(M, E, k, 1), E, block)
    x, w = whole((M, K), 1, 1), whole((E, N, K), 2, 1)  # sums of at most 2^20
    dy = whole((r.cap, N), 3, 1)
    expert = torch.from_numpy(np.repeat(r.eob[:r.npp // block], block)).long().cuda()
    live = torch.from_numpy(r.live).cuda()
    token = torch.from_numpy(np.where(r.live, r.sid[:r.npp], 0) // k).long().cuda()
    y = amr.grouped_gemm(x, w, *r.meta, k, block, out_dtype=torch.float32)
    dx = amr.grouped_gemm_dx(dy, w, *r.meta, M, k, block, out_dtype=torch.float32)
    dw = amr.grouped_gemm_dw(dy, x, E, *r.meta, k, block)
    want = torch.zeros_like(w, dtype=torch.float32)
    for i in range(r.npp):
        if not live[i]:
            assert not y[i].any() and not dx[i].any()
            continue
        e, t = int(expert[i]), int(token[i])
        xs, ws, ds = x[t].double(), w[e].double(), dy[i].double()
        assert torch.equal(y[i].double(), (ws * xs).sum(1))
        assert torch.equal(dx[i].double(), (ws * ds[:, None]).sum(0))
        want[e] += dy[i].float()[:, None] * x[t].float()
    assert torch.equal(dw.float(), want)


@pytest.mark.parametrize("M,E,k,K,N,block", [
    (20, 6, 2, 203, 77, 256), (20, 6, 2, 200, 72, 1024), (300, 2, 1, 64, 600, 512), (700, 3, 1, 203, 600, 64),
    (4000, 2, 1, 64, 2100, 128), (2000, 100, 2, 64, 520, 2048), (500, 40, 2, 64, 264, 48), (1500, 300, 1, 67, 130, 32),
    (900, 300, 1, 72, 136, 96), (64, 64, 1, 40, 2048, 4096)])
def test_choices_of_tiles(M, E, k, K, N, block):
    """Tiles chosen by the sizes: few and many rows an expert, blocks of one tile and of many."""
    r = Routed(ids_of(M, E, k, 3, 0.05), E, block)
    x, w, dy = whole((M, K), 1, 1), whole((E, N, K), 2, 1), whole((r.cap, N), 3, 1)
    live = np.flatnonzero(r.live)
    expert = r.eob[live // block]
    y = amr.grouped_gemm(x, w, *r.meta, k, block, out_dtype=torch.float32)
    dx = amr.grouped_gemm_dx(dy, w, *r.meta, M, k, block, out_dtype=torch.float32)
    dw = amr.grouped_gemm_dw(dy, x, E, *r.meta, k, block, out_dtype=torch.float32)
    pad = torch.from_numpy(~r.live).cuda()
    assert not y[:r.npp][pad].any() and not dx[:r.npp][pad].any()
    for e in range(E):
        at = torch.from_numpy(live[expert == e]).cuda()
        a, b, d = x[torch.from_numpy(r.sid[live[expert == e]] // k).long().cuda()].double(), w[e].double(), dy[at].double()
        assert torch.equal(y[at].double(), a @ b.t())
        assert torch.equal(dx[at].double(), d @ b)
        assert torch.equal(dw[e].double(), d.t() @ a)


def test_most_experts_and_picks():
    M, E, k, K, N, block = 3, 4096, 64, 40, 24, 16
    ids = ids_of(M, E, k, 2)
    ids[0, -1], ids[1, 0] = E - 1, 0
    r = Routed(ids, E, block)
    x, w, v = whole((M, K), 1), whole((E, N, K), 2), whole((M, k), 3, 2, torch.float32)
    y = amr.grouped_gemm(x, w, *r.meta, k, block)
    rows = amr.slot_rows(r.meta[0], r.meta[2], M, k)
    out = amr.combine(y, rows, v, out_dtype=torch.float32)
    p = (w[r.ids.long()].double() * x[:, None, None, :].double()).sum(-1)  # [M, k, N], below 256: exact in BF16
    assert torch.equal(out.double(), (p * v[:, :, None].double()).sum(1))
    dout = whole((M, N), 4)
    dy, dv = amr.combine_backward(dout, rows, r.meta[0], r.meta[2], weights=v, y=y)
    assert torch.equal(dv.double(), (p * dout[:, None, :].double()).sum(-1))
    dw = amr.grouped_gemm_dw(dy, x, E, *r.meta, k, block, out_dtype=torch.float32)
    want = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
    for t in range(M):
        for j in range(k):
            want[ids[t, j]] += (v[t, j] * dout[t].double())[:, None] * x[t].double()
    assert torch.equal(dw.double(), want)
    # the same products from 4-bit weights: groups with a 7 in them have the scale 1
    w[:, :, 0::32] = 7
    q = amr.int4_quantize(w, 32)
    assert (q.scales[:, :, :2] == 1).all()
    p = (w[r.ids.long()].double() * x[:, None, None, :].double()).sum(-1)
    got = amr.int4_matvec(x, q, r.ids)
    assert torch.equal(got, p.to(got.dtype))
    got = amr.int4_matvec(x, q, r.ids, weights=v)
    assert torch.equal(got, (p * v[:, :, None].double()).sum(1).to(got.dtype))


@pytest.mark.parametrize("mode", ["plain", "sum"])
def test_longest_int4_rows(mode):
    K, N, E, M, k = 262144, 6, 3, 2, 2
    w, x = whole((E, N, K), 1, 7), whole((M, K), 2, 1)  # partial sums with 16 + c stay below 2^23
    w[:, :, 0::32] = 7
    q = amr.int4_quantize(w, 32)
    ids = torch.tensor([[0, 2], [1, 1]], dtype=torch.int32, device="cuda")
    v = torch.tensor([[1.0, 2.0], [-1.0, 3.0]], device="cuda")
    p = (w[ids.long()].double() * x[:, None, None, :].double()).sum(-1)
    got = amr.int4_matvec(x, q, ids, weights=v if mode == "sum" else None)
    want = (p * v[:, :, None].double()).sum(1) if mode == "sum" else p
    assert torch.equal(got, want.to(got.dtype))


def test_layer_without_a_token():
    E, k, H, I, block = 4, 2, 32, 16, 16
    x, w1, w2 = normal((0, H), torch.bfloat16, 1), normal((E, 2 * I, H), torch.bfloat16, 2), \
        normal((E, H, I), torch.bfloat16, 3)
    route = amr.route_sort(torch.zeros(0, E, device="cuda"), torch.zeros(E, device="cuda"), k, 2, 2, block)
    v = route.weights.clone().requires_grad_()
    for leaf in (x, w1, w2):
        leaf.requires_grad_()
    out = amr.experts_train(x, w1, w2, route._replace(weights=v), block)
    assert out.shape == (0, H)
    out.sum().backward()
    assert x.grad.shape == (0, H) and v.grad.shape == (0, k) and not w1.grad.any() and not w2.grad.any()


def test_int4_without_a_token():
    q = amr.int4_quantize(normal((3, 8, 40), torch.bfloat16, 1), 32)
    x, ids = torch.zeros(0, 40, device="cuda").bfloat16(), torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    assert amr.int4_matvec(x, q, ids).shape == (0, 2, 8)
    assert amr.int4_matvec(x, q, ids, gated=True).shape == (0, 2, 4)
    assert amr.int4_matvec(x, q, ids, weights=torch.zeros(0, 2, device="cuda")).shape == (0, 8)
    empty = amr.int4_quantize(torch.zeros(0, 40, device="cuda"), 32)
    assert empty.codes.shape == (0, 64) and empty.scales.shape == (0, 4)


def test_dropped_tokens_hold_anything():
    """Tokens without a pick hold NaN, in the input, the weights and the output's gradient."""
    M, E, k, H, I, block = 21, 3, 2, 40, 24, 32
    ids = ids_of(M, E, k, 5)
    gone = np.arange(M) % 4 == 1
    ids[gone] = -1
    r = Routed(ids, E, block)
    x, w1, w2 = normal((M, H), torch.bfloat16, 1), normal((E, 2 * I, H), torch.bfloat16, 2, H ** -0.5), \
        normal((E, H, I), torch.bfloat16, 3, I ** -0.5)
    v, dout = torch.rand(M, k, device="cuda"), normal((M, H), torch.bfloat16, 4)

    def run(value):
        at = torch.from_numpy(gone).cuda()
        a, b, c = x.clone(), v.clone(), dout.clone()
        a[at], b[at], c[at] = value, value, value
        leaves = [t.clone().requires_grad_() for t in (a, w1, w2, b)]
        out = amr.experts_train(*leaves[:3], amr.RouteSortOutput(r.ids, leaves[3], *r.meta), block)
        out.backward(c)
        assert not out[at].any() and not leaves[0].grad[at].any() and not leaves[3].grad[at].any()
        return [out, *(t.grad for t in leaves)]
    for a, b in zip(run(0.0), run(float("nan"))):
        assert a.isfinite().all() and torch.equal(a, b)


def test_ranks_of_an_expert_parallel_layer():
    """The outputs of ranks that own a range of the experts add up to the layer's."""
    M, E, k, H, I, block = 50, 16, 4, 64, 32, 16
    x, w1, w2 = whole((M, H), 1, 1), whole((E, 2 * I, H), 2, 1), whole((E, H, I), 3, 1)
    logits, bias = normal((M, E), torch.float32, 4), torch.zeros(E, device="cuda")
    dout = normal((M, H), torch.bfloat16, 5)

    def layer(route, a, b):
        leaves = [t.clone().requires_grad_() for t in (a, b)]
        amr.experts_train(x, *leaves, route, block).backward(dout)
        rows = amr.slot_rows(route.sorted_ids, route.num_post_pad, M, k)
        y = amr.grouped_gemm(amr.swiglu(amr.grouped_gemm(x, a, *route[2:], k, block), route.num_post_pad), b,
                             *route[2:], k, block, tokens=M)
        picks = torch.where((rows >= 0)[:, :, None], y[rows.clamp(min=0).long()], 0)  # a row for each pick
        return picks, [t.grad for t in leaves]
    route = amr.route_sort(logits, bias, k, 4, 2, block)
    want, grads = layer(route, w1, w2)
    total = torch.zeros_like(want)
    for begin, count in ((0, 5), (5, 1), (6, 10)):
        local = amr.route_sort(logits, bias, k, 4, 2, block, local=(begin, count))
        here = slice(begin, begin + count)
        picks, mine = layer(local, w1[here].contiguous(), w2[here].contiguous())
        total += picks  # each pick is one rank's
        for a, b in zip(mine, grads):
            assert torch.equal(a, b[here])
    assert torch.equal(total, want)


def test_replayed_decode_step():
    """A captured step of int4 products reads the ids of each replay, dropped ones among them."""
    M, E, k, H, I = 2, 12, 3, 200, 48
    up = amr.int4_quantize(normal((E, 2 * I, H), torch.bfloat16, 1, H ** -0.5), 64)
    down = amr.int4_quantize(normal((E, H, I), torch.bfloat16, 2, I ** -0.5), 32)
    x, v = normal((M, H), torch.bfloat16, 3), torch.rand(M, k, device="cuda")
    ids = torch.from_numpy(ids_of(M, E, k, 1)).cuda()

    def step():
        return amr.int4_matvec(amr.int4_matvec(x, up, ids, gated=True), down, ids, weights=v)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(2, 6):
        ids.copy_(torch.from_numpy(ids_of(M, E, k, seed, 0.3)))
        x.copy_(normal((M, H), torch.bfloat16, seed))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want) and f64(held).any()
