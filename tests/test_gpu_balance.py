"""Balance loss, counts and the router's gradient on the GPU against the
float64 oracle (oracle/balance.py)."""
import numpy as np
import pytest

from oracle import balance as ob

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
amr = pytest.importorskip("align_moe_route_amd")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(M, E, k, B, masked, dtype, seed, spread=1.5):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((M, E)) * spread).to(DT[dtype])
    ids = np.argsort(-(rng.random((M, E)) if M * E < 1 << 22 else x.double().numpy()), axis=1)[:, :k].astype(np.int32)
    ids = np.sort(ids, axis=1)
    ids[rng.random(ids.shape) < 0.05] = -1
    ids[rng.random(ids.shape) < 0.02] = E
    off = None
    if B > 1:
        off = np.concatenate([[0], np.sort(rng.integers(0, M + 1, B - 1)), [M]]).astype(np.int32)
    mask = (rng.random(M) >= masked) if masked else None
    return x, ids, off, mask


def gpu(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def xmax(x64, mask):
    x = x64 if mask is None else x64[np.asarray(mask) != 0]
    x = np.abs(x[np.isfinite(x)])
    return min(float(x.max()), 200.0) if x.size else 0.0  # past that every score is 0, 1 or shifted


def check_forward(x, ids, off, mask, coef=0.3):
    out = amr.balance_loss(x.cuda(), gpu(ids), coef, seq_offsets=gpu(off), mask=gpu(mask))
    x64 = x.double().numpy()
    loss, counts, tokens, shares = ob.balance(x64, ids, coef, off, mask)
    assert np.array_equal(out.counts.cpu().numpy(), counts)
    assert np.array_equal(out.tokens.cpu().numpy(), tokens)
    E = x.shape[1]
    rel = ob.share_bound(xmax(x64, mask), E, int(tokens[:-1].max()))
    got = out.shares.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(shares))
    ok = ~np.isnan(shares)
    assert (np.abs(got - shares)[ok] <= (rel * shares + ob.FLUSH)[ok]).all()
    if np.isnan(loss):
        assert np.isnan(out.loss.item())
    else:
        assert abs(out.loss.item() - loss) <= (rel + 4 * ob.U) * abs(loss) + ob.FLUSH
    return out


SHAPES = [  # M, E, k, B, masked, dtype
    (1, 2, 1, 1, 0, "f32"), (1, 896, 16, 1, 0, "bf16"), (4, 64, 4, 1, 0, "f32"), (3, 7, 7, 1, 0, "bf16"),
    (5, 1, 1, 1, 0, "f32"), (65, 33, 5, 4, 0.3, "f32"), (512, 896, 16, 1, 0, "bf16"), (1000, 250, 8, 9, 0.1, "bf16"),
    (777, 897, 16, 3, 0.2, "f32"), (300, 1030, 3, 7, 0, "f32"), (64, 4096, 64, 5, 0.5, "f32"),
    (130, 4095, 16, 2, 0, "bf16"), (9000, 96, 6, 300, 0.1, "bf16"), (20, 16, 2, 60, 0.4, "f32"),
    (2048, 640, 8, 1, 0.9, "bf16"), (700, 3000, 8, 2, 0, "f32"), (41, 500, 4, 1, 0, "f32"), (50, 1600, 4, 3, 0, "bf16"),
    # sixteen lanes a row (one to four column groups, whole and cut) and more picks than lanes
    (333, 61, 7, 5, 0.2, "bf16"), (1500, 128, 8, 1, 0, "bf16"), (700, 190, 16, 40, 0.1, "f32"), (260, 256, 2, 2, 0, "f32"),
    (90, 100, 17, 3, 0.1, "f32"), (50, 64, 64, 1, 0, "bf16"), (77, 256, 33, 2, 0.3, "bf16"), (5000, 3, 2, 7, 0.1, "bf16"),
    # many short sequences of a wide router: two walkers a column in the second kernel
    (2000, 4000, 4, 70, 0.1, "bf16"),
]


@pytest.mark.parametrize("M,E,k,B,masked,dtype", SHAPES)
def test_balance(M, E, k, B, masked, dtype):
    print(f"[gpu] balance M={M} E={E} k={k} B={B} masked={masked} {dtype}", flush=True)
    x, ids, off, mask = make(M, E, k, B, masked, dtype, M + E)
    check_forward(x, ids, off, mask)


def check_backward(x, ids, off, mask, grad_w=True, balance=True, grad_loss=1.7, coef=0.3, seed=0):
    M, E = x.shape
    k = ids.shape[1]
    gw = np.random.default_rng(seed).standard_normal((M, k)).astype(np.float32) if grad_w else None
    x64 = x.double().numpy()
    counts = None
    bal = None
    if balance:
        _, counts, tokens, _ = ob.balance(x64, ids, coef, off, mask)
        bal = amr.BalanceOutput(None, gpu(counts.astype(np.int32)), gpu(tokens.astype(np.int32)), None)
    got = amr.router_backward(x.cuda(), gpu(ids), grad_weights=gpu(gw), balance=bal, coef=coef,
                              grad_loss=None if grad_loss is None else torch.full((1,), grad_loss, device="cuda"),
                              seq_offsets=gpu(off), mask=gpu(mask))
    assert got.dtype == x.dtype
    gl = 1.0 if grad_loss is None else float(np.float32(grad_loss))
    ref, size = ob.backward(x64, ids, float(np.float32(coef)), gl, gw, counts, off, mask)
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    half = 2.0 ** -8 if x.dtype == torch.bfloat16 else ob.U
    err = ob.grad_bound(xmax(x64, mask), E) * size + ob.FLUSH * max(1.0, float(np.nanmax(size)) * E)
    assert (np.abs(got - ref)[ok] <= (err + half * (np.abs(ref) + err))[ok]).all()
    if mask is not None:
        assert (got[np.asarray(mask) == 0] == 0).all()


@pytest.mark.parametrize("M,E,k,B,masked,dtype", SHAPES)
def test_backward(M, E, k, B, masked, dtype):
    print(f"[gpu] router backward M={M} E={E} k={k} B={B} masked={masked} {dtype}", flush=True)
    x, ids, off, mask = make(M, E, k, B, masked, dtype, M + E + 1)
    check_backward(x, ids, off, mask)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("grad_w,balance", [(True, False), (False, True), (False, False)])
def test_backward_terms(grad_w, balance, dtype):
    x, ids, off, mask = make(200, 384, 8, 3, 0.1, dtype, 4)
    check_backward(x, ids, off, mask, grad_w, balance, grad_loss=None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E", [48, 129, 300, 896, 1500])
def test_extreme_rows(E, dtype):
    """Rows of the type's lowest value, infinities, far-off rows whose scores
    underflow, and NaN or infinities in masked rows."""
    x, ids, _, _ = make(24, E, 4, 1, 0, dtype, E)
    low = torch.finfo(DT[dtype]).min
    x[0, :] = low
    x[1, :] = float("-inf")
    x[2, 1:] = float("-inf")
    x[3, ::2] = low
    x[4, :] = x[4] - 1000.0
    x[5, :] = x[5] - 80.0
    x[6, :] = x[6] - 40.0
    x[7, :] = x[7] + 60.0
    x[8, 3] = float("inf")
    x[9, :] = float("nan")
    x[10, 0] = float("inf")
    x[10, 1] = float("-inf")
    x[11, :] = float("-inf")
    x[11, 2] = -100.0
    x[12, 5] = torch.finfo(DT[dtype]).max
    mask = np.ones(24, bool)
    mask[9] = mask[10] = False
    out = check_forward(x, ids, None, mask)
    assert np.isfinite(out.loss.item())
    check_backward(x, ids, None, mask)
    check_forward(x, ids, np.array([0, 9, 11, 24], np.int32), mask)  # a sequence of masked rows only
    check_backward(x, ids, np.array([0, 9, 11, 24], np.int32), mask)


def test_unmasked_nan_is_not_hidden():
    x, ids, _, _ = make(12, 64, 4, 1, 0, "f32", 0)
    x[3, 7] = float("nan")
    off = np.array([0, 2, 6, 12], np.int32)
    out = check_forward(x, ids, off, None)
    assert np.isnan(out.loss.item()) and not np.isnan(out.shares[0].cpu().numpy()).any()
    ids[3] = np.arange(4)
    check_backward(x, ids, off, None, balance=False)


def test_everything_masked_and_no_tokens():
    x, ids, _, _ = make(10, 32, 4, 1, 0, "f32", 0)
    out = check_forward(x, ids, None, np.zeros(10, bool))
    assert out.loss.item() == 0.0
    check_backward(x, ids, None, np.zeros(10, bool))
    e = torch.empty(0, 32, device="cuda")
    i = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    out = amr.balance_loss(e, i, seq_offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert out.loss.item() == 0.0 and out.tokens.tolist() == [0, 0, 0] and not out.counts.any()
    assert amr.router_backward(e, i).shape == (0, 32)


def test_repeated_ids_add_up():
    x, ids, _, _ = make(40, 50, 4, 1, 0, "f32", 2)
    ids[:, 1] = ids[:, 0]
    ids[5] = 7
    check_forward(x, ids, None, None)
    check_backward(x, ids, None, None)


def test_same_inputs_same_bits_on_other_streams():
    x, ids, off, mask = make(5000, 300, 8, 11, 0.1, "bf16", 3)
    gx, gi, go, gm = x.cuda(), gpu(ids), gpu(off), gpu(mask)
    a = amr.balance_loss(gx, gi, seq_offsets=go, mask=gm)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append((amr.balance_loss(gx, gi, seq_offsets=go, mask=gm),
                         amr.router_backward(gx, gi, balance=a, seq_offsets=go, mask=gm)))
    torch.cuda.synchronize()
    for o, g in outs:
        assert all(torch.equal(p, q) for p, q in zip(a, o)) and torch.equal(g, outs[0][1])


def test_replayed_from_a_graph():
    x, ids, off, mask = make(600, 200, 8, 4, 0.1, "f32", 6)
    gx, gi, go, gm = x.cuda(), gpu(ids), gpu(off), gpu(mask)
    gw = torch.randn(600, 8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = amr.balance_loss(gx, gi, 0.1, seq_offsets=go, mask=gm)
        grad = amr.router_backward(gx, gi, grad_weights=gw, balance=out, coef=0.1, seq_offsets=go, mask=gm)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            amr.balance_loss(gx, gi, 0.1, seq_offsets=go, mask=gm, out=out)
            amr.router_backward(gx, gi, grad_weights=gw, balance=out, coef=0.1, seq_offsets=go, mask=gm, out=grad)
    for i in range(4):
        gx.copy_(torch.randn(600, 200, device="cuda"))
        gw.normal_()
        graph.replay()
        want = amr.balance_loss(gx, gi, 0.1, seq_offsets=go, mask=gm)
        wgrad = amr.router_backward(gx, gi, grad_weights=gw, balance=want, coef=0.1, seq_offsets=go, mask=gm)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)) and torch.equal(grad, wgrad)


def test_offsets_past_32_bits():
    """More than 2^31 logits: the last tokens' gradients, and the shares of a constant matrix."""
    M, E, k = 600000, 4096, 2
    x = torch.zeros(M, E, dtype=torch.bfloat16, device="cuda")
    ids = torch.randint(0, E, (M, k), dtype=torch.int32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0))
    out = amr.balance_loss(x, ids, 1.0)
    counts = torch.bincount(ids.reshape(-1).long(), minlength=E)
    assert torch.equal(out.counts[0].long(), counts) and out.tokens.tolist() == [M, 1]
    # equal shares; the chunks' sums add up to 2400 equal terms in FP32
    assert bool(((out.shares * E - 1).abs() <= 2600 * ob.U).all())
    assert abs(out.loss.item() - 1.0) <= 2700 * ob.U
    x[-5:] = torch.randn(5, E, device="cuda").bfloat16()
    gw = torch.randn(M, k, device="cuda")
    got = amr.router_backward(x, ids, grad_weights=gw)
    x64, i5 = x[-5:].double().cpu().numpy(), ids[-5:].cpu().numpy()
    ref, size = ob.backward(x64, i5, 1.0, 1.0, gw[-5:].cpu().numpy())
    err = ob.grad_bound(np.abs(x64).max(), E) * size + ob.FLUSH
    assert (np.abs(got[-5:].double().cpu().numpy() - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err)).all()
