"""`stream=` of the 4-bit and balance entry points: what a call on another stream
than the current one allocates, fills, reads and writes."""
import numpy as np
import pytest

from oracle import balance as ob
from oracle import mxfp4 as om

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
amr = pytest.importorskip("align_moe_route_amd")

PAUSE = 20_000_000  # cycles of a busy stream, about 10 ms: longer than the host takes for the calls behind it


@pytest.mark.parametrize("default", [False, True])
def test_workspace_is_filled_on_its_stream(monkeypatch, default):
    monkeypatch.setattr(amr, "_ws_cache", {})
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    want = torch.cuda.default_stream() if default else s
    made_on = []
    zeros = torch.zeros

    def spy(*args, **kw):
        made_on.append(torch.cuda.current_stream().cuda_stream)
        return zeros(*args, **kw)

    x = torch.randn(300, 40, device="cuda")
    ids = torch.randint(0, 40, (300, 3), dtype=torch.int32, device="cuda")
    plain = amr.balance_loss(x, ids, workspace=torch.empty(amr.balance_workspace_bytes(300, 40, 3), dtype=torch.uint8,
                                                           device="cuda"))
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "zeros", spy)
    with torch.cuda.stream(other):
        got = amr.balance_loss(x, ids, stream=want)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert made_on == [want.cuda_stream]
    assert all(torch.equal(p, q) for p, q in zip(plain, got))


def test_outputs_leave_what_the_current_stream_still_reads():
    """The current stream has yet to copy a freed tensor when a call on another
    stream allocates its outputs."""
    x = torch.randn(4096, 4096, device="cuda")
    want = amr.mxfp4_quantize(x)
    old = torch.full_like(want.codes, 7)
    copy = torch.empty_like(old)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(PAUSE)
    copy.copy_(old)
    del old
    got = amr.mxfp4_quantize(x, stream=s)
    torch.cuda.synchronize()
    assert bool((copy == 7).all())
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)


def test_inputs_and_outputs_are_held_until_their_stream_has_passed():
    """Temporaries dropped at once, before the call's stream has started: what is
    allocated in their place must not reach the results."""
    g = torch.Generator(device="cuda").manual_seed(0)
    M, E, k, block, N, K = 512, 8, 2, 32, 64, 512
    xs = [torch.randn(M, K, device="cuda", generator=g) for _ in range(2)]
    logits = torch.randn(M, E, device="cuda", generator=g)
    ids = torch.stack([torch.randperm(E, device="cuda", generator=g)[:k].sort().values for _ in range(M)]).int()
    meta = amr.sort_from_ids(ids, E, block)
    w = amr.mxfp4_quantize(torch.randn(E, N, K, device="cuda", generator=g))
    gw = torch.randn(M, k, device="cuda", generator=g)
    npp = int(meta.num_post_pad)

    def calls(stream, fresh):
        q = amr.mxfp4_quantize(fresh(xs[0]), stream=stream)
        y = amr.grouped_gemm_mxfp4(q, w, *(fresh(t) for t in meta), k, block, out_dtype=torch.float32, stream=stream)
        bal = amr.balance_loss(fresh(logits), fresh(ids), stream=stream)
        grad = amr.router_backward(fresh(logits), fresh(ids), grad_weights=fresh(gw), balance=bal, stream=stream)
        return y[:npp], bal.loss, bal.counts, bal.shares, grad

    want = calls(None, lambda t: t)
    s = torch.cuda.Stream()
    amr.balance_loss(logits, ids, stream=s)  # its workspace
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(PAUSE)
    kept = []

    def fresh(t):
        c = t.clone()
        torch.cuda.current_stream().synchronize()  # made before the call; the call's stream is still busy
        return c

    got = calls(s, fresh)
    for t in (xs[0], logits, ids, gw, *meta, *got):  # blocks of every size that was dropped
        kept += [torch.full_like(t, 1) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    # and the references themselves
    c, sc, xv = om.quantize(xs[0].double().cpu().numpy())
    ref, ab = om.product(c, sc, w.codes.cpu().numpy(), w.scales.cpu().numpy(), meta.sorted_ids.cpu().numpy(),
                         meta.expert_of_block.cpu().numpy(), npp, M, k, block)
    assert (np.abs(want[0].double().cpu().numpy() - ref) <= om.tolerance(ref, ab, K, False)).all()
    loss, counts, _, _ = ob.balance(logits.double().cpu().numpy(), ids.cpu().numpy(), 1.0)
    assert np.array_equal(want[2].cpu().numpy(), counts) and abs(want[1].item() - loss) < 1e-4
