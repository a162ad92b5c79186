"""The experts' entry points on two streams that are held until both have all their calls:
what the calls of one stream write is not what the other's read."""
import pytest
import torch

from test_gpu_experts_streams import calls, parts

pytestmark = pytest.mark.gpu
PAUSE = 200_000_000  # cycles of a busy stream, about 100 ms: longer than the calls take to issue


def test_two_streams_with_calls_in_turn():
    p, npp = parts()
    other = {n: t.clone() for n, t in p.items()}
    other["x"], other["v"], other["dout"] = -2 * p["x"], p["v"] + 1, p["dout"] * 3
    want = [calls(q, npp, None, lambda t: t) for q in (p, other)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(PAUSE)
    got = [[], []]
    for _ in range(3):
        for i, (s, q) in enumerate(zip(streams, (p, other))):
            with torch.cuda.stream(s):
                got[i].append(calls(q, npp, None, lambda t: t))
    assert not any(s.query() for s in streams)  # neither has begun
    torch.cuda.synchronize()
    for one, w in zip(got, want):
        for again in one:
            for i, (a, b) in enumerate(zip(again, w)):
                assert torch.equal(a, b), i
    assert not torch.equal(want[0][4], want[1][4])
