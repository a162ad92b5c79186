"""Fine-tune the router of a mixture of experts whose experts are frozen in 4 bits.

    python examples/finetune_router.py --steps 60

The experts' two weight matrices are quantised once (mxfp4_quantize).  A step
routes a batch (route_sort_train), quantises its rows, runs both grouped products
over the routing metadata (grouped_gemm_mxfp4, the second on rows in sorted
order), mixes the experts' outputs by the routing weights, and trains the router's
matrix on the distance to a teacher's outputs plus the balance loss.  Only the
routing weights and the balance loss carry gradients, so the backward pass through
the layer is router_backward and one product.  All data is synthetic.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import align_moe_route_amd as amr  # noqa: E402


class FrozenExperts:
    """Gated experts in 4-bit rows: y = W2 . (silu(W1g x) * W1u x)."""

    def __init__(self, E, hidden, inner, generator):
        def make(n, k):
            w = torch.randn(E, n, k, device="cuda", generator=generator) * k ** -0.5
            return amr.mxfp4_quantize(w.bfloat16())
        self.inner = inner
        self.w1, self.w2 = make(2 * inner, hidden), make(hidden, inner)

    @torch.no_grad()
    def __call__(self, x, route, k, block):
        """x [M, hidden] bfloat16 -> the picked experts' outputs [M, k, hidden] float32."""
        M = x.shape[0]
        meta = (route.sorted_ids, route.expert_of_block, route.num_post_pad)
        h = amr.grouped_gemm_mxfp4(amr.mxfp4_quantize(x), self.w1, *meta, k, block)
        act = torch.nn.functional.silu(h[:, :self.inner]) * h[:, self.inner:]
        y = amr.grouped_gemm_mxfp4(amr.mxfp4_quantize(act), self.w2, *meta, k, block, tokens=M,
                                   out_dtype=torch.float32)
        # rows back to slots; padding rows and rows past num_post_pad land in a spare row
        row = torch.arange(y.shape[0], device=y.device)
        slot = torch.where(row < route.num_post_pad, route.sorted_ids.long(), M * k)
        out = torch.empty(M * k + 1, y.shape[1], device=y.device)
        out[slot] = y
        return out[:M * k].view(M, k, -1)


def run(steps=60, tokens=512, E=64, k=8, hidden=512, inner=192, block=32, coef=0.01, lr=0.004, seed=0, report=print):
    """Trains and returns the (distance, balance loss) of every step."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    experts = FrozenExperts(E, hidden, inner, g)
    teacher = torch.randn(E, hidden, device="cuda", generator=g) * hidden ** -0.5
    router = (teacher + 0.7 * torch.randn(E, hidden, device="cuda", generator=g) * hidden ** -0.5).requires_grad_()
    bias = torch.zeros(E, device="cuda")
    shape = (k, 1, 1, block)
    optimizer = torch.optim.Adam([router], lr=lr)
    history = []
    for step in range(steps):
        x = torch.randn(tokens, hidden, device="cuda", generator=g).bfloat16()
        with torch.no_grad():
            want = amr.route_sort(3.0 * (x.float() @ teacher.T), bias, *shape)
            target = (want.weights[:, :, None] * experts(x, want, k, block)).sum(1)
        route, balance = amr.route_sort_train(3.0 * (x.float() @ router.T), bias, *shape, balance_coef=coef)
        got = (route.weights[:, :, None] * experts(x, route, k, block)).sum(1)
        distance = ((got - target) ** 2).mean() / (target ** 2).mean()
        optimizer.zero_grad()
        (distance + balance.loss.sum()).backward()
        optimizer.step()
        history.append((distance.detach(), balance.loss.detach()[0]))
        if report and (step % 10 == 0 or step == steps - 1):
            c = balance.counts[0].float()
            report(f"step {step:3d}  distance {history[-1][0].item():.4f}  balance {history[-1][1].item():.5f}"
                   f"  tokens an expert {c.min().item():.0f}..{c.max().item():.0f}")
    return [(float(d), float(b)) for d, b in history]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args()
    run(a.steps, a.tokens)
