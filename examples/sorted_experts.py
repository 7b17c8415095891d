"""Tokens sorted by expert, as a prompt or a training step uses them.

``serve``: a layer's experts in 4-bit block floating point next to the dense bf16 block: the
same router, the same routes, the error and the times of one step at several batch sizes.

``train``: a small MoE layer whose tokens are sorted by expert, multiplied expert by expert,
and brought back with the router's weights, all with gradients, fitted to a fixed target.

    python examples/sorted_experts.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch
from torch.autograd.function import once_differentiable

from routed_expert_ffn_top_gb300 import moe, synthetic as syn


# --------------------------------------------------------------------------------- autograd
class SortTokens(torch.autograd.Function):
    """Rows of x [M,H] in sorted order [M*k,H]."""

    @staticmethod
    def forward(ctx, x, route_row):
        ctx.save_for_backward(route_row)
        return moe.moe_token_sort(x, route_row)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_rows):
        (route_row,) = ctx.saved_tensors
        return moe.moe_token_sort_grad(grad_rows.contiguous(), route_row), None


class UnsortTokens(torch.autograd.Function):
    """The weighted sum [M,H] of each token's rows."""

    @staticmethod
    def forward(ctx, rows, route_row, weights):
        ctx.save_for_backward(rows, route_row, weights)
        return moe.moe_token_unsort(rows, route_row, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        rows, route_row, weights = ctx.saved_tensors
        grad_rows, grad_weights = moe.moe_token_unsort_grad(grad_out.contiguous(), rows, route_row, weights)
        return grad_rows, None, grad_weights


class SortedExperts(torch.nn.Module):
    """Router, then gated expert MLPs over sorted rows (fp32)."""

    def __init__(self, H, I, E, k):
        super().__init__()
        self.E, self.k = E, k
        self.router = torch.nn.Parameter(torch.randn(H, E) * 0.1)
        self.w_gate = torch.nn.Parameter(torch.randn(E, H, I) * H ** -0.5)
        self.w_up = torch.nn.Parameter(torch.randn(E, H, I) * H ** -0.5)
        self.w_down = torch.nn.Parameter(torch.randn(E, I, H) * I ** -0.5)

    def route(self, x):
        top = (x @ self.router).topk(self.k, dim=1)
        return top.indices.to(torch.int32), torch.softmax(top.values, dim=1)

    def forward(self, x):
        ids, weights = self.route(x)
        offsets, _, route_row = moe.moe_token_plan(ids, self.E)
        rows = SortTokens.apply(x, route_row)
        out = []
        bounds = offsets.tolist()
        for e in range(self.E):
            r = rows[bounds[e]:bounds[e + 1]]
            out.append((torch.nn.functional.silu(r @ self.w_gate[e]) * (r @ self.w_up[e])) @ self.w_down[e])
        return UnsortTokens.apply(torch.cat(out), route_row, weights)


def train(M=256, H=64, I=96, E=8, k=2, steps=60, device="cuda", seed=0):
    """Losses of a few steps of gradient descent towards a fixed random target."""
    torch.manual_seed(seed)
    layer = SortedExperts(H, I, E, k).to(device)
    x = torch.randn(M, H, device=device)
    target = torch.tanh(x @ torch.randn(H, H, device=device) * H ** -0.5)
    opt = torch.optim.Adam(layer.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        loss = (layer(x) - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


# ---------------------------------------------------------------------------------- serving
def _time(fn, n=20, replay=False):
    """us of a call, or of its launches replayed from a graph."""
    for _ in range(3):
        fn()
    if replay:
        fn = moe.capture_graph(lambda stream: fn()).replay
        fn()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(n):
        fn()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / n * 1e3


def serve(H=2048, I=768, E=128, k=8, sizes=(1, 21, 256), device="cuda", seed=0, replay=False):
    """Per batch size: (tokens, relative error of the 4-bit step against the bf16 block, us of the
    bf16 block, us of router and 4-bit step), called or replayed from a graph."""
    wl = syn.Workload("sorted_experts", H=H, I=I, E=E, k=k, b=0, M=max(sizes))
    dense = syn.make_layer(wl, seed=seed, device=device)
    four = moe.microscale_layer(dense)
    found = []
    for M in sizes:
        h = syn.make_hidden(wl, M=M, seed=seed, device=device)
        work, work4 = moe.alloc_workspace(dense, M, k, 0), moe.microscale_workspace(four, M, k)

        def block():
            return moe.moe_decode_block(h, dense, k, 0, workspace=work)[0]

        def step():
            ids, weights = moe.moe_route_topk(h, dense["w_router"], dense["bias"], k)
            return moe.moe_microscale_ffn(h, four, ids, weights, workspace=work4)

        a, b = block().double(), step().double()
        if moe.moe_read_device_status(work4):
            raise RuntimeError("device status set")
        found.append((M, float((a - b).norm() / a.norm()), _time(block, replay=replay),
                      _time(step, replay=replay)))
    return found


def main():
    for replay, how in ((False, "called"), (True, "replayed")):
        for M, err, t16, t4 in serve(replay=replay):
            print("%5d tokens, %-8s: bf16 block %7.1f us, router and 4-bit step %7.1f us (%s is faster), "
                  "relative difference %.3f" % (M, how, t16, t4, "bf16" if t16 < t4 else "4-bit", err))
    losses = train()
    print("training: loss %.4f -> %.4f in %d steps" % (losses[0], losses[-1], len(losses)))


if __name__ == "__main__":
    main()
