"""Training a layer's experts over tokens sorted by expert, in 16 bits, with 8-bit checkpoints.

``ExpertMLP``: the gated expert MLPs of a layer as one function with gradients. The tokens are
sorted by expert, multiplied by the experts' weights group by group, and brought back with the
router's weights. Between the passes it keeps x, g and u in 8 bits (and y, which the router's
gradient needs); p is computed again and the sorted rows are restored from the tokens. What goes from
call to call is of x's type, so outputs and gradients pass three to four roundings to it.

``train``: a few steps of it towards a fixed target; ``memory``: what it keeps, beside 16 bits.

    python examples/grouped_experts.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch
from torch.autograd.function import once_differentiable

from routed_expert_ffn_top_gb300 import moe


class ExpertMLP(torch.autograd.Function):
    """out [M,H] of x [M,H], its routes' plan (offsets, route_row) and router weights [M,k] fp32, and
    w_gate, w_up [E,H,I], w_down [E,I,H] of x's type; `code`: the checkpoints' type; `work`: the calls'
    status word, which the caller reads.  Without one every call waits for its result and raises what
    the device found."""

    @staticmethod
    def forward(ctx, x, weights, w_gate, w_up, w_down, offsets, route_row, code, work=None):
        rows = moe.moe_token_sort(x, route_row)
        p, codes, scales = moe.moe_grouped_gated_product(rows, w_gate, w_up, offsets, checkpoint=code, workspace=work)
        y = moe.moe_grouped_product(p, w_down, offsets, workspace=work)
        ctx.save_for_backward(*moe.moe_checkpoint_quantize(x, dtype=code), codes, scales, y, weights, w_gate, w_up, w_down,
                              offsets, route_row)
        ctx.work = work
        return moe.moe_token_unsort(y, route_row, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        x8, xs, codes, scales, y, weights, w_gate, w_up, w_down, offsets, route_row = ctx.saved_tensors
        work, I = ctx.work, w_gate.shape[2]
        need_x, need_weights, need_gate, need_up, need_down = ctx.needs_input_grad[:5]
        grad_x = grad_gate = grad_up = grad_down = None
        grad_y, grad_weights = moe.moe_token_unsort_grad(grad_out.contiguous(), y, route_row, weights)
        if need_x or need_gate or need_up or need_down:
            grad_gu, p = moe.moe_grouped_gated_product_grad(grad_y, w_down, offsets, codes, scales, workspace=work)
        if need_down:
            grad_down = moe.moe_grouped_weight_grad(p, grad_y, offsets, dtype=w_down.dtype, workspace=work)
        if need_gate or need_up:
            rows = moe.moe_checkpoint_dequantize(x8, xs, dtype=y.dtype, route_row=route_row)
        if need_gate:
            grad_gate = moe.moe_grouped_weight_grad(rows, grad_gu[:, :I], offsets, dtype=w_gate.dtype, workspace=work)
        if need_up:
            grad_up = moe.moe_grouped_weight_grad(rows, grad_gu[:, I:], offsets, dtype=w_up.dtype, workspace=work)
        if need_x:
            grad_rows = moe.moe_grouped_product(grad_gu, (w_gate, w_up), offsets, transposed=True, workspace=work)
            grad_x = moe.moe_token_sort_grad(grad_rows, route_row)
        return grad_x, grad_weights if need_weights else None, grad_gate, grad_up, grad_down, None, None, None, None


class GroupedExperts(torch.nn.Module):
    """Router (fp32), then the experts."""

    def __init__(self, H, I, E, k, dtype=torch.bfloat16, code=torch.float8_e4m3fn):
        super().__init__()
        self.E, self.k, self.code = E, k, code
        self.router = torch.nn.Parameter(torch.randn(H, E) * 0.1)
        self.w_gate = torch.nn.Parameter((torch.randn(E, H, I) * H ** -0.5).to(dtype))
        self.w_up = torch.nn.Parameter((torch.randn(E, H, I) * H ** -0.5).to(dtype))
        self.w_down = torch.nn.Parameter((torch.randn(E, I, H) * I ** -0.5).to(dtype))
        self.register_buffer("work", torch.zeros(moe.MOE_GROUPED_STATUS_BYTES, dtype=torch.uint8), persistent=False)

    def forward(self, x):
        top = (x.float() @ self.router).topk(self.k, dim=1)
        offsets, _, route_row = moe.moe_token_plan(top.indices.to(torch.int32), self.E)
        return ExpertMLP.apply(x, torch.softmax(top.values, dim=1), self.w_gate, self.w_up, self.w_down, offsets, route_row,
                               self.code, self.work)


def train(M=512, H=128, I=192, E=8, k=2, steps=60, device="cuda", seed=0, code=torch.float8_e4m3fn):
    """Losses of a few steps of gradient descent towards a fixed random target."""
    torch.manual_seed(seed)
    layer = GroupedExperts(H, I, E, k, code=code).to(device)
    x = torch.randn(M, H, device=device).to(torch.bfloat16)
    target = torch.tanh(x.float() @ torch.randn(H, H, device=device) * H ** -0.5)
    opt = torch.optim.Adam(layer.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        loss = (layer(x).float() - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    if moe.moe_read_device_status(layer.work):
        raise RuntimeError("device status set")
    return losses


def memory(M=8192, H=2048, I=768, k=8):
    """Bytes kept between the passes for M tokens: (in 16 bits: sorted rows, g, u, p and y; in 8)."""
    R = M * k

    def eight(rows, cols):  # codes, and scales in rows of whole 16 bytes
        return rows * (cols + -(-cols // 512) * 16)
    return 2 * R * (2 * H + 3 * I), eight(M, H) + eight(R, 2 * I) + 2 * R * H


def main():
    for code in (torch.float8_e4m3fn, torch.int8):
        losses = train(code=code)
        print("%s: loss %.4f -> %.4f in %d steps" % (code, losses[0], losses[-1], len(losses)))
    a, b = memory()
    print("kept between the passes for 8192 tokens: %.0f MB in 16 bits, %.0f MB with checkpoints" % (a / 1e6, b / 1e6))


if __name__ == "__main__":
    main()
