"""Plain fp64 forms of the grouped products and of the 8-bit checkpoint (torch, any device)."""
import torch

LARGEST = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def groups(sizes):
    return torch.tensor([0] + list(torch.tensor(sizes).cumsum(0)), dtype=torch.int32)


def spans(offsets):
    b = offsets.tolist()
    return [(e, b[e], b[e + 1]) for e in range(len(b) - 1)]


def product(rows, w, offsets, transposed=False):
    """fp64 rows times their expert's weights; zero past the last group."""
    y = torch.zeros((rows.shape[0], w.shape[1 if transposed else 2]), dtype=torch.float64, device=rows.device)
    for e, lo, hi in spans(offsets):
        m = w[e].double()
        y[lo:hi] = rows[lo:hi].double() @ (m.t() if transposed else m)
    return y


def weight_grad(rows, grads, offsets):
    out = torch.zeros((len(offsets) - 1, rows.shape[1], grads.shape[1]), dtype=torch.float64, device=rows.device)
    for e, lo, hi in spans(offsets):
        out[e] = rows[lo:hi].double().t() @ grads[lo:hi].double()
    return out


def gate(g, u):
    return g * torch.sigmoid(g) * u


def gate_grad(q, g, u):
    s = torch.sigmoid(g)
    return torch.cat((q * u * s * (1 + g * (1 - s)), q * g * s), 1)


def code_values(dtype):
    """The nonnegative codes' values in order."""
    if dtype is torch.int8:
        return torch.arange(128, dtype=torch.float64)
    return torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def quantise(x, dtype):
    """[R, C] -> (codes of `dtype` [R, C], scale bytes [R, pitch]) from the definition."""
    R, C = x.shape
    b = x.double().cpu().reshape(R, -1, 32)
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad.unsqueeze(-1), torch.zeros_like(b), b)
    amax = b.abs().amax(-1)
    # powers of two in order, the first that brings the largest magnitude within the codes
    power = torch.arange(-127, 128, dtype=torch.float64)
    X = torch.searchsorted(LARGEST[dtype] * torch.exp2(power), amax).double() - 127
    v = b * torch.exp2(-X).unsqueeze(-1)
    grid = code_values(dtype)
    mid = (grid[1:] + grid[:-1]) / 2
    at = torch.searchsorted(mid, v.abs().contiguous())  # a tie stays low
    tie = (at < len(mid)) & (v.abs() == mid[at.clamp(max=len(mid) - 1)]) & (at % 2 == 1)
    at = at + tie.long()
    if dtype is torch.int8:
        codes = torch.where(v < 0, -at, at).to(torch.int8)
    else:
        sign = torch.signbit(b) & ~bad.unsqueeze(-1)
        codes = (at | (sign.long() << 7)).to(torch.uint8).view(torch.float8_e4m3fn)
    scales = torch.zeros((R, -(-C // 512) * 16), dtype=torch.uint8)
    scales[:, :C // 32] = torch.where(bad, 255, (X + 127).to(torch.int64)).to(torch.uint8)
    return codes.reshape(R, C), scales


def values(codes, scales):
    """fp64 values of a checkpoint."""
    R, C = codes.shape
    s = scales[:, :C // 32].double()
    s = torch.where(s == 255, torch.full_like(s, float("nan")), torch.exp2(s - 127))
    return (codes.float().double().reshape(R, -1, 32) * s.unsqueeze(-1)).reshape(R, C)
