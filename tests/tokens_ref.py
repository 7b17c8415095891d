"""Plain fp64 forms of the token sort and of 4-bit block floating point (CPU, torch)."""
import torch

VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def plan(ids, E):
    """(offsets, row_route, route_row) by a loop over the routes."""
    flat = ids.reshape(-1).tolist()
    order = [r for e in range(E) for r, i in enumerate(flat) if i == e] if len(flat) * E < 50000 else \
        sorted((r for r, i in enumerate(flat) if 0 <= i < E), key=lambda r: flat[r])
    n = len(order)
    dropped = [r for r, i in enumerate(flat) if not 0 <= i < E]
    offsets = [0] * (E + 1)
    for r in order:
        offsets[flat[r] + 1] += 1
    for e in range(E):
        offsets[e + 1] += offsets[e]
    route_row = [0] * len(flat)
    for row, r in enumerate(order):
        route_row[r] = row
    for i, r in enumerate(dropped):
        route_row[r] = ~(n + i)
    t = torch.int32
    return (torch.tensor(offsets, dtype=t), torch.tensor(order + [-1] * len(dropped), dtype=t),
            torch.tensor(route_row, dtype=t).reshape(ids.shape))


def at_rows(route_row):
    """(rows [M*k] owned by each route, live [M*k])."""
    f = route_row.reshape(-1).long()
    return torch.where(f < 0, ~f, f), f >= 0


def quantise(x):
    """fp64 [..., C] -> (codes uint8 [..., C] one per value, scale bytes [..., C/32]) from the
    definition."""
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    amax = torch.where(bad, torch.ones_like(amax), amax)
    _, e = torch.frexp(amax)
    X = torch.where(amax > 0, (e - 1 - 2).double(), torch.full_like(amax, -127.0)).clamp(-127, 127)
    v = torch.where(bad.unsqueeze(-1), torch.zeros_like(b), b) * torch.exp2(-X).unsqueeze(-1)
    mid = (VALUES[1:] + VALUES[:-1]) / 2
    low = torch.searchsorted(mid, v.abs().contiguous())  # a tie stays low
    tie = (low < 7) & (v.abs() == mid[low.clamp(max=6)]) & (low % 2 == 1)
    code = (low + tie.long()) | (torch.signbit(v).long() << 3)
    byte = torch.where(bad, torch.full_like(X, 255.0), X + 127)
    return code.reshape(x.shape).to(torch.uint8), byte.to(torch.uint8)


def pack(code, byte):
    """One code per value and scale bytes to the stored layout."""
    codes = code[..., 0::2] | (code[..., 1::2] << 4)
    nb = byte.shape[-1]
    scales = torch.zeros(byte.shape[:-1] + (-(-nb // 16) * 16,), dtype=torch.uint8)
    scales[..., :nb] = byte
    return codes.contiguous(), scales


def values(codes, scales):
    """fp64 values of stored codes and scales."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    v = VALUES[c & 7] * (1 - 2 * (c >> 3)).double()
    nb = v.shape[-1] // 32
    s = torch.exp2(scales[..., :nb].double() - 127)
    s = torch.where(scales[..., :nb] == 255, torch.full_like(s, float("nan")), s)
    return (v.reshape(*v.shape[:-1], nb, 32) * s.unsqueeze(-1)).flatten(-2)


def product(x, w, offsets):
    """fp64 rows [R,K] in groups times w [E,N,K]; rows past the last group are zero."""
    y = torch.zeros((x.shape[0], w.shape[1]), dtype=torch.float64)
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            y[lo:hi] = x[lo:hi] @ w[e].T
    return y
