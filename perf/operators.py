"""Timed cases of the token sort and of the microscaled (4-bit) experts.

The operators, per call of `run`:

* ``route``: the forward pass of sorting -- the plan (stable order of the routes by expert),
  the token rows copied into that order, and the experts' rows brought back with their weights;
* ``grad``: the gradients of the way there and back;
* ``quantise``: a matrix to 4-bit codes with one power-of-two scale per 32 and back to values;
* ``product``: token rows quantised into sorted order, then the grouped product with 4-bit
  weights;
* ``experts``: the whole 4-bit expert step of a layer -- plan, quantised sort, gate/up product
  with SiLU, down product, and the weighted way back.

With ``own`` false `run` computes them in elementary torch operations in 32 bits; with
``own`` true it calls this package's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 32
# the magnitudes of a 4-bit code (one sign, two exponent bits, one mantissa bit)
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decoded token of a 128-expert layer: launch latency is what counts
        {"name": "route_1", "op": "route", "M": 1, "k": 8, "E": 128, "H": 2048, "dtype": "bf16", "drop": 0.0},
        # a prompt of 8192 tokens through the same layer
        {"name": "route_8192", "op": "route", "M": 8192, "k": 8, "E": 128, "H": 2048, "dtype": "bf16", "drop": 0.0},
        # a small ragged training micro-batch in 32 bits, odd width, dropped routes
        {"name": "grad_77_odd", "op": "grad", "M": 77, "k": 5, "E": 24, "H": 1033, "dtype": "f32", "drop": 0.05},
        # a training micro-batch of 8192 tokens
        {"name": "grad_8192", "op": "grad", "M": 8192, "k": 8, "E": 128, "H": 2048, "dtype": "bf16", "drop": 0.0},
        # the activations of 21 tokens
        {"name": "quantise_21", "op": "quantise", "M": 21, "H": 2048, "dtype": "bf16"},
        # one layer's gate and up weights, quantised once when a model is loaded
        {"name": "quantise_weights", "op": "quantise", "M": 128 * 1536, "H": 2048, "dtype": "bf16"},
        # one token's gate/up product alone
        {"name": "product_1", "op": "product", "M": 1, "k": 8, "E": 128, "N": 1536, "K": 2048, "dtype": "bf16", "drop": 0.0},
        # a ragged middle: odd row count, widths that end inside every tile, 32-bit results
        {"name": "product_517_odd", "op": "product", "M": 517, "k": 3, "E": 20, "N": 1000, "K": 1184, "dtype": "f32", "drop": 0.05},
        # the down product of a 4096-wide layer over a long prompt
        {"name": "product_4096", "op": "product", "M": 4096, "k": 8, "E": 64, "N": 4096, "K": 1536, "dtype": "bf16", "drop": 0.0},
        # the layer at one token, at 21 tokens and over a prompt of 8192 tokens
        {"name": "experts_1", "op": "experts", "M": 1, "k": 8, "E": 128, "H": 2048, "I": 768, "dtype": "bf16", "drop": 0.0},
        {"name": "experts_21", "op": "experts", "M": 21, "k": 8, "E": 128, "H": 2048, "I": 768, "dtype": "bf16", "drop": 0.0},
        {"name": "experts_8192", "op": "experts", "M": 8192, "k": 8, "E": 128, "H": 2048, "I": 768, "dtype": "bf16", "drop": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "grad", "quantise", "product", "experts"))
    c = {"op": op}
    if op == "quantise":
        c.update(M=_log(rng, 1, 65536), H=BLOCK * _log(rng, 1, 128), dtype=rng.choice(("bf16", "f16", "f32")))
    else:
        E = 8 * _log(rng, 1, 32)
        c.update(M=_log(rng, 1, 4096), k=rng.randint(1, 8), E=E, drop=rng.choice((0.0, 0.0, 0.05)))
    if op in ("route", "grad"):
        c.update(H=rng.choice((_log(rng, 64, 4096), 8 * _log(rng, 8, 512))), dtype=rng.choice(("bf16", "bf16", "f16", "f32")))
    elif op == "product":
        c.update(N=rng.choice((_log(rng, 32, 2048), 64 * rng.randint(1, 32))), K=BLOCK * _log(rng, 2, 64),
                 dtype=rng.choice(("bf16", "bf16", "f16", "f32")))
    elif op == "experts":
        c.update(H=BLOCK * _log(rng, 4, 64), I=BLOCK * rng.randint(2, 32), dtype="bf16")
    for key in ("H", "N", "K"):
        if c.get(key) == 3072:
            c[key] += BLOCK
    if c["M"] * c.get("k", 1) == 3072:
        c["M"] += 1
    return c


# --------------------------------------------------------------------------- plain forms
def _plain_quantise(x):
    """fp32 [R, C] -> (code values fp32 [R, C], scale exponents int32 [R, C/32])."""
    R, C = x.shape
    b = x.reshape(R, C // BLOCK, BLOCK)
    amax = b.abs().amax(-1)
    mant, e = torch.frexp(amax)  # amax = mant 2^e with mant in [0.5, 1)
    e = torch.where(amax > 0, e - 1 - 2, torch.full_like(e, -127)).clamp(-127, 127)
    v = torch.ldexp(torch.ldexp(b, (-e // 2).unsqueeze(-1)), (-e - (-e // 2)).unsqueeze(-1))
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6.0)  # round to even on each binade's grid
    return torch.copysign(q, v).reshape(R, C), e


def _power(e):
    """2^e in 32 bits for int exponents."""
    return torch.ldexp(torch.ones(e.shape, device=e.device), e)


def _pack(q, e):
    """Code values and exponents to bytes: two codes a byte, scale rows padded to 16 bytes."""
    grid = torch.tensor(MAGNITUDES, device=q.device)
    code = torch.searchsorted(grid, q.abs()).to(torch.uint8) | (torch.signbit(q).to(torch.uint8) << 3)
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
    nb = e.shape[1]
    scales = torch.zeros((q.shape[0], -(-nb // 16) * 16), dtype=torch.uint8, device=q.device)
    scales[:, :nb] = (e + 127).to(torch.uint8)
    return codes, scales


def _values(codes, scales):
    """fp32 values of packed codes [..., C/2] and scale bytes [..., pitch]."""
    lut = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=codes.device)
    v = torch.stack((lut[(codes & 15).long()], lut[(codes >> 4).long()]), -1).flatten(-2)
    nb = v.shape[-1] // BLOCK
    s = _power(scales[..., :nb].int() - 127)
    return (v.unflatten(-1, (nb, BLOCK)) * s.unsqueeze(-1)).flatten(-2)


def _plain_plan(ids, E):
    flat = ids.reshape(-1)
    R = flat.numel()
    valid = (flat >= 0) & (flat < E)
    key = torch.where(valid, flat, E)
    order = torch.sort(key, stable=True).indices  # row -> route, dropped routes last
    rows = torch.empty(R, dtype=torch.int64, device=ids.device)
    rows[order] = torch.arange(R, device=ids.device)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    counts.index_add_(0, key.long(), torch.ones_like(rows))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = counts[:E].cumsum(0)
    route_row = torch.where(valid, rows, -1 - rows).to(torch.int32).reshape(ids.shape)
    row_route = torch.where(valid[order], order, -1).to(torch.int32)
    return offsets, row_route, route_row


def _gather_rows(rows, route_row):
    """fp32 [M, k, H]: the row of every route, zero for a dropped one."""
    r = rows.float()[route_row.clamp(min=0).long()]
    return torch.where((route_row >= 0).unsqueeze(-1), r, 0.0)


def _plain_product(x, offsets, codes, scales):
    """fp32 rows x [R, K] in groups times the weights of each group's expert: fp32 [R, N]."""
    counts = offsets[1:] - offsets[:-1]
    used = counts.nonzero()[:, 0]
    R, N = x.shape[0], codes.shape[1]
    y = torch.zeros((R, N), device=x.device)
    if used.numel() == 0:
        return y
    cap = int(counts.max())
    i = torch.arange(cap, device=x.device)
    at = offsets[used].unsqueeze(1) + i  # [used, cap] rows, past a group's end: clamped, unused
    w = _values(codes[used], scales[used])
    z = torch.bmm(x[at.clamp(max=R - 1).long()], w.transpose(1, 2))
    keep = i < counts[used].unsqueeze(1)
    y[at[keep].long()] = z[keep]
    return y


def _plain_unsort(rows, route_row, weights, residual):
    return (_gather_rows(rows, route_row) * weights.unsqueeze(-1)).sum(1) + residual.float()


# --------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)
    return g


def _routing(case, g):
    """top-k ids and weights of a softmax router whose experts are unevenly loved; a share of
    the routes (and one whole token) dropped, as by a capacity limit."""
    M, k, E = case["M"], min(case["k"], case["E"]), case["E"]
    logits = torch.randn((M, E), generator=g, device="cuda") * 0.9
    logits += torch.randn((E,), generator=g, device="cuda") * 0.5
    top = logits.topk(k, dim=1)
    ids = top.indices.to(torch.int32)
    if case["drop"]:
        ids[torch.rand((M, k), generator=g, device="cuda") < case["drop"]] = -1
        ids[M // 2] = -1
    return ids.contiguous(), top.values.softmax(1).contiguous()


def _normal(shape, g, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _weights(E, N, K, g):
    codes, scales = [], []
    step = max(1, (1 << 26) // (N * K))
    for at in range(0, E, step):
        n = min(step, E - at)
        c, s = _pack(*_plain_quantise(_normal((n * N, K), g, torch.bfloat16, 0.02).float()))
        codes.append(c.reshape(n, N, K // 2))
        scales.append(s.reshape(n, N, -1))
    return torch.cat(codes), torch.cat(scales)


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    s = {"op": case["op"], "dtype": dt, "work": torch.zeros(4096, dtype=torch.uint8, device="cuda")}
    if case["op"] == "quantise":
        # a spread of magnitudes over the blocks, as channels of a layer have
        M, H = case["M"], case["H"]
        gain = torch.exp2(torch.randint(-3, 4, (M, H // BLOCK, 1), generator=g, device="cuda").float())
        s["x"] = (torch.randn((M, H // BLOCK, BLOCK), generator=g, device="cuda") * gain).reshape(M, H).to(dt)
        return s
    M, E = case["M"], case["E"]
    s["E"] = E
    s["ids"], s["w"] = _routing(case, g)
    R = s["ids"].numel()
    if case["op"] in ("route", "grad"):
        H = case["H"]
        s["rows"] = _normal((R, H), g, dt)
        if case["op"] == "route":
            s["x"], s["residual"] = _normal((M, H), g, dt), _normal((M, H), g, dt)
        else:
            s["grad_out"], s["grad_in"] = _normal((M, H), g, dt, 0.1), _normal((R, H), g, dt, 0.1)
            s["route_row"] = _plain_plan(s["ids"], E)[2]
    elif case["op"] == "product":
        s["x"] = _normal((M, case["K"]), g, torch.bfloat16)
        s["codes"], s["scales"] = _weights(E, case["N"], case["K"], g)
    else:
        H, I = case["H"], case["I"]
        s["x"], s["residual"] = _normal((M, H), g, torch.bfloat16), _normal((M, H), g, torch.bfloat16)
        layer = s["layer"] = {"H": H, "I": I, "E": E}
        layer["gate_up_codes"], layer["gate_up_scales"] = _weights(E, 2 * I, H, g)
        layer["down_codes"], layer["down_scales"] = _weights(E, H, I, g)
        # the call's workspace: sorted rows, quantised rows of both products, expert outputs
        s["work"] = torch.zeros((1 << 20) + R * (4 * H + 2 * I), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------- one pass
def _run_plain(s):
    dt = s["dtype"]
    if s["op"] == "quantise":
        q, e = _plain_quantise(s["x"].float())
        return {"values": (q.unflatten(-1, (-1, BLOCK)) * _power(e).unsqueeze(-1)).flatten(-2).to(dt)}
    if s["op"] == "grad":
        rr, w = s["route_row"], s["w"]
        live = (rr >= 0).unsqueeze(-1)
        d = s["grad_out"].float().unsqueeze(1)
        at = torch.where(rr >= 0, rr, -1 - rr).reshape(-1).long()
        grad_rows = torch.empty_like(s["rows"])
        grad_rows[at] = torch.where(live, d * w.unsqueeze(-1), 0.0).flatten(0, 1).to(dt)
        grad_w = (_gather_rows(s["rows"], rr) * d).sum(-1)
        return {"grad_rows": grad_rows, "grad_weights": grad_w, "grad_x": _gather_rows(s["grad_in"], rr).sum(1).to(dt)}
    offsets, row_route, route_row = _plain_plan(s["ids"], s["E"])
    k = s["ids"].shape[1]
    live = (row_route >= 0).unsqueeze(-1)
    if s["op"] == "route":
        rows = torch.where(live, s["x"][(row_route.clamp(min=0) // k).long()], 0.0)
        out = _plain_unsort(s["rows"], route_row, s["w"], s["residual"]).to(dt)
        return {"offsets": offsets, "row_route": row_route, "route_row": route_row, "rows": rows, "out": out}
    q, e = _plain_quantise(s["x"].float())
    x = (q.unflatten(-1, (-1, BLOCK)) * _power(e).unsqueeze(-1)).flatten(-2)
    rows = torch.where(live, x[(row_route.clamp(min=0) // k).long()], 0.0)
    if s["op"] == "product":
        return {"y": _plain_product(rows, offsets, s["codes"], s["scales"]).to(dt)}
    layer = s["layer"]
    y = _plain_product(rows, offsets, layer["gate_up_codes"], layer["gate_up_scales"])
    g, u = y.chunk(2, 1)
    q, e = _plain_quantise(g / (1 + torch.exp(-g)) * u)
    p = (q.unflatten(-1, (-1, BLOCK)) * _power(e).unsqueeze(-1)).flatten(-2)
    y = _plain_product(p, offsets, layer["down_codes"], layer["down_scales"]).to(dt)
    return {"out": _plain_unsort(y, route_row, s["w"], s["residual"]).to(dt)}


def _run_own(s):
    from routed_expert_ffn_top_gb300 import moe
    dt = s["dtype"]
    if s["op"] == "quantise":
        codes, scales = moe.moe_microscale_quantize(s["x"])
        return {"values": moe.moe_microscale_dequantize(codes, scales, dtype=dt)}
    if s["op"] == "grad":
        grad_rows, grad_w = moe.moe_token_unsort_grad(s["grad_out"], s["rows"], s["route_row"], s["w"])
        return {"grad_rows": grad_rows, "grad_weights": grad_w, "grad_x": moe.moe_token_sort_grad(s["grad_in"], s["route_row"])}
    if s["op"] == "experts":
        return {"out": moe.moe_microscale_ffn(s["x"], s["layer"], s["ids"], s["w"], residual=s["residual"], workspace=s["work"])}
    offsets, row_route, route_row = moe.moe_token_plan(s["ids"], s["E"])
    if s["op"] == "route":
        rows = moe.moe_token_sort(s["x"], route_row)
        out = moe.moe_token_unsort(s["rows"], route_row, s["w"], residual=s["residual"])
        return {"offsets": offsets, "row_route": row_route, "route_row": route_row, "rows": rows, "out": out}
    codes, scales = moe.moe_microscale_quantize(s["x"], route_row=route_row)
    return {"y": moe.moe_microscale_product(codes, scales, s["codes"], s["scales"], offsets=offsets, dtype=dt, workspace=s["work"])}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
    four = 0.5 + 1 / BLOCK  # bytes of a 4-bit value with its share of a scale
    M = case["M"]
    if case["op"] == "quantise":
        n = M * case["H"]
        return {"bytes": n * (2 * size + four), "flops": 3 * n}
    k = min(case["k"], case["E"])
    R = M * k
    if case["op"] == "route":
        H = case["H"]
        return {"bytes": 4 * R * 4 + 4 * (case["E"] + 1) + (M * H + R * H) * size + (R * H + 2 * M * H) * size, "flops": 2 * R * H}
    if case["op"] == "grad":
        H = case["H"]
        return {"bytes": 12 * R + (M + 2 * R) * H * size + (R + M) * H * size, "flops": 4 * R * H}
    # experts that a token's routes reach when they spread evenly
    used = case["E"] * (1 - (1 - k / case["E"]) ** M)
    if case["op"] == "product":
        N, K = case["N"], case["K"]
        return {"bytes": 4 * R + M * K * 2 + used * N * K * four + R * N * size, "flops": 2 * R * N * K}
    H, I = case["H"], case["I"]
    return {"bytes": 8 * R + 3 * M * H * 2 + used * 3 * H * I * four, "flops": 2 * R * 3 * H * I}


# ---------------------------------------------------------------------------- in 64 bits
def _exact_quantise(x):
    """float64 [R, C] -> float64 values, from the definition: X = floor(log2 max|x|) - 2, each
    x / 2^X to the nearest of the code values, ties to the one of even code, 6 at most."""
    b = x.reshape(x.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    X = torch.full_like(amax, -127.0)
    pos = amax > 0
    est = torch.floor(torch.log2(amax[pos]))
    est = torch.where(torch.exp2(est) > amax[pos], est - 1, est)
    est = torch.where(torch.exp2(est + 1) <= amax[pos], est + 1, est)
    X[pos] = (est - 2).clamp(-127, 127)
    v = b * torch.exp2(-X)
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    low = torch.searchsorted(mid, v.abs().contiguous(), right=False)  # a tie stays at the lower code
    tie = (low < 7) & (v.abs() == mid[low.clamp(max=6)]) & (low % 2 == 1)
    q = grid[low + tie.long()]
    return (torch.where(v < 0, -q, q) * torch.exp2(X)).reshape(x.shape)


def _exact_weights(codes, scales, e):
    """float64 [N, K] weights of expert e."""
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device=codes.device)
    c = codes[e]
    n, half = c.shape
    v = torch.empty((n, 2 * half), dtype=torch.float64, device=c.device)
    v[:, 0::2] = grid[(c & 7).long()] * (1 - 2 * ((c >> 3) & 1).double())
    v[:, 1::2] = grid[((c >> 4) & 7).long()] * (1 - 2 * (c >> 7).double())
    s = torch.exp2(scales[e][:, : 2 * half // BLOCK].double() - 127)
    return v * s.repeat_interleave(BLOCK, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quantise":
        return {"values": torch.cat([_exact_quantise(c.double()) for c in s["x"].split(32768)])}
    ids, w = s["ids"].cpu().reshape(-1), s["w"].double()
    M, k = s["w"].shape
    E, R = s["E"], M * k
    by = [[] for _ in range(E)]
    for r, e in enumerate(ids.tolist()):
        if 0 <= e < E:
            by[e].append(r)
    order = [r for rs in by for r in rs]
    n = len(order)
    row = torch.full((R,), -1, dtype=torch.int64)
    row[order] = torch.arange(n)
    order, row = torch.tensor(order, dtype=torch.int64).cuda(), row.cuda()
    token = order // k
    if s["op"] == "grad":
        H = s["rows"].shape[1]
        grad_rows = torch.zeros((R, H), dtype=torch.float64, device="cuda")
        grad_rows[:n] = s["grad_out"].double()[token] * w.reshape(-1)[order].unsqueeze(1)
        grad_w = torch.zeros(R, dtype=torch.float64, device="cuda")
        grad_w[order] = (s["grad_out"].double()[token] * s["rows"][:n].double()).sum(1)
        grad_x = torch.zeros((M, H), dtype=torch.float64, device="cuda").index_add_(0, token, s["grad_in"][:n].double())
        return {"grad_rows": grad_rows, "grad_weights": grad_w.reshape(M, k), "grad_x": grad_x}
    if s["op"] == "route":
        H = s["rows"].shape[1]
        rows = torch.zeros((R, H), dtype=torch.float64, device="cuda")
        rows[:n] = s["x"].double()[token]
        out = s["residual"].double().index_add_(0, token, s["rows"][:n].double() * w.reshape(-1)[order].unsqueeze(1))
        return {"offsets": None, "row_route": None, "route_row": None, "rows": rows, "out": out}
    x = _exact_quantise(s["x"].double())
    experts = s["op"] == "experts"
    codes, scales = (s["layer"]["gate_up_codes"], s["layer"]["gate_up_scales"]) if experts else (s["codes"], s["scales"])
    N = codes.shape[1]
    y = torch.zeros((R, N), dtype=torch.float64, device="cuda")
    out = s["residual"].double() if experts else None
    at = 0
    for e, rs in enumerate(by):
        if not rs:
            continue
        t = token[at:at + len(rs)]
        z = x[t] @ _exact_weights(codes, scales, e).T
        if not experts:
            y[at:at + len(rs)] = z
        else:
            g, u = z[:, : N // 2], z[:, N // 2:]
            p = _exact_quantise(g / (1 + torch.exp(-g)) * u)
            z = p @ _exact_weights(s["layer"]["down_codes"], s["layer"]["down_scales"], e).T
            out.index_add_(0, t, z * w.reshape(-1)[order[at:at + len(rs)]].unsqueeze(1))
        at += len(rs)
    return {"out": out} if experts else {"y": y}
