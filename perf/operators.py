"""Cases and plain forms of the layers that stand beside the memory layer in a recurrent stack.

The operators: the short causal convolution (`conv`: prompts, `conv_token`: one token a sequence), the selective state
space scan (`scan`, `scan_token`), and the gated feed-forward projections with their gradient (`gated`, `gated_grad`).
Every case is one call as a serving or training program makes it.  Where `own` is false `run` computes the
plain form, in 32 bits from elementary torch operations; where it is true it calls the framework.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"


def _t(name):
    return torch.bfloat16 if name == BF16 else torch.float32


def listed():
    return [
        # Eight long prompts in front of a scan; x is one half of a fused input projection, so its rows are strided.
        dict(name="conv 8 prompts", op="conv", B=8, T=4096, D=4096, K=4, dtype=BF16, wide=2, act="silu", ragged=False, state=True),
        # Prompts of different lengths, one of them empty, an odd channel count, full precision, no activation.
        dict(name="conv ragged odd f32", op="conv", B=5, T=1021, D=1537, K=3, dtype=F32, wide=1, act="none", ragged=True, state=True),
        # One decode token for 64 sequences whose windows sit in a pool of 96 slots.
        dict(name="conv token 64", op="conv_token", B=64, D=4096, K=4, dtype=BF16, wide=2, act="silu", pool=96),
        # A batch of prompts: enough independent channels to fill the card without a split over time.
        dict(name="scan 16 prompts", op="scan", B=16, T=2048, D=4096, N=16, G=1, dtype=BF16, gate=True, ragged=False, state=False),
        # One long prompt: few channels, so the work has to be split over time.
        dict(name="scan 1 long prompt", op="scan", B=1, T=32768, D=2048, N=16, G=1, dtype=BF16, gate=True, ragged=False, state=True),
        # Ragged prompts in full precision, odd sizes, two groups of channels that share B and C, no gate.
        dict(name="scan ragged odd f32", op="scan", B=3, T=777, D=1002, N=12, G=2, dtype=F32, gate=False, ragged=True, state=True),
        # The latency of one decode token for one sequence.
        dict(name="scan token 1", op="scan_token", B=1, D=2048, N=16, G=1, dtype=BF16, gate=True, pool=0),
        # A decode batch whose states sit in a pool, some rows of the batch being padding.
        dict(name="scan token 256", op="scan_token", B=256, D=4096, N=16, G=1, dtype=BF16, gate=True, pool=320),
        # The feed-forward block of a decode step: four tokens, all the weights.
        dict(name="gated 4 tokens", op="gated", M=4, D=2048, F=8192, act="silu"),
        # The same block over a batch of prompts.
        dict(name="gated 16384 tokens", op="gated", M=16384, D=2048, F=8192, act="silu"),
        # Its gradient in a training step of a small layer, ragged token count.
        dict(name="gated grad 1000 tokens", op="gated_grad", M=1000, D=1024, F=2736, act="gelu"),
        # Its gradient in a training step of a large batch.
        dict(name="gated grad 32768 tokens", op="gated_grad", M=32768, D=2048, F=8192, act="silu"),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n - (n % 384 == 0)  # a size that tiles of 128 and of 96 both divide is moved off them


def draw(rng):
    op = rng.choice(["conv", "conv_token", "scan", "scan", "scan_token", "gated", "gated_grad"])
    dtype = rng.choice([BF16, BF16, F32])
    if op == "conv":
        D, B = _log(rng, 64, 8192), _log(rng, 1, 32)
        T = min(_log(rng, 1, 32768), (1 << 27) // (B * D))
        return dict(op=op, B=B, T=max(1, T), D=D, K=rng.randint(2, 8), dtype=dtype, wide=rng.choice([1, 2]),
                    act=rng.choice(["silu", "none"]), ragged=rng.random() < 0.4, state=rng.random() < 0.6)
    if op == "conv_token":
        B = _log(rng, 1, 512)
        return dict(op=op, B=B, D=_log(rng, 64, 8192), K=rng.randint(2, 8), dtype=dtype, wide=rng.choice([1, 2]),
                    act=rng.choice(["silu", "none"]), pool=rng.choice([0, B + B // 4 + 1]))
    if op in ("scan", "scan_token"):
        G = rng.choice([1, 1, 2, 4])
        D, N, B = _log(rng, 64, 8192) // G * G, rng.choice([4, 7, 8, 12, 16, 16, 16, 32, 64, 100, 128]), _log(rng, 1, 32)
        if op == "scan_token":
            B = min(_log(rng, 1, 512), (1 << 26) // (D * N))
            return dict(op=op, B=B, D=D, N=N, G=G, dtype=dtype, gate=rng.random() < 0.7,
                        pool=rng.choice([0, B + B // 4 + 1]))
        T = min(_log(rng, 1, 32768), (1 << 30) // (B * D * N))
        return dict(op=op, B=B, T=max(1, T), D=D, N=N, G=G, dtype=dtype, gate=rng.random() < 0.7,
                    ragged=rng.random() < 0.4, state=rng.random() < 0.6)
    D, F = 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 1536)
    M = min(_log(rng, 1, 32768), (1 << 38) // (D * F))
    return dict(op=op, M=M, D=D, F=F, act=rng.choice(["silu", "gelu"]))


def _cells(case):
    """(b, t) pairs of the case that hold a token, in the mean: a ragged batch's lengths are spread evenly."""
    n = case["B"] * case.get("T", 1)
    return n * (0.5 if case.get("ragged") else 1.0)


def work(case):
    op = case["op"]
    if op.startswith("gated"):
        M, D, F = case["M"], case["D"], case["F"]
        if op == "gated":
            return {"bytes": 2.0 * (M * D + 2 * F * D + M * F), "flops": 4.0 * M * D * F}
        # the gradient recomputes both projections, then has two products of the same size as the two together
        return {"bytes": 2.0 * (2 * M * D + 4 * F * D + M * F), "flops": 12.0 * M * D * F}
    es = 2 if case["dtype"] == BF16 else 4
    B, D, n = case["B"], case["D"], _cells(case)
    out = B * case.get("T", 1) * D * es
    if op.startswith("conv"):
        K = case["K"]
        carried = B * D * (K - 1) * es * (2 if case.get("state", True) else 1)
        return {"bytes": n * D * es + out + carried + D * (K + 1) * 4.0, "flops": n * D * (2.0 * K + 4)}
    N, G = case["N"], case["G"]
    carried = 4.0 * B * D * N * (2 if case.get("state", True) else 1)
    reads = n * es * (D * (3 if case["gate"] else 2) + 2 * G * N)
    return {"bytes": reads + out + carried + 4.0 * D * (N + 2), "flops": n * D * (7.0 * N + 8)}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _lengths(case, g):
    """Lengths from 0 to T, the first sequence full and the last one empty where there are three or more."""
    B, T = case["B"], case["T"]
    n = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    n[0] = T
    if B >= 3:
        n[-1] = 0
    return n


def _slots(case, g):
    """Distinct slots of the pool in random order; about one row in sixteen of a batch of 16 or more is padding."""
    if not case["pool"]:
        return None
    s = torch.randperm(case["pool"], generator=g, device="cuda")[: case["B"]].to(torch.int32)
    if case["B"] >= 16:
        s[3::16] = -1
    return s


def prepare(case, seed):
    g = _gen(seed)
    rn = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s = dict(case)
    op = case["op"]
    if op.startswith("gated"):
        M, D, F = case["M"], case["D"], case["F"]
        s["x"] = rn(M, D).bfloat16()
        s["w"] = (rn(2 * F, D) * D ** -0.5).bfloat16()
        if op == "gated_grad":
            s["dh"] = rn(M, F).bfloat16()
        return s
    dt, B, D = _t(case["dtype"]), case["B"], case["D"]
    token = op.endswith("_token")
    lead = (B,) if token else (B, case["T"])
    s["lengths"] = _lengths(case, g) if case.get("ragged") else None
    s["slots"] = _slots(case, g) if token else None
    rows = case["pool"] if token and case["pool"] else B
    if op.startswith("conv"):
        K = case["K"]
        s["x"] = rn(*lead, case["wide"] * D).to(dt)[..., :D]
        s["w"] = (rn(D, K) * K ** -0.5).to(dt)
        s["bias"] = (rn(D) * 0.1).to(dt)
        s["state"] = rn(rows, K - 1, D).to(dt) if case.get("state", True) else None
        s["state_out"] = torch.zeros((rows, K - 1, D), dtype=dt, device="cuda")
        return s
    N, G = case["N"], case["G"]
    s["x"] = rn(*lead, D).to(dt)
    # the low-rank step-size features and B and C come out of one projection, as its slices
    rank = max(1, D // 64)
    wide = rn(*lead, rank + 2 * G * N).to(dt)
    s["B_"] = wide[..., rank : rank + G * N].unflatten(-1, (G, N))
    s["C_"] = wide[..., rank + G * N :].unflatten(-1, (G, N))
    s["dt"] = (rn(*lead, D) * 0.5).to(dt)
    # step sizes between 0.001 and 0.1 before the input's own part, decay rates 1 .. N
    step = torch.exp(torch.rand(D, generator=g, device="cuda") * math.log(100.0) + math.log(0.001))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(0.1 * rn(D, N))
    s["skip"] = 1.0 + 0.1 * rn(D)
    s["z"] = rn(*lead, 2 * D).to(dt)[..., D:] if case["gate"] else None
    s["state"] = rn(rows, D, N) if case.get("state", True) else None
    s["state_out"] = torch.zeros((rows, D, N), device="cuda")
    return s


def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import sparse_state_linear_sdm_gb300 as sdm

    op = s["op"]
    if op == "gated":
        return sdm.project_gated(s["x"], s["w"], activation=s["act"])
    if op == "gated_grad":
        return sdm.project_gated_backward(s["x"], s["w"], s["dh"], activation=s["act"])
    if op == "conv":
        return sdm.causal_conv(s["x"], s["w"], s["bias"], state=s["state"], state_out=s["state_out"],
                               activation=s["act"], lengths=s["lengths"])
    if op == "conv_token":
        return sdm.causal_conv_step(s["x"], s["w"], s["bias"], state=s["state"], state_out=s["state_out"],
                                    activation=s["act"], slots=s["slots"])
    if op == "scan":
        return sdm.selective_scan(s["x"], s["dt"], s["A"], s["B_"], s["C_"], D=s["skip"], z=s["z"],
                                  dt_bias=s["dt_bias"], state=s["state"], state_out=s["state_out"],
                                  lengths=s["lengths"])
    return sdm.selective_step(s["x"], s["dt"], s["A"], s["B_"], s["C_"], D=s["skip"], z=s["z"],
                              dt_bias=s["dt_bias"], state=s["state"], state_out=s["state_out"], slots=s["slots"])


# ---- plain forms ----


def _act(g, act):
    """(act(g), act'(g)) in 32 bits; gelu is the exact one, g Phi(g)."""
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    p = 0.5 * (1.0 + torch.erf(g * 0.5 ** 0.5))
    return g * p, p + g * torch.exp(-0.5 * g * g) * (2.0 * math.pi) ** -0.5


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-v.abs()))


def _plain(s):
    op = s["op"]
    if op.startswith("gated"):
        x, w = s["x"].float(), s["w"].float()
        F = s["F"]
        gate, up = x @ w[:F].T, x @ w[F:].T
        a, da = _act(gate, s["act"])
        if op == "gated":
            return (a * up).bfloat16()
        dh = s["dh"].float()
        d = torch.cat([dh * up * da, dh * a], dim=1)
        return (d @ w).bfloat16(), (d.T @ x).bfloat16()
    if op == "conv":
        return _plain_conv(s)
    if op == "conv_token":
        return _plain_conv_token(s)
    return _plain_scan(s) if op == "scan" else _plain_scan_token(s)


def _plain_conv(s):
    x, w, K, T = s["x"].float(), s["w"].float(), s["K"], s["T"]
    before = s["state"].float() if s["state"] is not None else x.new_zeros(x.shape[0], K - 1, x.shape[2])
    u = torch.cat([before, x], dim=1)
    y = (u.unfold(1, K, 1) * w).sum(-1) + s["bias"].float()
    if s["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    n = s["lengths"]
    last = torch.arange(K - 1, device=x.device)
    if n is None:
        s["state_out"].copy_(u[:, T:])
    else:
        y = torch.where((torch.arange(T, device=x.device) < n[:, None])[..., None], y, 0.0)
        at = (n.long()[:, None] + last)[..., None].expand(-1, -1, x.shape[2])
        s["state_out"].copy_(u.gather(1, at))
    return y.to(s["x"].dtype), s["state_out"]


def _rows(s):
    """The rows of the batch that hold a sequence, and their places in the pool."""
    if s["slots"] is None:
        at = torch.arange(s["B"], device=s["x"].device)
        return torch.ones_like(at, dtype=torch.bool), at
    return s["slots"] >= 0, s["slots"].long().clamp(min=0)


def _plain_conv_token(s):
    x, w = s["x"].float(), s["w"].float()
    live, at = _rows(s)
    u = torch.cat([s["state"][at].float(), x[:, None]], dim=1)
    y = (u * w.T).sum(1) + s["bias"].float()
    if s["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    y = torch.where(live[:, None], y, 0.0)
    _put(s["state_out"], u[:, 1:].to(s["state"].dtype), live, at)
    return y.to(s["x"].dtype), s["state_out"]


def _put(pool, rows, live, at):
    """rows[b] to pool[at[b]] where live[b]; a padding row writes a live one's value where that one goes."""
    if bool(live.numel() == pool.shape[0]):
        pool.copy_(rows)
        return
    first = live.int().argmax().view(1)
    pool[torch.where(live, at, at.index_select(0, first))] = torch.where(
        live.view(-1, *[1] * (rows.dim() - 1)), rows, rows.index_select(0, first))


def _gated_out(s, y, x):
    y = y + s["skip"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z / (1.0 + torch.exp(-z)))
    return y


def _recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1: windows of about sqrt(T) tokens side by side, then window after window."""
    T = a.shape[1]
    w = math.isqrt(T - 1) + 1
    n = -(-T // w)
    if n * w > T:
        a = torch.cat([a, a.new_ones(a.shape[0], n * w - T, *a.shape[2:])], dim=1)
        b = torch.cat([b, b.new_zeros(b.shape[0], n * w - T, *b.shape[2:])], dim=1)
    a, b = a.unflatten(1, (n, w)), b.unflatten(1, (n, w))
    for j in range(1, w):
        b[:, :, j].addcmul_(a[:, :, j], b[:, :, j - 1])
        a[:, :, j].mul_(a[:, :, j - 1])
    for c in range(1, n):
        b[:, c].addcmul_(a[:, c], b[:, c - 1, -1:])
    return b.flatten(1, 2)[:, :T]


def _plain_scan(s):
    x, D, G, N, T = s["x"].float(), s["D"], s["G"], s["N"], s["T"]
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    if s["lengths"] is not None:
        valid = (torch.arange(T, device=x.device) < s["lengths"][:, None])[..., None]
        delta = torch.where(valid, delta, 0.0)
    Bm = s["B_"].float().repeat_interleave(D // G, dim=2)
    Cm = s["C_"].float().repeat_interleave(D // G, dim=2) if G > 1 else s["C_"].float()
    a = torch.exp(delta[..., None] * s["A"])
    b = (delta * x)[..., None] * (Bm if G > 1 else s["B_"].float())
    if s["state"] is not None:
        b[:, 0] += a[:, 0] * s["state"]
    b = _recurrence(a, b)
    y = _gated_out(s, (b * Cm).sum(-1), x)
    if s["lengths"] is not None:
        y = torch.where(valid, y, 0.0)
    s["state_out"].copy_(b[:, -1])
    return y.to(s["x"].dtype), s["state_out"]


def _plain_scan_token(s):
    x, D, G = s["x"].float(), s["D"], s["G"]
    live, at = _rows(s)
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    Bm = s["B_"].float().repeat_interleave(D // G, dim=1)
    Cm = s["C_"].float().repeat_interleave(D // G, dim=1)
    h = torch.exp(delta[..., None] * s["A"]) * s["state"][at] + (delta * x)[..., None] * Bm
    y = torch.where(live[:, None], _gated_out(s, (h * Cm).sum(-1), x), 0.0)
    _put(s["state_out"], h, live, at)
    return y.to(s["x"].dtype), s["state_out"]


# ---- the definitions in 64 bits ----


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("gated"):
        return _exact_gated(s)
    if op.startswith("conv"):
        return _exact_conv(s)
    return _exact_scan(s)


def _exact_gated(s):
    if 12.0 * s["M"] * s["D"] * s["F"] > 1.0e13:
        return None
    x, w, F = s["x"].double(), s["w"].double(), s["F"]
    g, u = x @ w[:F].T, x @ w[F:].T
    if s["act"] == "silu":
        p = torch.sigmoid(g)
        slope = p + g * p * (1 - p)
    else:
        p = torch.special.ndtr(g)
        slope = p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if s["op"] == "gated":
        return g * p * u
    dh = s["dh"].double()
    dg, du = dh * u * slope, dh * g * p
    return dg @ w[:F] + du @ w[F:], torch.cat([dg.T @ x, du.T @ x])


def _exact_conv(s):
    token = s["op"] == "conv_token"
    x = s["x"].double()
    x = x[:, None] if token else x
    n = s["lengths"].tolist() if s["lengths"] is not None else [x.shape[1]] * x.shape[0]
    slots = s["slots"].tolist() if s["slots"] is not None else list(range(x.shape[0]))
    w, bias, K = s["w"].double(), s["bias"].double(), s["K"]
    y, out = torch.zeros_like(x), torch.zeros(s["state_out"].shape, dtype=torch.float64, device=x.device)
    for b, (length, slot) in enumerate(zip(n, slots)):
        if slot < 0:
            continue
        old = s["state"][slot].double() if s["state"] is not None else x.new_zeros(K - 1, x.shape[2])
        u = torch.cat([old, x[b, :length]])
        acc = bias.expand(length, -1).clone()
        for j in range(K):
            acc += u[j : j + length] * w[:, j]
        y[b, :length] = acc * torch.sigmoid(acc) if s["act"] == "silu" else acc
        out[slot] = u[length:]
    return (y[:, 0] if token else y), out


def _exact_scan(s):
    token = s["op"] == "scan_token"
    if not token and s["T"] * (1.0 + s["B"] * s["D"] * s["N"] / 4.0e6) > 6.0e4:
        return None  # over about 20 seconds token by token
    lead = lambda v: v[:, None] if token else v  # noqa: E731
    x, dt, Bm, Cm = (lead(s[k]) for k in ("x", "dt", "B_", "C_"))
    n, T, D, G = x.shape[0], x.shape[1], s["D"], s["G"]
    A, skip, bias = s["A"].double(), s["skip"].double(), s["dt_bias"].double()
    slots = s["slots"].long() if s["slots"] is not None else torch.arange(n, device=x.device)
    live = slots >= 0
    h = s["state"][slots.clamp(min=0)].double() if s["state"] is not None else A.new_zeros(n, D, s["N"])
    y = torch.zeros(n, T, D, dtype=torch.float64, device=x.device)
    for t in range(T):
        xt = x[:, t].double()
        delta = torch.logaddexp(dt[:, t].double() + bias, A.new_zeros(()))
        new = h * torch.exp(delta[..., None] * A)
        new = new + (delta * xt).view(n, G, D // G, 1).mul(Bm[:, t].double()[:, :, None]).view_as(h)
        ok = live if s["lengths"] is None else live & (s["lengths"] > t)
        h = torch.where(ok[:, None, None], new, h)
        o = (h.view(n, G, D // G, -1) * Cm[:, t].double()[:, :, None]).sum(-1).view(n, D) + skip * xt
        if s["z"] is not None:
            zt = lead(s["z"])[:, t].double()
            o = o * zt * torch.sigmoid(zt)
        y[:, t] = torch.where(ok[:, None], o, 0.0)
    out = torch.zeros(s["state_out"].shape, dtype=torch.float64, device=x.device)
    out[slots[live]] = h[live]
    return (y[:, 0] if token else y), out
