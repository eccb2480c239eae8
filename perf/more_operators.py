"""Cases and plain forms of a linear attention layer's operators: the attention itself and what stands around it.

The operators: linear attention with a decay for each head (`linear`: prompts, `linear_token`: one token a sequence), the
norms after and before a block with its gate, residual and residual scale in one pass (`norm`) and their gradient
(`norm_grad`), and a projection with bias, activation and residual in its epilogue (`project`) and its gradient
(`project_grad`).  Every case is one call as a serving or training program makes it.  Where `own` is false `run` computes
the plain form, in 32 bits from elementary torch operations; where it is true it calls the framework.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
EPS = 1e-6


def _t(name):
    return torch.bfloat16 if name == BF16 else torch.float32


def listed():
    return [
        # Eight long prompts; q, k and v are slices of one projection, every token and head has its decay.
        dict(name="linear 8 prompts", op="linear", B=8, T=4096, H=16, Hk=16, dk=128, dv=128, dtype=BF16, decay="token",
             ragged=False, state=False),
        # One long prompt continued from a state: eight heads leave the card short, so the work is split over time.
        dict(name="linear 1 long prompt", op="linear", B=1, T=32768, H=8, Hk=8, dk=128, dv=128, dtype=BF16, decay="token",
             ragged=False, state=True),
        # Prompts of different lengths, one of them empty, in full precision: odd sizes, heads that share queries and
        # keys, a fixed decay for each head.
        dict(name="linear ragged odd f32", op="linear", B=3, T=777, H=6, Hk=2, dk=50, dv=37, dtype=F32, decay="head",
             ragged=True, state=True),
        # The latency of one decode token of one sequence.
        dict(name="linear token 1", op="linear_token", B=1, H=16, Hk=16, dk=64, dv=64, dtype=BF16, decay="token", pool=0),
        # A decode batch whose states sit in a pool, some rows of the batch being padding.
        dict(name="linear token 256", op="linear_token", B=256, H=16, Hk=16, dk=128, dv=128, dtype=BF16, decay="token",
             pool=320),
        # Between two blocks of a decode step: the residual addition and the next block's norm.
        dict(name="norm 4 tokens", op="norm", M=4, D=2048, groups=1, x=BF16, r=BF16, w=BF16, after=False, gate=False,
             scale=False, residual=True, before=True),
        # Between two blocks of a batch of prompts, a norm on either side and a full-precision residual stream.
        dict(name="norm 16384 tokens", op="norm", M=16384, D=2048, groups=1, x=BF16, r=F32, w=F32, after=True, gate=False,
             scale=True, residual=True, before=True),
        # A training step's gradient of the norm and gate over the heads of an attention's output.
        dict(name="head norm grad 16384", op="norm_grad", M=16384, D=2048, groups=16, x=BF16, r=BF16, w=F32, after=True,
             gate=True, scale=False, residual=False, before=False),
        # The gradient of everything at once, rows of an odd width, a token count that divides nothing.
        dict(name="norm grad ragged", op="norm_grad", M=4099, D=1537, groups=1, x=BF16, r=F32, w=F32, after=True, gate=True,
             scale=True, residual=True, before=True),
        # The last projection of a feed-forward block in a decode step: four tokens, all the weights.
        dict(name="project 4 tokens", op="project", M=4, D=8192, N=2048, act="none", bias=False, residual=True),
        # The same projection over a batch of prompts.
        dict(name="project 16384 tokens", op="project", M=16384, D=8192, N=2048, act="none", bias=False, residual=True),
        # The gradient of a first projection with bias and gelu, ragged token count.
        dict(name="project grad 1000 tokens", op="project_grad", M=1000, D=1024, N=2736, act="gelu", bias=True,
             residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_token", "norm", "norm_grad", "project", "project_grad"])
    if op.startswith("linear"):
        share = rng.choice([1, 1, 2, 4])
        H = share * _log(rng, 1, 16)
        dk, dv = (rng.choice([16, 32, 50, 64, 64, 80, 100, 128, 128, 128, 256]) for _ in range(2))
        c = dict(op=op, H=H, Hk=H // share, dk=dk, dv=dv, dtype=rng.choice([BF16, BF16, F32]),
                 decay=rng.choice(["token", "token", "head", "none"]))
        if op == "linear_token":
            B = min(_log(rng, 1, 512), max(1, (1 << 26) // (H * dk * dv)))
            return dict(c, B=B, pool=rng.choice([0, B + B // 4 + 1]))
        B = _log(rng, 1, 32)
        T = min(_log(rng, 1, 32768), (1 << 32) // (B * H * dk * dv), (1 << 26) // (B * H * max(dk, dv)))
        return dict(c, B=B, T=max(1, T), ragged=rng.random() < 0.4, state=rng.random() < 0.6)
    if op.startswith("norm"):
        by_head = rng.random() < 0.4
        groups = _log(rng, 2, 32) if by_head else 1
        D = groups * rng.choice([32, 64, 96, 128, 256]) if by_head else _log(rng, 32, 8192)
        M = min(_log(rng, 1, 32768), (1 << 25) // D)
        after, gate = by_head or rng.random() < 0.5, rng.random() < 0.5
        residual = not by_head and rng.random() < 0.8
        x = rng.choice([BF16, BF16, F32])
        return dict(op=op, M=M, D=D, groups=groups, x=x, r=rng.choice([x, F32]) if residual else x, w=rng.choice([BF16, F32]),
                    after=after, gate=gate, scale=residual and rng.random() < 0.5, residual=residual, before=not by_head)
    D, N = 8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 1024)
    M = min(_log(rng, 1, 32768), (1 << 36) // (D * N))
    return dict(op=op, M=M, D=D, N=N, act=rng.choice(["none", "silu", "gelu"]), bias=rng.random() < 0.5,
                residual=op == "project" and rng.random() < 0.5)


def _es(name):
    return 2 if name == BF16 else 4


def work(case):
    op = case["op"]
    if op.startswith("project"):
        M, D, N = case["M"], case["D"], case["N"]
        b = 2.0 * N if case["bias"] else 0.0
        if op == "project":
            return {"bytes": 2.0 * (M * D + N * D + M * N * (2 if case["residual"] else 1)) + b, "flops": 2.0 * M * D * N}
        # the gradient of an activation recomputes the projection, then has two products of its size
        return {"bytes": 2.0 * (2 * M * D + 2 * N * D + M * N) + 2 * b,
                "flops": (4.0 if case["act"] == "none" else 6.0) * M * D * N}
    if op.startswith("norm"):
        n, D, ex, er, ew = case["M"] * case["D"], case["D"], _es(case["x"]), _es(case["r"]), _es(case["w"])
        weights = ew * D * (case["after"] + case["scale"] + case["before"])
        inner = case["after"] or case["gate"] or case["scale"]
        if op == "norm":
            new = case["residual"] or inner  # the stream behind the addition is an output too
            b = n * (ex * (1 + case["gate"] + case["before"]) + er * (case["residual"] + new))
            return {"bytes": float(b + weights), "flops": 12.0 * n}
        # x and the gate, y's and the stream's gradients and the stream in, theirs out
        b = n * ex * ((1 if inner else 0) + case["gate"] + case["before"])
        b += n * er * (1 + case["before"])
        b += n * (ex * ((1 if inner or case["x"] != case["r"] or not case["residual"] else 0) + case["gate"]) + er * case["residual"])
        return {"bytes": float(b + 2 * weights), "flops": 30.0 * n}
    B, H, Hk, dk, dv = (case[k] for k in ("B", "H", "Hk", "dk", "dv"))
    T = case.get("T", 1)
    n, es = B * T * (0.5 if case.get("ragged") else 1.0), _es(case["dtype"])
    decays = 4.0 * (n * H if case["decay"] == "token" else H if case["decay"] == "head" else 0)
    states = 4.0 * B * H * dk * dv * (2 if case.get("state", True) else 1)
    return {"bytes": n * es * (2 * Hk * dk + H * dv) + B * T * H * dv * es + decays + states, "flops": 4.0 * n * H * dk * dv}


# ---- what a program has in hand ----


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
    if op.startswith("linear"):
        return _prepare_linear(s, g, rn)
    if op.startswith("norm"):
        return _prepare_norm(s, rn)
    M, D, N = case["M"], case["D"], case["N"]
    s["inp"] = rn(M, D).bfloat16()
    s["wt"] = (rn(N, D) * D ** -0.5).bfloat16()
    s["bias_"] = (rn(N) * 0.1).bfloat16() if case["bias"] else None
    s["res"] = rn(M, N).bfloat16() if case["residual"] else None
    s["dy"] = rn(M, N).bfloat16() if op == "project_grad" else None
    return s


def _prepare_linear(s, g, rn):
    B, H, Hk, dk, dv, dt = s["B"], s["H"], s["Hk"], s["dk"], s["dv"], _t(s["dtype"])
    token = s["op"] == "linear_token"
    lead = (B,) if token else (B, s["T"])
    # queries, keys and values come out of one projection, as its slices
    wide = rn(*lead, 2 * Hk * dk + H * dv).to(dt)
    s["q"] = wide[..., : Hk * dk].unflatten(-1, (Hk, dk))
    s["k"] = wide[..., Hk * dk : 2 * Hk * dk].unflatten(-1, (Hk, dk))
    s["v"] = wide[..., 2 * Hk * dk :].unflatten(-1, (H, dv))
    # heads forget at rates from 1/1000 to 1/2 a token
    rate = torch.exp(torch.rand(H, generator=g, device="cuda") * math.log(500.0) + math.log(0.001))
    s["g"] = None
    if s["decay"] == "token":
        s["g"] = -rate * torch.exp(0.5 * rn(*lead, H))
    elif s["decay"] == "head":
        s["g"] = torch.log1p(-rate)
    s["lengths"] = _lengths(s, g) if s.get("ragged") else None
    s["slots"] = _slots(s, g) if token else None
    rows = s["pool"] if token and s["pool"] else B
    s["S"] = rn(rows, H, dk, dv) if s.get("state", True) else None
    s["S_out"] = torch.zeros((rows, H, dk, dv), device="cuda")
    return s


def _prepare_norm(s, rn):
    M, D = s["M"], s["D"]
    x, r, w = _t(s["x"]), _t(s["r"]), _t(s["w"])
    s["inp"] = rn(M, D).to(x)
    s["res"] = (2.0 * rn(M, D)).to(r) if s["residual"] else None
    s["z"] = rn(M, 2 * D).to(x)[:, D:] if s["gate"] else None  # one half of a wider projection
    s["w_after"] = (1.0 + 0.1 * rn(D)).to(w) if s["after"] else None
    s["w_scale"] = (0.5 + 0.1 * rn(D)).to(w) if s["scale"] else None
    s["w_before"] = (1.0 + 0.1 * rn(D)).to(w) if s["before"] else None
    if s["op"] == "norm_grad":
        # what the forward pass left, and the gradients of its two outputs
        s["stream"] = _stream(s)[0].to(r)
        s["dy"] = rn(M, D).to(x) if s["before"] else None
        s["dr"] = rn(M, D).to(r)
    return s


def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import sparse_state_linear_sdm_gb300 as sdm

    op = s["op"]
    if op == "linear":
        return sdm.linear_attention(s["q"], s["k"], s["v"], s["g"], state=s["S"], state_out=s["S_out"], lengths=s["lengths"])
    if op == "linear_token":
        return sdm.linear_attention_step(s["q"], s["k"], s["v"], s["g"], state=s["S"], state_out=s["S_out"],
                                         slots=s["slots"])
    if op == "norm":
        if not s["before"] and not s["residual"]:
            return sdm.gated_norm(s["inp"], s["w_after"], s["z"], groups=s["groups"], eps=EPS)
        y, r = sdm.residual_norm(s["inp"], s["res"], s["w_before"], after=s["w_after"], gate=s["z"], scale=s["w_scale"],
                                 eps=EPS)
        return (y, r) if _moves(s) else y
    if op == "norm_grad":
        if not s["before"] and not s["residual"]:
            dx, dw, dz = sdm.gated_norm_backward(s["inp"], s["w_after"], s["dr"], s["z"], groups=s["groups"], eps=EPS)
            return {"dx": dx, "dz": dz, "dafter": dw}
        dx, dres, dw, dafter, dz, dscale = sdm.residual_norm_backward(
            s["inp"], s["stream"], s["dy"], s["dr"], s["w_before"], after=s["w_after"], gate=s["z"], scale=s["w_scale"],
            residual=s["residual"], eps=EPS)
        return {"dx": dx, "dres": dres, "dbefore": dw, "dafter": dafter, "dz": dz, "dscale": dscale}
    if op == "project":
        return sdm.project(s["inp"], s["wt"], s["bias_"], s["res"], activation=s["act"])
    return sdm.project_backward(s["inp"], s["wt"], s["dy"], s["bias_"], activation=s["act"])


# ---- plain forms ----


def _plain(s):
    op = s["op"]
    if op == "linear":
        return _plain_linear(s)
    if op == "linear_token":
        return _plain_token(s)
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_grad":
        return _plain_norm_grad(s)
    x, w = s["inp"].float(), s["wt"].float()
    z = x @ w.T
    if s["bias_"] is not None:
        z = z + s["bias_"].float()
    a, da = _act(z, s["act"])
    if op == "project":
        return (a if s["res"] is None else a + s["res"].float()).bfloat16()
    dz = s["dy"].float() if da is None else s["dy"].float() * da
    return (dz @ w).bfloat16(), (dz.T @ x).bfloat16(), None if s["bias_"] is None else dz.sum(0).bfloat16()


def _act(z, act):
    """(act(z), act'(z)) in 32 bits; gelu is the exact one, z Phi(z)."""
    if act == "none":
        return z, None
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return z * p, p * (1.0 + z * (1.0 - p))
    p = 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5))
    return z * p, p + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5


def _heads(t, H):
    """[B, T, h, d] -> [B, H, T, d] in 32 bits, each of the h heads for H / h of them."""
    return t.float().transpose(1, 2).repeat_interleave(H // t.shape[2], dim=1)


def _plain_linear(s, C=64):
    """In chunks of C tokens: within a chunk the masked products of its queries and keys, between chunks the state in
    front of each, as a product over the chunks before it.  Sums of decays are held in 64 bits."""
    B, T, H, dk, dv = s["B"], s["T"], s["H"], s["dk"], s["dv"]
    q, k, v = _heads(s["q"], H) * dk ** -0.5, _heads(s["k"], H), _heads(s["v"], H)
    dev, n = q.device, -(-T // C)
    g = torch.zeros(B, H, T, dtype=torch.float64, device=dev)
    if s["g"] is not None:
        g = g + (s["g"].double().transpose(1, 2) if s["g"].dim() == 3 else s["g"].double()[:, None])
    if s["lengths"] is not None:
        valid = (torch.arange(T, device=dev) < s["lengths"][:, None])[:, None]
        g = torch.where(valid, g, 0.0)
        k, v = torch.where(valid[..., None], k, 0.0), torch.where(valid[..., None], v, 0.0)
    pad = n * C - T
    q, k, v = (torch.nn.functional.pad(t, (0, 0, 0, pad)).unflatten(2, (n, C)) for t in (q, k, v))
    G = torch.cumsum(torch.nn.functional.pad(g, (0, pad)).unflatten(2, (n, C)), -1)
    ahead = torch.ones(C, C, dtype=torch.bool, device=dev).triu(1)
    P = (q @ k.transpose(-1, -2)) * torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(ahead, -math.inf)).float()
    o = P @ v
    kv = (k * torch.exp(G[..., -1:] - G).float()[..., None]).transpose(-1, -2) @ v   # what a chunk adds to the state
    end = torch.cumsum(G[..., -1], -1)                                               # decay up to each chunk's end
    start = end - G[..., -1]
    late = torch.ones(n + 1, n, dtype=torch.bool, device=dev).triu(0)                # chunks not before this one
    until = torch.cat([start, end[..., -1:]], -1)
    L = torch.exp((until[..., :, None] - end[..., None, :]).masked_fill(late, -math.inf)).float()
    S = (L @ kv.flatten(3)).unflatten(3, (dk, dv))
    if s["S"] is not None:
        S = S + torch.exp(until).float()[..., None, None] * s["S"][:, :, None]
    o = o + (q * torch.exp(G).float()[..., None]) @ S[:, :, :n]
    o = o.flatten(2, 3)[:, :, :T].transpose(1, 2)
    if s["lengths"] is not None:
        o = torch.where(valid.transpose(1, 2)[..., None], o, 0.0)
    s["S_out"].copy_(S[:, :, n])
    return o.to(s["v"].dtype), s["S_out"]


def _rows(s):
    """The rows of the batch that hold a sequence, and their places in the pool."""
    if s["slots"] is None:
        at = torch.arange(s["B"], device=s["q"].device)
        return torch.ones_like(at, dtype=torch.bool), at
    return s["slots"] >= 0, s["slots"].long().clamp(min=0)


def _plain_token(s):
    H, dk = s["H"], s["dk"]
    q, k, v = (_heads(s[n][:, None], H)[:, :, 0] for n in ("q", "k", "v"))
    live, at = _rows(s)
    S = s["S"][at]
    if s["g"] is not None:
        S = torch.exp(s["g"] if s["g"].dim() == 2 else s["g"][None])[..., None, None] * S
    S = S + k[..., None] * v[..., None, :]
    o = (q[..., None] * S).sum(-2) * dk ** -0.5
    o = torch.where(live[:, None, None], o, 0.0)
    if live.numel() == s["S_out"].shape[0]:
        s["S_out"].copy_(S)
    else:  # a padding row writes a live one's state where that one goes
        first = live.int().argmax().view(1)
        s["S_out"][torch.where(live, at, at.index_select(0, first))] = torch.where(live[:, None, None, None], S,
                                                                                    S.index_select(0, first))
    return o.to(s["v"].dtype), s["S_out"]


def _moves(s):
    """Whether the stream behind the block is another one than its input."""
    return s["residual"] or s["after"] or s["gate"] or s["scale"]


def _inverse_rms(t, groups):
    """1 / rms over each group of channels, for every channel of it."""
    i = torch.rsqrt(t.unflatten(-1, (groups, -1)).square().mean(-1) + EPS)
    return i.repeat_interleave(t.shape[-1] // groups, -1)


def _stream(s):
    """The stream behind the block, in 32 bits, and what its gradient takes of the way there."""
    x = s["inp"].float()
    i = n = gate = None
    a = x
    if s["after"]:
        i = _inverse_rms(x, s["groups"])
        a = n = x * i * s["w_after"].float()
    if s["gate"]:
        z = s["z"].float()
        gate = z / (1.0 + torch.exp(-z))
        a = a * gate
    r = a * s["w_scale"].float() if s["scale"] else a
    return (r + s["res"].float() if s["residual"] else r), (x, i, n, gate, a)


def _plain_norm(s):
    r = _stream(s)[0]
    if not s["before"]:
        return r.to(_t(s["r"]))
    y = (r * _inverse_rms(r, 1) * s["w_before"].float()).to(s["inp"].dtype)
    return (y, r.to(_t(s["r"]))) if _moves(s) else y


def _norm_slope(d, w, x, i, groups):
    """(gradient to x, gradient to w) of x i w for the gradient d, where i is 1 / rms over groups of channels."""
    dw = d * x * i
    d = d * w
    mean = (d * x).unflatten(-1, (groups, -1)).mean(-1).repeat_interleave(x.shape[-1] // groups, -1)
    return i * (d - x * (i * i) * mean), dw.sum(0)


def _plain_norm_grad(s):
    out = {"dx": None, "dres": None, "dbefore": None, "dafter": None, "dz": None, "dscale": None}
    xt, wt = s["inp"].dtype, _t(s["w"])
    x, i, n, gate, a = _stream(s)[1]
    d = s["dr"].float()
    if s["before"]:
        r = s["stream"].float()
        more, dw = _norm_slope(s["dy"].float(), s["w_before"].float(), r, _inverse_rms(r, 1), 1)
        d, out["dbefore"] = d + more, dw.to(wt)
    if s["residual"]:
        out["dres"] = d.to(_t(s["r"]))
    if s["scale"]:
        out["dscale"] = (d * a).sum(0).to(wt)
        d = d * s["w_scale"].float()
    if s["gate"]:
        z = s["z"].float()
        p = 1.0 / (1.0 + torch.exp(-z))
        out["dz"] = (d * (n if s["after"] else x) * p * (1.0 + z * (1.0 - p))).to(xt)
        d = d * gate
    if s["after"]:
        d, dw = _norm_slope(d, s["w_after"].float(), x, i, s["groups"])
        out["dafter"] = dw.to(wt)
    out["dx"] = d.to(xt)
    return out


# ---- the definitions in 64 bits ----


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("linear"):
        return _exact_linear(s)
    if op == "norm":
        return _exact_norm(s)
    if op == "norm_grad":
        return _exact_norm_grad(s)
    return _exact_project(s)


def _exact_linear(s):
    """Token by token."""
    token = s["op"] == "linear_token"
    B, T, H, Hk, dk, dv = s["B"], s.get("T", 1), s["H"], s["Hk"], s["dk"], s["dv"]
    if T * (1.0 + B * H * dk * dv / 2.0e6) > 1.2e5:
        return None  # over about 20 seconds
    q, k, v = (s[n][:, None] if token else s[n] for n in ("q", "k", "v"))
    decay = torch.ones(B, T, H, dtype=torch.float64, device=q.device)
    if s["g"] is not None:
        decay = decay * torch.exp(s["g"].double().view(B, T, H) if s["decay"] == "token" else s["g"].double())
    slots = s["slots"].long() if s["slots"] is not None else torch.arange(B, device=q.device)
    live = slots >= 0
    length = s["lengths"] if s["lengths"] is not None else torch.full((B,), T, device=q.device)
    S = torch.zeros(B, H, dk, dv, dtype=torch.float64, device=q.device)
    if s["S"] is not None:
        S = S + s["S"][slots.clamp(min=0)].double()
    o = torch.zeros(B, T, H, dv, dtype=torch.float64, device=q.device)
    of = torch.arange(H, device=q.device) // (H // Hk)
    for t in range(T):
        kt, vt, qt = k[:, t].double()[:, of], v[:, t].double(), q[:, t].double()[:, of]
        new = torch.addcmul(S * decay[:, t, :, None, None], kt[..., None], vt[:, :, None])
        ok = live & (length > t)
        S = torch.where(ok[:, None, None, None], new, S)
        o[:, t] = torch.where(ok[:, None, None], torch.matmul(qt[:, :, None], S)[:, :, 0] / math.sqrt(dk), 0.0)
    out = torch.zeros(s["S_out"].shape, dtype=torch.float64, device=q.device)
    out[slots[live]] = S[live]
    return (o[:, 0] if token else o), out


def _exact_forward(s):
    """The stream behind the block and the output, differentiable in every input of `leaf`."""
    leaf = {n: s[n].double().requires_grad_() for n in ("inp", "res", "z", "w_after", "w_scale", "w_before")
            if s[n] is not None}
    M, D = s["M"], s["D"]
    h = leaf["inp"]
    if s["after"]:
        parts = h.reshape(M, s["groups"], D // s["groups"])
        h = (parts / torch.sqrt((parts ** 2).mean(2, keepdim=True) + EPS)).reshape(M, D) * leaf["w_after"]
    if s["gate"]:
        h = h * leaf["z"] * torch.sigmoid(leaf["z"])
    if s["scale"]:
        h = h * leaf["w_scale"]
    if s["residual"]:
        h = leaf["res"] + h
    return leaf, h


def _exact_norm(s):
    with torch.no_grad():
        leaf, h = _exact_forward(s)
        if not s["before"]:
            return h
        y = h / torch.sqrt((h ** 2).mean(1, keepdim=True) + EPS) * leaf["w_before"]
        return (y, h) if _moves(s) else y


def _exact_norm_grad(s):
    """By torch's differentiation of the definition, at the stream that the forward pass kept."""
    with torch.enable_grad():
        leaf, h = _exact_forward(s)
        d, dw = s["dr"].double(), None
        if s["before"]:
            r = s["stream"].double().requires_grad_()
            y = r / torch.sqrt((r ** 2).mean(1, keepdim=True) + EPS) * leaf["w_before"]
            more, dw = torch.autograd.grad(y, [r, leaf["w_before"]], s["dy"].double())
            d = d + more
        names = [n for n in ("inp", "res", "z", "w_after", "w_scale") if n in leaf]
        got = dict(zip(names, torch.autograd.grad(h, [leaf[n] for n in names], d)))
    return {"dx": got["inp"], "dres": got.get("res"), "dbefore": dw, "dafter": got.get("w_after"), "dz": got.get("z"),
            "dscale": got.get("w_scale")}


def _exact_project(s):
    if 6.0 * s["M"] * s["D"] * s["N"] > 1.0e13:
        return None
    x, w = s["inp"].double(), s["wt"].double()
    z = torch.matmul(x, w.transpose(0, 1))
    if s["bias_"] is not None:
        z += s["bias_"].double()
    p = torch.sigmoid(z) if s["act"] == "silu" else torch.special.ndtr(z)
    if s["op"] == "project":
        y = z if s["act"] == "none" else z * p
        return y if s["res"] is None else y + s["res"].double()
    dz = s["dy"].double()
    if s["act"] == "silu":
        dz = dz * (p + z * p * (1 - p))
    elif s["act"] == "gelu":
        dz = dz * (p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    return dz @ w, dz.T @ x, None if s["bias_"] is None else dz.sum(0)
