"""Blocks of linear attention, served and trained a little: a norm, one projection to queries, keys, values, gates and
decays, linear attention, the norm of its heads with their gate, and a projection back onto the stream; between blocks the
residual addition and the next norm are one call.

  python examples/linear_stack.py

runs a batch of prompts of different lengths through two blocks, decodes tokens from the carried states, and takes a few
gradient steps on what follows the attention.  Weights are random: the point is how the calls fit together.
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import sparse_state_linear_sdm_gb300 as sdm  # noqa: E402

BF16 = torch.bfloat16


class LinearBlock:
    """One block and its weights.  D: model width; H heads of dv values, Hk of them with queries and keys of dk columns."""

    def __init__(self, D=256, H=4, Hk=2, dk=64, dv=64, F=512, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rn = lambda *s, scale=1.0: torch.randn(s, generator=g, device=device) * scale  # noqa: E731
        w = lambda n, k: rn(n, k, scale=k ** -0.5).to(BF16)  # noqa: E731
        self.D, self.H, self.Hk, self.dk, self.dv = D, H, Hk, dk, dv
        self.norm, self.head_norm, self.scale = (torch.ones(n, device=device) for n in (D, H * dv, D))
        self.w_in = w(2 * Hk * dk + 2 * H * dv, D)                # queries, keys, values, gates
        self.b_in = torch.zeros(self.w_in.shape[0], dtype=BF16, device=device)
        self.w_decay = w(8 * ((H + 7) // 8), D)
        self.rate = torch.exp(torch.rand(H, generator=g, device=device) * 4.0 - 5.0)   # 0.007 .. 0.4 a token
        self.w_out = w(D, H * dv)
        self.mlp_norm, self.w_up, self.w_down = torch.ones(D, device=device), w(F, D), w(D, F)

    def state(self, nb: int):
        return torch.zeros((nb, self.H, self.dk, self.dv), dtype=torch.float32, device=self.norm.device)

    def _split(self, n):
        """q, k, v, gate, decay of normed tokens n [..., D]."""
        p = sdm.project(n, self.w_in, self.b_in)
        a, b = self.Hk * self.dk, self.H * self.dv
        q, k, v = (p[..., i:j].unflatten(-1, (h, -1)) for i, j, h in ((0, a, self.Hk), (a, 2 * a, self.Hk), (2 * a, 2 * a + b, self.H)))
        k = (k.float() * torch.rsqrt(k.float().square().sum(-1, keepdim=True) + 1e-6)).to(BF16)
        decay = -self.rate * torch.nn.functional.softplus(sdm.project(n, self.w_decay)[..., :self.H].float())
        return q, k, v, p[..., 2 * a + b:], decay

    def _finish(self, x, o, gate):
        """The stream behind the block, x [..., D] before it."""
        y = sdm.gated_norm(o.flatten(-2), self.head_norm, gate, groups=self.H)
        n, x = sdm.residual_norm(sdm.project(y, self.w_out), x, self.mlp_norm, scale=self.scale)
        return sdm.project(sdm.project(n, self.w_up, activation="gelu"), self.w_down, residual=x)

    def prompt(self, x, state, lengths=None):
        """x [B, T, D] -> [B, T, D], the state continued."""
        q, k, v, gate, decay = self._split(sdm.residual_norm(x, weight=self.norm)[0])
        o, _ = sdm.linear_attention(q, k, v, decay, state=state, lengths=lengths)
        return self._finish(x, o, gate)

    def step(self, x, state, slots=None):
        """One decode token of every sequence: x [B, D] -> [B, D]; slots: the rows of `state` the sequences have."""
        q, k, v, gate, decay = self._split(sdm.residual_norm(x, weight=self.norm)[0])
        o, _ = sdm.linear_attention_step(q, k, v, decay, state=state, slots=slots)
        return self._finish(x, o, gate)


def finish_loss(block, o, gate, x, target):
    """Half the squared distance of a block's stream (up to its addition) to `target`, and its gradients to the output
    projection, the residual scale, the head norm, the attention's output, the gate and the stream before it."""
    flat = o.flatten(-2)
    y = sdm.gated_norm(flat, block.head_norm, gate, groups=block.H)
    p = sdm.project(y, block.w_out)
    n, r = sdm.residual_norm(p, x, block.mlp_norm, scale=block.scale)
    diff = n.float() - target
    dp, dx, dweight, _, _, dscale = sdm.residual_norm_backward(p, r, diff.to(BF16), None, block.mlp_norm, scale=block.scale)
    dy, dw, _ = sdm.project_backward(y, block.w_out, dp)
    do, dhead, dgate = sdm.gated_norm_backward(flat, block.head_norm, dy, gate, groups=block.H)
    return 0.5 * diff.square().sum().item(), dict(w_out=dw, scale=dscale, mlp_norm=dweight, head_norm=dhead,
                                                  o=do.view_as(o), gate=dgate, x=dx)


def main():
    blocks = [LinearBlock(seed=i) for i in range(2)]
    nb, T, new = 4, 96, 16
    x = torch.randn(nb, T, blocks[0].D, device="cuda").to(BF16)
    states = [b.state(nb) for b in blocks]
    y = x
    for b, st in zip(blocks, states):
        y = b.prompt(y, st)
    tok = y[:, -1].contiguous()
    for _ in range(new):
        for b, st in zip(blocks, states):
            tok = b.step(tok, st)
    print(f"prompt of {nb} x {T} tokens, {new} tokens decoded: last token's rms "
          f"{tok.float().square().mean().sqrt().item():.3f}")
    ragged = blocks[0].prompt(x, blocks[0].state(nb), lengths=torch.tensor([96, 40, 0, 7], dtype=torch.int32, device="cuda"))
    print(f"ragged prompts: {tuple(ragged.shape)}")
    b = blocks[0]
    q, k, v, gate, decay = b._split(sdm.residual_norm(x, weight=b.norm)[0])
    o, _ = sdm.linear_attention(q, k, v, decay)
    target = torch.randn(x.shape, device="cuda")
    losses = []
    for _ in range(6):
        loss, g = finish_loss(b, o, gate, x, target)
        losses.append(loss)
        b.w_out = (b.w_out.float() - 1e-3 * g["w_out"].float()).to(BF16)
        b.scale = b.scale - 1e-3 * g["scale"]
    print("losses: " + ", ".join(f"{v:.1f}" for v in losses))


if __name__ == "__main__":
    main()
