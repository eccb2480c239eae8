"""A hybrid recurrent block, served and trained a little: a short causal convolution and a selective state space
scan, the sparse delta memory, and a gated feed-forward layer, each with a residual connection.

  python examples/hybrid_stack.py

runs a batch of prompts of different lengths through the block, then decodes tokens from the carried states, then takes
a few gradient steps on the feed-forward layer.  Weights are random: the point is how the calls fit together.
The plain projections between them are torch products.
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


class HybridBlock:
    """One block and its weights.  D: model width; `inner` channels of N states in the scan; H memory heads of S*S
    slots and d_v columns, W written and R read a token; F feed-forward columns."""

    def __init__(self, D=256, inner=512, N=16, K=4, H=2, S=16, d_v=64, W=8, R=8, F=768, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rn = lambda *s, scale=1.0: (torch.randn(s, generator=g, device=device) * scale)  # noqa: E731
        self.D, self.inner, self.N, self.K, self.H, self.S, self.d_v, self.W, self.R, self.F = (
            D, inner, N, K, H, S, d_v, W, R, F)
        self.rank = max(8, D // 16)
        w = lambda n, k: rn(n, k, scale=k ** -0.5).to(BF16)  # noqa: E731
        self.w_in, self.w_mix = w(2 * inner, D), w(D, inner)
        self.w_conv, self.b_conv = rn(inner, K, scale=K ** -0.5).to(BF16), torch.zeros(inner, dtype=BF16, device=device)
        self.w_x, self.w_dt = w(self.rank + 2 * N, inner), w(inner, self.rank)
        step = torch.exp(torch.rand(inner, generator=g, device=device) * 4.6 - 6.9)  # 0.001 .. 0.1
        self.dt_bias = step + torch.log(-torch.expm1(-step))
        self.A = -torch.arange(1, N + 1, device=device, dtype=torch.float32).repeat(inner, 1)
        self.skip = torch.ones(inner, device=device)
        self.w_kq, self.w_v, self.w_gates = w(4 * H * S, D), w(H * d_v, D), w(2 * H, D)
        self.w_mem = w(D, H * d_v)
        self.M0 = rn(H, S * S, d_v, scale=0.02)
        self.w_gate_up, self.w_down = w(2 * F, D), w(D, F)

    def states(self, nb: int) -> dict:
        """Fresh states of nb sequences."""
        dev = self.M0.device
        M = torch.empty((nb, self.H, self.S * self.S, self.d_v), dtype=torch.float32, device=dev)
        return dict(conv=torch.zeros((nb, self.K - 1, self.inner), dtype=BF16, device=dev),
                    scan=torch.zeros((nb, self.inner, self.N), dtype=torch.float32, device=dev),
                    memory=sdm.init_state_from_M0(M, self.M0))

    @staticmethod
    def _norm(x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(BF16)

    def _memory_inputs(self, x):
        """v [B, H, T, d_v], alpha, beta [B, H, T] of tokens x [B, T, D]."""
        nb, T, _ = x.shape
        v = (x @ self.w_v.T).view(nb, T, self.H, self.d_v).transpose(1, 2).contiguous()
        gates = torch.sigmoid((x @ self.w_gates.T).float()).view(nb, T, 2, self.H).transpose(1, 3)
        return v, gates[:, :, 0].contiguous(), gates[:, :, 1].contiguous()

    def prompt(self, x, st, lengths=None):
        """x [B, T, D] -> [B, T, D], the states in `st` continued.  lengths (int32 [B]) end the convolution and the
        scan of each sequence; the memory takes whole prompts, so it is run on full ones only."""
        n = self._norm(x)
        xz = n @ self.w_in.T                                      # the convolution reads one half in place
        c, _ = sdm.causal_conv(xz[..., :self.inner], self.w_conv, self.b_conv, state=st["conv"], lengths=lengths)
        p = c @ self.w_x.T                                        # step features, B and C: slices of one product
        r, N = self.rank, self.N
        y, _ = sdm.selective_scan(c, p[..., :r] @ self.w_dt.T, self.A, p[..., r:r + N], p[..., r + N:], D=self.skip,
                                  z=xz[..., self.inner:], dt_bias=self.dt_bias, state=st["scan"], lengths=lengths)
        x = x + y @ self.w_mix.T
        if lengths is None:
            n = self._norm(x)
            kp, qp = sdm.project_kq(n, self.w_kq, self.H, self.S)
            o, _, _ = sdm.forward(kp, qp, *self._memory_inputs(n), None, self.W, self.R, M=st["memory"])
            x = x + o.transpose(1, 2).reshape(*x.shape[:2], -1).to(BF16) @ self.w_mem.T
        h = sdm.project_gated(self._norm(x), self.w_gate_up)
        return x + h @ self.w_down.T

    def step(self, x, st, memory_step):
        """One decode token of every sequence: x [B, D] -> [B, D]; memory_step: sdm.DecodeStep on st["memory"]."""
        n = self._norm(x)
        xz = n @ self.w_in.T
        c, _ = sdm.causal_conv_step(xz[:, :self.inner], self.w_conv, self.b_conv, state=st["conv"])
        p = c @ self.w_x.T
        r, N = self.rank, self.N
        y, _ = sdm.selective_step(c, p[:, :r] @ self.w_dt.T, self.A, p[:, r:r + N], p[:, r + N:], D=self.skip,
                                  z=xz[:, self.inner:], dt_bias=self.dt_bias, state=st["scan"])
        x = x + y @ self.w_mix.T
        n = self._norm(x).unsqueeze(1)
        kp, qp = sdm.project_kq(n, self.w_kq, self.H, self.S)
        o = memory_step(kp, qp, *self._memory_inputs(n))
        x = x + o.transpose(1, 2).reshape(x.shape[0], -1).to(BF16) @ self.w_mem.T
        h = sdm.project_gated(self._norm(x), self.w_gate_up)
        return x + h @ self.w_down.T


def train_feed_forward(block: HybridBlock, x, target, steps=8, lr=2.0):
    """Gradient steps on the feed-forward layer's weights for the mean squared distance of its output to `target`;
    returns the losses.  The forward pass keeps its input; the gradient recomputes the projections from it."""
    losses = []
    for _ in range(steps):
        h = sdm.project_gated(x, block.w_gate_up)
        diff = (h @ block.w_down.T).float() - target
        losses.append(diff.square().mean().item())
        dy = (diff * (2.0 / diff.numel())).to(BF16)
        dh = dy @ block.w_down
        _, dw = sdm.project_gated_backward(x, block.w_gate_up, dh)
        block.w_down = (block.w_down.float() - lr * (dy.T @ h).float()).to(BF16)
        block.w_gate_up = (block.w_gate_up.float() - lr * dw.float()).to(BF16)
    return losses


def main():
    block = HybridBlock()
    nb, T, new = 4, 96, 16
    x = torch.randn(nb, T, block.D, device="cuda").to(BF16)
    st = block.states(nb)
    y = block.prompt(x, st)
    memory = sdm.DecodeStep(st["memory"], block.W, block.R)
    tok = y[:, -1]
    for _ in range(new):
        tok = block.step(tok, st, memory)
    print(f"prompt of {nb} x {T} tokens, {new} tokens decoded from the carried states: "
          f"last token's rms {tok.float().square().mean().sqrt().item():.3f}")
    ragged = block.prompt(x, block.states(nb), lengths=torch.tensor([96, 40, 0, 7], dtype=torch.int32, device="cuda"))
    print(f"ragged prompts: {tuple(ragged.shape)}")
    xs = x.reshape(-1, block.D)
    losses = train_feed_forward(block, xs, torch.randn(xs.shape, device="cuda") * 0.5)
    print("feed-forward losses: " + ", ".join(f"{v:.4f}" for v in losses))


if __name__ == "__main__":
    main()
