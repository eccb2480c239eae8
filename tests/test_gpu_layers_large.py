"""The convolution, the scan and the gated projections where element offsets pass 2^31, and inside a CUDA graph.

The last tokens of a long input are compared with the same tokens run alone: the arithmetic of a token does not
depend on where it stands, so the convolution and the projections agree bit for bit (the projections' gradient, whose
reduction is split differently for few tokens, is held to the 64-bit definition and its bound instead); the scan's states here decay to
nothing within ten tokens (steps of about 1.3 at a rate of 64), so the tokens after them agree to rounding."""
import numpy as np
import pytest
import torch

import layers_ref as ref
import sparse_state_linear_sdm_gb300 as sdm

pytestmark = pytest.mark.gpu

T, D = 540_000, 4096  # 2.2e9 elements


@pytest.fixture(scope="module")
def long_input():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    return torch.randn((1, T, D), generator=g, device="cuda", dtype=torch.bfloat16)


def test_convolution_past_32_bit_offsets(long_input):
    x = long_input
    w = torch.randn(D, 4, device="cuda").bfloat16()
    y, _ = sdm.causal_conv(x, w)
    st = x[:, T - 40 - 3:T - 40].contiguous()
    tail, _ = sdm.causal_conv(x[:, T - 40:], w, state=st)
    assert torch.equal(y[:, T - 40:], tail)


def test_scan_past_32_bit_offsets(long_input):
    x = long_input
    A = torch.full((D, 4), -64.0, device="cuda")
    bc = torch.randn((1, T, 4), device="cuda").bfloat16()
    bias = torch.ones(D, device="cuda")
    run = lambda a: sdm.selective_scan(a(x), a(x), A, a(bc), a(bc), dt_bias=bias,  # noqa: E731
                                       state_out=torch.empty(1, D, 4, device="cuda"))
    y, st = run(lambda v: v)
    tail, ts = run(lambda v: v[:, T - 40:])
    assert torch.allclose(y[:, T - 30:].float(), tail[:, 10:].float(), rtol=2.0 ** -7, atol=1e-6)
    assert torch.allclose(st, ts, rtol=1e-5, atol=1e-7)


def test_gated_past_32_bit_offsets():
    M, d, F = 270_000, 64, 8192  # 2.2e9 outputs
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn((M, d), generator=g, device="cuda").bfloat16()
    w = torch.randn((2 * F, d), generator=g, device="cuda").bfloat16()
    h = sdm.project_gated(x, w)
    assert torch.equal(h[M - 300:], sdm.project_gated(x[M - 300:].contiguous(), w))
    dx, _ = sdm.project_gated_backward(x, w, h)
    host = lambda t: t[M - 300:].double().cpu().numpy()  # noqa: E731
    want, _, bound, _ = ref.gated_grad(host(x), w.double().cpu().numpy(), host(h), "silu")
    assert (np.abs(host(dx) - want) <= bound + ref.ROUND["bf16"] * (np.abs(want) + bound)).all()


def test_layers_replay_from_a_graph():
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, w, dh = rn(300, 128).bfloat16(), rn(144, 128).bfloat16(), rn(300, 72).bfloat16()
    u, dt, A, bc = rn(1, 700, 64), rn(1, 700, 64), -torch.exp(rn(64, 16)), rn(1, 700, 16)
    k = rn(64, 4)
    ws = torch.empty(sdm.selective_scan_workspace_size(1, 700, 64, 16), dtype=torch.uint8, device="cuda")

    def run():
        c, _ = sdm.causal_conv(u, k)
        y, _ = sdm.selective_scan(c, dt, A, bc, bc, workspace=ws)
        h = sdm.project_gated(x, w)
        return (c, y, h, *sdm.project_gated_backward(x, w, dh))

    want = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
