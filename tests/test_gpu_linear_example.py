"""The blocks of examples/linear_stack.py: linear attention, norms and projections together, as they are served and trained."""
import importlib.util
import os

import pytest
import torch

import sparse_state_linear_sdm_gb300 as sdm

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "linear_stack.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("linear_stack", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _x(*shape, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("T", [40, 300])
def test_prompt_then_tokens_is_the_longer_prompt(example, T):
    """The two differ by bf16 roundings between the layers (2^-8 each, some ten of them in a row); 1/16 of the output's size
    bounds them with room, and a wrong state is off by its whole size."""
    blocks = [example.LinearBlock(seed=s) for s in (3, 4)]
    x = _x(3, T, blocks[0].D)
    whole = x
    for b in blocks:
        whole = b.prompt(whole, b.state(3))
    states = [b.state(3) for b in blocks]
    y = x[:, :T - 6].contiguous()
    for b, st in zip(blocks, states):
        y = b.prompt(y, st)
    outs = [y]
    for t in range(T - 6, T):
        tok = x[:, t].contiguous()
        for b, st in zip(blocks, states):
            tok = b.step(tok, st)
        outs.append(tok.unsqueeze(1))
    got = torch.cat(outs, 1).float()
    off = (got - whole.float()).norm(dim=-1) / whole.float().norm(dim=-1)
    assert off.max() < 1 / 16, off.max().item()


def test_sequences_in_slots_and_ragged_prompts(example):
    b = example.LinearBlock(seed=5)
    x = _x(2, 150, b.D)
    ln = torch.tensor([150, 33], dtype=torch.int32, device="cuda")
    st = b.state(2)
    b.prompt(x, st, lengths=ln)
    alone = b.state(1)
    b.prompt(x[1:, :33].contiguous(), alone, lengths=ln[1:])
    assert torch.equal(st[1:], alone)                             # padding changes nothing
    pool = torch.zeros(5, *st.shape[1:], device="cuda")
    slots = torch.tensor([4, 1], dtype=torch.int32, device="cuda")
    pool[slots.long()] = st
    tok = x[:, -1].contiguous()
    assert torch.equal(b.step(tok, pool, slots), b.step(tok, st)) and torch.equal(pool[slots.long()], st)


def test_gradients_against_torch(example):
    """Against torch's differentiation of the same steps in 64 bits.  The kernels round seven tensors of the chain to bf16 (y,
    p, r, n's gradient, dp, dy, and each result), each by 2^-8 / sqrt(3) of its norm in the mean: 2^-8 * sqrt(7 / 3) < 0.006 of a
    result's norm; 0.02 is three times that."""
    b = example.LinearBlock(seed=7)
    o, gate, x = _x(2, 50, b.H, b.dv), _x(2, 50, b.H * b.dv, seed=2), _x(2, 50, b.D, seed=3)
    target = _x(2, 50, b.D, seed=4).float()
    loss, got = example.finish_loss(b, o, gate, x, target)
    leaf = {n: t.double().requires_grad_() for n, t in
            dict(o=o, gate=gate, x=x, w_out=b.w_out, scale=b.scale, mlp_norm=b.mlp_norm, head_norm=b.head_norm).items()}
    h = leaf["o"] / (leaf["o"].square().mean(-1, keepdim=True) + 1e-6).sqrt()
    y = h.flatten(-2) * leaf["head_norm"] * torch.nn.functional.silu(leaf["gate"])
    r = leaf["x"] + leaf["scale"] * (y @ leaf["w_out"].T)
    n = r / (r.square().mean(-1, keepdim=True) + 1e-6).sqrt() * leaf["mlp_norm"]
    want = 0.5 * (n - target).square().sum()
    want.backward()
    assert abs(loss - want.item()) < 0.01 * want.item()
    for name, t in got.items():
        w = leaf[name].grad
        off = ((t.double() - w).norm() / w.norm()).item()
        assert off < 0.02, (name, off)


def test_example_runs(example, capsys):
    example.main()
    assert "losses" in capsys.readouterr().out


def test_a_decode_step_replays_from_a_graph(example):
    """A block's step, every call of it captured: the state goes on from token to token."""
    b = example.LinearBlock(seed=9)
    x, st = _x(4, b.D), b.state(4)
    kept = [b.step(x, st).clone() for _ in range(3)]
    st.zero_()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b.step(x, b.state(4))
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = b.step(x, st)
    st.zero_()
    for want in kept:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
