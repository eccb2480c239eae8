"""The hybrid block of examples/hybrid_stack.py: the layers together as they are served and trained."""
import importlib.util
import os

import pytest
import torch

import sparse_state_linear_sdm_gb300 as sdm

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_stack.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("hybrid_stack", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_prompt_then_tokens_is_the_longer_prompt(example):
    """The decoded tokens match the longer prompt's last ones.  The two differ by bf16 roundings of the products
    between the layers (2^-8 each, some ten of them in a row) and where such a rounding changes a memory slot's
    rank; 1/8 of the output's size bounds both with room, and a wrong state is off by its whole size."""
    block = example.HybridBlock(seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(3, 40, block.D, generator=g, device="cuda").bfloat16()
    whole = block.prompt(x, block.states(3))
    st = block.states(3)
    first = block.prompt(x[:, :34].contiguous(), st)
    memory = sdm.DecodeStep(st["memory"], block.W, block.R)
    outs = [block.step(x[:, t].contiguous(), st, memory).unsqueeze(1) for t in range(34, 40)]
    got = torch.cat([first, *outs], 1).float()
    for t in range(40):
        d = (got[:, t] - whole[:, t].float()).norm() / whole[:, t].float().norm()
        assert d < 0.125, (t, d.item())


def test_ragged_prompts_end_where_they_end(example):
    block = example.HybridBlock(seed=5)
    x = torch.randn(2, 24, block.D, device="cuda").bfloat16()
    ln = torch.tensor([24, 9], dtype=torch.int32, device="cuda")
    st = block.states(2)
    block.prompt(x, st, lengths=ln)
    alone = block.states(1)
    block.prompt(x[1:, :9].contiguous(), alone, lengths=ln[1:])
    assert torch.equal(st["conv"][1:], alone["conv"])
    assert torch.allclose(st["scan"][1:], alone["scan"], rtol=0.02, atol=0.02)


def test_feed_forward_learns(example):
    block = example.HybridBlock(seed=7)
    x = torch.randn(256, block.D, device="cuda").bfloat16()
    losses = example.train_feed_forward(block, x, 0.5 * torch.randn(256, block.D, device="cuda"))
    assert losses[-1] < losses[0]


def test_example_runs(example, capsys):
    example.main()
    assert "feed-forward losses" in capsys.readouterr().out
