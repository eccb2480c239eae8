"""Linear attention at the ends of its ranges: the longest prompts that a call takes, and what their cuts leave."""
import numpy as np
import pytest
import torch

import mixer_ref as ref
import sparse_state_linear_sdm_gb300 as sdm

pytestmark = pytest.mark.gpu

LONGEST = 2 ** 31 - 1 - 1024  # tokens


@pytest.mark.parametrize("dtype, d", [(torch.float32, 1), (torch.bfloat16, 1), (torch.bfloat16, 8)],
                         ids=["token by token", "copied", "chunks"])
def test_the_longest_prompt(dtype, d):
    """One head of 2^31 - 1025 tokens is cut into segments, and the last one's length on top of its start would pass 2^31.
    Decays of 1 leave nothing of what is 200 tokens back, so every output but the last ones is the same up to its roundings
    (three of at most 2^-8 on either side), and those and the state are the definition's over the last 200 tokens.
    bf16 goes in chunks whatever d (copied to rows of 16 bytes where it is 1), so its bound is the chunks'.  d = 1: queries
    and keys with strides of 0; d = 8: q, k and v are the same rows."""
    torch.cuda.empty_cache()
    code = 2 if dtype == torch.bfloat16 else 4
    need = LONGEST * 2 * code * d + sdm.linear_attention_workspace_size(dtype, 1, LONGEST, 1, 1, d, d)
    if torch.cuda.mem_get_info()[0] < need + (4 << 30):
        pytest.skip(f"needs {need >> 30} GB")
    v = torch.full((1, LONGEST, 1, d), 0.5, dtype=dtype, device="cuda")
    torch.manual_seed(5)
    v[0, -5:, 0] = torch.randn(5, d, device="cuda").to(dtype)
    q = k = v if d == 8 else torch.ones(1, 1, 1, 1, dtype=dtype, device="cuda").expand(1, LONGEST, 1, 1)
    o = torch.full_like(v, float("nan"))
    decay, state = torch.full((1,), -1.0, device="cuda"), torch.zeros(1, 1, d, d, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sdm.linear_attention(q, k, v, decay, scale=1.0, state=state, out=o, dev_err=err)
    assert err.item() == 0
    one = o[0, 200, 0].float()
    for part in o[0, 200:-5, 0].split(1 << 27):              # no token is left out, wherever it is
        assert ((part.float() - one).abs().amax(0) <= 6 * ref.H * one.abs()).all()
    n = 200                                                  # e^-200 of the state: nothing
    h = lambda t: t[:, -n:].double().cpu().numpy()           # noqa: E731
    want, wstate, eo, es = ref.linear(h(q), h(k), h(v), np.full((1, n, 1), -1.0), 1.0, np.zeros((1, 1, d, d)),
                                      chunked=dtype == torch.bfloat16)
    off = np.abs(h(o) - want)[:, n // 2:] / (eo + ref.ROUND["bf16" if code == 2 else "f32"] * (np.abs(want) + eo))[:, n // 2:]
    assert off.max() <= 1, off.max()
    off = np.abs(state.double().cpu().numpy() - wstate) / (es + ref.U * np.abs(wstate))
    assert off.max() <= 1, off.max()
