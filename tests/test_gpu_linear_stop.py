"""Linear attention on the tensor cores when a copy does not come: the block stops, waits for what it has under way and reports,
the other blocks' work is right, and a new state is written whole or not at all (sdm_test_linear_stall; the waits' limit is
1 ms).  Nothing here faults or hangs: every wait is bounded."""
import ctypes
import time

import pytest
import torch

import sparse_state_linear_sdm_gb300 as sdm
from test_gpu_linear import _case
from test_mixer_abi import BF16, LinearArgs, P, SZ

pytestmark = pytest.mark.gpu

WHOLE = ("bf16", 2, 700, 2, 2, 128, 128, "token", True, None, 0, "dense")    # 6 chunks, 4 blocks
CUT = ("bf16", 1, 2048, 2, 2, 64, 128, "token", True, None, 0, "dense")      # 8 segments of 2 chunks


def _stall(a, o, state_out, pass_, block, chunk, load):
    B, T, Hk, dk = a["q"].shape
    H, dv = a["v"].shape[2:]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = sdm.linear_attention_workspace_size(torch.bfloat16, B, T, H, Hk, dk, dv)
    ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")
    args = LinearArgs(**{x: a[y].data_ptr() for x, y in (("q", "q"), ("k", "k"), ("v", "v"), ("g", "decay"), ("state", "state"))},
                      **{f"{x}_bs": a[y].stride(0) for x, y in (("q", "q"), ("k", "k"), ("v", "v"), ("g", "decay"))},
                      **{f"{x}_ts": a[y].stride(1) for x, y in (("q", "q"), ("k", "k"), ("v", "v"), ("g", "decay"))},
                      state_out=state_out.data_ptr(), lengths=None, slots=None, o=o.data_ptr(), dtype=BF16, B=B, T=T, H=H,
                      Hk=Hk, dk=dk, dv=dv, n_slots=B, scale=dk ** -0.5)
    f = sdm.lib().sdm_test_linear_stall
    f.argtypes = [P, P, SZ, *[ctypes.c_int] * 4, ctypes.c_ulonglong, P, P]
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    status = f(ctypes.byref(args), ws.data_ptr(), n, pass_, block, chunk, load, 1_000_000, err.data_ptr(),
               torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == 0 and time.perf_counter() - t0 < 1.5      # no wait of a drain has run into its 2 s
    return err.item()


def _run(c, in_place, *where):
    """(o, state) of a clean call, the state before, and o and state after a stall there; the call after it is clean again."""
    a = _case(c)
    o, st = sdm.linear_attention(**a, state_out=torch.zeros_like(a["state"]))
    before = a["state"].clone() if in_place else torch.full_like(st, 7.0)
    out = torch.full_like(o, 3.0)
    state_out = a["state"] if in_place else before.clone()
    assert _stall(a, out, state_out, *where) == sdm.SDM_DEV_TIMEOUT
    got = state_out.clone()
    if in_place:
        a["state"].copy_(before)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o2, st2 = sdm.linear_attention(**a, state_out=torch.zeros_like(st), dev_err=err)
    assert err.item() == 0 and torch.equal(o2, o) and torch.equal(st2, st)
    return o, st, before, out, got


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("chunk,load", [(0, 2), (0, 0), (0, 1), (1, 1), (2, 0), (3, 2), (5, 0), (5, 1)])
def test_a_sequence_in_one_piece(chunk, load, in_place):
    o, st, before, out, got = _run(WHOLE, in_place, 0, 1, chunk, load)
    rest = [(0, 0), (1, 0), (1, 1)]                            # block 1: sequence 0, head 1
    for b, h in rest:
        assert torch.equal(out[b, :, h], o[b, :, h]) and torch.equal(got[b, h], st[b, h])
    late = (chunk, load) == (5, 1)                             # q of the last chunk: the state is already known
    assert torch.equal(got[0, 1], (st if late else before)[0, 1])


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("chunk,load", [(0, 1), (0, 0), (1, 0)])
def test_the_end_of_a_segment(chunk, load, in_place):
    """Segment 3 of head 1: its end is not known, so neither are the later ones' beginnings nor the new state."""
    o, st, before, out, got = _run(CUT, in_place, 1, 7, chunk, load)
    assert torch.equal(out[:, :, 0], o[:, :, 0]) and torch.equal(got[0, 0], st[0, 0])
    assert torch.equal(out[:, :1024, 1], o[:, :1024, 1]) and torch.equal(got[0, 1], before[0, 1])


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("seg,chunk,load", [(7, 0, 0), (7, 1, 2), (7, 1, 1), (2, 0, 2), (2, 1, 0), (0, 1, 1)])
def test_a_segment(seg, chunk, load, in_place):
    """A segment's outputs depend on itself alone, and the new state on the last one."""
    o, st, before, out, got = _run(CUT, in_place, 2, seg * 2, chunk, load)
    assert torch.equal(out[:, :, 1], o[:, :, 1]) and torch.equal(got[0, 1], st[0, 1])
    others = [t for t in range(2048) if t // 256 != seg]
    assert torch.equal(out[:, others, 0], o[:, others, 0])
    lost = seg == 7 and (chunk, load) != (1, 1)
    assert torch.equal(got[0, 0], (before if lost else st)[0, 0])
