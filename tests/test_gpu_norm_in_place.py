"""Gradients of the norms written over the tensors they come from: dx, dgate and dresidual may lie exactly over an input of the
same row size (sdm_residual_norm_backward), and are then bit for bit what they are in memory of their own."""
import ctypes

import pytest
import torch

import sparse_state_linear_sdm_gb300 as sdm
from test_gpu_norm import _case
from test_mixer_abi import BF16, F32, SILU, NormArgs, NormGrads, P, SZ

pytestmark = pytest.mark.gpu

CODES = {torch.float32: F32, torch.bfloat16: BF16}
CASES = [
    # x, residual, weights, M, D, groups, parts (after, gate, scale, residual, weight), layout
    ("bf16", "bf16", "bf16", 2000, 2048, 1, "rw", "dense"),       # the next row ahead; more rows than teams
    ("bf16", "bf16", "bf16", 900, 2047, 1, "rw", "dense"),        # rows off 16 bytes
    ("bf16", "bf16", "f32", 700, 8192, 1, "rw", "dense"),         # no row ahead
    ("bf16", "bf16", "f32", 400, 16384, 1, "rw", "dense"),
    ("bf16", "bf16", "f32", 400, 8191, 1, "agsrw", "dense"),
    ("bf16", "bf16", "bf16", 3000, 1000, 1, "agsrw", "dense"),
    ("f32", "f32", "f32", 3000, 500, 1, "agsrw", "dense"),
    ("bf16", "bf16", "f32", 700, 6000, 1, "agsrw", "dense"),      # sums in shared memory
    ("bf16", "bf16", "f32", 4000, 2048, 16, "ag", "dense"),       # heads of 128
    ("bf16", "bf16", "f32", 4000, 150, 6, "ag", "dense"),
    ("f32", "f32", "f32", 9000, 40, 1, "sr", "dense"),            # no norm after it: the rest decides at run time
    ("bf16", "bf16", "bf16", 5000, 264, 1, "gsr", "dense"),
]
IDS = [f"{c[0]}-{c[3]}x{c[4]}.{c[5]}-{c[6]}" for c in CASES]
# output -> the inputs it may lie over here; every pair of a row, and three at once
OVER = ([{"dx": "x"}, {"dx": "dy"}, {"dx": "r"}, {"dx": "dr"}, {"dx": "gate"}, {"dgate": "gate"}, {"dgate": "x"}, {"dgate": "dr"},
         {"dresidual": "dr"}, {"dresidual": "r"}, {"dresidual": "dy"}, {"dresidual": "x"}]
        + [{"dx": "x", "dgate": "gate", "dresidual": "dr"}, {"dx": "dr", "dgate": "x", "dresidual": "r"},
           {"dx": "dy", "dresidual": "dr"}, {"dx": "gate", "dgate": "dr"}])


def _gradients(t, weights, c, over):
    """Every output of the C entry for the tensors t = {x, gate, r, dy, dr} (copied first); `over` as in OVER."""
    t = {n: v if v is None else v.clone() for n, v in t.items()}
    x = t["x"]
    M, D = x.shape
    wt = next(v.dtype for v in weights.values() if v is not None)
    like = dict(dx=x, dgate=t["gate"], dresidual=t["dr"] if "r" in c[6] else None)
    out = {n: None if v is None else (t[over[n]] if n in over else torch.full_like(v, 3.0)) for n, v in like.items()}
    for n, of in (("dafter", "after"), ("dscale", "scale"), ("dweight", "weight")):
        out[n] = None if weights[of] is None else torch.empty(D, dtype=wt, device="cuda")
    at = lambda v: None if v is None else v.data_ptr()  # noqa: E731
    rs = lambda v: 0 if v is None else v.stride(0)      # noqa: E731
    args = NormArgs(x=at(x), residual=None, gate=at(t["gate"]), x_rs=rs(x), residual_rs=0, gate_rs=rs(t["gate"]),
                    after=at(weights["after"]), scale=at(weights["scale"]), weight=at(weights["weight"]),
                    x_dtype=CODES[x.dtype], r_dtype=CODES[t["dr"].dtype], w_dtype=CODES[wt], act=SILU, M=M, D=D, groups=c[5],
                    eps=1e-6)
    grads = NormGrads(r=at(t["r"]), dy=at(t["dy"]), dr=at(t["dr"]), r_rs=rs(t["r"]), dy_rs=rs(t["dy"]), dr_rs=rs(t["dr"]),
                      **{n: at(v) for n, v in out.items()})
    ws = torch.empty(sdm.residual_norm_backward_workspace_size(M, D, c[5]), dtype=torch.uint8, device="cuda")
    f = sdm.lib().sdm_residual_norm_backward
    f.argtypes = [P, P, P, SZ, P]
    assert f(ctypes.byref(args), ctypes.byref(grads), ws.data_ptr(), ws.numel(),
             torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_gradients_over_their_inputs(c):
    a, dy, dr = _case(c)
    weights = {n: a[n] for n in ("after", "scale", "weight")}
    has_weight = a["weight"] is not None
    r = sdm.residual_norm(**a)[1]
    t = dict(x=a["x"], gate=a["gate"], r=r if has_weight else None, dy=dy if has_weight else None, dr=dr)
    want = _gradients(t, weights, c, {})
    got = sdm.residual_norm_backward(a["x"], r, t["dy"], dr, a["weight"], after=a["after"], gate=a["gate"], scale=a["scale"],
                                     residual=a["residual"] is not None, groups=c[5])
    for n, v in zip(("dx", "dresidual", "dweight", "dafter", "dgate", "dscale"), got):
        assert v is None or torch.equal(v, want[n]), n
    ran = 0
    for over in OVER:
        if any(t[i] is None or want[n] is None or t[i].dtype != want[n].dtype for n, i in over.items()):
            continue
        ran += 1
        for n, v in _gradients(t, weights, c, over).items():
            assert v is None or torch.equal(v, want[n]), (over, n)
    assert ran >= 3
