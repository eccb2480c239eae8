"""Host checks of the entry point that stops linear attention's copies: bad arguments launch nothing.  No GPU needed."""
import ctypes

import sparse_state_linear_sdm_gb300 as sdm
from test_mixer_abi import AT, BF16, EINVAL, EUNSUPPORTED, F32, LINEAR, LinearArgs, P, SZ

I, ULL = ctypes.c_int, ctypes.c_ulonglong


def stall(pass_=0, block=0, chunk=0, load=0, wait=1_000_000, err=AT[10], **kw):
    f = sdm.lib().sdm_test_linear_stall
    f.argtypes = [P, P, SZ, I, I, I, I, ULL, P, P]
    args = LinearArgs(**{**LINEAR, "dtype": BF16, "T": 64, **kw})
    return f(ctypes.byref(args), AT[9], 1 << 20, pass_, block, chunk, load, wait, err, None)


def test_stall_rejects_bad_arguments_without_launching():
    for kw in (dict(pass_=-1), dict(pass_=3), dict(block=-1), dict(chunk=-1), dict(load=-1), dict(load=3), dict(wait=10),
               dict(wait=2_000_000_000), dict(err=None), dict(B=0)):
        assert stall(**kw) == EINVAL, kw
    for kw in (dict(T=1), dict(T=4), dict(dtype=F32), dict(dk=200), dict(q=AT[0] + 2, q_ts=33)):   # token by token
        assert stall(**kw) == EUNSUPPORTED, kw
    f = sdm.lib().sdm_test_linear_stall
    assert f(None, None, 0, 0, 0, 0, 0, 1_000_000, AT[10], None) == EINVAL
