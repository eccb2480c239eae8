"""Host checks of the convolution, scan and gated entry points: bad arguments are refused before anything is
launched, and calls with nothing to do return at once.  No GPU needed."""
import ctypes

import pytest
import torch

import sparse_state_linear_sdm_gb300 as sdm

OK, EINVAL, EALIGN, EUNSUPPORTED, ENOSPACE = 0, -1, -2, -6, -7
FAKE, ODD = 0x10000, 0x10001  # never dereferenced on these paths
F32, BF16 = 0, 1
P, I, LL, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t


def conv(x=FAKE, bs=64, ts=16, dt=BF16, w=FAKE, bias=FAKE, wdt=BF16, B=2, T=4, D=16, K=4, act=1, state=FAKE,
         out=FAKE, rows=2, lengths=None, slots=None, y=FAKE, err=None):
    f = sdm.lib().sdm_causal_conv
    f.argtypes = [P, LL, LL, I, P, P, I, I, I, I, I, I, P, P, I, P, P, P, P, P]
    return f(x, bs, ts, dt, w, bias, wdt, B, T, D, K, act, state, out, rows, lengths, slots, y, err, None)


def test_conv_refusals():
    assert conv(B=0) == EINVAL
    assert conv(T=-1) == EINVAL
    assert conv(D=0) == EINVAL
    assert conv(K=1) == EINVAL
    assert conv(dt=3) == EINVAL
    assert conv(wdt=-1) == EINVAL
    assert conv(act=2) == EINVAL
    assert conv(K=9) == EUNSUPPORTED
    assert conv(B=1 << 20, T=1 << 12, rows=1 << 20) == EUNSUPPORTED
    assert conv(rows=1) == EINVAL                       # two sequences, one row, no slots
    assert conv(slots=FAKE, rows=0) == EINVAL
    assert conv(x=ODD) == EALIGN
    assert conv(y=None) == EALIGN
    assert conv(w=None) == EALIGN
    assert conv(state=ODD) == EALIGN
    assert conv(dt=F32, x=0x10002) == EALIGN
    assert conv(lengths=0x10002) == EALIGN
    assert conv(T=0) == OK                              # in place and no token: nothing to do
    assert conv(T=0, out=None, x=None, y=None) == OK


SCAN = dict(x=FAKE, dt=FAKE, Bm=FAKE, Cm=FAKE, z=FAKE, x_bs=64, x_ts=16, dt_bs=64, dt_ts=16, B_bs=32, B_ts=8, C_bs=32,
            C_ts=8, z_bs=64, z_ts=16, A=FAKE, D=FAKE, dt_bias=FAKE, state=FAKE, state_out=FAKE, lengths=0, slots=0,
            y=FAKE, dtype=BF16, B=2, T=4, Dm=16, N=8, G=1, softplus=1, n_slots=2)


class ScanArgs(ctypes.Structure):
    """sdm_ssm_args."""
    _fields_ = ([(n, P) for n in ("x", "dt", "Bm", "Cm", "z")]
                + [(n, LL) for n in ("x_bs", "x_ts", "dt_bs", "dt_ts", "B_bs", "B_ts", "C_bs", "C_ts", "z_bs", "z_ts")]
                + [(n, P) for n in ("A", "D", "dt_bias", "state", "state_out", "lengths", "slots", "y")]
                + [(n, I) for n in ("dtype", "B", "T", "Dm", "N", "G", "softplus", "n_slots")])


def scan(ws=0, ws_bytes=0, err=None, **kw):
    f = sdm.lib().sdm_selective_scan
    f.argtypes = [P, P, SZ, P, P]
    return f(ctypes.byref(ScanArgs(**{**SCAN, **kw})), ws, ws_bytes, err, None)


def test_scan_needs_its_arguments():
    f = sdm.lib().sdm_selective_scan
    f.argtypes = [P, P, SZ, P, P]
    assert f(None, None, 0, None, None) == EINVAL


def test_scan_refusals():
    assert scan(B=0) == EINVAL
    assert scan(T=-1) == EINVAL
    assert scan(N=0) == EINVAL
    assert scan(G=3) == EINVAL                          # 16 channels in 3 groups
    assert scan(dtype=2) == EINVAL
    assert scan(N=129) == EUNSUPPORTED
    assert scan(B=1 << 16, T=1 << 16, n_slots=1 << 16) == EUNSUPPORTED
    assert scan(n_slots=1) == EINVAL
    assert scan(slots=FAKE, n_slots=0) == EINVAL
    assert scan(A=0) == EALIGN
    assert scan(x=0) == EALIGN
    assert scan(z=ODD) == EALIGN
    assert scan(state=0x10002) == EALIGN
    assert scan(dtype=F32, Bm=0x10002) == EALIGN
    assert scan(y=0) == EALIGN
    assert scan(T=0) == OK
    need = sdm.selective_scan_workspace_size(1, 4096, 64, 16)
    long = dict(B=1, T=4096, Dm=64, N=16, n_slots=1)
    assert need > 0
    assert scan(**long) == EALIGN                       # a workspace is needed
    assert scan(ws=FAKE, ws_bytes=need - 1, **long) == ENOSPACE
    assert scan(ws=0x10008, ws_bytes=need, **long) == EALIGN


def test_scan_workspace_sizes():
    size = sdm.selective_scan_workspace_size
    assert size(1, 1, 64, 16) == 0 and size(1, 40, 64, 16) == 0          # too short to cut
    assert size(16, 4096, 8192, 16) == 0                                 # channels enough
    assert size(0, 4096, 64, 16) == 0 and size(1, 4096, 63, 16, 2) == 0  # no such sizes
    assert size(1, 1 << 20, 8192, 128) % 4 == 0


def test_gated_refusals():
    f = sdm.lib().sdm_project_gated
    f.argtypes = [P, P, LL, I, I, I, P, P, P]
    call = lambda x=FAKE, w=FAKE, M=8, D=64, F=64, act=1, h=FAKE: f(x, w, M, D, F, act, h, None, None)  # noqa: E731
    assert call(M=-1) == EINVAL and call(D=0) == EINVAL and call(F=0) == EINVAL
    assert call(act=0) == EINVAL and call(act=3) == EINVAL
    assert call(D=60) == EUNSUPPORTED and call(F=68) == EUNSUPPORTED
    assert call(M=1 << 31) == EUNSUPPORTED
    assert call(x=0x10008) == EALIGN and call(w=None) == EALIGN and call(h=None) == EALIGN
    assert call(M=0, x=None, h=None) == OK
    b = sdm.lib().sdm_project_gated_backward
    b.argtypes = [P, P, P, LL, I, I, I, P, P, P, SZ, P, P]
    need = sdm.project_gated_backward_workspace_size(8, 64, 64)
    grad = lambda dh=FAKE, dx=FAKE, dw=FAKE, ws=FAKE, n=need, D=64: b(  # noqa: E731
        FAKE, FAKE, dh, 8, D, 64, 1, dx, dw, ws, n, None, None)
    assert need >= 8 * 2 * 64 * 2
    assert grad(dh=None) == EALIGN and grad(dx=0x10008) == EALIGN and grad(dw=None) == EALIGN and grad(ws=None) == EALIGN
    assert grad(n=need - 1) == ENOSPACE and grad(D=68) == EUNSUPPORTED
    assert sdm.project_gated_backward_workspace_size(0, 64, 64) == 0


def test_python_calls_refuse_host_tensors():
    x = torch.zeros(2, 3, 8)
    for call in (lambda: sdm.causal_conv(x, torch.zeros(8, 4)),
                 lambda: sdm.causal_conv_step(x[:, 0], torch.zeros(8, 4), state=torch.zeros(2, 3, 8)),
                 lambda: sdm.selective_scan(x, x, torch.zeros(8, 4), x, x),
                 lambda: sdm.project_gated(x, torch.zeros(16, 8)),
                 lambda: sdm.project_gated_backward(x, torch.zeros(16, 8), x)):
        with pytest.raises(TypeError):
            call()


EOVERLAP = -9
FAR = 0x4000000  # past every tensor at FAKE


def test_conv_refuses_an_output_over_another_tensor():
    """A prompt's strips read tokens that other threads' outputs would replace.  Nothing here is launched."""
    apart = dict(w=FAR, bias=FAR + 0x1000, state=FAR + 0x2000, out=FAR + 0x4000)
    long = dict(apart, B=1, T=4096, ts=16, bs=4096 * 16, rows=1)
    nbytes = 4096 * 16 * 2
    assert conv(**long) == EOVERLAP                                          # y is x
    assert conv(**dict(long, y=FAKE + nbytes - 16)) == EOVERLAP              # x's last bytes
    assert conv(**dict(long, y=FAKE - nbytes + 16)) == EOVERLAP              # and its first
    assert conv(**dict(long, T=9, bs=9 * 16)) == EOVERLAP
    assert conv(**dict(apart, y=FAKE, ts=32, bs=128)) == EOVERLAP            # a slice's rows, not where y's are
    assert conv(**dict(apart, T=1, y=FAKE, bs=32)) == EOVERLAP
    for name in ("w", "bias", "state", "out"):
        assert conv(**dict(long, y=apart[name])) == EOVERLAP, name
    assert conv(**dict(long, y=FAR + 0x8000, lengths=FAR + 0x8000)) == EOVERLAP
    assert conv(**dict(long, y=FAR + 0x8000, slots=FAR + 0x8004)) == EOVERLAP


def test_new_states_over_what_the_call_reads_are_refused():
    """One sequence's new state would replace what another still reads.  Nothing here is launched."""
    apart = dict(w=FAR, bias=FAR + 0x1000, y=FAR + 0x8000)
    row = 3 * 16 * 2                                     # a sequence's state of the convolution, in bytes
    assert conv(**apart, state=FAR + 0x2000, out=FAR + 0x2000 + row) == EOVERLAP
    assert conv(**apart, state=FAR + 0x2000 + row, out=FAR + 0x2000) == EOVERLAP
    for over in (FAKE, FAR, FAR + 0x1000):
        assert conv(**apart, state=FAR + 0x2000, out=over) == EOVERLAP, hex(over)
    assert conv(**apart, state=FAR + 0x2000, out=FAR + 0x4000, lengths=FAR + 0x4000) == EOVERLAP
    assert conv(T=0, **apart, state=FAR + 0x2000, out=FAR + 0x2000 + row) == EOVERLAP
    apart = dict(A=FAR, D=FAR + 0x1000, dt_bias=FAR + 0x1800, y=FAR + 0x8000)
    row = 16 * 8 * 4
    for T in (1, 4):
        assert scan(**apart, T=T, state=FAR + 0x2000, state_out=FAR + 0x2000 + row) == EOVERLAP
        assert scan(**apart, T=T, state=FAR + 0x2000 + row, state_out=FAR + 0x2000) == EOVERLAP
        for over in (FAKE, FAR, FAR + 0x1000, FAR + 0x1800):
            assert scan(**apart, T=T, state=FAR + 0x4000, state_out=over) == EOVERLAP, hex(over)
        assert scan(**apart, T=T, state=0, state_out=FAR + 0x2000, slots=FAR + 0x2000) == EOVERLAP


def test_scan_refuses_outputs_over_another_tensor():
    """y may be x, dt or z, but not begin elsewhere in them, nor lie over what every block reads.  Nothing here is
    launched."""
    apart = dict(x=FAR, dt=FAR + 0x10000, z=FAR + 0x20000, Bm=FAR + 0x30000, Cm=FAR + 0x40000, A=FAR + 0x50000,
                 D=FAR + 0x60000, dt_bias=FAR + 0x70000, state=FAR + 0x80000, state_out=FAR + 0x90000,
                 lengths=FAR + 0xA0000, slots=FAR + 0xB0000)
    for T in (1, 4):
        for name in ("Bm", "Cm", "A", "D", "dt_bias", "state", "state_out", "lengths", "slots"):
            assert scan(**apart, T=T, y=apart[name]) == EOVERLAP, name
        for name in ("x", "dt", "z"):
            assert scan(**apart, T=T, y=apart[name] + 16) == EOVERLAP, name
            assert scan(**{**apart, name + "_bs": 16 * T + 16}, T=T, y=apart[name]) == EOVERLAP, name
    assert scan(**apart, z_ts=32, z_bs=128, y=apart["z"]) == EOVERLAP        # half of a wider projection
    need = sdm.selective_scan_workspace_size(1, 4096, 64, 16)
    big = {n: FAR + (i << 24) for i, n in enumerate(apart)}
    long = dict(big, B=1, T=4096, Dm=64, N=16, n_slots=1, y=FAR + (20 << 24), ws_bytes=need, x_ts=64, dt_ts=64, z_ts=64)
    for name in (*big, "y"):
        assert scan(ws=long[name], **long) == EOVERLAP, name


def test_gated_refuses_outputs_over_another_tensor():
    """Tiles of x and w are read while others' outputs are written.  Nothing here is launched."""
    f = sdm.lib().sdm_project_gated
    f.argtypes = [P, P, LL, I, I, I, P, P, P]
    for M in (4, 40):                                    # few tokens, and tiles
        n = M * 64 * 2
        for h in (FAKE, FAKE + n - 16, FAKE - n + 16, FAR, FAR + 128 * 64 * 2 - 16):
            assert f(FAKE, FAR, M, 64, 64, 1, h, None, None) == EOVERLAP, (M, hex(h))
    b = sdm.lib().sdm_project_gated_backward
    b.argtypes = [P, P, P, LL, I, I, I, P, P, P, SZ, P, P]
    need = sdm.project_gated_backward_workspace_size(40, 64, 64)
    at = dict(x=FAR, w=FAR + (1 << 20), dh=FAR + (2 << 20), dx=FAR + (3 << 20), dw=FAR + (4 << 20), ws=FAR + (5 << 20))

    def grad(**kw):
        a = {**at, **kw}
        return b(a["x"], a["w"], a["dh"], 40, 64, 64, 1, a["dx"], a["dw"], a["ws"], need, None, None)

    for out, over in (("dx", ("x", "w", "dw", "ws")), ("dw", ("x", "w", "dx", "ws")), ("ws", ("x", "w", "dh", "dx", "dw"))):
        for name in over:
            assert grad(**{out: at[name]}) == EOVERLAP, (out, name)
            assert grad(**{out: at[name] + 16}) == EOVERLAP, (out, name)
    assert b(None, FAR, None, 0, 64, 64, 1, None, FAR, None, 0, None, None) == EOVERLAP


def test_prompts_whose_token_indexes_would_wrap_are_refused():
    """The last strip, chunk or tile of a prompt just under 2^31 tokens ends past 2^31.  Nothing here is launched."""
    for T in (0x7FFFFFFF, 0x7FFFFFFF - 64):
        assert conv(B=1, T=T, D=1, rows=1) == EUNSUPPORTED
    for T in (0x7FFFFFFF, 0x7FFFFFFF - 20):
        for Dm in (1, 1 << 20):                          # cut into many chunks, and whole
            assert scan(B=1, T=T, Dm=Dm, n_slots=1) == EUNSUPPORTED
    assert sdm.selective_scan_workspace_size(1, 0x7FFFFFFF, 1, 16) > 0
