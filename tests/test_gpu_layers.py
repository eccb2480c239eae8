"""The short causal convolution and the selective state space scan against their 64-bit definitions
(layers_ref.py, which derives the tolerances from the arithmetic).

Inputs are exact in their type, so the reference sees the kernel's own inputs."""
import numpy as np
import pytest
import torch

import layers_ref as ref
import sparse_state_linear_sdm_gb300 as sdm

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _check(got, want, bound, dtype, label):
    g = _host(got)
    tol = bound + ref.ROUND[dtype] * (np.abs(want) + bound) + 1e-37
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (f"{label}: {int(bad.sum())} of {bad.size} outside, worst "
                           f"{float(np.nanmax(np.abs(g - want) / tol)):.2f} of the tolerance")


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *shape: torch.randn(shape, generator=g, device="cuda")


def _slots(nb, pool, seed):
    if not pool:
        return None
    s = torch.from_numpy(np.random.RandomState(seed).permutation(pool)[:nb].astype(np.int32))
    if nb > 2:
        s[1] = -1
    return s.cuda()


# ---- convolution ----

CONV = [
    # dtype, B, T, D, K, act, columns before x in its rows, columns after, state, lengths, pool
    ("bf16", 2, 37, 64, 4, "silu", 0, 64, True, None, 0),
    ("bf16", 1, 1, 8, 2, "none", 0, 0, True, None, 0),
    ("bf16", 3, 130, 24, 8, "silu", 8, 0, True, (130, 5, 0), 0),      # lengths under the window, and zero
    ("bf16", 2, 33, 31, 4, "silu", 0, 0, False, None, 0),             # D not a multiple of a piece
    ("bf16", 2, 19, 40, 3, "silu", 3, 2, True, (19, 1), 0),           # rows that start off 16 bytes
    ("f32", 3, 65, 20, 5, "none", 0, 4, True, (64, 65, 2), 0),
    ("f32", 2, 9, 7, 6, "silu", 1, 0, True, None, 0),
    ("f32", 4, 40, 16, 4, "silu", 0, 0, True, (40, 3, 0, 17), 9),     # states in a pool, one padding row
    ("bf16", 5, 1, 96, 4, "silu", 0, 96, True, None, 11),             # a decode token
    ("bf16", 2, 1030, 256, 7, "silu", 0, 0, True, None, 0),
    ("f32", 1, 3, 4, 8, "none", 0, 0, True, None, 0),                 # fewer tokens than the window
]


def _conv_case(c, seed=3):
    dtype, B, T, D, K, act, before, after, state, lengths, pool = c
    rn, ty = _gen(seed), TYPES[dtype]
    x = rn(B, T, before + D + after).to(ty)[..., before:before + D]
    w, bias = (rn(D, K) * 0.5).to(ty), rn(D).to(ty)
    slots = _slots(B, pool, seed)
    st = rn(pool or B, K - 1, D).to(ty) if state else None
    ln = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return x, w, bias, st, act, ln, slots


@pytest.mark.parametrize("c", CONV, ids=[f"{c[0]}-{c[1]}x{c[2]}x{c[3]}-K{c[4]}" for c in CONV])
def test_conv_against_its_definition(c):
    x, w, bias, st, act, ln, slots = _conv_case(c)
    want, wstate, bound = ref.conv(_host(x), _host(w), _host(bias), _host(st), act, _host(ln), _host(slots))
    out_state = None if st is None else torch.zeros_like(st)
    y, written = sdm.causal_conv(x, w, bias, state=st, state_out=out_state, activation=act, lengths=ln, slots=slots)
    _check(y, want, bound, c[0], "y")
    if st is None:
        assert written is None
        return
    assert written is out_state
    live = np.arange(st.shape[0]) if slots is None else np.array([s for s in _host(slots).astype(int) if s >= 0])
    assert np.array_equal(_host(out_state)[live], wstate[live])  # inputs are only moved
    rest = np.setdiff1d(np.arange(st.shape[0]), live)
    assert not _host(out_state)[rest].any()                      # other slots are not touched
    inplace = st.clone()
    y2, same = sdm.causal_conv(x, w, bias, state=inplace, activation=act, lengths=ln, slots=slots)
    assert same is inplace and torch.equal(y2, y)
    assert np.array_equal(_host(inplace), wstate)


@pytest.mark.parametrize("dtype,w_dtype", [("bf16", "f32"), ("f32", "bf16")])
def test_conv_weights_of_another_type_and_no_bias(dtype, w_dtype):
    rn = _gen(8)
    x, w = rn(2, 21, 32).to(TYPES[dtype]), rn(32, 4).to(TYPES[w_dtype])
    y, none = sdm.causal_conv(x, w)
    want, _, bound = ref.conv(_host(x), _host(w), np.zeros(32), None, "silu")
    assert none is None
    _check(y, want, bound, dtype, "y")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_conv_in_pieces_and_token_by_token_is_one_call(dtype):
    rn, ty = _gen(4), TYPES[dtype]
    B, T, D, K = 3, 23, 48, 4
    x, w, bias, st = rn(B, T, D).to(ty), rn(D, K).to(ty), rn(D).to(ty), rn(B, K - 1, D).to(ty)
    whole, end = sdm.causal_conv(x, w, bias, state=st, state_out=torch.empty_like(st))
    carried, parts = st.clone(), []
    for t0, t1 in ((0, 1), (1, 3), (3, 14), (14, 14), (14, 20)):
        parts.append(sdm.causal_conv(x[:, t0:t1], w, bias, state=carried)[0])
    for t in range(20, T):
        parts.append(sdm.causal_conv_step(x[:, t], w, bias, state=carried)[0].unsqueeze(1))
    assert torch.equal(torch.cat(parts, 1), whole)
    assert torch.equal(carried, end)


def test_conv_reads_nothing_past_a_length_or_of_a_padding_row():
    rn = _gen(5)
    x, w, bias = rn(3, 40, 16), rn(16, 4), rn(16)
    st = rn(4, 3, 16)
    ln = torch.tensor([7, 40, 0], dtype=torch.int32, device="cuda")
    slots = torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    clean = sdm.causal_conv(x, w, bias, state=st, state_out=torch.zeros_like(st), lengths=ln, slots=slots)
    x[0, 7:], x[1], x[2] = float("nan"), float("inf"), float("nan")
    st[1], st[3] = float("nan"), float("nan")
    dirty = sdm.causal_conv(x, w, bias, state=st, state_out=torch.zeros_like(st), lengths=ln, slots=slots)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])
    assert not dirty[0][0, 7:].any() and not dirty[0][1:].any()


def test_lengths_outside_the_prompt_are_clamped():
    rn = _gen(6)
    x, w, bias = rn(2, 9, 8), rn(8, 3), rn(8)
    ln = torch.tensor([-4, 1000], dtype=torch.int32, device="cuda")
    y, _ = sdm.causal_conv(x, w, bias, lengths=ln)
    assert not y[0].any() and torch.equal(y[1:], sdm.causal_conv(x[1:], w, bias)[0])


# ---- scan ----

SCAN = [
    # dtype, B, T, Dm, N, G, gate, skip, bias, softplus, lengths, pool, columns before x
    ("bf16", 2, 37, 64, 16, 1, True, True, True, True, None, 0, 0),
    ("f32", 1, 2, 8, 1, 1, False, False, False, False, None, 0, 0),
    ("f32", 2, 50, 30, 5, 2, True, True, True, True, (50, 13), 0, 1),     # odd sizes, rows off 16 bytes
    ("bf16", 3, 33, 129, 16, 1, False, True, True, True, (0, 33, 16), 0, 0),
    ("bf16", 2, 19, 96, 8, 3, True, True, True, True, None, 0, 0),
    ("f32", 2, 41, 24, 32, 1, True, True, True, True, None, 0, 0),
    ("bf16", 1, 40, 40, 64, 2, True, False, True, True, None, 0, 0),
    ("f32", 1, 35, 17, 128, 1, True, True, True, True, None, 0, 0),
    ("bf16", 1, 35, 24, 100, 1, True, True, True, True, None, 0, 0),
    ("f32", 4, 21, 16, 12, 1, True, True, True, True, (21, 5, 0, 20), 7, 0),
    ("f32", 1, 700, 16, 16, 1, True, True, True, True, None, 0, 0),       # long enough to be cut in chunks
    ("bf16", 2, 530, 24, 7, 1, False, True, True, True, (530, 129), 5, 0),
    ("f32", 3, 400, 8, 4, 1, True, True, True, True, (0, 127, 400), 0, 0),
    ("bf16", 6, 1, 96, 16, 1, True, True, True, True, None, 9, 0),        # one decode token
    ("f32", 3, 1, 10, 5, 2, True, True, True, False, None, 0, 1),
    ("f32", 2, 1, 12, 128, 1, False, False, False, True, None, 0, 0),
    ("bf16", 3, 1, 33, 100, 1, True, True, True, True, (1, 0, 1), 0, 0),
]


def _scan_case(c, seed=11):
    dtype, B, T, Dm, N, G, gate, skip, bias, softplus, lengths, pool, before = c
    rn, ty = _gen(seed), TYPES[dtype]
    k = dict(x=rn(B, T, before + Dm).to(ty)[..., before:], dt=(rn(B, T, Dm) * 0.5).to(ty))
    wide = rn(B, T, 3 + 2 * G * N).to(ty)
    k["B"] = wide[..., 3:3 + G * N].unflatten(-1, (G, N))
    k["C"] = wide[..., 3 + G * N:].unflatten(-1, (G, N))
    k["A"] = -torch.exp(rn(Dm, N)) if softplus else -0.5 - 0.1 * rn(Dm, N).abs()
    if not softplus:
        k["dt"] = k["dt"].abs()
    k["D"] = rn(Dm) if skip else None
    k["z"] = rn(B, T, before + Dm).to(ty)[..., before:] if gate else None
    k["dt_bias"] = rn(Dm) - 1.0 if bias else None
    if bias and not softplus:
        k["dt_bias"] = k["dt_bias"].abs()
    k["state"] = rn(pool or B, Dm, N)
    k["dt_softplus"] = softplus
    k["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    k["slots"] = _slots(B, pool, seed)
    return k


def _scan_ref(k):
    return ref.scan(*(_host(k[n]) for n in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "state")),
                    k["dt_softplus"], _host(k["lengths"]), _host(k["slots"]))


@pytest.mark.parametrize("c", SCAN, ids=[f"{c[0]}-{c[1]}x{c[2]}x{c[3]}-N{c[4]}-G{c[5]}" for c in SCAN])
def test_scan_against_its_definition(c):
    k = _scan_case(c)
    want, wstate, ey, es = _scan_ref(k)
    out_state = torch.zeros_like(k["state"])
    y, written = sdm.selective_scan(**k, state_out=out_state)
    assert written is out_state
    _check(y, want, ey, c[0], "y")
    slots = k["slots"]
    live = np.arange(k["state"].shape[0]) if slots is None else np.array([s for s in _host(slots).astype(int) if s >= 0])
    _check(out_state[torch.from_numpy(live).cuda()], wstate[live], es[live], "f32", "state")
    rest = np.setdiff1d(np.arange(k["state"].shape[0]), live)
    assert not _host(out_state)[rest].any()
    inplace = k["state"].clone()
    y2, same = sdm.selective_scan(**{**k, "state": inplace})
    assert same is inplace and torch.equal(y2, y)
    at = torch.from_numpy(live).cuda()
    assert torch.equal(inplace[at], out_state[at])
    assert torch.equal(inplace[torch.from_numpy(rest).cuda()], k["state"][torch.from_numpy(rest).cuda()])


def test_scan_without_a_state_starts_from_zero():
    k = _scan_case(SCAN[0])
    zero = {**k, "state": torch.zeros_like(k["state"])}
    a, end = sdm.selective_scan(**zero, state_out=torch.empty_like(k["state"]))
    b, none = sdm.selective_scan(**{**k, "state": None})
    assert none is None and torch.equal(a, b)
    c, kept = sdm.selective_scan(**{**k, "state": None}, state_out=torch.empty_like(k["state"]))
    assert torch.equal(c, a) and torch.equal(kept, end)


def _cut(k, t0, t1, state):
    part = {n: (v[:, t0:t1] if n in ("x", "dt", "B", "C", "z") and v is not None else v) for n, v in k.items()}
    part["state"] = state
    return part


@pytest.mark.parametrize("c", [SCAN[0], SCAN[4], SCAN[5]], ids=["N16", "N8-G3", "N32"])
def test_scan_in_pieces_continues_exactly(c):
    k = _scan_case(c)
    T = k["x"].shape[1]
    whole, end = sdm.selective_scan(**k, state_out=torch.empty_like(k["state"]))
    st, parts = k["state"].clone(), []
    for t0, t1 in ((0, 2), (2, T // 2), (T // 2, T // 2), (T // 2, T)):
        parts.append(sdm.selective_scan(**_cut(k, t0, t1, st))[0])
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(st, end)


@pytest.mark.parametrize("c", [SCAN[0], SCAN[2], SCAN[7]], ids=["bf16", "f32-G2", "N128"])
def test_prompt_then_tokens_is_the_longer_prompt(c):
    k = {**_scan_case(c), "lengths": None}
    T = k["x"].shape[1]
    want, wstate, ey, es = _scan_ref(k)
    st = k["state"].clone()
    sdm.selective_scan(**_cut(k, 0, T - 4, st))
    for t in range(T - 4, T):
        one = {n: (v[:, t] if n in ("x", "dt", "B", "C", "z") and v is not None else v) for n, v in k.items()}
        one.pop("lengths")
        one["state"] = st
        y, _ = sdm.selective_step(**one)
        _check(y, want[:, t], ey[:, t], c[0], f"token {t}")
    _check(st, wstate, es, "f32", "state")


def test_scan_reads_nothing_past_a_length_or_of_a_padding_row():
    for c in (SCAN[9], SCAN[11]):
        k = _scan_case(c)
        out = lambda: sdm.selective_scan(**k, state_out=torch.zeros_like(k["state"]))  # noqa: E731
        clean = out()
        ln, slots = k["lengths"].tolist(), k["slots"].tolist()
        for b, n in enumerate(ln):
            n = 0 if slots[b] < 0 else n
            for name in ("x", "dt", "B", "C", "z"):
                if k[name] is not None:
                    k[name][b, n:] = float("nan")
        free = [s for s in range(k["state"].shape[0]) if s not in slots]
        k["state"][free] = float("nan")
        dirty = out()
        assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


def test_scan_decays_that_vanish_and_steps_of_zero():
    k = _scan_case(SCAN[5])
    k["A"][:, 0], k["A"][:, 1] = -3.0e38, 0.0      # forgotten at once, and never
    k["dt"][0, 3] = -3.0e38                         # softplus 0: the token changes nothing
    k["z"][0, 5] = -200.0                           # a closed gate
    y, st = sdm.selective_scan(**k, state_out=torch.empty_like(k["state"]))
    assert torch.isfinite(st[1]).all() and torch.isfinite(y[1]).all()
    assert torch.isfinite(y[0, :3]).all() and (y[0, 5].abs() < 1e-30).all()


@pytest.mark.parametrize("T", [1, 64, 400])
def test_steps_of_size_zero_keep_the_state_bit_for_bit(T):
    """softplus of a very negative number is 0: a decay of exactly 1, over one token, many, and many in chunks."""
    rn = _gen(17)
    k = dict(x=rn(2, T, 40), dt=torch.full((2, T, 40), -3.0e38, device="cuda"), A=-torch.exp(rn(40, 16)),
             B=rn(2, T, 16), C=rn(2, T, 16), state=rn(2, 40, 16))
    y, st = sdm.selective_scan(**k, state_out=torch.empty_like(k["state"]))
    assert torch.equal(st, k["state"])


def test_slots_outside_the_pool_are_reported_and_skipped():
    k = _scan_case(SCAN[9])
    good = k["slots"].clone()
    good[2] = -1
    bad = k["slots"].clone()
    bad[2] = 7
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = sdm.selective_scan(**{**k, "slots": good}, state_out=torch.zeros_like(k["state"]), dev_err=err)
    assert err.item() == 0
    got = sdm.selective_scan(**{**k, "slots": bad}, state_out=torch.zeros_like(k["state"]), dev_err=err)
    assert err.item() == sdm.SDM_DEV_INDEX_RANGE
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    x, w, bias, st, act, ln, slots = _conv_case(CONV[7])
    slots[2] = 9
    err.zero_()
    y, _ = sdm.causal_conv(x, w, bias, state=st, lengths=ln, slots=slots, dev_err=err)
    assert err.item() == sdm.SDM_DEV_INDEX_RANGE and not y[2].any()


def test_layers_on_another_stream():
    k = _scan_case(SCAN[10])
    want, wend = sdm.selective_scan(**k, state_out=torch.empty_like(k["state"]))
    x, w, bias, st, act, ln, slots = _conv_case(CONV[0])
    cwant, _ = sdm.causal_conv(x, w, bias, state=st.clone())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got, end = sdm.selective_scan(**k, state_out=torch.empty_like(k["state"]))
        cgot, _ = sdm.causal_conv(x, w, bias, state=st.clone())
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(end, wend) and torch.equal(cgot, cwant)


def test_layer_calls_refuse_what_they_cannot_run():
    rn = _gen(1)
    x, w = rn(2, 5, 16), rn(16, 4)
    with pytest.raises(TypeError):
        sdm.causal_conv(x.cpu(), w)
    with pytest.raises(TypeError):
        sdm.causal_conv(x.half(), w)
    with pytest.raises(ValueError):
        sdm.causal_conv(x, w, activation="gelu")
    with pytest.raises(ValueError):
        sdm.causal_conv(x.transpose(1, 2), rn(5, 4))          # channels not dense
    with pytest.raises(ValueError):
        sdm.causal_conv(x, rn(15, 4))
    with pytest.raises(ValueError):
        sdm.causal_conv(x, w, state=rn(2, 4, 16))             # K-1 rows are wanted
    with pytest.raises(ValueError):
        sdm.causal_conv(x, w, slots=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(sdm.SDMError):
        sdm.causal_conv(x, rn(16, 9))
    with pytest.raises(sdm.SDMError):
        sdm.causal_conv(x, rn(16, 1))
    with pytest.raises(ValueError):
        sdm.causal_conv_step(x[:, 0], w, state=None)
    k = _scan_case(SCAN[5])
    for name, bad in (("A", k["A"][:, :-1]), ("dt", k["dt"].bfloat16()), ("B", k["B"][:, :-1]), ("D", k["D"].double()),
                      ("state", k["state"][:1]), ("z", k["z"].transpose(1, 2))):
        with pytest.raises((TypeError, ValueError)):
            sdm.selective_scan(**{**k, name: bad})
    big = {**k, "A": rn(24, 129), "B": rn(2, 41, 129), "C": rn(2, 41, 129), "state": None}
    with pytest.raises(sdm.SDMError):
        sdm.selective_scan(**big)
    chunked = _scan_case(SCAN[10])
    with pytest.raises(sdm.SDMError):
        sdm.selective_scan(**chunked, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


# ---- outputs that share memory with inputs ----


def _expects_overlap(call):
    with pytest.raises(ValueError, match="overlaps"):
        call()


def test_conv_output_over_its_input():
    """Up to eight tokens y may be x; a longer prompt's may not, nor may it touch another tensor of the call."""
    for T, dtype in ((1, "bf16"), (4, "f32"), (8, "bf16"), (8, "f32")):
        rn, ty = _gen(21), TYPES[dtype]
        x, w, st = rn(3, T, 512).to(ty), rn(512, 4).to(ty), rn(3, 3, 512).to(ty)
        want, end = sdm.causal_conv(x, w, state=st, state_out=torch.empty_like(st))
        got, kept = sdm.causal_conv(x, w, state=st, state_out=torch.empty_like(st), out=x)
        assert got is x and torch.equal(got, want) and torch.equal(kept, end)
    rn = _gen(22)
    w = rn(512, 4)
    for T in (9, 1000):
        x = rn(1, T, 512)
        kept = x.clone()
        _expects_overlap(lambda: sdm.causal_conv(x, w, out=x))
        assert torch.equal(x, kept)
    both = rn(1, 16, 512)
    _expects_overlap(lambda: sdm.causal_conv(both[:, 5:15], w, out=both[:, :10]))
    _expects_overlap(lambda: sdm.causal_conv(rn(1, 4, 512), w, out=w.view(1, 4, 512)))


def test_conv_output_between_the_rows_of_its_input():
    """Memory that lies between the sequences of a strided x is not x's: y may be there."""
    rn = _gen(23)
    wide = rn(2, 3, 40, 64)
    x, room = wide[:, 0], wide[0, 1:]
    w = rn(64, 4)
    want, _ = sdm.causal_conv(x, w)
    got, _ = sdm.causal_conv(x, w, out=room)
    assert got is room and torch.equal(got, want)


def test_new_states_over_old_ones():
    """The same rows or others, not some of both."""
    rn = _gen(24)
    x, w, pool = rn(2, 6, 32), rn(32, 4), rn(3, 3, 32)
    _expects_overlap(lambda: sdm.causal_conv(x, w, state=pool[:2], state_out=pool[1:]))
    _expects_overlap(lambda: sdm.causal_conv_step(x[:, 0], w, state=pool[1:], state_out=pool[:2]))
    k = _scan_case(SCAN[5])
    pool = rn(3, *k["state"].shape[1:])
    _expects_overlap(lambda: sdm.selective_scan(**{**k, "state": pool[:2]}, state_out=pool[1:]))
    both = rn(4, *k["state"].shape[1:])
    both[:2] = k["state"]
    want, end = sdm.selective_scan(**k, state_out=torch.empty_like(k["state"]))
    got, _ = sdm.selective_scan(**{**k, "state": both[:2]}, state_out=both[2:])     # side by side
    assert torch.equal(got, want) and torch.equal(both[2:], end) and torch.equal(both[:2], k["state"])


def _dense_scan(T, dtype, seed=25):
    rn, ty = _gen(seed), TYPES[dtype]
    return dict(x=rn(2, T, 48).to(ty), dt=rn(2, T, 48).to(ty), z=rn(2, T, 48).to(ty), A=-torch.exp(rn(48, 16)),
                B=rn(2, T, 16).to(ty), C=rn(2, T, 16).to(ty), state=rn(2, 48, 16))


@pytest.mark.parametrize("T", [1, 70, 700])
@pytest.mark.parametrize("name", ["x", "dt", "z"])
def test_scan_output_over_x_dt_or_z(name, T):
    for dtype in ("bf16", "f32"):
        k = _dense_scan(T, dtype)
        want, end = sdm.selective_scan(**k, state_out=torch.empty_like(k["state"]))
        got, st = sdm.selective_scan(**k, state_out=torch.empty_like(k["state"]), out=k[name])
        assert got is k[name] and torch.equal(got, want) and torch.equal(st, end)


def test_scan_output_over_anything_else():
    k = _dense_scan(33, "f32")
    wide = torch.zeros(2, 34, 48, device="cuda")
    _expects_overlap(lambda: sdm.selective_scan(**{**k, "x": wide[:, 1:]}, out=wide.view(-1)[:2 * 33 * 48].view(2, 33, 48)))
    flat = torch.zeros(2 * 33 * 48, device="cuda")
    _expects_overlap(lambda: sdm.selective_scan(**{**k, "B": flat[:2 * 33 * 16].view(2, 33, 16)}, out=flat.view(2, 33, 48)))
    _expects_overlap(lambda: sdm.selective_scan(**{**k, "state": flat[:2 * 48 * 16].view(2, 48, 16)},
                                                out=flat.view(2, 33, 48)))


# ---- prompts cut in chunks ----

CUT = [
    # dtype, B, T, Dm, N, G, gate, skip, bias, softplus, lengths, pool, columns before x
    ("bf16", 1, 1000, 256, 16, 1, True, True, True, True, None, 0, 0),           # one long prompt, 16-byte rows
    ("bf16", 1, 300, 40, 32, 1, True, True, True, True, None, 0, 0),
    ("f32", 1, 300, 40, 32, 2, True, False, True, True, None, 0, 0),
    ("bf16", 2, 330, 48, 64, 1, False, True, True, True, (330, 101), 4, 0),
    ("f32", 2, 300, 33, 64, 1, True, True, False, True, None, 0, 1),
    ("bf16", 1, 290, 24, 100, 1, True, True, True, True, None, 0, 0),
    ("f32", 3, 310, 24, 100, 2, True, True, True, True, (310, 64, 0), 5, 0),
    ("bf16", 1, 350, 32, 128, 2, True, True, True, True, None, 0, 0),
    ("f32", 1, 300, 18, 128, 1, False, False, False, True, None, 0, 0),
    ("bf16", 2, 400, 300, 16, 2, True, True, True, True, None, 0, 0),            # groups of 150: a part of a tile
    ("f32", 2, 300, 402, 12, 3, True, True, True, True, (299, 300), 3, 0),       # of 134
    ("f32", 1, 500, 270, 16, 1, True, True, True, True, None, 0, 2),
    ("bf16", 4, 200, 96, 8, 3, True, True, True, True, (200, 199, 31, 33), 0, 0),
    ("bf16", 1, 450, 64, 16, 1, True, True, True, False, None, 0, 0),            # without softplus
]


@pytest.mark.parametrize("c", CUT, ids=[f"{c[0]}-{c[1]}x{c[2]}x{c[3]}-N{c[4]}-G{c[5]}" for c in CUT])
def test_scan_in_chunks_against_its_definition(c):
    """States that remember hundreds of tokens (rates of about 0.01 in the first half of the channels, steps of about
    0.3), so that a wrong join of the chunks would show, and states that forget within a chunk.  The bound per token
    covers the join's own roundings: a chunk's sum of c <= 64 step sizes is off by at most c U of itself, which moves its
    decay by c U |A| sum, under the 6 U a token for the slow channels and scaled by the decay itself for the others."""
    k = _scan_case(c, seed=31)
    k["A"][:c[3] // 2] *= 0.01
    assert sdm.selective_scan_workspace_size(c[1], c[2], c[3], c[4], c[5]) > 0
    want, wstate, ey, es = _scan_ref(k)
    y, out_state = sdm.selective_scan(**k, state_out=torch.zeros_like(k["state"]))
    _check(y, want, ey, c[0], "y")
    slots = k["slots"]
    live = np.arange(k["state"].shape[0]) if slots is None else np.array([s for s in _host(slots).astype(int) if s >= 0])
    at = torch.from_numpy(live).cuda()
    _check(out_state[at], wstate[live], es[live], "f32", "state")
    inplace = k["state"].clone()
    y2, _ = sdm.selective_scan(**{**k, "state": inplace})
    assert torch.equal(y2, y) and torch.equal(inplace[at], out_state[at])
    rest = np.setdiff1d(np.arange(k["state"].shape[0]), live)
    rest = torch.from_numpy(rest).cuda()
    assert torch.equal(inplace[rest], k["state"][rest]) and not out_state[rest].any()


# ---- errors and empty batches ----


def test_an_output_that_does_not_fit_is_an_out_of_memory_error():
    x = torch.zeros(1 << 20, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(1 << 21, 8, dtype=torch.bfloat16, device="cuda")       # h: 2 TB
    with pytest.raises(torch.OutOfMemoryError):
        sdm.project_gated(x, w)


def test_a_flag_without_a_truth_value_is_its_own_error():
    k = _scan_case(SCAN[5])
    with pytest.raises(ValueError, match="ambiguous"):
        sdm.selective_scan(**{**k, "dt_softplus": np.array([True, False])})


def test_a_batch_of_no_sequences():
    """An empty batch has an empty output and leaves the states alone, as the projections' does."""
    rn = _gen(26)
    x, w = rn(0, 7, 16), rn(16, 4)
    y, st = sdm.causal_conv(x, w)
    assert y.shape == (0, 7, 16) and y.dtype == x.dtype and st is None
    pool, none = rn(3, 3, 16), torch.empty(0, dtype=torch.int32, device="cuda")
    kept = pool.clone()
    y, st = sdm.causal_conv_step(rn(0, 16), w, state=pool, slots=none)
    assert y.shape == (0, 16) and st is pool and torch.equal(pool, kept)
    y, st = sdm.causal_conv(x, w, state=rn(0, 3, 16), lengths=none)
    assert y.shape == (0, 7, 16) and st.shape == (0, 3, 16)
    A, pool = -torch.exp(rn(16, 4)), rn(2, 16, 4)
    y, st = sdm.selective_scan(x, x, A, rn(0, 7, 4), rn(0, 7, 4), state=pool, slots=none)
    assert y.shape == (0, 7, 16) and st is pool
    y, st = sdm.selective_step(rn(0, 16), rn(0, 16), A, rn(0, 1, 4), rn(0, 1, 4), state=rn(0, 16, 4))
    assert y.shape == (0, 16) and st.shape == (0, 16, 4)
    with pytest.raises(ValueError):
        sdm.causal_conv(x, rn(15, 4))
    with pytest.raises(TypeError):
        sdm.selective_scan(x, x, A.double(), rn(0, 7, 4), rn(0, 7, 4))


# ---- growing states ----


@pytest.mark.parametrize("softplus", [True, False])
def test_scan_of_growing_states_in_chunks(softplus):
    """A chunk's whole factor, e^96 and e^1900 here, passes the largest float; the states do not: nothing grows from 0,
    and 1e-30 to 5e11.  The bound is the definition's, which takes the factors token by token."""
    T, Dm, N = 700, 24, 16
    assert sdm.selective_scan_workspace_size(1, T, Dm, N, 1) > 0
    rn = _gen(33)
    dt = torch.full((1, T, Dm), 20.0 if softplus else -20.0, device="cuda")
    A = torch.full((Dm, N), 2.0 if softplus else -2.0, device="cuda")
    B, C = rn(1, T, N), rn(1, T, N)
    y, st = sdm.selective_scan(torch.zeros(1, T, Dm, device="cuda"), dt, A, B, C, dt_softplus=softplus,
                               state=torch.zeros(1, Dm, N, device="cuda"))
    assert not y.any() and not st.any()

    T = 80                                      # two chunks of 48 and 32 tokens
    dt = torch.zeros(1, T, Dm, device="cuda")
    dt[:, :48] = 1.0 if softplus else -1.0
    if softplus:                                # log(e - 1): a step of 1; and one of 0
        dt = torch.where(dt > 0, 0.5413248546129181, -200.0)
    state = torch.full((1, Dm, N), 1e-30, device="cuda")
    k = dict(x=torch.zeros(1, T, Dm, device="cuda"), dt=dt, A=A, B=B[:, :T].contiguous().unsqueeze(2),
             C=C[:, :T].contiguous().unsqueeze(2), D=None, z=None, dt_bias=None, state=state, dt_softplus=softplus,
             lengths=None, slots=None)
    assert sdm.selective_scan_workspace_size(1, T, Dm, N, 1) > 0
    want, wstate, ey, es = _scan_ref(k)
    y, st = sdm.selective_scan(**k, state_out=torch.empty_like(state))
    assert wstate.max() > 1e11
    _check(y, want, ey, "f32", "y")
    _check(st, wstate, es, "f32", "state")
