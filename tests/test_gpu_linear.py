"""Linear attention, prompts and single tokens, against its 64-bit definition (mixer_ref.py, which derives the tolerances
from the arithmetic).  Inputs are exact in their type, so the reference sees the kernel's own inputs."""
import numpy as np
import pytest
import torch

import mixer_ref as ref
import sparse_state_linear_sdm_gb300 as sdm

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _check(got, want, bound, dtype, label):
    g = _host(got)
    assert g.shape == want.shape
    tol = bound + ref.ROUND[dtype] * (np.abs(want) + bound) + 1e-37
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (f"{label}: {int(bad.sum())} of {bad.size} outside, worst "
                           f"{float(np.nanmax(np.abs(g - want) / tol)):.2f} of the tolerance")


def _check_norm(got, want, dtype, label):
    """In norm: an output of bf16 has its own rounding, the state's and the masked products', each even and of at most
    2^-8, so 2^-8 / sqrt(3) in the mean: 2^-8 with all three; twice that here.  fp32 has some hundreds of roundings of
    2^-24 that add up in squares: 2^-20 covers 256 of them in a row."""
    if want.size:
        off = np.linalg.norm(_host(got) - want) / max(np.linalg.norm(want), 1e-30)
        assert off < (2.0 ** -7 if dtype == "bf16" else 2.0 ** -20), f"{label}: {off:.3e} of its norm off"


CASES = [
    # dtype, B, T, H, Hk, dk, dv, decay, state, lengths, pool, layout
    ("f32", 2, 19, 4, 2, 16, 16, "token", True, None, 0, "wide"),
    ("f32", 1, 2, 1, 1, 1, 1, "token", True, None, 0, "dense"),
    ("f32", 3, 33, 6, 3, 50, 37, "head", True, (33, 7, 0), 0, "wide"),      # odd sizes
    ("f32", 2, 40, 2, 1, 128, 128, "token", True, None, 0, "odd"),          # rows off 16 bytes
    ("f32", 2, 31, 2, 2, 256, 250, "none", False, None, 0, "dense"),
    ("f32", 4, 48, 2, 2, 64, 96, "token", True, (48, 16, 17, 1), 7, "wide"),
    ("f32", 1, 500, 2, 2, 64, 64, "token", True, None, 0, "dense"),         # cut into segments
    ("f32", 2, 333, 3, 1, 33, 20, "head", True, (333, 100), 5, "wide"),
    ("f32", 1, 300, 1, 1, 200, 129, "token", True, None, 0, "dense"),
    ("f32", 2, 50, 2, 1, 32, 32, "token", True, None, 0, "expanded"),       # the same keys for every token
    ("bf16", 2, 20, 4, 2, 64, 64, "token", True, None, 0, "wide"),          # too short for chunks
    ("bf16", 2, 31, 2, 2, 50, 40, "token", True, None, 0, "wide"),
    ("bf16", 2, 128, 4, 4, 128, 128, "token", True, None, 0, "wide"),       # one chunk
    ("bf16", 1, 127, 2, 1, 128, 64, "token", True, None, 0, "wide"),
    ("bf16", 1, 129, 2, 1, 64, 128, "head", True, None, 0, "wide"),
    ("bf16", 2, 33, 2, 2, 16, 8, "none", False, None, 0, "dense"),
    ("bf16", 3, 300, 4, 2, 80, 104, "token", True, (300, 131, 0), 5, "wide"),
    ("bf16", 4, 257, 2, 2, 64, 64, "token", True, (256, 257, 1, 129), 0, "wide"),
    ("bf16", 1, 1100, 2, 2, 128, 128, "token", True, None, 0, "wide"),      # cut into segments of chunks
    ("bf16", 2, 900, 1, 1, 128, 250, "token", True, (900, 300), 0, "wide"), # two column tiles, and no multiple of 8
    ("bf16", 1, 400, 2, 2, 128, 256, "head", True, None, 0, "wide"),
    ("bf16", 2, 150, 4, 2, 50, 37, "token", True, (150, 33), 0, "wide"),    # copied to rows of 16 bytes
    ("bf16", 1, 700, 2, 1, 100, 36, "token", True, None, 3, "wide"),
    ("bf16", 2, 140, 2, 2, 64, 64, "token", True, None, 0, "odd"),          # rows off 16 bytes: token by token
    ("bf16", 2, 140, 2, 2, 60, 64, "token", True, None, 0, "odd"),
    ("bf16", 2, 140, 2, 2, 64, 64, "token", True, None, 0, "expanded"),
    ("bf16", 1, 140, 2, 2, 192, 64, "token", True, None, 0, "wide"),        # too many rows for the tiles
    ("bf16", 5, 1, 4, 2, 64, 64, "token", True, None, 9, "wide"),           # one token
    ("f32", 3, 1, 2, 1, 50, 37, "head", True, None, 0, "odd"),
    ("bf16", 3, 1, 2, 2, 256, 256, "none", True, (1, 0, 1), 0, "wide"),
    ("f32", 2, 1, 1, 1, 128, 33, "token", False, None, 0, "dense"),
]
IDS = [f"{c[0]}-{c[1]}x{c[2]}-H{c[3]}.{c[4]}-{c[5]}x{c[6]}-{c[11]}" for c in CASES]


def _case(c, seed=3):
    dtype, B, T, H, Hk, dk, dv, decay, state, lengths, pool, layout = c
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rn, ty = (lambda *s: torch.randn(s, generator=g, device="cuda")), TYPES[dtype]
    n = 2 * Hk * dk + H * dv
    first = 1 if layout == "odd" else 0
    wide = rn(B, T, first + n + (2 if layout == "odd" else 0)).to(ty)[..., first:]
    q, k, v = (t.unflatten(-1, (h, d)) for t, h, d in
               ((wide[..., :Hk * dk], Hk, dk), (wide[..., Hk * dk:2 * Hk * dk], Hk, dk), (wide[..., 2 * Hk * dk:n], H, dv)))
    if layout == "dense":
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    if layout == "expanded":
        k = k[:, :1].expand(B, T, Hk, dk)
    a = dict(q=q, k=k, v=v)
    rate = torch.exp(torch.rand(H, generator=g, device="cuda") * 6.0 - 6.0)    # 0.0025 .. 1
    a["decay"] = {"none": None, "head": -rate, "token": -rate * torch.exp(rn(B, T, H))}[decay]
    a["state"] = rn(pool or B, H, dk, dv) if state else None
    a["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    slots = None
    if pool:
        s = torch.from_numpy(np.random.RandomState(seed).permutation(pool)[:B].astype(np.int32))
        if B > 2:
            s[1] = -1
        slots = s.cuda()
    a["slots"] = slots
    return a


def _ref(a, scale=None, dtype="bf16"):
    B, T, Hk, dk = a["q"].shape
    H, dv = a["v"].shape[2:]
    g = np.zeros((B, T, H)) if a["decay"] is None else np.broadcast_to(_host(a["decay"]), (B, T, H))
    st = np.zeros((B, H, dk, dv)) if a["state"] is None else _host(a["state"])
    return ref.linear(*(_host(a[n]) for n in ("q", "k", "v")), g, dk ** -0.5 if scale is None else scale, st,
                      _host(a["lengths"]), _host(a["slots"]), chunked=dtype == "bf16")


def _live(a):
    rows = a["state"].shape[0] if a["state"] is not None else a["q"].shape[0]
    live = list(range(rows)) if a["slots"] is None else [s for s in a["slots"].tolist() if s >= 0]
    return live, [s for s in range(rows) if s not in live]


@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_linear_against_its_definition(c):
    a = _case(c)
    want, wstate, eo, es = _ref(a, dtype=c[0])
    rows = wstate.shape[0]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept = torch.full((rows, *wstate.shape[1:]), 7.0, device="cuda")
    o, written = sdm.linear_attention(**a, state_out=kept, dev_err=err)
    assert err.item() == 0 and written is kept and o.dtype == TYPES[c[0]]
    _check(o, want, eo, c[0], "o")
    _check_norm(o, want, c[0], "o")
    live, rest = _live(a)
    _check(kept[live], wstate[live], es[live], "f32", "state")
    _check_norm(kept[live], wstate[live], "f32", "state")
    assert (kept[rest] == 7.0).all()                       # other rows are not touched
    if a["state"] is None:
        o2, none = sdm.linear_attention(**a)
        assert none is None and torch.equal(o2, o)
        return
    inplace = a["state"].clone()
    o2, same = sdm.linear_attention(**{**a, "state": inplace})
    assert same is inplace and torch.equal(o2, o) and torch.equal(inplace[live], kept[live])
    assert torch.equal(inplace[rest], a["state"][rest])


def test_scale_and_decays_of_one_row():
    a = _case(CASES[0])
    want, _, eo, _ = _ref(a, scale=-0.3, dtype="f32")
    run = lambda x, **kw: sdm.linear_attention(**x, **kw, state_out=torch.empty_like(a["state"]))[0]  # noqa: E731
    _check(run(a, scale=-0.3), want, eo, "f32", "o")
    a["decay"] = a["decay"][:1, :1, :].expand(2, 19, 4)      # both strides 0
    row = {**a, "decay": a["decay"][0, 0].contiguous()}
    assert torch.equal(run(a), run(row))


@pytest.mark.parametrize("c", [CASES[0], CASES[6], CASES[18], CASES[21]], ids=["f32", "f32-cut", "tiles-cut", "copied"])
def test_prompt_in_pieces_and_tokens_is_the_longer_prompt(c):
    a = _case(c)
    T = a["q"].shape[1]
    a["lengths"] = None
    want, wstate, eo, es = _ref(a, dtype=c[0])
    st = a["state"].clone()
    cuts = [0, T // 3, T // 3, T // 2, T - 3]
    for t0, t1 in zip(cuts, cuts[1:]):
        part = {n: (v[:, t0:t1] if n in ("q", "k", "v", "decay") else v) for n, v in a.items()}
        o, _ = sdm.linear_attention(**{**part, "state": st})
        _check(o, want[:, t0:t1], eo[:, t0:t1] + ref.H * np.abs(eo[:, t0:t1]), c[0], f"tokens {t0} to {t1}")
    for t in range(T - 3, T):
        o, same = sdm.linear_attention_step(a["q"][:, t], a["k"][:, t], a["v"][:, t], a["decay"][:, t], state=st,
                                            slots=a["slots"])
        assert same is st and o.shape == want[:, t].shape
        _check(o, want[:, t], eo[:, t], c[0], f"token {t}")
    live, _ = _live(a)
    _check(st[live], wstate[live], es[live], "f32", "state")


@pytest.mark.parametrize("c", [CASES[5], CASES[16], CASES[17], CASES[19], CASES[21], CASES[29]],
                         ids=["f32", "tiles", "tiles-64", "columns", "copied", "token"])
def test_nothing_past_a_length_or_of_a_padding_row_is_read(c):
    a = _case(c)
    run = lambda: sdm.linear_attention(**a, state_out=torch.zeros_like(a["state"]))  # noqa: E731
    clean = run()
    slots = a["slots"].tolist() if a["slots"] is not None else list(range(c[1]))
    for b, n in enumerate(a["lengths"].tolist()):
        n = 0 if slots[b] < 0 else n
        for name in ("q", "k", "v", "decay"):
            if a[name] is not None and a[name].dim() > 1:
                a[name][b, n:] = float("nan") if b % 2 else float("inf")
        assert not clean[0][b, n:].any()
    a["state"][_live(a)[1]] = float("nan")
    dirty = run()
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


def test_rows_of_a_padding_sequence_are_not_read():
    for c in (CASES[16], CASES[5]):
        a = _case(c)
        clean = sdm.linear_attention(**a, state_out=torch.zeros_like(a["state"]))
        for name in ("q", "k", "v", "decay"):
            a[name][1] = float("nan")
        dirty = sdm.linear_attention(**a, state_out=torch.zeros_like(a["state"]))
        assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1]) and not dirty[0][1].any()


@pytest.mark.parametrize("c", [CASES[0], CASES[6], CASES[12], CASES[18], CASES[21], CASES[27]],
                         ids=["f32", "f32-cut", "tiles", "tiles-cut", "copied", "token"])
def test_decays_that_forget_everything_or_nothing(c):
    """-inf and very strong decays leave nothing of what was before, 0 everything; rows after them are the definition's."""
    a = _case(c)
    T = a["q"].shape[1]
    a["decay"][:, T // 2:] *= 0.0
    a["decay"][0, T // 3, 0] = float("-inf")
    a["decay"][0, 0, 1] = -3.0e38
    a["decay"][-1, T - 1, 0] = -60.0
    a["decay"][-1, :, -1] = -9.0                            # forgets within a token or two, all along
    want, wstate, eo, es = _ref(a, dtype=c[0])
    o, st = sdm.linear_attention(**a, state_out=torch.zeros_like(a["state"]))
    _check(o, want, eo, c[0], "o")
    live, _ = _live(a)
    _check(st[live], wstate[live], es[live], "f32", "state")


@pytest.mark.parametrize("c", [CASES[6], CASES[18]], ids=["f32-cut", "tiles-cut"])
def test_states_that_grow(c):
    """A segment's whole factor passes the largest float; nothing grows from 0, and 1e-30 to 1e10."""
    a = _case(c)
    T = a["q"].shape[1]
    a["decay"] = torch.full_like(a["decay"], 100.0 / T * 1.5)
    a["k"] = torch.zeros_like(a["k"])
    a["state"].zero_()
    o, st = sdm.linear_attention(**a, state_out=torch.empty_like(a["state"]))
    assert not o.any() and not st.any()
    a["state"].fill_(1e-30)
    a["decay"] = torch.full_like(a["decay"], 92.0 / T)
    want, wstate, eo, es = _ref(a, dtype=c[0])
    o, st = sdm.linear_attention(**a, state_out=torch.empty_like(a["state"]))
    assert wstate.max() > 1e9
    _check(o, want, eo, c[0], "o")
    _check(st, wstate, es, "f32", "state")


@pytest.mark.parametrize("name", ["q", "k", "v", "decay"])
def test_a_nan_stays_where_the_definition_has_it(name):
    """A token's own output for q; everything of the head from there on for k and decay; of the column for v, where the
    tensor cores (a chunk's products with v are taken whole) have it for the chunk's other tokens too."""
    for c in (CASES[0], CASES[6], CASES[12], CASES[18], CASES[21]):
        a = _case(c)
        a["lengths"] = None
        T, at = a["q"].shape[1], a["q"].shape[1] // 2 + 3
        where = (0, at, 0) if name == "decay" else (0, at, 0, 3)
        a[name] = a[name].clone()
        a[name][where] = float("nan")
        share = c[3] // c[4] if name in ("q", "k") else 1
        o, st = sdm.linear_attention(**a, state_out=torch.empty_like(a["state"]))
        bad = torch.isnan(o)
        if name == "q":
            assert bad[0, at, :share].all() and not torch.isnan(st).any()
            bad[0, at, :share] = False
        elif name == "v":
            assert bad[0, at:, 0, 3].all() and torch.isnan(st[0, 0, :, 3]).all()
            first = at // 128 * 128 if c[0] == "bf16" else at
            assert not bad[0, :first].any()
            bad[0, first:, 0, 3] = False
        else:
            assert bad[0, at:, :share].all() and torch.isnan(st[0, :share]).any()
            bad[0, at:, :share] = False
        assert not bad.any()


def test_slots_outside_the_pool_are_reported_and_skipped():
    for c in (CASES[5], CASES[16], CASES[27]):
        a = _case(c)
        good, bad = a["slots"].clone(), a["slots"].clone()
        good[2], bad[2] = -1, a["state"].shape[0]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        want = sdm.linear_attention(**{**a, "slots": good}, state_out=torch.zeros_like(a["state"]), dev_err=err)
        assert err.item() == 0
        got = sdm.linear_attention(**{**a, "slots": bad}, state_out=torch.zeros_like(a["state"]), dev_err=err)
        assert err.item() == sdm.SDM_DEV_INDEX_RANGE
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_no_sequences_and_no_tokens():
    for dtype in TYPES.values():
        z = lambda *s: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        o, st = sdm.linear_attention(z(0, 7, 2, 16), z(0, 7, 2, 16), z(0, 7, 4, 8))
        assert o.shape == (0, 7, 4, 8) and st is None
        pool = torch.randn(3, 4, 16, 8, device="cuda")
        kept = pool.clone()
        o, st = sdm.linear_attention_step(z(0, 2, 16), z(0, 2, 16), z(0, 4, 8), state=pool,
                                          slots=torch.empty(0, dtype=torch.int32, device="cuda"))
        assert o.shape == (0, 4, 8) and st is pool and torch.equal(pool, kept)
        o, st = sdm.linear_attention(z(3, 0, 2, 16), z(3, 0, 2, 16), z(3, 0, 4, 8), state=pool,
                                     state_out=torch.empty_like(pool))
        assert o.shape == (3, 0, 4, 8) and torch.equal(st, pool)


def test_other_streams_and_workspaces():
    for c in (CASES[6], CASES[18], CASES[22]):
        a = _case(c)
        want, end = sdm.linear_attention(**a, state_out=torch.zeros_like(a["state"]))
        torch.cuda.synchronize()
        B, T, Hk, dk = a["q"].shape
        need = sdm.linear_attention_workspace_size(TYPES[c[0]], B, T, c[3], Hk, dk, c[6])
        assert need > 0
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            got, st = sdm.linear_attention(**a, state_out=torch.zeros_like(a["state"]), workspace=ws)
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(st, end)
        with pytest.raises(sdm.SDMError):
            sdm.linear_attention(**a, state_out=torch.zeros_like(a["state"]), workspace=ws[:need - 16])


def test_calls_replay_from_graphs_that_share_a_workspace():
    a, b = _case(CASES[18]), _case(CASES[22])
    size = max(sdm.linear_attention_workspace_size(torch.bfloat16, x["q"].shape[0], x["q"].shape[1], x["v"].shape[2],
                                                   x["q"].shape[2], x["q"].shape[3], x["v"].shape[3]) for x in (a, b))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    calls = [lambda x=x, s=torch.zeros_like(x["state"]): sdm.linear_attention(**x, state_out=s, workspace=ws)
             for x in (a, b)]
    want = [[t.clone() for t in f()] for f in calls]
    torch.cuda.synchronize()
    graphs, got = [], []
    for f in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(f())
        graphs.append(g)
    for i in (0, 1, 1, 0):
        for t in got[i]:
            t.fill_(3.0)
        graphs[i].replay()
        torch.cuda.synchronize()
        live = _live((a, b)[i])[0]
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1][live], want[i][1][live])


def test_refusals():
    a = _case(CASES[0])
    for name, bad in (("k", a["k"][:, :, :1]), ("v", a["v"].bfloat16()), ("q", a["q"].half()), ("q", a["q"].cpu()),
                      ("decay", a["decay"].double()), ("decay", a["decay"][:, :, :2]), ("state", a["state"][:1]),
                      ("state", a["state"].bfloat16()), ("v", a["v"].transpose(2, 3)),
                      ("lengths", torch.zeros(3, dtype=torch.int32, device="cuda")),
                      ("slots", torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            sdm.linear_attention(**{**a, name: bad})
    with pytest.raises(ValueError):
        sdm.linear_attention(**{**a, "state": None, "slots": torch.zeros(2, dtype=torch.int32, device="cuda")})
    with pytest.raises(ValueError):
        sdm.linear_attention_step(a["q"][:, 0], a["k"][:, 0], a["v"][:, 0], state=None)
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    with pytest.raises(sdm.SDMError):
        sdm.linear_attention(z(1, 2, 3, 8), z(1, 2, 3, 8), z(1, 2, 4, 8))      # 3 heads of keys for 4
    with pytest.raises(sdm.SDMError):
        sdm.linear_attention(z(1, 2, 1, 257), z(1, 2, 1, 257), z(1, 2, 1, 8))
    with pytest.raises(sdm.SDMError):
        sdm.linear_attention(z(1, 2, 1, 8), z(1, 2, 1, 8), z(1, 2, 1, 300))


def test_outputs_over_inputs_are_refused():
    v = torch.randn(2, 40, 4, 16, device="cuda")
    for over in range(3):
        three = [v.clone() for _ in range(3)]
        with pytest.raises(ValueError, match="overlaps"):
            sdm.linear_attention(*three, out=three[over])
    pool = torch.randn(3, 4, 16, 16, device="cuda")
    for T in (1, 40):
        with pytest.raises(ValueError, match="overlaps"):
            sdm.linear_attention(v[:, :T], v[:, :T], v[:, :T], state=pool[:2], state_out=pool[1:])


def test_offsets_past_32_bits():
    """The last tokens of a long prompt whose values pass 2^31 elements are those of the same tokens run alone from
    the state that a strong decay leaves of the ones before: nothing."""
    T, H = 270_000, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    v = torch.randn((1, T, H, 128), generator=g, device="cuda", dtype=torch.bfloat16)
    qk = torch.randn((1, T, 1, 256), generator=g, device="cuda", dtype=torch.bfloat16)
    q, k = qk[..., :128], qk[..., 128:]
    decay = torch.full((H,), -20.0, device="cuda")
    o, st = sdm.linear_attention(q, k, v, decay, state_out=torch.empty(1, H, 128, 128, device="cuda"))
    n = T - 40
    tail, ts = sdm.linear_attention(q[:, n:], k[:, n:], v[:, n:], decay, state_out=torch.empty_like(st))
    assert torch.allclose(o[:, n + 5:].float(), tail[:, 5:].float(), rtol=2.0 ** -6, atol=2.0 ** -6)
    assert torch.allclose(st, ts, rtol=1e-4, atol=1e-5)
    # token by token (keys of an odd address), over the same values
    odd = torch.empty(T * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(1, T, 1, 128).copy_(k)
    o2, st2 = sdm.linear_attention(q, odd, v, decay, state_out=torch.empty_like(st), out=o)
    assert torch.allclose(o2[:, n + 5:].float(), tail[:, 5:].float(), rtol=2.0 ** -6, atol=2.0 ** -6)
    assert torch.allclose(st2, ts, rtol=1e-4, atol=1e-5)


@pytest.mark.parametrize("c", [
    ("bf16", 1, 1500, 2, 1, 100, 36, "token", True, (1400,), 3, "wide"),    # copied rows, cut into segments
    ("bf16", 3, 1290, 2, 2, 64, 128, "token", True, (1290, 1, 700), 0, "wide"),
    ("bf16", 1, 1152, 3, 3, 128, 64, "head", False, None, 0, "dense"),
    ("bf16", 160, 40, 4, 4, 32, 16, "token", True, None, 0, "wide"),        # many small heads: one by one below 64
    ("bf16", 160, 64, 4, 4, 32, 16, "token", True, None, 0, "wide"),        # and a chunk from 64 on
], ids=lambda c: f"{c[1]}x{c[2]}-H{c[3]}-{c[5]}x{c[6]}")
def test_linear_where_its_form_changes(c):
    a = _case(c, seed=11)
    want, wstate, eo, es = _ref(a)
    kept = torch.full(wstate.shape, 7.0, device="cuda")
    o, _ = sdm.linear_attention(**a, state_out=kept)
    live, _ = _live(a)
    _check(o, want, eo, "bf16", "o")
    _check_norm(o, want, "bf16", "o")
    _check(kept[live], wstate[live], es[live], "f32", "state")
    _check_norm(kept[live], wstate[live], "f32", "state")


@pytest.mark.parametrize("dtype, T, dk", [("f32", 20, 64), ("f32", 500, 64), ("bf16", 100, 64), ("bf16", 1500, 128)])
def test_a_sequence_without_tokens_keeps_its_state_bit_for_bit(dtype, T, dk):
    a = _case((dtype, 2, T, 2, 2, dk, 64, "token", True, (T, 0), 0, "wide"))
    kept = torch.empty_like(a["state"])
    o, _ = sdm.linear_attention(**a, state_out=kept)
    assert torch.equal(kept[1], a["state"][1]) and (o[1] == 0).all()


@pytest.mark.parametrize("B,T,H,d", [(1, 16384, 8, 128), (4, 1024, 16, 128), (2, 4096, 16, 64)])
def test_long_prompts_many_times(B, T, H, d):
    """The chunks' warps meet in any order; results and errors do not depend on it."""
    a = _case(("bf16", B, T, H, H, d, d, "token", True, None, 0, "wide"))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, again = torch.empty_like(a["state"]), torch.empty_like(a["state"])
    o, _ = sdm.linear_attention(**a, state_out=kept, dev_err=err)
    for i in range(200):
        o2, _ = sdm.linear_attention(**a, state_out=again, dev_err=err)
        assert torch.equal(o2, o) and torch.equal(again, kept), i
    assert err.item() == 0
