"""The norms with gate, residual and residual scale, and their gradient, against the 64-bit definition (mixer_ref.py, which
derives the tolerances; test_mixer_ref.py holds its gradient to differences)."""
import numpy as np
import pytest
import torch

import mixer_ref as ref
import sparse_state_linear_sdm_gb300 as sdm

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
NAMES = {torch.float32: "f32", torch.bfloat16: "bf16"}


def _host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _check(got, want, bound, label):
    g = _host(got)
    assert g.shape == want.shape, label
    tol = bound + ref.ROUND[NAMES[got.dtype]] * (np.abs(want) + bound) + 1e-37
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (f"{label}: {int(bad.sum())} of {bad.size} outside, worst "
                           f"{float(np.nanmax(np.abs(g - want) / tol)):.2f} of the tolerance")


CASES = [
    # x, residual, weights, M, D, groups, parts: after, gate, scale, residual, weight; layout
    ("bf16", "bf16", "bf16", 5, 64, 1, "agsrw", "dense"),
    ("bf16", "f32", "f32", 7, 256, 1, "agsrw", "wide"),
    ("f32", "f32", "f32", 3, 40, 1, "agsrw", "wide"),
    ("bf16", "bf16", "f32", 9, 100, 1, "rw", "dense"),
    ("bf16", "f32", "bf16", 4, 1537, 1, "agsrw", "wide"),          # an odd width
    ("f32", "f32", "bf16", 2, 777, 1, "rw", "odd"),
    ("bf16", "bf16", "bf16", 1, 1, 1, "agsrw", "dense"),
    ("bf16", "bf16", "f32", 33, 512, 4, "ag", "wide"),             # heads of 128
    ("f32", "f32", "f32", 17, 96, 3, "ag", "dense"),
    ("bf16", "bf16", "bf16", 40, 150, 6, "ag", "wide"),            # heads of 25
    ("bf16", "f32", "f32", 12, 192, 3, "agsr", "dense"),
    ("bf16", "bf16", "bf16", 6, 2048, 1, "w", "dense"),            # a norm alone
    ("f32", "f32", "f32", 6, 30, 1, "w", "odd"),
    ("bf16", "bf16", "f32", 6, 128, 1, "gsr", "dense"),
    ("bf16", "bf16", "f32", 6, 128, 1, "asw", "dense"),
    ("bf16", "f32", "f32", 5, 600, 1, "sr", "wide"),
    ("bf16", "bf16", "bf16", 3, 3000, 1, "agsrw", "dense"),
    ("bf16", "f32", "f32", 3, 4100, 1, "agsrw", "dense"),
    ("f32", "f32", "f32", 2, 8000, 1, "arw", "dense"),
    ("bf16", "bf16", "bf16", 2, 16384, 1, "agsrw", "dense"),
    ("bf16", "f32", "bf16", 2, 16383, 1, "rw", "odd"),
    ("bf16", "bf16", "bf16", 37, 400, 1, "agsrw", "dense"),        # two rows a block, two warps each
    ("bf16", "f32", "f32", 38, 301, 1, "agsrw", "wide"),
    ("f32", "f32", "f32", 11, 1536, 4, "ag", "dense"),             # heads of 384
    ("bf16", "bf16", "bf16", 1300, 64, 1, "agsrw", "dense"),       # more rows than the card holds at once ...
    ("bf16", "f32", "f32", 3000, 1030, 1, "agsrw", "dense"),
    ("bf16", "bf16", "f32", 30000, 24, 2, "ag", "dense"),
    ("f32", "f32", "f32", 2500, 513, 1, "rw", "dense"),
    ("bf16", "bf16", "f32", 700, 8000, 1, "agsrw", "dense"),
    ("bf16", "bf16", "bf16", 900, 2500, 1, "rw", "dense"),
]
IDS = [f"{c[0]}-{c[1]}-{c[2]}-{c[3]}x{c[4]}.{c[5]}-{c[6]}-{c[7]}" for c in CASES]


def _case(c, seed=4):
    x, r, w, M, D, groups, parts, layout = c
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731

    def rows(ty):
        if layout == "dense":
            return rn(M, D).to(TYPES[ty])
        first, more = (1, 1) if layout == "odd" else (8, 16)
        return rn(M, first + D + more).to(TYPES[ty])[:, first:first + D]

    vec = lambda on: (1.0 + 0.2 * rn(D)).to(TYPES[w]) if on in parts else None  # noqa: E731
    a = dict(x=rows(x), residual=rows(r) if "r" in parts else None, weight=vec("w"), after=vec("a"),
             gate=rows(x) if "g" in parts else None, scale=vec("s"), groups=groups)
    return a, rows(x), rows(r if "r" in parts else x)


def _ref(a, eps=1e-6, act="silu"):
    return ref.norm(*(_host(a[n]) for n in ("x", "residual", "weight", "after", "gate", "scale")), a["groups"], eps, act)


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_norm_against_its_definition(c, act):
    if act == "none" and ("g" not in c[6] or c[3] > 100):
        pytest.skip("the same as silu")
    a, _, _ = _case(c)
    wy, wr, ey, er = _ref(a, act=act)
    y, r = sdm.residual_norm(**a, activation=act)
    if a["weight"] is None:
        assert y is None
    else:
        assert y.dtype == a["x"].dtype
        _check(y, wy, ey, "y")
    if set(c[6]) == {"w"}:
        assert r is a["x"]
    else:
        assert r.dtype == (a["x"] if a["residual"] is None else a["residual"]).dtype
        _check(r, wr, er, "r")
    if "a" in c[6] and not set(c[6]) & set("srw"):
        assert torch.equal(sdm.gated_norm(a["x"], a["after"], a["gate"], groups=a["groups"], activation=act), r)


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_norm_gradient_against_its_definition(c, act):
    if act == "none" and ("g" not in c[6] or c[3] > 100):
        pytest.skip("the same as silu")
    a, dy, dr = _case(c)
    r = sdm.residual_norm(**a, activation=act)[1]
    has = {n: a[n] is not None for n in a if n != "groups"}
    args = dict(weight=a["weight"], after=a["after"], gate=a["gate"], scale=a["scale"], residual=has["residual"],
                groups=a["groups"], activation=act)
    got = sdm.residual_norm_backward(a["x"], r, dy if has["weight"] else None, dr, **args)
    got = dict(zip(("dx", "dresidual", "dweight", "dafter", "dgate", "dscale"), got))
    h = [_host(t) for t in (a["x"], r, dy if has["weight"] else None, dr, a["weight"], a["after"], a["gate"], a["scale"])]
    want = ref.norm_grad(*h, a["groups"], 1e-6, act)
    size = ref.norm_grad(*h, a["groups"], 1e-6, act, size=True)
    for name, t in got.items():
        if not has.get(name[1:], name == "dx"):
            assert t is None, name
            continue
        assert t.dtype == {"dx": a["x"], "dgate": a["x"], "dresidual": r}.get(name, next(
            v for v in (a["weight"], a["after"], a["scale"], a["x"]) if v is not None)).dtype
        rows = c[3] if name in ("dweight", "dafter", "dscale") else 0
        _check(t, want[name], (256 + rows) * ref.U * size[name], name)
    if "a" in c[6] and not set(c[6]) & set("srw"):
        dx, dw, dz = sdm.gated_norm_backward(a["x"], a["after"], dr, a["gate"], groups=a["groups"], activation=act)
        assert torch.equal(dx, got["dx"]) and torch.equal(dw, got["dafter"]) and torch.equal(dz, got["dgate"])
    again = sdm.residual_norm_backward(a["x"], r, dy if has["weight"] else None, dr, **args)
    assert all(u is None or torch.equal(u, v) for u, v in zip(again, got.values()))


def test_gradients_that_are_absent_or_broadcast():
    a, dy, dr = _case(CASES[1])
    r = sdm.residual_norm(**a)[1]
    args = dict(weight=a["weight"], after=a["after"], gate=a["gate"], scale=a["scale"])
    zero = sdm.residual_norm_backward(a["x"], r, dy, torch.zeros_like(dr), **args)
    none = sdm.residual_norm_backward(a["x"], r, dy, None, **args)
    assert all(torch.equal(u, v) for u, v in zip(zero, none))
    one = dy[:1].expand_as(dy)                               # a row for all, as a sum's gradient comes
    got = sdm.residual_norm_backward(a["x"], r, one, dr, **args)
    want = sdm.residual_norm_backward(a["x"], r, one.contiguous(), dr, **args)
    assert all(torch.equal(u, v) for u, v in zip(got, want))


def test_one_tensor_for_equal_gradients():
    """Without a block in between, dx and dresidual are the same values: one tensor where their types are the same."""
    a, dy, dr = _case(CASES[3])
    r = sdm.residual_norm(**a)[1]
    g = sdm.residual_norm_backward(a["x"], r, dy, dr, a["weight"])
    assert g[0] is g[1]
    a, dy, dr = _case(("bf16", "f32", "f32", 9, 100, 1, "rw", "dense"))
    r = sdm.residual_norm(**a)[1]
    g = sdm.residual_norm_backward(a["x"], r, dy, dr, a["weight"])
    assert g[0].dtype == torch.bfloat16 and g[1].dtype == torch.float32 and torch.equal(g[0], g[1].bfloat16())
    x = a["x"]
    y, same = sdm.residual_norm(x, weight=a["weight"])       # a norm alone: r is x
    dx = sdm.residual_norm_backward(x, None, dy, None, a["weight"], residual=False)
    with_r = sdm.residual_norm_backward(x, same, dy, None, a["weight"], residual=False)
    assert same is x and torch.equal(dx[0], with_r[0]) and dx[1] is None and torch.equal(dx[2], with_r[2])


def test_rows_of_zeros_large_values_and_no_rows():
    for x_type in TYPES.values():
        x = torch.randn(6, 96, device="cuda").to(x_type)
        x[1], x[2], x[3] = 0.0, 1e18, 1e-18
        w = torch.ones(96, device="cuda")
        y, _ = sdm.residual_norm(x, weight=w, eps=1e-6)
        assert not y[1].any() and torch.isfinite(y).all() and (y[2] - 1).abs().max() < 0.01
        g = sdm.residual_norm_backward(x, None, torch.ones_like(x), None, w, residual=False)
        assert torch.isfinite(g[0]).all() and torch.isfinite(g[2]).all()
        none = x[:0]
        y, r = sdm.residual_norm(none, none, w, after=w, gate=none)
        assert y.shape == (0, 96) and r.shape == (0, 96)
        g = sdm.residual_norm_backward(none, none, none, none, w, after=w, gate=none)
        assert g[0].shape == (0, 96) and not g[2].any() and not g[3].any() and g[2].shape == (96,)


def test_a_row_does_not_reach_another():
    a, dy, dr = _case(("bf16", "f32", "f32", 50, 300, 1, "agsrw", "dense"))
    clean = sdm.residual_norm(**a)
    args = dict(weight=a["weight"], after=a["after"], gate=a["gate"], scale=a["scale"])
    gclean = sdm.residual_norm_backward(a["x"], clean[1], dy, dr, **args)
    a["x"][7], a["gate"][9], a["residual"][20] = float("nan"), float("inf"), float("nan")
    dirty = sdm.residual_norm(**a)
    gdirty = sdm.residual_norm_backward(a["x"], dirty[1], dy, dr, **args)
    rest = [i for i in range(50) if i not in (7, 9, 20)]
    for u, v in zip((*clean, *gclean[:2], gclean[4]), (*dirty, *gdirty[:2], gdirty[4])):
        assert torch.equal(u[rest], v[rest])


def test_the_stream_in_place_and_outputs_over_inputs():
    a, _, _ = _case(("bf16", "f32", "f32", 70, 264, 1, "asrw", "dense"))
    wy, wr = sdm.residual_norm(**a)
    y, r = sdm.residual_norm(**a, residual_out=a["residual"], out=a["x"])
    assert r is a["residual"] and y is a["x"] and torch.equal(y, wy) and torch.equal(r, wr)
    a, _, _ = _case(("f32", "f32", "f32", 6, 64, 1, "asrw", "dense"))
    wide = torch.zeros(7, 64, device="cuda")
    with pytest.raises(ValueError, match="overlaps"):
        sdm.residual_norm(**{**a, "x": wide[1:]}, out=wide[:6])
    with pytest.raises(ValueError, match="overlaps"):
        sdm.residual_norm(**a, out=wide[:6], residual_out=wide[1:])
    flat = torch.zeros(6 * 64, device="cuda")
    with pytest.raises(ValueError, match="overlaps"):
        sdm.residual_norm(**{**a, "weight": flat[:64]}, out=flat.view(6, 64))


def test_norm_on_other_streams_in_graphs_and_of_batches():
    a, dy, dr = _case(("bf16", "f32", "f32", 60, 264, 1, "agsrw", "dense"))
    args = dict(weight=a["weight"], after=a["after"], gate=a["gate"], scale=a["scale"])
    y, r = sdm.residual_norm(**a)
    want = (y, r, *sdm.residual_norm_backward(a["x"], r, dy, dr, **args))
    three = {n: v.view(3, 20, 264) if torch.is_tensor(v) and v.dim() == 2 else v for n, v in a.items()}
    y3, r3 = sdm.residual_norm(**three)
    assert y3.shape == (3, 20, 264) and torch.equal(y3.view(60, 264), y) and torch.equal(r3.view(60, 264), r)
    ws = torch.full((sdm.residual_norm_backward_workspace_size(60, 264),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    def run():
        y, r = sdm.residual_norm(**a)
        return (y, r, *sdm.residual_norm_backward(a["x"], r, dy, dr, **args, workspace=ws))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        for t in got:
            t.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want))


def test_norm_refuses_what_it_cannot_run():
    a, dy, dr = _case(("bf16", "f32", "f32", 6, 64, 1, "agsrw", "dense"))
    x, w = a["x"], a["weight"]
    for kw in (dict(x=x.cpu()), dict(x=x.half()), dict(residual=a["residual"].double()), dict(weight=w[:-1]),
               dict(weight=w.bfloat16()), dict(gate=a["gate"].float()), dict(gate=a["gate"][:3]), dict(groups=3),
               dict(groups=2), dict(activation="gelu"), dict(x=x.t(), residual=None, gate=None),
               dict(residual=a["residual"][:5])):
        with pytest.raises((TypeError, ValueError)):
            sdm.residual_norm(**{**a, **kw})
    f = x.float()
    with pytest.raises(TypeError):
        sdm.residual_norm(f, x, w)                           # a stream narrower than its block
    with pytest.raises(ValueError):
        sdm.residual_norm(x)
    with pytest.raises(ValueError):
        sdm.gated_norm(x, None)
    with pytest.raises(sdm.SDMError):
        sdm.residual_norm(x, weight=w, eps=-1.0)
    with pytest.raises(sdm.SDMError):
        sdm.residual_norm(torch.zeros(2, 16392, device="cuda"), weight=torch.zeros(16392, device="cuda"))
    r = sdm.residual_norm(**a)[1]
    args = dict(weight=w, after=a["after"], gate=a["gate"], scale=a["scale"])
    for pos, kw in (((x, r, None, dr), args), ((x, None, dy, dr), args), ((x, r, None, None), {}), ((x, r, dy, dr), {}),
                    ((x, r, dy[:3], dr), args), ((x, r, dy, dr.bfloat16()), args)):
        with pytest.raises((TypeError, ValueError)):
            sdm.residual_norm_backward(*pos, **kw)
    with pytest.raises(sdm.SDMError):
        sdm.residual_norm_backward(x, r, dy, dr, **args, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


def test_norm_past_32_bit_offsets():
    M, D = 560_000, 4096  # 2.3e9 elements
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn((M, D), generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.rand(D, generator=g, device="cuda")
    y, _ = sdm.residual_norm(x, weight=w)
    assert torch.equal(y[M - 300:], sdm.residual_norm(x[M - 300:], weight=w)[0])
    dx = sdm.gated_norm_backward(x, w, y)[0]
    assert torch.equal(dx[M - 300:], sdm.gated_norm_backward(x[M - 300:], w, y[M - 300:])[0])


def test_memory_for_an_output_that_there_is_not():
    x, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        sdm.residual_norm(x, weight=w, residual_out=torch.empty_like(x))
    with pytest.raises(ValueError):
        sdm.residual_norm(x, x.clone(), out=torch.empty_like(x))
