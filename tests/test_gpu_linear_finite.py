"""Linear attention where values are not finite: nothing of a later token reaches an earlier one."""
import numpy as np
import pytest
import torch

import mixer_ref as ref
import sparse_state_linear_sdm_gb300 as sdm
from test_gpu_linear import CASES, _case, _host, _live, _ref

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
FORMS = {"f32": 0, "f32-cut": 6, "lengths": 16, "tiles": 12, "tiles-64": 13, "tiles-cut": 18, "two-column-tiles": 20,
         "columns-copied": 19, "copied": 21, "copied-100": 22, "token by token": 23, "no-decay": 15}


def _run(a):
    return sdm.linear_attention(**a, state_out=None if a["state"] is None else torch.zeros_like(a["state"]))


def _places(T, dv):
    """(token, column, value): every border of a chunk's blocks, columns twice, the last token, the last column."""
    spots = [(t, (7 * i + 3) % (dv - 1), (NAN, INF, -INF)[i % 3]) for i, t in enumerate((0, 31, 32, 63, 64, 96, 127, 128, T // 2))]
    spots += [(T // 3, 1, INF), (T // 3 + 1, 1, NAN), (T - 1, dv - 1, NAN)]
    return [s for s in spots if s[0] < T]


def _check_rest(o2, o, bad, eo, dtype, columns):
    """What is not spoilt: other columns bit for bit, the spoilt ones' earlier tokens within the definition's bound twice (the
    one run's and the other's), for they may be formed in another order."""
    rest = ~columns.expand_as(o)
    assert torch.equal(o2[rest], o[rest])
    got, clean, keep = _host(o2), _host(o), ~bad.cpu().numpy()
    tol = 2 * (eo + ref.ROUND[dtype] * (np.abs(clean) + 2 * eo)) + 1e-37
    assert (np.abs(got - clean) <= tol)[keep].all()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("form", FORMS)
def test_a_value_reaches_its_column_from_its_token_on(form, in_place):
    c = CASES[FORMS[form]]
    a = _case(c)
    T, dv = a["v"].shape[1], a["v"].shape[3]
    o, st = _run(a)
    eo = _ref(a, dtype=c[0])[2]
    a["v"] = a["v"].clone()
    n = T if a["lengths"] is None else int(a["lengths"][0])
    bad = torch.zeros_like(o, dtype=torch.bool)
    for t, col, x in _places(n, dv):
        a["v"][0, t, 0, col] = x
        bad[0, t:n, 0, col] = True
    if in_place and a["state"] is not None:
        a["state"] = a["state"].clone()
        o2, st2 = sdm.linear_attention(**a)
        live = _live(a)[0]
        kept = torch.zeros_like(st)
        kept[live] = st2[live]
        st2 = kept
    else:
        o2, st2 = _run(a)
    assert not torch.isfinite(o2[bad]).any()
    _check_rest(o2, o, bad, eo, c[0], bad.any(1, keepdim=True))
    if st is None:
        return
    slot = 0 if a["slots"] is None else int(a["slots"][0])
    hit = torch.zeros_like(st, dtype=torch.bool)
    hit[slot, 0, :, :] = bad[0, n - 1, 0]
    assert not torch.isfinite(st2[hit]).any()
    assert torch.equal(st2[~hit], st[~hit])


@pytest.mark.parametrize("form", FORMS)
def test_values_of_one_token_alone(form):
    """All of a token's values at once, at the first, a middle and the last token: the ones before it are as they were."""
    c = CASES[FORMS[form]]
    a = _case(c)
    a["lengths"] = None
    T = a["v"].shape[1]
    o, _ = _run(a)
    eo = _ref(a, dtype=c[0])[2]
    live = [b for b in range(o.shape[0]) if a["slots"] is None or int(a["slots"][b]) >= 0]
    for t, x in ((0, NAN), (T // 2 + 1, INF), (T - 1, -INF)):
        b = {**a, "v": a["v"].clone()}
        b["v"][:, t] = x
        o2, st2 = _run(b)
        bad = torch.zeros_like(o, dtype=torch.bool)
        bad[live, t:] = True
        assert not torch.isfinite(o2[bad]).any()
        _check_rest(o2, o, bad, eo, c[0], bad.any(1, keepdim=True))
        assert st2 is None or not torch.isfinite(st2[_live(a)[0]]).any()


def test_growth_past_the_largest_float_spoils_no_earlier_token():
    """Finite values whose weighted products pass the largest float: the state is not finite from then on, earlier outputs are."""
    a = _case(CASES[12])
    T = a["v"].shape[1]
    a["decay"] = torch.zeros_like(a["decay"])
    o, _ = _run(a)
    a["decay"][:, T - 4:] = 60.0
    o2, st2 = _run(a)
    assert torch.equal(o2[:, :T - 4], o[:, :T - 4]) and not torch.isfinite(st2).any()


def test_a_key_that_is_not_finite_changes_no_earlier_token():
    for form in ("tiles", "tiles-cut", "copied", "two-column-tiles"):
        a = _case(CASES[FORMS[form]])
        a["lengths"] = None
        o, _ = _run(a)
        T = a["k"].shape[1]
        a["k"] = a["k"].clone()
        a["k"][0, T - 2, 0, 3] = INF
        a["v"] = a["v"].clone()
        a["v"][0, T - 1, 0, 2] = NAN
        o2, _ = _run(a)
        o2[0, :, 0, 2] = o[0, :, 0, 2]
        assert torch.equal(o2[:, :T - 2], o[:, :T - 2])
