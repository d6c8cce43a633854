"""The scan's rates and steps at the ends of their ranges: rates that are not finite, steps of nothing."""
from __future__ import annotations

import pytest
import torch

import ssm_ref as ref
from test_ssm import INF, ccv, cuda, make, path, pool  # noqa: F401

pytestmark = pytest.mark.gpu
NAN = float("nan")
# form, heads, channels a head, states, decays a state, segment
FORMS = [("recurrent", 3, 64, 128, False, None), ("recurrent", 40, 1, 16, True, None), ("recurrent", 40, 1, 100, True, None),
         ("chunked", 3, 64, 128, False, 0), ("chunked", 3, 64, 64, False, 1), ("scan", 40, 1, 16, True, 0), ("scan", 40, 1, 16, True, 1),
         ("scan", 35, 1, 100, True, 0), ("scan", 3, 8, 16, False, 0), ("scan", 3, 8, 16, False, 1)]
LENGTHS = [[1], [33], [64], [128], [129, 5, 300]]


def call(ccv, t, lengths, **kw):  # noqa: F811
    on = cuda(t)
    h, p = t["x"].shape[1:]
    state = pool(len(lengths), h, p, t["B"].shape[2], 50).cuda()
    starts = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")
    init = torch.ones(len(lengths), dtype=torch.bool, device="cuda")
    out = ccv.ssm_fwd(*(on[k] for k in ("x", "dt", "A", "B", "C")), state, starts, None, init, D=on["D"], z=on["z"],
                      dt_bias=on["dt_bias"], **kw)
    return out, state


@pytest.mark.parametrize("form,heads,dim,states,per,segment", FORMS)
@pytest.mark.parametrize("lengths", LENGTHS)
def test_a_rate_that_is_no_number_shows(ccv, path, form, heads, dim, states, per, segment, lengths):  # noqa: F811
    """Its head's outputs and state are NaN (with a decay a state that state, and the outputs), the others as without it."""
    path(form, segment)
    t = make(sum(lengths), heads, dim, 1, states, 51, per_state=per)
    out, state = call(ccv, t, lengths)
    t["A"][1] = NAN
    got, after = call(ccv, t, lengths)
    assert bool(got[:, 1].isnan().all()) and bool(after[:, 1].isnan().all())
    keep = [i for i in range(heads) if i != 1]
    assert torch.equal(got[:, keep], out[:, keep]) and torch.equal(after[:, keep], state[:, keep])
    if per:
        t = make(sum(lengths), heads, dim, 1, states, 51, per_state=per)
        t["A"][1, 2] = NAN
        got, after = call(ccv, t, lengths)
        assert bool(got[:, 1].isnan().all()) and bool(after[:, 1, :, 2].isnan().all())
        rest = [i for i in range(states) if i != 2]
        assert torch.equal(after[:, 1][:, :, rest], state[:, 1][:, :, rest])


@pytest.mark.parametrize("form,heads,dim,states,per,segment", FORMS)
@pytest.mark.parametrize("lengths", LENGTHS)
def test_a_rate_of_minus_infinity_leaves_nothing(ccv, path, form, heads, dim, states, per, segment, lengths):  # noqa: F811
    """exp(-inf) is 0: a head's state is its last token's term alone, however the tokens fall into tiles."""
    path(form, segment)
    t = make(sum(lengths), heads, dim, 1, states, 52, per_state=per)
    out, state = call(ccv, t, lengths)
    t["A"][1] = -INF
    got, after = call(ccv, t, lengths)
    keep = [i for i in range(heads) if i != 1]
    assert torch.equal(got[:, keep], out[:, keep]) and torch.equal(after[:, keep], state[:, keep])
    d = ref.steps(t["dt"], t["dt_bias"], True, (0.0, INF))[:, 1]
    term = (d[:, None] * t["x"][:, 1].double())[..., None] * t["B"][:, 0].double()[:, None]  # (tokens, dim, states)
    c = t["C"][:, 0].double()[:, None]
    want = (term * c).sum(-1) + t["D"][1].double() * t["x"][:, 1].double()
    # the products' bounds of the other tests, with nothing carried from token to token
    bound = (ref.OUT_MAG + ref.STATE_MAG) * (term * c).abs().sum(-1) + 2.0 ** -20 * (t["D"][1] * t["x"][:, 1].double()).abs()
    ref.assert_out(got[:, 1], want, bound)
    last = [sum(lengths[:i + 1]) - 1 for i in range(len(lengths))]
    ref.assert_state(after[:, 1], term[last], 2 * term[last].abs())


@pytest.mark.parametrize("form,heads,dim,states,per,segment", FORMS)
def test_a_step_of_nothing_leaves_the_state(ccv, path, form, heads, dim, states, per, segment):  # noqa: F811
    """Steps of 0 keep the state as it is whatever the rate, minus infinity among them, and add nothing."""
    path(form, segment)
    t = make(300, heads, dim, 1, states, 53, per_state=per, kind=torch.float32)
    t["dt"].zero_()
    t["dt_bias"] = None
    t["A"][1] = -INF
    got, after = call(ccv, t, [300], dt_softplus=False)
    first = pool(1, heads, dim, states, 50).cuda()
    assert torch.equal(after, first)
    c, s = t["C"].double().repeat_interleave(heads, 1), first[0].cpu().double()
    want = torch.einsum("hpn,thn->thp", s, c) + t["D"].double()[:, None] * t["x"].double()
    size = torch.einsum("hpn,thn->thp", s.abs(), c.abs())
    ref.assert_out(got, want, ref.OUT_MAG * size + 2.0 ** -20 * (t["D"][:, None] * t["x"].double()).abs())


@pytest.mark.parametrize("per_state", [False, True])
def test_update_with_rates_at_the_ends(ccv, per_state):  # noqa: F811
    h, p, n = (40, 1, 16) if per_state else (3, 64, 128)
    t = make(2, h, p, 1, n, 54, per_state=per_state, kind=torch.float32)
    t["A"][0], t["A"][1] = NAN, -INF
    t["dt_bias"] = None
    t["dt"][0, 1] = 0.0
    t["dt"][1, 1] = 0.25
    on, state = cuda(t), pool(2, h, p, n, 55).cuda()
    first = state.clone()
    out = ccv.ssm_update(*(on[k] for k in ("x", "dt", "A", "B", "C")), state, dt_softplus=False)
    assert bool(state[:, 0].isnan().all()) and bool(out[:, 0].isnan().all()) and bool(state[:, 2:].isfinite().all())
    assert torch.equal(state[0, 1], first[0, 1])
    term = 0.25 * t["x"][1, 1].double()[:, None] * t["B"][1, 0].double()
    ref.assert_state(state[1, 1], term, 2 * term.abs())
