"""How many bits of a state the scan's forms keep.

State, in the 2-norm, where the errors of the terms d x B add up as the terms do.  A term is off by the step's error (the
logarithm and the addition of the bias, 2^-22 on average), its decay's (an exponential of 2 units, 2^-23), two products
and, in the chunked form, three bf16 parts (2^-25 each), and by a truncated sum's share (2^-24 of the sum in each of its
last 24 steps of 16 products, which add up to 2^-22 on average).  Less than 2^-21 in all, which is allowed.  With two
parts of the weighted tokens a term has 16 bits and one for the sign of the rest, 2^-18.5 on average: six times as much.

That is the chunked form, whose decays go by sums of pairs of floats and whose state is rounded once in 128 tokens.  The
forms that go token by token multiply what they hold by a decay at every token.  The decay is off by up to 2 units in the last
place of a value in [1/2, 1) (2 * 2^-24 = 2^-23), not of both signs where steps are alike, so what is k <= n tokens old is
off by k 2^-23 besides: 2^-21 + n 2^-23 is allowed there.

That is the chunked form, whose decays go by sums of pairs of floats and whose state is rounded once in 128 tokens.  The
forms that go token by token multiply what they hold by a decay at every token.  The decay is off by up to 2 units in the last
place of a value in [1/2, 1) (2 * 2^-24 = 2^-23), not of both signs where steps are alike, so what is k <= n tokens old is
off by k 2^-23 besides: 2^-21 + n 2^-23 is allowed there.

The first test confirms on the host that the formulas with three parts are far below the bound and with two above it;
the others run the kernels.
"""
from __future__ import annotations

import pytest
import torch

import ssm_ref as ref
from test_ssm import BF16, INF, ccv, cuda, make, path, pool  # noqa: F401

STATE = 2.0 ** -21


def whole(t, n, start):
    """The final states of one sequence in 64 bits."""
    d = ref.steps(t["dt"], t["dt_bias"], True, (0.0, INF))
    a = t["A"] if t["A"].dim() == 2 else t["A"][:, None]
    return ref.ssm_tokens(t["x"][:n], d[:n], a, t["B"][:n], t["C"][:n], start.double())[2]


def off(got, want):
    return float((got.detach().cpu().double() - want).norm() / want.norm())


def cut(x, parts):
    """x as the sum of its first so many bf16 parts."""
    rest, out = x.float(), torch.zeros_like(x)
    for _ in range(parts):
        part = rest.to(BF16).float()
        out, rest = out + part.double(), rest - part
    return out


def chunked(t, n, start, parts):
    """The chunked form's states, its weighted tokens cut to so many parts; sums in 64 bits, states kept in 32."""
    d = ref.steps(t["dt"], t["dt_bias"], True, (0.0, INF))
    s, rep = start.double(), t["x"].shape[1] // t["B"].shape[1]
    b = t["B"].double().repeat_interleave(rep, 1)
    for at in range(0, n, 128):
        to = min(at + 128, n)
        g = (d[at:to] * t["A"].double()).cumsum(0)
        w = cut(((g[-1] - g).exp() * d[at:to])[..., None] * t["x"][at:to].double(), parts)
        s = (g[-1].exp()[:, None, None] * s + torch.einsum("thp,thn->hpn", w, b[at:to])).float().double()
    return s


@pytest.mark.parametrize("n", [1, 128, 300, 1000])
def test_bound_tells_the_parts(n):
    t = make(n, 2, 64, 1, 128, 80 + n)
    start = pool(1, 2, 64, 128, 81)[0] * 0
    want = whole(t, n, start)
    assert off(chunked(t, n, start, 3), want) < STATE / 4
    assert off(chunked(t, n, start, 2), want) > 3 * STATE


@pytest.mark.gpu
@pytest.mark.parametrize("form,segment,heads,dim,groups,states,per", [
    ("chunked", 0, 4, 64, 2, 128, False), ("chunked", 1, 4, 64, 2, 128, False), ("chunked", 3, 3, 64, 1, 64, False),
    ("chunked", 0, 2, 80, 1, 96, False), ("recurrent", 0, 4, 64, 2, 128, False), ("scan", 0, 6, 8, 1, 16, False),
    ("scan", 0, 100, 1, 1, 16, True), ("scan", 1, 100, 1, 1, 16, True), ("recurrent", 0, 100, 1, 1, 16, True)])
@pytest.mark.parametrize("n", [1, 128, 300, 1000])
@pytest.mark.parametrize("init", [True, False])
def test_prompt(ccv, path, form, segment, heads, dim, groups, states, per, n, init):  # noqa: F811
    path(form, segment)
    t = make(n, heads, dim, groups, states, 82 + n, per_state=per, kind=torch.float32)
    start = pool(1, heads, dim, states, 83) * (0.2 if init else 0.0)
    want, got, on = whole(t, n, start[0]), start.cuda(), cuda(t)
    ccv.ssm_fwd(*(on[k] for k in ("x", "dt", "A", "B", "C")), got, torch.tensor([0, n], dtype=torch.int32, device="cuda"), None,
                torch.tensor([True], device="cuda"), dt_bias=on["dt_bias"])
    allowed = STATE + (0 if form == "chunked" else n * 2.0 ** -23)
    assert off(got[0], want) < allowed
    for h in range(heads if dim > 1 else 0):  # and no head is worse than all together by more than chance
        assert off(got[0, h], want[h]) < 2 * allowed


@pytest.mark.gpu
@pytest.mark.parametrize("heads,dim,states,per", [(4, 64, 128, False), (100, 1, 16, True)])
def test_update(ccv, heads, dim, states, per):  # noqa: F811
    t = make(6, heads, dim, 1, states, 84, per_state=per, kind=torch.float32)
    start = 0.2 * pool(1, heads, dim, states, 85)
    want, got = whole(t, 6, start[0]), start.cuda()
    on = {k: v[None] if k in ("x", "dt", "B", "C") else v for k, v in cuda(t).items()}
    ccv.ssm_update(*(on[k] for k in ("x", "dt", "A", "B", "C")), got, dt_bias=on["dt_bias"])
    assert off(got[0], want) < STATE
