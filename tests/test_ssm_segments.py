"""Arguments of ssm_fwd in the token scan, and in both forms that cut sequences into segments: lines, padding, no states,
steps' limits, offsets and lines that are wrong, values that are not finite before, in and after a cut."""
from __future__ import annotations

import pytest
import torch

from test_ssm import BF16, INF, ccv, check_fwd, cuda, make, path  # noqa: F401

pytestmark = pytest.mark.gpu
# form, segment, heads, channels a head, states, decays a state
CALLS = [("scan", 0, 40, 1, 16, True), ("scan", 1, 40, 1, 16, True), ("scan", 2, 5, 8, 24, True), ("scan", 0, 6, 4, 16, False),
         ("scan", 1, 6, 4, 16, False), ("chunked", 1, 2, 64, 128, False), ("chunked", 2, 3, 80, 64, False)]
CASES = pytest.mark.parametrize("form,segment,heads,dim,states,per", CALLS)


@CASES
def test_lines_and_padding(ccv, path, form, segment, heads, dim, states, per):  # noqa: F811
    """Lines in another order than the sequences, one of them skipped; tokens past the last sequence stay as they are."""
    path(form, segment)
    lengths = [100, 330, 300, 0, 129, 700]
    t = make(sum(lengths) + 9, heads, dim, 1, states, 70, per_state=per, gated=True)
    lines = torch.tensor([5, -1, 0, 2, 3, 8], dtype=torch.int32)
    for init in ([True, True, False, True, True, True], None):
        check_fwd(ccv, t, lengths, init=init, lines=lines, num_lines=9, channels=dim == 1)
    check_fwd(ccv, t, lengths, state=False, channels=dim == 1)


@CASES
@pytest.mark.parametrize("kw", [{"dt_softplus": False, "dt_limit": (0.001, 0.1)}, {"dt_limit": (0.01, 0.02)}, {"dt_limit": (0.0, 0.05)},
                                {"dt_limit": (0.02, INF)}])
def test_steps(ccv, path, form, segment, heads, dim, states, per, kw):  # noqa: F811
    path(form, segment)
    for kind in (BF16, torch.float32):
        t = make(300, heads, dim, 1, states, 71, per_state=per, kind=kind)
        check_fwd(ccv, t, [300], init=[True], channels=dim == 1, **kw)
    t["dt_bias"] = t["D"] = None
    check_fwd(ccv, t, [300], init=[True], channels=dim == 1, **kw)


@CASES
def test_strong_decays(ccv, path, form, segment, heads, dim, states, per):  # noqa: F811
    """Decays that leave nothing of a state within a token, and ones that leave it as it is, over a cut."""
    path(form, segment)
    t = make(300, heads, dim, 1, states, 72, per_state=per, strong=True)
    t["dt_bias"] += 3
    check_fwd(ccv, t, [300], init=[True], channels=dim == 1)
    t["A"][0], t["A"][1] = 0.0, -1e4
    check_fwd(ccv, t, [299], init=[True], channels=dim == 1)


@CASES
def test_bad_offsets_and_lines(ccv, path, form, segment, heads, dim, states, per):  # noqa: F811
    path(form, segment)
    t = cuda(make(300, heads, dim, 1, states, 73, per_state=per))
    state = torch.zeros(2, heads, dim, states, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda starts, lines: ccv.ssm_fwd(*(t[k] for k in ("x", "dt", "A", "B", "C")), state,  # noqa: E731
                                             torch.tensor(starts, dtype=torch.int32, device="cuda"),
                                             torch.tensor(lines, dtype=torch.int32, device="cuda"), err_count=err)
    for starts, lines in (([0, 301], [0]), ([-1, 200], [0]), ([200, 100], [0]), ([0, 200], [2]), ([0, 200], [-7])):
        before = int(err)
        call(starts, lines)
        assert int(err) > before, (starts, lines)
        assert not bool(state.any())
    before = int(err)
    call([0, 300], [-1])
    assert not bool(state.any()) and int(err) == before


@CASES
@pytest.mark.parametrize("what", ["x", "B", "C", "dt"])
@pytest.mark.parametrize("at", [3, 201, 290])
def test_not_finite_reaches_later_segments_only(ccv, path, form, segment, heads, dim, states, per, what, at):  # noqa: F811
    """As without segments: tokens before it, other sequences and (for x and dt) other heads are as without it, and later
    tokens are not finite where the formulas carry it."""
    path(form, segment)
    t = make(900, heads, dim, 1, states, 74, per_state=per)
    starts = torch.tensor([0, 600, 900], dtype=torch.int32, device="cuda")
    at *= 2

    def call(t):
        on = cuda(t)
        state = torch.zeros(2, heads, dim, states, device="cuda")
        out = ccv.ssm_fwd(*(on[k] for k in ("x", "dt", "A", "B", "C")), state, starts, D=on["D"], dt_bias=on["dt_bias"])
        return out, state

    out, state = call(t)
    p, n = dim // 2, states // 2
    t[what][(at, 1, p) if what == "x" else (at, 1) if what == "dt" else (at, 0, n)] = float("nan")
    got, after = call(t)
    same = lambda a, b: torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))  # noqa: E731
    assert same(got[:at], out[:at]) and same(got[600:], out[600:]) and torch.equal(after[1], state[1])
    if what in ("x", "dt"):
        other = [i for i in range(heads) if i != 1]
        assert same(got[:, other], out[:, other]) and torch.equal(after[0, other], state[0, other])
    if what == "x":
        assert bool(got[at:600, 1, p].isnan().all()) and bool(after[0, 1, p].isnan().all())
        rest = [i for i in range(dim) if i != p]
        assert same(got[:, 1, rest], out[:, 1, rest]) and torch.equal(after[0, 1, rest], state[0, 1, rest])
    elif what == "dt":
        assert bool(got[at:600, 1].isnan().all()) and bool(after[0, 1].isnan().all())
    elif what == "B":
        assert bool(got[at:600].isnan().all()) and bool(after[0, ..., n].isnan().all())
    else:
        assert bool(got[at].isnan().all()) and same(got[at + 1:], out[at + 1:]) and torch.equal(after, state)
