"""The scan's rates at the ends of their range."""
from __future__ import annotations

import pytest
import torch

from test_ssm import ccv, cuda, make, path, pool  # noqa: F401

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
