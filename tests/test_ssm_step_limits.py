"""min(max(d, lo), hi) of the scan's steps where the limits cross or leave fp32's range."""
from __future__ import annotations

import pytest
import torch

import ssm_ref as ref
from test_ssm import INF, ccv, cuda, make, path, pool  # noqa: F401

pytestmark = pytest.mark.gpu


def run(ccv, t, limit, update):  # noqa: F811
    on = cuda(t)
    n, h, p = t["x"].shape
    args = tuple(on[k] for k in ("x", "dt", "A", "B", "C"))
    kw = {"D": on["D"], "dt_bias": on["dt_bias"], "dt_limit": limit}
    if update:
        state = pool(n, h, p, t["B"].shape[2], 60).cuda()
        return ccv.ssm_update(*args, state, **kw), state
    state = pool(1, h, p, t["B"].shape[2], 60).cuda()
    starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    return ccv.ssm_fwd(*args, state, starts, None, torch.tensor([True], device="cuda"), **kw), state


@pytest.mark.parametrize("form,per_state", [("recurrent", False), ("recurrent", True), ("chunked", False), ("scan", True)])
@pytest.mark.parametrize("update", [False, True])
def test_limits_that_cross(ccv, path, form, per_state, update):  # noqa: F811
    """The upper one holds: every step is 0.05, below the lower limit or not."""
    path(form)
    h, p, n = (40, 1, 16) if per_state else (3, 64, 128)
    t = make(70, h, p, 1, n, 61, per_state=per_state)
    want = run(ccv, t, (0.05, 0.05), update)
    for limit in ((0.06, 0.05), (3.0, 0.05), (INF, 0.05)):
        got = run(ccv, t, limit, update)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    if not update:
        d = torch.full(t["dt"].shape, 0.05)
        out, bound, state, mag = ref.ssm_tokens(t["x"], d, t["A"] if per_state else t["A"][:, None], t["B"], t["C"],
                                                pool(1, h, p, n, 60)[0].double(), t["D"])
        ref.assert_out(want[0], out, bound)
        ref.assert_state(want[1][0], state, mag)


@pytest.mark.parametrize("limit", [(0.0, 1e300), (-1e300, INF), (-1e300, 1e300)])
def test_limits_past_fp32_are_none(ccv, limit):  # noqa: F811
    t = make(70, 3, 64, 1, 128, 62)
    for update in (False, True):
        want, got = run(ccv, t, (0.0, INF), update), run(ccv, t, limit, update)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
