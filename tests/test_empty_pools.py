"""A pool without lines, or with lines without room, is a pool: its rows are refused one by one or have no tokens."""
from __future__ import annotations

import pytest
import torch

from test_ssm import BF16, ccv, cuda, make  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("place", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_histories(ccv, place, masked):  # noqa: F811
    logits = torch.randn(3, 1000, device="cuda")
    kw = {"repetition": torch.full((3,), 2.0, device="cuda")}
    if masked:
        kw["mask"] = torch.zeros(3, 32, dtype=torch.int32, device="cuda")
    for lines, size, indices, skipped in ((0, 8, (0, -1, 5), 3), (0, 0, (-1, -1, -1), 3), (2, 0, (1, -1, 2), 2)):
        err, given = i32(0), logits.clone()
        out = given if place else torch.full_like(logits, 7.0)
        before = out.clone()
        ccv.logits_process(given, i32(*[0] * (lines * size)).reshape(lines, size), i32(*[0] * lines), None, i32(*indices), out=out,
                           err_count=err, **kw)
        rows = slice(3 - skipped, 3) if skipped < 3 else slice(0, 3)
        assert torch.equal(out[rows], before[rows])
        assert (int(err) > 0) == any(i >= lines for i in indices)
        if skipped < 3:
            want = torch.full_like(logits[0], -torch.inf) if masked else logits[0]
            assert torch.equal(out[0], want)


def test_states(ccv):  # noqa: F811
    for heads, dim, states, per in ((2, 64, 128, False), (40, 1, 16, True)):
        for length in (40, 2):
            t = cuda(make(length, heads, dim, 1, states, 90, per_state=per))
            state = torch.zeros(0, heads, dim, states, device="cuda")
            args = tuple(t[k] for k in ("x", "dt", "A", "B", "C"))
            for lines, counted in ((i32(0), True), (i32(-1), False)):
                err, out = i32(0), torch.full_like(t["x"], 7.0)
                ccv.ssm_fwd(*args, state, i32(0, length), lines, out=out, err_count=err)
                assert bool((out == 7).all()) and (int(err) > 0) == counted
                err = i32(0)
                ccv.ssm_update(*(a[None] if a.shape[0] == length and k != 2 else a for k, a in enumerate(args)), state, lines,
                               out=out[None], err_count=err)
                assert bool((out == 7).all()) and (int(err) > 0) == counted
