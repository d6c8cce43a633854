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
