"""The example layer's way back from speculative steps: decode, prefill and a new first step after settle.

Tolerance as in test_linear_layer.
"""
from __future__ import annotations

import pytest
import torch

from test_linear_layer import hidden_states, ints, ll, make, near  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture
def kept(ll):  # noqa: F811
    """A layer after speculative steps of two rows and one that has decoded what was kept, with the last counts."""
    x = hidden_states(90)
    spec, plain = make(ll, 3), make(ll, 3)
    fresh, lines = torch.zeros(2, dtype=torch.bool, device="cuda"), ints(2, 0)
    for net in (spec, plain):
        net.prefill(x[:40], x[:40], ints(0, 25, 40), lines, fresh)
    counts = None
    for step, keep in enumerate(((3, 1), (2, 4), (1, 3))):
        fed = torch.stack([x[40 + step:44 + step], x[50 + step:54 + step]])
        spec.verify(fed, fed, lines, counts)
        counts = ints(*keep)
        for t in range(4):
            for row in range(2):
                if t < keep[row]:
                    plain.decode(fed[row:row + 1, t], fed[row:row + 1, t], lines[row:row + 1])
    return spec, plain, lines, counts, x


def test_decode_after_settle(kept):
    spec, plain, lines, counts, x = kept
    spec.settle(lines, counts)
    near(spec.state[lines.long()].flatten(1), plain.state[lines.long()].flatten(1), "state")
    for t in range(3):
        fed = torch.stack([x[60 + t], x[70 + t]])
        got, res = spec.decode(fed, fed, lines)
        want, want_res = plain.decode(fed, fed, lines)
        near(got, want, f"token {t}")
        near(res, want_res, f"residual {t}")


def test_prefill_after_settle(kept):
    spec, plain, lines, counts, x = kept
    spec.settle(lines, counts)
    yes = torch.ones(2, dtype=torch.bool, device="cuda")
    got, _ = spec.prefill(x[60:85], x[60:85], ints(0, 20, 25), lines, yes)
    want, _ = plain.prefill(x[60:85], x[60:85], ints(0, 20, 25), lines, yes)
    near(got, want, "second prompt")


def test_first_step_after_settle_and_with_a_new_row(kept):
    """Settled rows and a row that has only been prefilled take a first step together."""
    spec, plain, lines, counts, x = kept
    spec.settle(lines, counts)
    no = torch.zeros(1, dtype=torch.bool, device="cuda")
    for net in (spec, plain):
        net.prefill(x[75:88], x[75:88], ints(0, 13), ints(1), no)
    rows = torch.cat([lines, ints(1)])
    fed = torch.stack([x[60:64], x[64:68], x[68:72]])
    got, _ = spec.verify(fed, fed, rows, None)
    for t in range(4):
        want, _ = plain.decode(fed[:, t].contiguous(), fed[:, t].contiguous(), rows)
        near(got[:, t], want, f"token {t}")


def test_settling_some_rows_leaves_the_others(kept):
    spec, plain, lines, counts, x = kept
    before = spec.state.clone(), spec.conv_state.clone()
    spec.settle(lines[:1], counts[:1])
    others = torch.ones(spec.state.shape[0], dtype=torch.bool, device="cuda")
    others[lines[0].long()] = False
    assert torch.equal(spec.state[others], before[0][others])
    assert torch.equal(spec.conv_state[others[:3]], before[1][others[:3]])
    fed = x[60:64][None]
    got, _ = spec.verify(fed, fed, lines[1:], counts[1:])  # the other row goes on speculating
    for t in range(4):
        want, _ = plain.decode(fed[:, t], fed[:, t], lines[1:])
        near(got[:, t], want, f"token {t}")
