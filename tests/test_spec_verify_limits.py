"""spec_verify at the ends of its arguments' ranges."""
from __future__ import annotations

import pytest
import torch

from test_spec_verify import ccv, check, make  # noqa: F401

pytestmark = pytest.mark.gpu
INF = float("inf")
TINY = [1e-45, 1e-41, 1e-39, 4e-39, 5e-39, 1.2e-38, 1e-30, 1e-6]
HUGE = [1e6, 1e30, 1e38, 3.4e38, INF]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("v", [7, 2050, 40001])
def test_temperatures(ccv, dtype, draft, v):  # noqa: F811
    """A row with the least temperature takes the largest logit, one with the largest draws evenly."""
    t = torch.tensor(TINY + HUGE)
    d = make(len(t), 3, v, v, dtype, draft)
    d["tokens"][::2, 0] = d["logits"][::2, 0].float().argmax(-1)
    check(ccv, d, temperature=t)


def test_least_temperature_is_greedy(ccv):  # noqa: F811
    d = make(4, 2, 999, 3, torch.float32, draft=False)
    cold = check(ccv, d, temperature=torch.full((4,), 1e-45))
    greedy = check(ccv, d, temperature=torch.zeros(4))
    assert torch.equal(cold[0], greedy[0]) and torch.equal(cold[1], greedy[1])


def test_masked_logits_with_infinite_temperature(ccv):  # noqa: F811
    """-inf stays impossible; the rest is even, the type's lowest value too."""
    d = make(2, 1, 64, 5, torch.float32, draft=False)
    d["tokens"][:] = 3
    d["logits"][:, :, 8:] = -INF
    d["logits"][:, :, 4] = torch.finfo(torch.float32).min / 2
    d["uniform"][:] = torch.tensor([[0.12], [0.13]])      # either side of 1 / 8
    d["noise"][:] = 1.0
    d["noise"][:, 8:] = 1e-9                               # would win if they had any probability
    d["noise"][:, 4] = 0.5
    got = ccv.spec_verify(*(d[n].cuda() for n in ("logits", "tokens", "uniform", "noise")),
                          temperature=torch.full((2,), INF, device="cuda"))
    assert got[0].tolist() == [[3, 4], [4, -1]] and got[1].tolist() == [2, 1]


def test_negative_and_nan_temperatures_are_greedy(ccv):  # noqa: F811
    d = make(3, 2, 500, 6)
    on = [d[n].cuda() for n in ("logits", "tokens", "uniform", "noise", "probs")]
    want = ccv.spec_verify(*on, temperature=torch.zeros(3, device="cuda"))
    got = ccv.spec_verify(*on, temperature=torch.tensor([-1.0, float("nan"), -INF], device="cuda"))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
