"""gdr_fwd on inputs that are not finite, in every form: a token's output does not depend on later tokens.

What comes before the token, the other rows of the state and the other sequences
have the bits of a run on finite inputs; from the token on, what it reaches is
not finite.
"""
from __future__ import annotations

import pytest
import torch

from test_gdr import ccv, dev, inputs, path  # noqa: F401

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
LENGTHS, STARTS = [70, 150, 30], [0, 70, 220, 250]  # the second sequence gets the value


def call(ccv, d, pool):  # noqa: F811
    dd, state = dev(d), pool.cuda().clone()
    starts = torch.tensor(STARTS, dtype=torch.int32, device="cuda")
    init = torch.tensor([True, True, False], device="cuda")
    out = ccv.gdr_fwd(dd["q"], dd["k"], dd["v"], dd["g"], dd["beta"], state, starts, None, init)
    torch.cuda.synchronize()
    return out.cpu(), state.cpu()


def make(dk, dv, seed):
    d, g = inputs(250, 2, 4, dk, dv, seed)
    return d, 0.3 * torch.randn(3, 4, dv, dk, generator=g)


def same_bits(a, b):
    assert torch.equal(a.contiguous().view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32),
                       b.contiguous().view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32))


def check(ccv, dk, dv, poison, token, heads, rows, last=None):  # noqa: F811
    """`heads` and `rows` (index tensors) are what the value at `token` of the second sequence reaches, up to token `last`."""
    d, pool = make(dk, dv, 7 + dk + token)
    want, want_state = call(ccv, d, pool)
    bad = {k: v.clone() for k, v in d.items()}
    bad_pool = pool.clone()
    poison(bad, bad_pool, 70 + token)
    got, state = call(ccv, bad, bad_pool)
    hit = torch.zeros(want.shape, dtype=torch.bool)
    end = 220 if last is None else 70 + last + 1
    for h in heads:
        hit[70 + token:end, h, rows] = True
    same_bits(got[~hit], want[~hit])
    assert not bool(got[hit].float().isfinite().any())
    hit_state = torch.zeros(state.shape, dtype=torch.bool)
    if last is None:
        for h in heads:
            hit_state[1, h, rows] = True
    same_bits(state[~hit_state], want_state[~hit_state])
    assert not bool(state[hit_state].isfinite().any())


DIMS = [(128, 128), (64, 64), (40, 130), (128, 256)]
TOKENS = [0, 5, 31, 32, 40, 63, 64, 100, 149]


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_value(ccv, path, dk, dv, value):  # noqa: F811
    for token in TOKENS:
        def poison(d, pool, t):
            d["v"][t, 2, dv - 3] = value
        check(ccv, dk, dv, poison, token, [2], torch.tensor([dv - 3]))


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("value", [NAN, INF])
def test_key(ccv, path, dk, dv, value):  # noqa: F811
    for token in TOKENS:
        def poison(d, pool, t):
            d["k"][t, 1, dk // 2] = value
        check(ccv, dk, dv, poison, token, [2, 3], torch.arange(dv))


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("value", [NAN, INF])
def test_query(ccv, path, dk, dv, value):  # noqa: F811
    for token in TOKENS:
        def poison(d, pool, t):
            d["q"][t, 0, 3] = value
        check(ccv, dk, dv, poison, token, [0, 1], torch.arange(dv), last=token)


@pytest.mark.parametrize("name,value", [("g", NAN), ("beta", NAN), ("beta", INF)])
def test_gates(ccv, path, name, value):  # noqa: F811
    for token in TOKENS:
        def poison(d, pool, t):
            d[name][t, 3] = value
        check(ccv, 128, 128, poison, token, [3], torch.arange(128))


def test_initial_state(ccv, path):  # noqa: F811
    def poison(d, pool, t):
        pool[1, 1, 17, 5] = NAN
    check(ccv, 128, 128, poison, 0, [1], torch.tensor([17]))


def test_two_tokens(ccv, path):  # noqa: F811
    """Two values of one row and one of another: each row counts from its own first."""
    d, pool = make(128, 128, 3)
    want, want_state = call(ccv, d, pool)
    bad = {k: v.clone() for k, v in d.items()}
    for t, row in ((70 + 90, 4), (70 + 33, 4), (70 + 35, 100)):
        bad["v"][t, 0, row] = NAN
    got, state = call(ccv, bad, pool)
    hit = torch.zeros(want.shape, dtype=torch.bool)
    hit[70 + 33:220, 0, 4] = True
    hit[70 + 35:220, 0, 100] = True
    same_bits(got[~hit], want[~hit])
    assert bool(got[hit].isnan().all())
    hit_state = torch.zeros(state.shape, dtype=torch.bool)
    hit_state[1, 0, [4, 100]] = True
    same_bits(state[~hit_state], want_state[~hit_state])
    assert bool(state[hit_state].isnan().all())
