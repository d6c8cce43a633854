"""The selective state space layer's operators together: prefill, decode and speculative steps agree with one another.

All three compute the same function of the same tokens, each operator rounding
its output to bf16; the comparison is in the 2-norm of a row.  A row passes five
roundings of 2^-8 at most (projection, convolution, scan, norm, output), 2^-9.6
in the mean square each, which the norm and the products carry with gains near
1: 2^-6 of the row is five times what they add to.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sl():
    from causal_depthwise_conv1d_fwd_gb300 import build, ssm_layer

    build.build()
    return ssm_layer


def near(a, b, what):
    a, b = a.float(), b.float()
    off = (a - b).norm(dim=-1) / b.norm(dim=-1)
    assert float(off.max()) < 2.0 ** -6, (what, float(off.max()))


def make(sl, lines=3, steps=4):
    return sl.SelectiveStateLayer(192, 4, 64, 2, 64, lines, steps, seed=3)


def hidden_states(n):
    return torch.randn(n, 192, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_decode_continues_prefill(sl):
    x = hidden_states(190)
    whole, part = make(sl), make(sl)
    fresh = torch.zeros(1, dtype=torch.bool, device="cuda")
    want, want_res = whole.prefill(x, x, ints(0, 190), ints(1), fresh)
    part.prefill(x[:180], x[:180], ints(0, 180), ints(1), fresh)
    for t in range(180, 190):
        got, res = part.decode(x[t:t + 1], x[t:t + 1], ints(1))
        near(got, want[t:t + 1], f"token {t}")
        near(res, want_res[t:t + 1], f"residual {t}")
    near(part.state[1].flatten(1), whole.state[1].flatten(1), "state")


def test_prefill_in_two_calls(sl):
    x = hidden_states(240)
    whole, part = make(sl), make(sl)
    no, yes = (torch.full((2,), v, dtype=torch.bool, device="cuda") for v in (False, True))
    want, _ = whole.prefill(x, x, ints(0, 200, 240), ints(2, 0), no)
    a = torch.cat([x[:33], x[200:210]])
    part.prefill(a, a, ints(0, 33, 43), ints(2, 0), no)
    b = torch.cat([x[33:200], x[210:240]])
    got, _ = part.prefill(b, b, ints(0, 167, 197), ints(2, 0), yes)
    near(got, torch.cat([want[33:200], want[210:240]]), "second call")


def test_speculative_steps_follow_what_was_kept(sl):
    """Four tokens a step of which 1 to 4 stay: what is kept equals decoding those tokens one by one; settled, too."""
    x = hidden_states(64)
    spec, plain = make(sl, 2), make(sl, 2)
    fresh = torch.zeros(2, dtype=torch.bool, device="cuda")
    lines = ints(0, 1)
    for net in (spec, plain):
        net.prefill(x[:40], x[:40], ints(0, 25, 40), lines, fresh)
    counts = None
    for step, keep in enumerate(((4, 1), (2, 3), (1, 4), (3, 2))):
        fed = torch.stack([x[40 + step:44 + step], x[50 + step:54 + step]])
        got, _ = spec.verify(fed, fed, lines, counts)
        counts = ints(*keep)
        for t in range(4):
            rows = [r for r in range(2) if t < keep[r]]
            if rows:
                want, _ = plain.decode(fed[rows, t], fed[rows, t], ints(*rows))
                near(got[rows, t], want, f"step {step}, token {t}")
    spec.settle(lines, counts)
    for t in range(60, 62):
        fed = x[[t, t + 2]]
        near(spec.decode(fed, fed, lines)[0], plain.decode(fed, fed, lines)[0], f"after settle, token {t}")


def test_serving_example_keeps_what_may_follow(sl):
    kept = sl.serve()
    assert len(kept) == 2 and all(len(row) >= 5 for row in kept)
    assert all(t >= 0 and t % 2 == 0 for row in kept for t in row)
    assert kept == sl.serve()
