"""The operators together: a layer's prefill, decode and speculative steps agree with one another.

All three compute the same function of the same tokens, each operator rounding
its output to bf16; the comparison is in the 2-norm of a row.  A row passes five
roundings of 2^-9 (projection, convolution, delta rule, norm, output), which the
norm and the products carry with gains near 1: 2^-6 of the row is twice what
they add to if none cancels.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ll():
    from causal_depthwise_conv1d_fwd_gb300 import build, linear_layer

    build.build()
    return linear_layer


def near(a, b, what):
    a, b = a.float(), b.float()
    off = (a - b).norm(dim=-1) / b.norm(dim=-1)
    assert float(off.max()) < 2.0 ** -6, (what, float(off.max()))


def make(ll, lines=3, steps=4):
    return ll.LinearAttentionLayer(192, 2, 4, 64, lines, steps, seed=3)


def hidden_states(n):
    g = torch.Generator().manual_seed(5)
    return torch.randn(n, 192, generator=g).to(torch.bfloat16).cuda()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_decode_continues_prefill(ll):
    x = hidden_states(90)
    whole, part = make(ll), make(ll)
    fresh = torch.zeros(1, dtype=torch.bool, device="cuda")
    want, want_res = whole.prefill(x, x, ints(0, 90), ints(1), fresh)
    part.prefill(x[:80], x[:80], ints(0, 80), ints(1), fresh)
    for t in range(80, 90):
        got, res = part.decode(x[t:t + 1], x[t:t + 1], ints(1))
        near(got, want[t:t + 1], f"token {t}")
        near(res, want_res[t:t + 1], f"residual {t}")
    near(part.state[1].flatten(1), whole.state[1].flatten(1), "state")
    near(part.conv_state[1, :, :3].t(), whole.conv_state[1, :, :3].t(), "conv state")


def test_prefill_in_two_calls(ll):
    x = hidden_states(140)
    whole, part = make(ll), make(ll)
    no, yes = (torch.full((2,), v, dtype=torch.bool, device="cuda") for v in (False, True))
    want, _ = whole.prefill(x, x, ints(0, 100, 140), ints(2, 0), no)
    a = torch.cat([x[:33], x[100:110]])
    part.prefill(a, a, ints(0, 33, 43), ints(2, 0), no)
    b = torch.cat([x[33:100], x[110:140]])
    got, _ = part.prefill(b, b, ints(0, 67, 97), ints(2, 0), yes)
    near(got, torch.cat([want[33:100], want[110:140]]), "second call")


def test_speculative_steps_follow_what_was_kept(ll):
    """Four tokens a step of which 1 to 4 stay: what is kept equals decoding those tokens one by one."""
    x = hidden_states(64)
    spec, plain = make(ll, 2), make(ll, 2)
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


def test_serving_example_runs(ll):
    kept = ll.serve()
    assert len(kept) == 2 and all(len(row) >= 4 and min(row) >= 0 for row in kept)
    assert kept == ll.serve()
