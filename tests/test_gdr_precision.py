"""How many bits gdr_fwd's products carry, on inputs that show them.

`plain` inputs are those of the other tests.  On `erased` ones the keys have 2-norm 1
exactly, b is 1 and the values are 0, so every token takes its key's part of the
state away: d_i = -a_i S k_i, and the output for q_i = k_i is 0, the difference
of sums as large as d.

State, in the 2-norm.  Operands of 24 bits are off by 2^-25 of themselves on
average, T by up to 2^-21 of the products that it is made of, and a sum of
truncated steps loses 2^-24 of itself on average in each of its last 16 (the
products of the first parts, and of all parts of its second half): less than
2^-21 of the state for the errors of one token, which shrink with the state
afterwards.  2^-20 is allowed.  One part of an operand fewer (16 bits, 2^-18 on
average) costs 2^-19.5 to 2^-18, and adding the first parts first as much.
Output, in the 2-norm against that of d.  S, P and d have 16 bits there: three
roundings of 2^-18 at most and one product of two second parts, not all of one
sign: 2^-17 on average over both sums.  2^-15 is allowed; 8 bits anywhere cost
2^-10.5.

The first tests confirm these figures on the formulas with their operands cut to
so many parts, on the host; the others run the kernels.
"""
from __future__ import annotations

import pytest
import torch

import layer_ref as ref
from test_gdr import ccv, dev, inputs, path, split  # noqa: F401

BF16 = torch.bfloat16
STATE, OUT = 2.0 ** -20, 2.0 ** -15
WHOLE = {"S": 3, "R": 3, "T": 3, "d": 3, "S_out": 2, "P": 2, "d_out": 2}


def erased(n, hk, hv, dk, dv, seed):
    """(q, k, v, g, beta) of n tokens, and a pool of one line."""
    g = torch.Generator().manual_seed(seed)
    live = {128: 64, 64: 16}[dk]
    k = torch.zeros(n, hk, dk)
    for t in range(n):
        for h in range(hk):
            at = torch.randperm(dk, generator=g)[:live]
            k[t, h, at] = (torch.randint(0, 2, (live,), generator=g) * 2 - 1) * live ** -0.5
    k = k.to(BF16)
    d = {"q": k, "k": k, "v": torch.zeros(n, hv, dv, dtype=BF16), "g": -0.02 * torch.rand(n, hv, generator=g),
         "beta": torch.ones(n, hv)}
    return d, torch.randn(1, hv, dv, dk, generator=g)


def steps(d, start, scale, l2):
    """Token by token in 64 bits: outputs, final state, and every token's d."""
    out, _, state, _ = ref.gdr_tokens(*split(d, 0, d["v"].shape[0]), start.double(), scale, l2)
    if l2:
        return out, state, None
    s, ds, rep = start.double(), [], d["v"].shape[1] // d["k"].shape[1]
    for t in range(d["v"].shape[0]):
        k = d["k"][t].double().repeat_interleave(rep, 0)
        s = d["g"][t].double().exp()[:, None, None] * s
        ds.append(d["beta"][t].double()[:, None] * (d["v"][t].double() - torch.einsum("hvk,hk->hv", s, k)))
        s = s + ds[-1][..., None] * k[:, None]
    return out, state, torch.stack(ds)


def off(got, want, size):
    return float((got.detach().cpu().double() - want).norm() / size.norm())


# ------------------------------------------------------------- on the host ----

def cut(x, parts):
    """x as its first so many bf16 parts."""
    rest, out = x.float(), []
    for _ in range(parts):
        out.append(rest.to(BF16).float())
        rest = rest - out[-1]
    return [p.double() for p in out]


def chunked(q, k, v, g, b, s, parts):
    """One head's chunked form with each operand cut to its parts; sums in 64 bits, kept values in 32."""
    f32 = lambda x: x.float().double()  # noqa: E731
    outs = []
    for at in range(0, q.shape[0], 64):
        kk, qq, vv, gg, bb = (x[at:at + 64] for x in (k, q, v, g, b))
        run = gg.cumsum(0)
        decay = torch.exp(run[:, None] - run).tril()
        t = torch.linalg.inv(torch.eye(len(gg), dtype=torch.float64) + (bb[:, None] * (kk @ kk.T) * decay).tril(-1))
        p = (qq @ kk.T * decay).tril()
        sk = f32(sum(cut(s, parts["S"])) @ kk.T).T
        r = bb[:, None] * (vv - run.exp()[:, None] * sk)
        d = f32(sum(cut(t, parts["T"])) @ sum(cut(r, parts["R"])))
        out = run.exp()[:, None] * (sum(cut(s, parts["S_out"])) @ qq.T).T
        pp, dd = cut(p, parts["P"]), cut(d, parts["d_out"])
        for i, x in enumerate(pp):
            for j, y in enumerate(dd):
                if i + j < 2:
                    out = out + x @ y
        outs.append(out)
        s = f32(run[-1].exp() * s + sum(cut((run[-1] - run).exp()[:, None] * d, parts["d"])).T @ kk)
    return torch.cat(outs), s


def host_errors(d, start, scale, l2, parts):
    out, state, ds = steps(d, start, scale, l2)
    q, k = d["q"][:, 0].double(), d["k"][:, 0].double()
    if l2:
        q, k = (x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt() for x in (q, k))
    got, got_state = chunked(q * scale, k, d["v"][:, 0].double(), d["g"][:, 0].double(), d["beta"][:, 0].double(),
                             start[0].double(), {**WHOLE, **parts})
    return off(got_state[None], state, state), None if ds is None else off(got[:, None], out, ds)


@pytest.mark.parametrize("n", [129, 200])
def test_bounds_tell_the_parts_of_the_state(n):
    d, pool = erased(n, 1, 1, 128, 128, n)
    assert host_errors(d, pool[0], 1.0, False, {})[0] < STATE / 4
    for name in ("S", "R", "T", "d"):
        assert host_errors(d, pool[0], 1.0, False, {name: 2})[0] > STATE, name


@pytest.mark.parametrize("n", [70, 500])
def test_bounds_tell_the_parts_on_plain_inputs(n):
    d, g = inputs(n, 1, 1, 128, 128, n)
    pool = 0.3 * torch.randn(1, 1, 128, 128, generator=g)
    assert host_errors(d, pool[0], 128 ** -0.5, True, {})[0] < STATE / 4
    for name in ("R", "d"):
        assert host_errors(d, pool[0], 128 ** -0.5, True, {name: 2})[0] > STATE, name


@pytest.mark.parametrize("n", [64, 129])
def test_bounds_tell_the_parts_of_the_output(n):
    d, pool = erased(n, 1, 1, 128, 128, n + 1)
    assert host_errors(d, pool[0], 1.0, False, {})[1] < OUT / 4
    for name in ("S_out", "P", "d_out"):
        assert host_errors(d, pool[0], 1.0, False, {name: 1})[1] > 8 * OUT, name


# -------------------------------------------------------------- the kernels ----

def run(ccv, d, pool, scale, l2):  # noqa: F811
    dd, state = dev(d), pool.cuda().clone()
    starts = torch.tensor([0, d["v"].shape[0]], dtype=torch.int32, device="cuda")
    out = ccv.gdr_fwd(dd["q"], dd["k"], dd["v"], dd["g"], dd["beta"], state, starts,
                      has_initial_state=torch.tensor([True], device="cuda"), scale=scale, qk_l2norm=l2)
    return out, state


@pytest.mark.gpu
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 256)])
@pytest.mark.parametrize("n", [63, 64, 65, 129, 200])
def test_erased(ccv, path, n, dk, dv):  # noqa: F811
    n = n if dk == 128 else n // 2 + 33  # 64 keys are used up after half as many tokens
    d, pool = erased(n, 2, 4, dk, dv, n + dk)
    want, want_state, ds = steps(d, pool[0], 1.0, False)
    out, state = run(ccv, d, pool, 1.0, False)
    assert off(state[0], want_state, want_state) < STATE
    assert off(out, want, ds) < OUT
    for h in range(4):  # and no head is worse than all together by more than chance
        assert off(state[0, h], want_state[h], want_state[h]) < 2 * STATE
        assert off(out[:, h], want[:, h], ds[:, h]) < 2 * OUT


@pytest.mark.gpu
@pytest.mark.parametrize("n", [70, 129, 500])
@pytest.mark.parametrize("init", [True, False])
def test_plain(ccv, path, n, init):  # noqa: F811
    d, g = inputs(n, 2, 4, 128, 128, n)
    pool = (0.3 if init else 0.0) * torch.randn(1, 4, 128, 128, generator=g)
    want, want_state, _ = steps(d, pool[0], 128 ** -0.5, True)
    out, state = run(ccv, d, pool, None, True)
    assert off(state[0], want_state, want_state) < STATE
    # one rounding to bf16: 2^-9.2 of the output on average; 2^-9 is allowed
    assert off(out, want, want) < 2.0 ** -9


@pytest.mark.gpu
@pytest.mark.parametrize("t", [1, 6])
def test_update(ccv, t):  # noqa: F811
    """The recurrent form of decode has fp32 throughout."""
    d, pool = erased(8 * t, 2, 4, 128, 128, t)
    want_state, got = [], torch.cat([pool] * 8).cuda()
    for r in range(8):
        part = {n: x[r * t:(r + 1) * t] for n, x in d.items()}
        want_state.append(steps(part, pool[0], 1.0, False)[1])
    dd = {n: x.cuda().unflatten(0, (8, t)) for n, x in d.items()}
    ccv.gdr_update(dd["q"], dd["k"], dd["v"], dd["g"], dd["beta"], got, scale=1.0, qk_l2norm=False)
    want_state = torch.stack(want_state)
    assert off(got, want_state, want_state) < 2.0 ** -22
