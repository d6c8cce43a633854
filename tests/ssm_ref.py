"""Plain 64-bit implementations of the selective state space scan and of the logits' adjustment (not collected as tests).

The scan runs token by token and returns, beside each result, what bounds its error.  With u = d A, a = exp(u) and
w = |d x B| the sum of absolute values A_t = a A_{t-1} + w bounds |S_t|, and an error made at one token decays like the state:

* state: a term d x B has a relative error of 2^-21 (the step d, by expf and log1pf of a few units in 2^-24 each, and the
  product), and a sum of up to 128 products in 32 bits, truncated, loses at most 128 * 2^-24 = 2^-17: STATE_MAG of w.  A
  decay has a relative error of 2^-21 (1 + |u|): exp by 2 units, u by the step's error.  So
  mag_t = a mag_{t-1} + w + 2^-4 (1 + |u|) A_t, and the state is within STATE_MAG mag.
* out: one rounding to bf16 (at most 2^-8 of the value), and products whose operands carry 16 bits or more
  (2^-16 each, two of them at most in a product): 2^-15 of the sum of A_t |C|, which bounds every sum of products on the
  way; and the state's own error times |C|.  The gate multiplies both; its own error of 2^-20 is far below.
"""
from __future__ import annotations

import torch

OUT_RTOL, OUT_MAG, STATE_MAG = 2.0 ** -8, 2.0 ** -15, 2.0 ** -17


def steps(dt, bias, softplus, limit):
    d = dt.double()
    if bias is not None:
        d = d + bias.double()
    if softplus:
        d = torch.where(d > 20, d, torch.log1p(torch.exp(d.clamp(max=20))))
    lo, hi = limit
    return torch.where(d < lo, torch.full_like(d, lo), torch.where(d > hi, torch.full_like(d, hi), d))


def ssm_tokens(x, d, A, B, C, state, D=None, z=None, keep=None):
    """Tokens of one row or sequence: x (n, heads, dim), steps d (n, heads), A (heads, 1 or states), B, C (n, groups,
    states), state (heads, dim, states) float64.  Returns the outputs, their bound, the final state and its magnitude."""
    x, d, A, B, C = (t.double() for t in (x, d, A, B, C))
    rep = x.shape[1] // B.shape[1]
    B, C = B.repeat_interleave(rep, 1), C.repeat_interleave(rep, 1)
    out, bound = torch.zeros_like(x), torch.zeros_like(x)
    total, mag = state.abs(), torch.zeros_like(state)
    for t in range(x.shape[0]):
        u = (d[t][:, None] * A)[:, None]
        a, w = u.exp(), (d[t][:, None] * x[t])[..., None] * B[t][:, None]
        state = a * state + w
        total = a * total + w.abs()
        mag = a * mag + w.abs() + 2.0 ** -4 * (1 + u.abs()) * total
        out[t] = (state * C[t][:, None]).sum(-1)
        c = C[t][:, None].abs()
        bound[t] = ((OUT_MAG * total + STATE_MAG * mag) * c).sum(-1)
        if keep is not None:
            keep.append((state, mag))
    if D is not None:
        out = out + D.double()[:, None] * x
        bound = bound + 2.0 ** -20 * (D.double()[:, None] * x).abs()
    if z is not None:
        gate = z.double() * torch.sigmoid(z.double())
        out, bound = out * gate, bound * gate.abs()
    return out, bound, state, mag


def ssm_fwd(x, dt, A, B, C, state, starts, lines=None, init=None, D=None, z=None, dt_bias=None, dt_softplus=True,
            dt_limit=(0.0, float("inf")), pad=-1):
    """Outputs (NaN where nothing is written), bounds, the pool after the call and its magnitude."""
    d = steps(dt, dt_bias, dt_softplus, dt_limit)
    out, bound = torch.full(x.shape, float("nan"), dtype=torch.float64), torch.zeros(x.shape, dtype=torch.float64)
    pool = None if state is None else state.double().clone()
    mags = None if state is None else torch.zeros_like(pool)
    a = A if A.dim() == 2 else A[:, None]
    for i in range(len(starts) - 1):
        s, e = int(starts[i]), int(starts[i + 1])
        line = i if lines is None else int(lines[i])
        if line == pad or s == e:
            continue
        shape = (x.shape[1], x.shape[2], B.shape[2])
        first = pool[line] if state is not None and init is not None and bool(init[i]) else torch.zeros(shape, dtype=torch.float64)
        out[s:e], bound[s:e], last, mag = ssm_tokens(x[s:e], d[s:e], a, B[s:e], C[s:e], first, D, None if z is None else z[s:e])
        if state is not None:
            pool[line], mags[line] = last, mag
    return out, bound, pool, mags


def assert_within(got, ref, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    err = (got - ref).abs()
    bad = ~(err <= bound + 1e-37)
    if bool(bad.any()):
        i = int(bad.flatten().nonzero()[0])
        worst = float((err / (bound + 1e-37)).nan_to_num(1e9).max())
        raise AssertionError(f"{what}: {int(bad.sum())}/{bad.numel()} outside, worst {worst:.3g} times the bound; first at "
                             f"{i}: {float(got.flatten()[i]):.6e} vs {float(ref.flatten()[i]):.6e}")


def assert_out(got, ref, bound, what="out"):
    assert_within(got, ref, OUT_RTOL * ref.abs() + bound, what)


def assert_state(got, ref, mag, what="state"):
    assert_within(got, ref, STATE_MAG * mag, what)


def logits(x, history=None, lengths=None, prompts=None, indices=None, drafts=None, repetition=None, frequency=None,
           presence=None, bias_ids=None, bias=None, mask=None, pad=-1):
    """(batch, positions, vocab) in 64 bits, rows that are skipped as NaN; and what bounds its error: the sum of the
    terms' sizes, each term rounded a few times in 32 bits."""
    b, n, v = x.shape
    out, size = torch.full(x.shape, float("nan"), dtype=torch.float64), torch.zeros(x.shape, dtype=torch.float64)
    for r in range(b):
        line = r if indices is None else int(indices[r])
        if indices is not None and line == pad:
            continue
        ids, prompt = torch.empty(0, dtype=torch.int64), 0
        if history is not None:
            if not 0 <= line < history.shape[0]:
                continue
            told = min(max(int(lengths[line]), 0), history.shape[1])
            prompt = 0 if prompts is None else min(max(int(prompts[line]), 0), history.shape[1])
            ids = history[line, :told].long()
        good = (ids >= 0) & (ids < v)
        said = good & (torch.arange(len(ids)) >= prompt)
        seen = torch.bincount(ids[good], minlength=v) > 0
        count = torch.bincount(ids[said], minlength=v)
        for i in range(n):
            if i > 0 and drafts is not None:
                token = int(drafts[r, i - 1])
                if 0 <= token < v:
                    seen[token] = True
                    count[token] += 1
            y = x[r, i].double()
            rep = 1.0 if repetition is None else float(repetition[r])
            y = torch.where(seen, torch.where(y > 0, y / rep, y * rep), y)
            s = y.abs()
            f = (0.0 if frequency is None else float(frequency[r])) * count
            p = (0.0 if presence is None else float(presence[r])) * (count > 0)
            y, s = y - f - p, s + f.abs() + p.abs()
            if bias is not None:
                for token, value in zip(bias_ids[r].tolist(), bias[r].double().tolist()):
                    if 0 <= token < v:
                        y[token] += value
                        s[token] += abs(value)
            if mask is not None:
                at = torch.arange(v)
                may = (mask[r, i].long()[at // 32] >> (at % 32)) & 1 == 1
                y = torch.where(may, y, -torch.inf)
            out[r, i], size[r, i] = y, s
    return out, size
