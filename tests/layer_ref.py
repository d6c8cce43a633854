"""Plain 64-bit implementations of the linear-attention layer's operators (not collected as tests).

The gated delta rule runs token by token and returns, beside each result, what
bounds its error.  S is a contraction of each of its rows (b |k|^2 <= 2), so an
error made at one token only shrinks later, and a row's error is at most the
sum, decayed like the state, of what each token can add:

* state: a token adds a relative error of what it sums to the row,
  b |k| (|v| + a |S| |k|), and a rounding of the row itself, for which 2^-6 |S|
  is counted.  Operands carry at least 22 bits (2^-22) and a sum of 128
  products in 32 bits loses at most 128 * 2^-24 = 2^-17: STATE_MAG.
* out: one rounding to bf16 (at most 2^-9 of the value, 2^-8 is allowed) and
  three factors that the chunked form rounds to 11 bits (2^-11 at most each):
  the state, and the products and pseudo-values of the tokens since the chunk's
  start, whose sizes |S| + sum of decayed |d| |k| bounds, times |q|.
* out, over a whole sequence in the 2-norm: those roundings are independent, so
  they stay near 2^-9.2 of the output; 2^-8 is allowed, and 2^-11 of the bound
  above for outputs that are differences of larger terms.
"""
from __future__ import annotations

import torch

CHUNK = 64
OUT_RTOL, OUT_MAG, STATE_MAG = 2.0 ** -8, 3 * 2.0 ** -11, 2.0 ** -17


def gates(g, beta, a_log=None, dt_bias=None):
    if a_log is None:
        return g.double(), beta.double()
    x = g.double() + dt_bias.double()
    return -a_log.double().exp() * torch.nn.functional.softplus(x), torch.sigmoid(beta.double())


def gdr_tokens(q, k, v, g, beta, state, scale, qk_l2norm, keep=None):
    """Tokens of one row or sequence, (n, heads, dim) each, from state (heads_v, dim_v, dim_k) float64: the
    outputs, the final state, and the bounds' magnitudes (n, heads_v, dim_v) and (heads_v, dim_v)."""
    q, k, v = q.double(), k.double(), v.double()
    if qk_l2norm:
        q = q / (q.square().sum(-1, keepdim=True) + 1e-6).sqrt()
        k = k / (k.square().sum(-1, keepdim=True) + 1e-6).sqrt()
    q = q * scale
    rep = v.shape[1] // k.shape[1]
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    kn, qn = k.norm(dim=-1, keepdim=True), q.norm(dim=-1, keepdim=True)
    out, out_mag = torch.zeros_like(v), torch.zeros_like(v)
    mag = torch.zeros(state.shape[:2], dtype=torch.float64)
    for t in range(q.shape[0]):
        if t % CHUNK == 0:
            sums = state.norm(dim=-1)
        a, b = g[t].exp()[:, None], beta[t].abs()[:, None]
        state = a[..., None] * state
        size = state.norm(dim=-1)
        d = beta[t][:, None] * (v[t] - torch.einsum("hvk,hk->hv", state, k[t]))
        state = state + d[..., None] * k[t][:, None, :]
        mag = a * mag + b * kn[t] * (v[t].abs() + size * kn[t]) + 2.0 ** -6 * size
        sums = a * sums + d.abs() * kn[t]
        out[t] = torch.einsum("hvk,hk->hv", state, q[t])
        out_mag[t] = (OUT_MAG * sums + STATE_MAG * mag) * qn[t]
        if keep is not None:
            keep.append((state, mag))
    return out, out_mag, state, mag


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


def assert_out(got, ref, mag, what="out"):
    assert_within(got, ref, OUT_RTOL * ref.abs() + mag, what)
    off = (got.detach().cpu().double() - ref).norm()
    assert off <= OUT_RTOL * ref.norm() + mag.norm() / 3, (what, float(off), float(ref.norm()))


def assert_state(got, ref, mag, what="state"):
    assert_within(got, ref, STATE_MAG * mag[..., None], what)


def act(z, activation):
    if activation is None:
        return z
    return z * torch.sigmoid(z) if activation == "silu" else torch.sigmoid(z)


def rms(x, eps):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt()


def gated_rms_norm(x, gate, weight, eps, activation, before):
    x, z, w = x.double(), act(gate.double(), activation), weight.double()
    return rms(x, eps) * w * z if before else rms(x * z, eps) * w


def residual_rms_norm(x, residual, weight, post_weight, gate, scale, eps, offset):
    t = x.double()
    if post_weight is not None:
        t = rms(t, eps) * (post_weight.double() + offset)
    if gate is not None:
        t = t * gate.double()
    h = residual.double() + scale * t
    return rms(h, eps) * (weight.double() + offset), h, residual.double().abs() + abs(scale) * t.abs()


def spec_verify(logits, tokens, uniform, noise, probs=None, num_drafts=None, temperature=None):
    """Row by row, in 64 bits: (tokens, counts) as int32."""
    b, s = tokens.shape
    v = logits.shape[-1]
    out = torch.full((b, s + 1), -1, dtype=torch.int32)
    count = torch.zeros(b, dtype=torch.int32)
    x = logits.double()
    x = torch.where(torch.isnan(x), -torch.inf, x).clamp(max=torch.finfo(torch.float32).max)
    for r in range(b):
        n = s if num_drafts is None else int(num_drafts[r])
        if n < 0:
            continue
        temp = 1.0 if temperature is None else float(temperature[r])

        def p_of(i):
            best = x[r, i].max()
            if best == -torch.inf:
                return torch.zeros(v, dtype=torch.float64)
            if temp == 0:
                p = torch.zeros(v, dtype=torch.float64)
                p[int((x[r, i] == best).nonzero()[0])] = 1.0
                return p
            e = torch.exp((x[r, i] - best) / temp)
            return e / e.sum()

        kept = 0
        while kept < n:
            t = int(tokens[r, kept])
            if not 0 <= t < v:
                break
            q = 1.0 if probs is None else float(probs[r, kept, t])
            if not float(uniform[r, kept]) * q < float(p_of(kept)[t]):
                break
            kept += 1
        p = p_of(kept)
        if kept < n and temp != 0:
            if probs is not None:
                p = (p - probs[r, kept].double()).clamp_min(0)
            elif 0 <= int(tokens[r, kept]) < v:
                p[int(tokens[r, kept])] = 0
        score = p if temp == 0 else p / noise[r].double()
        out[r, :kept] = tokens[r, :kept]
        if float(score.max()) > 0:
            out[r, kept] = int(score.argmax())
        count[r] = kept + 1
    return out, count
