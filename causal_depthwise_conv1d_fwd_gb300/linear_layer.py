"""A linear-attention layer on the library's operators: an example of how they are
used together, and a small program for tests and profilers.

One layer takes normalised hidden states x and the residual stream and returns
both for the next block:

    mixed, z, b, a = x W_in
    q, k, v        = split(SiLU(causal_conv(mixed)))     ccv_fwd / ccv_update / ccv_update_spec
    o              = gated delta rule(q, k, v, a, b)     gdr_fwd / gdr_update
    y              = (norm(o) * SiLU(z)) W_out           gated_rms_norm
    x, residual    = norm(residual + y), residual + y    residual_rms_norm

The matrix products are torch's.  A sequence owns one line of the convolution's
pool and one of the delta rule's.  While it decodes speculatively it also owns
one delta-rule line for each token of a step (`step_lines`): a step writes the
state after every token, and the next one starts from the state after the last
token that spec_verify kept -- its counts go to ccv_update_spec and gdr_update
as num_accepted_tokens.  The sequence's own lines stay as they were before the
first step; `settle` brings them up to date, for decode, another prefill, or a
step together with sequences that have not begun to speculate.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import api, layer

BF16 = torch.bfloat16


class LinearAttentionLayer:
    """Weights and state pools of one layer; `steps` tokens at most a row and step."""

    def __init__(self, hidden: int, num_k_heads: int, num_v_heads: int, head_dim: int, lines: int,
                 steps: int = 1, width: int = 4, device="cuda", seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        self.hk, self.hv, self.d, self.width = num_k_heads, num_v_heads, head_dim, width
        self.qk, self.vd = num_k_heads * head_dim, num_v_heads * head_dim
        self.mixed = 2 * self.qk + self.vd

        def weight(*shape, std):
            return (std * torch.randn(*shape, generator=g)).to(BF16).to(device)

        self.w_in = weight(self.mixed + self.vd + 2 * num_v_heads, hidden, std=hidden ** -0.5)
        self.w_out = weight(hidden, self.vd, std=self.vd ** -0.5)
        self.conv_weight = weight(self.mixed, width, std=width ** -0.5)
        self.norm_weight = 1 + weight(head_dim, std=0.1)
        self.out_norm_weight = weight(hidden, std=0.1)  # used as 1 + weight
        self.a_log = torch.log(1 + 15 * torch.rand(num_v_heads, generator=g)).to(device)
        self.dt_bias = (torch.randn(num_v_heads, generator=g) - 3).to(device)
        # dim contiguous, as the convolution's decode kernel likes it; room for `steps` inputs
        self.conv_state = torch.zeros(lines, width - 2 + steps, self.mixed, dtype=BF16,
                                      device=device).transpose(1, 2)
        self.state = torch.zeros(lines * (1 + steps), num_v_heads, head_dim, head_dim, device=device)
        self.step_lines = (lines + torch.arange(lines * steps, dtype=torch.int32, device=device)
                           ).reshape(lines, steps)

    def _project(self, x):
        """(..., hidden) -> mixed, z, b, a."""
        return (x @ self.w_in.t()).split([self.mixed, self.vd, self.hv, self.hv], -1)

    def _heads(self, mixed):
        """(..., mixed) -> q, k, v as views of it."""
        q, k, v = mixed.split([self.qk, self.qk, self.vd], -1)
        return (q.unflatten(-1, (self.hk, self.d)), k.unflatten(-1, (self.hk, self.d)),
                v.unflatten(-1, (self.hv, self.d)))

    def _finish(self, o, z, residual) -> Tuple[torch.Tensor, torch.Tensor]:
        o = o.reshape(-1, self.hv, self.d)
        y = layer.gated_rms_norm(o, z.reshape(-1, self.vd).unflatten(-1, (self.hv, self.d)),
                                 self.norm_weight)
        return layer.residual_rms_norm(y.flatten(1) @ self.w_out.t(), residual,
                                       self.out_norm_weight, weight_offset=1.0)

    def prefill(self, x: torch.Tensor, residual: torch.Tensor, query_start_loc: torch.Tensor,
                lines: torch.Tensor, has_initial_state: torch.Tensor):
        """Varlen prompts, or their next parts: x, residual (total_tokens, hidden).
        After speculative steps a sequence is settled first."""
        mixed, z, b, a = self._project(x)
        mixed = api.ccv_fwd(mixed.t(), self.conv_weight, None, self.conv_state, query_start_loc,
                            lines, has_initial_state).t()
        o = layer.gdr_fwd(*self._heads(mixed), a, b, self.state, query_start_loc, lines,
                          has_initial_state, a_log=self.a_log, dt_bias=self.dt_bias)
        return self._finish(o, z, residual)

    def decode(self, x: torch.Tensor, residual: torch.Tensor, lines: torch.Tensor):
        """One token a row: x, residual (batch, hidden).  After speculative steps a
        row is settled first."""
        mixed, z, b, a = self._project(x)
        mixed = api.ccv_update(mixed, self.conv_state, self.conv_weight, None, "silu", lines)
        o = layer.gdr_update(*self._heads(mixed), a, b, self.state, lines, a_log=self.a_log,
                             dt_bias=self.dt_bias)
        return self._finish(o, z, residual)

    def verify(self, x: torch.Tensor, residual: torch.Tensor, lines: torch.Tensor,
               num_accepted_tokens: Optional[torch.Tensor]):
        """A speculative step: x, residual (batch, steps, hidden) hold the last
        token and the drafts after it.  num_accepted_tokens is what the step
        before kept of its own tokens (None: the first step after a prefill, a
        decode or a settle)."""
        batch, steps = x.shape[:2]
        mixed, z, b, a = self._project(x)
        mixed = api.ccv_update_spec(mixed.transpose(1, 2), self.conv_state, self.conv_weight, None,
                                    "silu", lines, num_accepted_tokens).transpose(1, 2)
        o = layer.gdr_update(*self._heads(mixed), a, b, self.state, lines, num_accepted_tokens,
                             self.step_lines[lines.long()], a_log=self.a_log, dt_bias=self.dt_bias)
        x, residual = self._finish(o, z, residual.flatten(0, 1))
        return x.unflatten(0, (batch, steps)), residual.unflatten(0, (batch, steps))

    def settle(self, lines: torch.Tensor, num_accepted_tokens: torch.Tensor):
        """Ends the rows' speculative steps: their lines become what they are
        after the tokens that the last step kept (1 or more of them)."""
        rows, last = lines.long(), num_accepted_tokens.long() - 1
        self.state[rows] = self.state[self.step_lines[rows, last].long()]
        window = last[:, None] + torch.arange(self.width - 1, device=last.device)
        self.conv_state[rows, :, :self.width - 1] = self.conv_state[rows].gather(
            2, window[:, None].expand(-1, self.mixed, -1))


def serve(device="cuda", hidden: int = 256, vocab: int = 1000, rounds: int = 3, seed: int = 0):
    """Two prompts through a layer, then speculative rounds: three drafts a row
    from a small random draft head, verified against the target head.  Returns the
    tokens that were kept, a list a row."""
    g = torch.Generator(device=device).manual_seed(seed)
    steps, batch = 4, 2
    net = LinearAttentionLayer(hidden, 2, 4, 64, batch, steps, device=device, seed=seed)
    embed = torch.randn(vocab, hidden, generator=g, device=device).to(BF16)
    head = torch.randn(vocab, hidden, generator=g, device=device).to(BF16) * (4 * hidden ** -0.5)
    lines = torch.arange(batch, dtype=torch.int32, device=device)

    prompts = [torch.randint(vocab, (n,), generator=g, device=device) for n in (100, 37)]
    starts = torch.tensor([0, 100, 137], dtype=torch.int32, device=device)
    x = embed[torch.cat(prompts)]
    fresh = torch.zeros(batch, dtype=torch.bool, device=device)
    out, _ = net.prefill(x, x, starts, lines, fresh)
    token = (out[starts[1:].long() - 1] @ head.t()).argmax(-1)  # the first new token, greedily
    kept, count = [[int(t)] for t in token], None
    for _ in range(rounds):
        drafts = torch.randint(vocab, (batch, steps - 1), generator=g, device=device,
                               dtype=torch.int32)
        drafts[:, 0] = (embed[token] @ head.t()).argmax(-1)  # a draft that is sometimes right
        fed = torch.cat([token[:, None], drafts], 1).long()
        out, _ = net.verify(embed[fed], embed[fed], lines, count)
        logits = (out @ head.t()).contiguous()
        tokens, count = layer.spec_verify(
            logits, drafts, torch.rand(batch, steps - 1, generator=g, device=device),
            torch.empty(batch, vocab, device=device).exponential_(generator=g))
        token = tokens.gather(1, count.long()[:, None] - 1)[:, 0].long()
        for row in range(batch):
            kept[row] += tokens[row, :int(count[row])].tolist()
    return kept
