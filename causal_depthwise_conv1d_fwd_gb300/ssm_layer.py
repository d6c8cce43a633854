"""A selective state space layer on the library's operators: an example of how they are
used together, and a small program for tests and profilers.

One layer takes normalised hidden states and the residual stream and returns both
for the next block:

    mixed, z, dt = h W_in
    x, B, C      = split(SiLU(causal_conv(mixed)))       ccv_fwd / ccv_update / ccv_update_spec
    y            = scan(x, dt, A, B, C) + D x            ssm_fwd / ssm_update
    u            = norm(y SiLU(z)) W_out                 gated_rms_norm
    h, residual  = norm(residual + u), residual + u      residual_rms_norm

The matrix products are torch's.  State lines, the lines of a speculative step and
`settle` are as in :mod:`.linear_layer`.  `serve` puts logits_process between the
target's logits and spec_verify: penalties for what a request has said, and a
mask of the tokens that may follow.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import api, layer, logits, ssm

BF16 = torch.bfloat16


class SelectiveStateLayer:
    """Weights and state pools of one layer; `steps` tokens at most a row and step."""

    def __init__(self, hidden: int, heads: int, head_dim: int, groups: int, dim_state: int,
                 lines: int, steps: int = 1, width: int = 4, device="cuda", seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.p, self.groups, self.n, self.width = heads, head_dim, groups, dim_state, width
        self.inner = heads * head_dim
        self.mixed = self.inner + 2 * groups * dim_state

        def weight(*shape, std):
            return (std * torch.randn(*shape, generator=g)).to(BF16).to(device)

        self.w_in = weight(self.mixed + self.inner + heads, hidden, std=hidden ** -0.5)
        self.w_out = weight(hidden, self.inner, std=self.inner ** -0.5)
        self.conv_weight = weight(self.mixed, width, std=width ** -0.5)
        self.norm_weight = 1 + weight(self.inner, std=0.1)
        self.out_norm_weight = weight(hidden, std=0.1)  # used as 1 + weight
        self.A = -(1 + 15 * torch.rand(heads, generator=g)).to(device)
        self.D = (1 + 0.1 * torch.randn(heads, generator=g)).to(device)
        self.dt_bias = (torch.randn(heads, generator=g) - 3).to(device)
        # dim contiguous, as the convolution's decode kernel likes it; room for `steps` inputs
        self.conv_state = torch.zeros(lines, width - 2 + steps, self.mixed, dtype=BF16,
                                      device=device).transpose(1, 2)
        self.state = torch.zeros(lines * (1 + steps), heads, head_dim, dim_state, device=device)
        self.step_lines = (lines + torch.arange(lines * steps, dtype=torch.int32, device=device)
                           ).reshape(lines, steps)

    def _project(self, h):
        """(.., hidden) -> mixed, z, dt."""
        return (h @ self.w_in.t()).split([self.mixed, self.inner, self.heads], -1)

    def _split(self, mixed):
        """(.., mixed) -> x, B, C as views of it."""
        x, b, c = mixed.split([self.inner, self.groups * self.n, self.groups * self.n], -1)
        return (x.unflatten(-1, (self.heads, self.p)), b.unflatten(-1, (self.groups, self.n)),
                c.unflatten(-1, (self.groups, self.n)))

    def _finish(self, y, z, residual) -> Tuple[torch.Tensor, torch.Tensor]:
        y = layer.gated_rms_norm(y.reshape(-1, self.inner), z.reshape(-1, self.inner),
                                 self.norm_weight, norm_before_gate=False)
        return layer.residual_rms_norm(y @ self.w_out.t(), residual, self.out_norm_weight,
                                       weight_offset=1.0)

    def prefill(self, h: torch.Tensor, residual: torch.Tensor, query_start_loc: torch.Tensor,
                lines: torch.Tensor, has_initial_state: torch.Tensor):
        """Varlen prompts, or their next parts: h, residual (total_tokens, hidden).
        After speculative steps a sequence is settled first."""
        mixed, z, dt = self._project(h)
        mixed = api.ccv_fwd(mixed.t(), self.conv_weight, None, self.conv_state, query_start_loc,
                            lines, has_initial_state).t()
        x, b, c = self._split(mixed)
        y = ssm.ssm_fwd(x, dt, self.A, b, c, self.state, query_start_loc, lines, has_initial_state,
                        D=self.D, dt_bias=self.dt_bias)
        return self._finish(y, z, residual)

    def decode(self, h: torch.Tensor, residual: torch.Tensor, lines: torch.Tensor):
        """One token a row: h, residual (batch, hidden).  After speculative steps a
        row is settled first."""
        mixed, z, dt = self._project(h)
        mixed = api.ccv_update(mixed, self.conv_state, self.conv_weight, None, "silu", lines)
        x, b, c = self._split(mixed)
        y = ssm.ssm_update(x, dt, self.A, b, c, self.state, lines, D=self.D, dt_bias=self.dt_bias)
        return self._finish(y, z, residual)

    def verify(self, h: torch.Tensor, residual: torch.Tensor, lines: torch.Tensor,
               num_accepted_tokens: Optional[torch.Tensor]):
        """A speculative step: h, residual (batch, steps, hidden) hold the last
        token and the drafts after it.  num_accepted_tokens is what the step
        before kept of its own tokens (None: the first step after a prefill, a
        decode or a settle)."""
        batch, steps = h.shape[:2]
        mixed, z, dt = self._project(h)
        mixed = api.ccv_update_spec(mixed.transpose(1, 2), self.conv_state, self.conv_weight, None,
                                    "silu", lines, num_accepted_tokens).transpose(1, 2)
        x, b, c = self._split(mixed)
        y = ssm.ssm_update(x, dt, self.A, b, c, self.state, lines, num_accepted_tokens,
                           self.step_lines[lines.long()], D=self.D, dt_bias=self.dt_bias)
        h, residual = self._finish(y, z, residual.flatten(0, 1))
        return h.unflatten(0, (batch, steps)), residual.unflatten(0, (batch, steps))

    def settle(self, lines: torch.Tensor, num_accepted_tokens: torch.Tensor):
        """Ends the rows' speculative steps: their lines become what they are
        after the tokens that the last step kept (1 or more of them)."""
        rows, last = lines.long(), num_accepted_tokens.long() - 1
        self.state[rows] = self.state[self.step_lines[rows, last].long()]
        window = last[:, None] + torch.arange(self.width - 1, device=last.device)
        self.conv_state[rows, :, :self.width - 1] = self.conv_state[rows].gather(
            2, window[:, None].expand(-1, self.mixed, -1))


def serve(device="cuda", hidden: int = 256, vocab: int = 1000, rounds: int = 4, seed: int = 0):
    """Two prompts through a layer, then speculative rounds: three drafts a row
    from a small random draft head, verified against the target head's logits
    after penalties and a mask that leaves the even tokens.  Returns the tokens
    that were kept, a list a row."""
    g = torch.Generator(device=device).manual_seed(seed)
    steps, batch = 4, 2
    net = SelectiveStateLayer(hidden, 4, 64, 1, 128, batch, steps, device=device, seed=seed)
    embed = torch.randn(vocab, hidden, generator=g, device=device).to(BF16)
    head = torch.randn(vocab, hidden, generator=g, device=device).to(BF16) * (4 * hidden ** -0.5)
    lines = torch.arange(batch, dtype=torch.int32, device=device)
    even = torch.full((batch, steps, (vocab + 31) // 32), 0x55555555, dtype=torch.int32, device=device)
    penalties = {"repetition": torch.full((batch,), 1.2, device=device),
                 "presence": torch.full((batch,), 0.5, device=device)}

    prompts = [torch.randint(vocab, (n,), generator=g, device=device) for n in (100, 37)]
    history = torch.zeros(batch, 256, dtype=torch.int32, device=device)
    for row, tokens in enumerate(prompts):
        history[row, :len(tokens)] = tokens
    told = torch.tensor([100, 37], dtype=torch.int32, device=device)
    prompt = told.clone()
    starts = torch.tensor([0, 100, 137], dtype=torch.int32, device=device)
    h = embed[torch.cat(prompts)]
    fresh = torch.zeros(batch, dtype=torch.bool, device=device)
    out, _ = net.prefill(h, h, starts, lines, fresh)
    first = (out[starts[1:].long() - 1] @ head.t()).contiguous()
    logits.logits_process(first, history, told, prompt, mask=even[:, 0], out=first, **penalties)
    token = first.argmax(-1)  # the first new token, greedily
    kept, count = [[int(t)] for t in token], None
    for row in range(batch):
        history[row, told[row]] = token[row]
    told += 1
    for _ in range(rounds):
        drafts = torch.randint(vocab // 2, (batch, steps - 1), generator=g, device=device,
                               dtype=torch.int32) * 2
        drafts[:, 0] = (embed[token] @ head.t()).argmax(-1)  # a draft that is sometimes right
        fed = torch.cat([token[:, None], drafts], 1).long()
        out, _ = net.verify(embed[fed], embed[fed], lines, count)
        target = logits.logits_process((out @ head.t()).contiguous(), history, told, prompt,
                                       draft_tokens=drafts, mask=even, **penalties)
        tokens, count = layer.spec_verify(
            target, drafts, torch.rand(batch, steps - 1, generator=g, device=device),
            torch.empty(batch, vocab, device=device).exponential_(generator=g))
        token = tokens.gather(1, count.long()[:, None] - 1)[:, 0].long()
        for row in range(batch):
            n = int(count[row])
            history[row, int(told[row]):int(told[row]) + n] = tokens[row, :n]
            kept[row] += tokens[row, :n].tolist()
        told += count
    return kept
