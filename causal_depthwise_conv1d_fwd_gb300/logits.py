"""Python binding of include/ccv_logits.h: the adjustment of logits before tokens
are chosen.  Argument marshalling only, as in :mod:`.layer`, whose words on
streams hold here, too."""
from __future__ import annotations

import struct
from typing import Optional

import torch

from .api import PAD_SLOT_ID, Launch, _elsewhere
from .layer import _BF16, _F32, _I32, _Tensor, _call, _device, _empty, _err, _made, _need, _vector

# struct ccv_logits_args of include/ccv_logits.h, packed into bytes as in :mod:`.layer`.
_LOGITS = struct.Struct("<" + "Qqq" * 2 + "Qq" + "QQQ" + "Qqq" + "QQQ" + "QQq" + "Qqq" + "i" * 9 + "4x")


def logits_process(logits: torch.Tensor, history: Optional[torch.Tensor] = None,
                   history_lengths: Optional[torch.Tensor] = None,
                   prompt_lengths: Optional[torch.Tensor] = None,
                   history_indices: Optional[torch.Tensor] = None,
                   draft_tokens: Optional[torch.Tensor] = None,
                   repetition: Optional[torch.Tensor] = None,
                   frequency: Optional[torch.Tensor] = None,
                   presence: Optional[torch.Tensor] = None,
                   bias_ids: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                   mask: Optional[torch.Tensor] = None, pad_slot_id: int = PAD_SLOT_ID,
                   out: Optional[torch.Tensor] = None, err_count: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Penalties for repeated tokens, a bias list and a grammar's mask, in that order.

    logits (batch, positions, vocab) or (batch, vocab), bf16 or fp32.  history
    (num_lines, size) int32 holds the tokens of requests, prompt first, of
    which history_lengths (num_lines) are there and prompt_lengths (num_lines,
    None: 0) are prompt; row b has line history_indices[b] (None: line b;
    pad_slot_id: the row is skipped).  draft_tokens (batch, positions - 1)
    int32: position i also follows drafts 0 .. i - 1.  repetition, frequency
    and presence (batch) fp32: a token seen before has its logit divided by
    repetition (multiplied, where it is not above 0); one said n > 0 times
    since the prompt loses frequency n + presence.  bias_ids int32 and bias
    fp32 (batch, size) are added; ids outside the vocabulary are passed over.
    mask (batch, positions, ceil(vocab / 32)) or (batch, ceil(vocab / 32))
    int32 has a 1 bit for every token that may follow; the others get -inf.
    Returns out, of logits' shape and bf16 or fp32 (None: a new tensor of
    logits' type; logits itself: in place).
    """
    if stream is not None:
        return _elsewhere(stream, logits, logits_process, logits, history, history_lengths,
                          prompt_lengths, history_indices, draft_tokens, repetition, frequency,
                          presence, bias_ids, bias, mask, pad_slot_id, out, err_count)
    dev, args, out, _ = _marshal(logits, history, history_lengths, prompt_lengths, history_indices,
                                 draft_tokens, repetition, frequency, presence, bias_ids, bias,
                                 mask, pad_slot_id, out, err_count)
    _call("logits_process", args, dev)
    return out


def prepare_logits_process(logits, history=None, history_lengths=None, prompt_lengths=None,
                           history_indices=None, draft_tokens=None, repetition=None,
                           frequency=None, presence=None, bias_ids=None, bias=None, mask=None,
                           pad_slot_id=PAD_SLOT_ID, out=None, err_count=None) -> Launch:
    """Validate and marshal a logits_process call once; returns a reusable Launch."""
    _, args, result, keep = _marshal(logits, history, history_lengths, prompt_lengths,
                                     history_indices, draft_tokens, repetition, frequency, presence,
                                     bias_ids, bias, mask, pad_slot_id, out, err_count)
    return Launch("logits_process", args, result, keep, _made((result,), (out,)))


def _marshal(logits, history, history_lengths, prompt_lengths, history_indices, draft_tokens,
             repetition, frequency, presence, bias_ids, bias, mask, pad_slot_id, out, err_count):
    dev = _device(logits)
    if not (dev >= 0 and logits.dtype in (_BF16, _F32)):
        _need(dev, logits, "logits", _BF16, _F32)
    shape, ls = logits.shape, logits.stride()
    if len(shape) == 2:
        b, n, v = shape[0], 1, shape[1]
        ls = (ls[0], 0, ls[1])
    elif len(shape) == 3:
        b, n, v = shape
    else:
        raise ValueError("logits must be (batch, positions, vocab) or (batch, vocab)")
    if out is None:
        out = _empty(shape, dtype=logits.dtype, device=logits.device)
    elif out is not logits:
        _need(dev, out, "out", _BF16, _F32)
        if out.shape != shape:
            raise ValueError("out must have logits' shape")
    os_ = out.stride() if len(shape) == 3 else (out.stride(0), 0, out.stride(1))
    if v > 1 and not ls[2] == os_[2] == 1:
        raise ValueError("logits and out must have stride 1 along vocab")
    hp = hs = lines = size = 0
    hl = pl = None
    if history is not None:
        if not isinstance(history, _Tensor) or history.dtype is not _I32 or history.get_device() != dev:
            _need(dev, history, "history", _I32)
        if history.dim() != 2 or (history.shape[1] > 1 and history.stride(1) != 1):
            raise ValueError("history must be (num_lines, size) with stride 1 along a line")
        lines, size = history.shape
        # an empty pool has no address, but is not none: any other one, which nothing reads
        hp, hs = history.data_ptr() or logits.data_ptr(), history.stride(0)
        if history_lengths is None:
            raise ValueError("history needs history_lengths")
        hl = _vector(dev, history_lengths, "history_lengths", _I32, lines) or hp
        pl = _vector(dev, prompt_lengths, "prompt_lengths", _I32, lines)
        if history_indices is None and lines < b:
            raise ValueError(f"history has {lines} lines, needs {b}")
    hi = _vector(dev, history_indices, "history_indices", _I32, b)
    dp, ds = 0, (0, 0)
    if draft_tokens is not None:
        _need(dev, draft_tokens, "draft_tokens", _I32)
        if draft_tokens.shape != (b, max(n - 1, 0)):
            raise ValueError("draft_tokens must be (batch, positions - 1)")
        dp, ds = draft_tokens.data_ptr(), draft_tokens.stride()
    rp, fp, pp = (_vector(dev, t, name, _F32, b) for t, name in
                  ((repetition, "repetition"), (frequency, "frequency"), (presence, "presence")))
    ip = bp = bs = count = 0
    if (bias_ids is None) != (bias is None):
        raise ValueError("bias_ids and bias go together")
    if bias is not None:
        _need(dev, bias, "bias", _F32)
        _need(dev, bias_ids, "bias_ids", _I32)
        if bias.dim() != 2 or bias.shape[0] != b or bias_ids.shape != bias.shape:
            raise ValueError("bias_ids and bias must be (batch, size), one shape")
        count = bias.shape[1]
        if count > 1 and not bias.stride(1) == bias_ids.stride(1) == 1:
            raise ValueError("bias_ids and bias must have stride 1 along a row")
        if b > 1 and count and bias.stride(0) != bias_ids.stride(0):
            raise ValueError("bias_ids and bias must have one row stride")
        ip, bp, bs = bias_ids.data_ptr(), bias.data_ptr(), bias.stride(0)
    mp, ms = 0, (0, 0)
    if mask is not None:
        _need(dev, mask, "mask", _I32)
        words = (v + 31) // 32
        if mask.shape != (*shape[:-1], words):
            raise ValueError(f"mask must be {(*shape[:-1], words)}")
        if words > 1 and mask.stride(-1) != 1:
            raise ValueError("mask must have stride 1 along its words")
        mp, ms = mask.data_ptr(), (mask.stride(0), mask.stride(1) if len(shape) == 3 else 0)
    packed = _LOGITS.pack(logits.data_ptr(), ls[0], ls[1], out.data_ptr(), os_[0], os_[1], hp, hs,
                          hi or 0, hl or 0, pl or 0, dp, *ds, rp or 0, fp or 0, pp or 0, ip, bp, bs,
                          mp, *ms, 1 if logits.dtype is _F32 else 0, 1 if out.dtype is _F32 else 0,
                          b, n, v, lines, size, count, pad_slot_id)
    keep = (logits, history, history_lengths, prompt_lengths, history_indices, draft_tokens,
            repetition, frequency, presence, bias_ids, bias, mask, out, err_count)
    return dev, (packed, _err(dev, err_count)), out, keep
