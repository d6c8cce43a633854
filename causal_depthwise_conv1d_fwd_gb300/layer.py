"""Python binding of include/ccv_layer.h: the operators a linear-attention layer
runs next to the causal convolution (gated delta rule, norms, draft
verification).  Argument marshalling only, as in :mod:`.api`."""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _lib
from .api import PAD_SLOT_ID, Launch, _index_vector, _need_cuda, _ptr

_ACTIVATIONS = {None: 0, "silu": 1, "swish": 1, "sigmoid": 2}


class ScratchLaunch(Launch):
    """A Launch whose call uses a workspace.  One that the binding allocated
    belongs to the plan: on a stream other than its own the allocator is told,
    and the plan must not run on two streams at once."""

    def __init__(self, name, args, result, keep, scratch: torch.Tensor):
        super().__init__(name, args, result, keep)
        self._scratch = scratch

    def _launch(self, stream):
        result = super()._launch(stream)
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=self.device)
            self._scratch.record_stream(stream)
        return result


def _workspace(given: Optional[torch.Tensor], size: int, device) -> torch.Tensor:
    if given is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    _need_cuda(given, "workspace", torch.uint8)
    if given.dim() != 1 or (given.numel() and given.stride(0) != 1):
        raise ValueError("workspace must be a contiguous 1-D tensor")
    return given


def _view(t: torch.Tensor, has_row: bool) -> _lib.HeadsView:
    st = t.stride()
    return _lib.HeadsView(t.data_ptr(), *(st if has_row else (0, *st)))


def _gdr_args(q, k, v, g, beta, state, scale, qk_l2norm, a_log, dt_bias, pad_slot_id, out,
              has_row: bool):
    """Checks shared by gdr_fwd and gdr_update; (..., heads, dim) tensors."""
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _need_cuda(t, name, torch.bfloat16)
        if t.dim() != (4 if has_row else 3):
            raise ValueError(f"{name} must be ({'batch, seqlen' if has_row else 'total_tokens'}, "
                             "heads, dim)")
    lead = v.shape[:-2]
    hv, dv = v.shape[-2:]
    hk, dk = k.shape[-2:]
    if q.shape != k.shape or k.shape[:-2] != lead:
        raise ValueError("q and k must have the same shape, and v the same tokens")
    if (a_log is None) != (dt_bias is None):
        raise ValueError("a_log and dt_bias go together")
    gate_dtype = torch.float32 if a_log is None else torch.bfloat16
    for t, name in ((g, "g"), (beta, "beta")):
        _need_cuda(t, name, gate_dtype)
        if t.shape != (*lead, hv):
            raise ValueError(f"{name} must have shape {(*lead, hv)}, got {tuple(t.shape)}")
    if beta.stride() != g.stride():
        raise ValueError("g and beta must have the same strides")
    if a_log is not None:
        for t, name in ((a_log, "a_log"), (dt_bias, "dt_bias")):
            _index_vector(t, name, torch.float32, hv)
            if t.numel() != hv:
                raise ValueError(f"{name} must have {hv} entries, got {t.numel()}")
    if state is not None:
        _need_cuda(state, "state", torch.float32)
        if state.dim() != 4 or state.shape[1:] != (hv, dv, dk):
            raise ValueError("state must be (num_lines, num_v_heads, dim_v, dim_k)")
        ss, lines = state.stride(), state.shape[0]
    else:
        ss, lines = (0, 0, 0, 0), 0
    if out is None:
        out = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    else:
        _need_cuda(out, "out", torch.bfloat16)
        if out.shape != v.shape:
            raise ValueError("out must have v's shape")
    gs = g.stride() if has_row else (0, *g.stride())
    args = _lib.GdrArgs(_view(q, has_row), _view(k, has_row), _view(v, has_row),
                        _view(out, has_row), g.data_ptr(), beta.data_ptr(), *gs,
                        a_log.data_ptr() if a_log is not None else None,
                        dt_bias.data_ptr() if dt_bias is not None else None,
                        state.data_ptr() if state is not None else None, *ss, lines, hk, hv, dk, dv,
                        dk ** -0.5 if scale is None and dk else float(scale or 0.0),
                        int(bool(qk_l2norm)), pad_slot_id)
    return args, out


def gdr_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
            beta: torch.Tensor, state: Optional[torch.Tensor], query_start_loc: torch.Tensor,
            cache_indices: Optional[torch.Tensor] = None,
            has_initial_state: Optional[torch.Tensor] = None, scale: Optional[float] = None,
            qk_l2norm: bool = True, a_log: Optional[torch.Tensor] = None,
            dt_bias: Optional[torch.Tensor] = None, pad_slot_id: int = PAD_SLOT_ID,
            out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
            err_count: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gated delta rule over varlen sequences (prefill), states updated in place.

    q, k are (total_tokens, num_k_heads, dim_k), v is (total_tokens,
    num_v_heads, dim_v), bf16 with any strides -- slices of a channel-last
    ccv_fwd output, for example.  g and beta are (total_tokens, num_v_heads):
    fp32 decay logarithm and write strength, or with a_log and dt_bias the
    bf16 projections they come from.  state is (num_lines, num_v_heads, dim_v,
    dim_k) fp32.  scale defaults to dim_k ** -0.5.  Returns out.
    """
    return prepare_gdr_fwd(q, k, v, g, beta, state, query_start_loc, cache_indices,
                           has_initial_state, scale, qk_l2norm, a_log, dt_bias, pad_slot_id, out,
                           workspace, err_count)(stream)


def prepare_gdr_fwd(q, k, v, g, beta, state, query_start_loc, cache_indices=None,
                    has_initial_state=None, scale=None, qk_l2norm=True, a_log=None, dt_bias=None,
                    pad_slot_id=PAD_SLOT_ID, out=None, workspace=None, err_count=None) -> Launch:
    """Validate and marshal a gdr_fwd call once; returns a reusable Launch."""
    args, out = _gdr_args(q, k, v, g, beta, state, scale, qk_l2norm, a_log, dt_bias, pad_slot_id,
                          out, has_row=False)
    qsl = _index_vector(query_start_loc, "query_start_loc", torch.int32, 1)
    batch, total = qsl.numel() - 1, v.shape[0]
    ci = _index_vector(cache_indices, "cache_indices", torch.int32, batch)
    hi = has_initial_state
    if hi is not None:
        if hi.dtype not in (torch.bool, torch.uint8):
            raise TypeError("has_initial_state must be bool or uint8")
        hi = _index_vector(hi, "has_initial_state", hi.dtype, batch)
    _need_cuda(err_count, "err_count", torch.int32)
    size = _lib.load().gdr_fwd_workspace(total, batch, args.num_k_heads, args.num_v_heads,
                                         args.dim_k, args.dim_v)
    scratch = _workspace(workspace, size, v.device)
    call = (ctypes.byref(args), _ptr(qsl), batch, _ptr(ci), _ptr(hi), total, _ptr(scratch),
            scratch.numel(), _ptr(err_count))
    return ScratchLaunch("gdr_fwd", call, out, (args, q, k, v, g, beta, state, qsl, ci, hi, a_log,
                                                dt_bias, out, scratch, err_count), scratch)


def gdr_update(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
               beta: torch.Tensor, state: torch.Tensor,
               state_indices: Optional[torch.Tensor] = None,
               num_accepted_tokens: Optional[torch.Tensor] = None,
               output_state_indices: Optional[torch.Tensor] = None,
               scale: Optional[float] = None, qk_l2norm: bool = True,
               a_log: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
               pad_slot_id: int = PAD_SLOT_ID, out: Optional[torch.Tensor] = None,
               err_count: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gated delta rule over the new tokens of each row (decode, speculative verify).

    q, k (batch, num_k_heads, dim_k) and v (batch, num_v_heads, dim_v), or
    with a seqlen axis after batch; g and beta alike without dim.  The row's
    state line state_indices[b] is updated in place; with
    output_state_indices (batch, steps >= seqlen) the state after token t goes
    to line [b, t] instead (-1: none), and with num_accepted_tokens the row
    starts from line [b, num_accepted_tokens[b] - 1].  Returns out with v's
    rank.
    """
    return prepare_gdr_update(q, k, v, g, beta, state, state_indices, num_accepted_tokens,
                              output_state_indices, scale, qk_l2norm, a_log, dt_bias, pad_slot_id,
                              out, err_count)(stream)


def prepare_gdr_update(q, k, v, g, beta, state, state_indices=None, num_accepted_tokens=None,
                       output_state_indices=None, scale=None, qk_l2norm=True, a_log=None,
                       dt_bias=None, pad_slot_id=PAD_SLOT_ID, out=None, err_count=None) -> Launch:
    """Validate and marshal a gdr_update call once; returns a reusable Launch."""
    squeeze = v.dim() == 3
    if squeeze:
        q, k, v, g, beta = (t.unsqueeze(1) for t in (q, k, v, g, beta))
        out = out.unsqueeze(1) if out is not None else None
    if state is None:
        raise TypeError("state must be a CUDA tensor")
    args, out = _gdr_args(q, k, v, g, beta, state, scale, qk_l2norm, a_log, dt_bias, pad_slot_id,
                          out, has_row=True)
    batch, seqlen = v.shape[:2]
    idx = _index_vector(state_indices, "state_indices", torch.int32, batch)
    nacc = _index_vector(num_accepted_tokens, "num_accepted_tokens", torch.int32, batch)
    oidx = output_state_indices
    _need_cuda(oidx, "output_state_indices", torch.int32)
    if oidx is not None and (oidx.dim() != 2 or oidx.shape[0] != batch):
        raise ValueError("output_state_indices must be (batch, steps)")
    _need_cuda(err_count, "err_count", torch.int32)
    ost = oidx.stride() if oidx is not None else (0, 0)
    call = (ctypes.byref(args), _ptr(idx), _ptr(nacc), _ptr(oidx), *ost,
            oidx.shape[1] if oidx is not None else 0, batch, seqlen, _ptr(err_count))
    return Launch("gdr_update", call, out.squeeze(1) if squeeze else out,
                  (args, q, k, v, g, beta, state, idx, nacc, oidx, a_log, dt_bias, out, err_count))


def gated_rms_norm(x: torch.Tensor, gate: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                   activation="silu", norm_before_gate: bool = True,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """RMS norm over the last dimension with a gate: norm(x) weight act(gate),
    or norm(x act(gate)) weight with norm_before_gate=False.  x, gate
    (tokens, heads, dim) or (tokens, dim) bf16; activation "silu", "sigmoid"
    or None.  Returns out."""
    return prepare_gated_rms_norm(x, gate, weight, eps, activation, norm_before_gate, out)(stream)


def prepare_gated_rms_norm(x, gate, weight, eps=1e-6, activation="silu", norm_before_gate=True,
                           out=None) -> Launch:
    """Validate and marshal a gated_rms_norm call once; returns a reusable Launch."""
    _need_cuda(x, "x", torch.bfloat16)
    _need_cuda(gate, "gate", torch.bfloat16)
    if activation not in _ACTIVATIONS:
        raise ValueError(f"unsupported activation: {activation!r}")
    if x.dim() not in (2, 3) or gate.shape != x.shape:
        raise ValueError("x and gate must be (tokens, heads, dim) or (tokens, dim), one shape")
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    else:
        _need_cuda(out, "out", torch.bfloat16)
        if out.shape != x.shape:
            raise ValueError("out must have x's shape")
    weight = _norm_weight(weight, "weight", x.shape[-1])
    tokens, heads, dim = x.shape if x.dim() == 3 else (x.shape[0], 1, x.shape[1])

    def view(t):
        st = t.stride()
        return _lib.HeadsView(t.data_ptr(), 0, st[0], st[1] if t.dim() == 3 else 0, st[-1])

    vx, vg, vo = view(x), view(gate), view(out)
    call = (ctypes.byref(vx), ctypes.byref(vg), _ptr(weight), ctypes.byref(vo), tokens, heads, dim,
            float(eps), _ACTIVATIONS[activation], int(bool(norm_before_gate)))
    return Launch("gated_rms_norm", call, out, (vx, vg, vo, x, gate, weight, out))


def _norm_weight(w: Optional[torch.Tensor], name: str, dim: int):
    if w is None:
        return None
    _need_cuda(w, name, torch.bfloat16)
    if w.shape != (dim,) or (dim > 1 and w.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {dim}")
    return w


def residual_rms_norm(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor,
                      post_weight: Optional[torch.Tensor] = None,
                      gate: Optional[torch.Tensor] = None, scale: float = 1.0, eps: float = 1e-6,
                      weight_offset: float = 0.0, out: Optional[torch.Tensor] = None,
                      residual_out: Optional[torch.Tensor] = None,
                      stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """What lies between two blocks, in one pass: h = residual + scale * t with
    t = x, normalised with post_weight and multiplied by gate when they are
    given; returns (norm(h) * (weight + weight_offset), h).

    x (tokens, dim) bf16; residual bf16 or fp32; gate (dim,) or (tokens, dim).
    residual_out may be residual and out may be x (in place).
    """
    return prepare_residual_rms_norm(x, residual, weight, post_weight, gate, scale, eps,
                                     weight_offset, out, residual_out)(stream)


def prepare_residual_rms_norm(x, residual, weight, post_weight=None, gate=None, scale=1.0,
                              eps=1e-6, weight_offset=0.0, out=None, residual_out=None) -> Launch:
    """Validate and marshal a residual_rms_norm call once; returns a reusable Launch."""
    _need_cuda(x, "x", torch.bfloat16)
    _need_cuda(residual, "residual")
    if residual.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"residual must be bfloat16 or float32, got {residual.dtype}")
    if x.dim() != 2 or residual.shape != x.shape:
        raise ValueError("x and residual must be (tokens, dim), one shape")
    tokens, dim = x.shape
    if weight is None:
        raise TypeError("weight must be a CUDA tensor")
    weight = _norm_weight(weight, "weight", dim)
    post_weight = _norm_weight(post_weight, "post_weight", dim)
    gst = (0, 0)
    if gate is not None:
        _need_cuda(gate, "gate", torch.bfloat16)
        if gate.shape not in ((dim,), (tokens, dim)):
            raise ValueError("gate must be (dim,) or (tokens, dim)")
        gst = (0, gate.stride(0)) if gate.dim() == 1 else gate.stride()
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if residual_out is None:
        residual_out = torch.empty(x.shape, dtype=residual.dtype, device=x.device)
    _need_cuda(out, "out", torch.bfloat16)
    _need_cuda(residual_out, "residual_out", residual.dtype)
    if out.shape != x.shape or residual_out.shape != x.shape:
        raise ValueError("out and residual_out must have x's shape")
    call = (_ptr(x), *x.stride(), _ptr(residual), *residual.stride(),
            int(residual.dtype == torch.float32), _ptr(weight), _ptr(post_weight), _ptr(gate), *gst,
            _ptr(out), *out.stride(), _ptr(residual_out), *residual_out.stride(), tokens, dim,
            float(scale), float(eps), float(weight_offset))
    return Launch("residual_rms_norm", call, (out, residual_out),
                  (x, residual, weight, post_weight, gate, out, residual_out))


def spec_verify(target_logits: torch.Tensor, draft_tokens: torch.Tensor, uniform: torch.Tensor,
                noise: torch.Tensor, draft_probs: Optional[torch.Tensor] = None,
                num_drafts: Optional[torch.Tensor] = None,
                temperature: Optional[torch.Tensor] = None,
                out_tokens: Optional[torch.Tensor] = None,
                num_accepted: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None,
                err_count: Optional[torch.Tensor] = None,
                stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Accept or reject drafted tokens against the target's probabilities.

    target_logits (batch, drafts + 1, vocab) bf16 or fp32, draft_tokens
    (batch, drafts) int32, uniform (batch, drafts) fp32 in [0, 1), noise
    (batch, vocab) fp32 exponentially distributed, draft_probs (batch, drafts,
    vocab) fp32 or None (certain drafts), num_drafts (batch) int32 or None,
    temperature (batch) fp32 or None (0: greedy).  Returns (tokens, count):
    int32 (batch, drafts + 1) with the kept drafts, the next token, then -1,
    and int32 (batch) kept drafts + 1 -- the num_accepted_tokens of the next
    ccv_update_spec and gdr_update.
    """
    return prepare_spec_verify(target_logits, draft_tokens, uniform, noise, draft_probs, num_drafts,
                               temperature, out_tokens, num_accepted, workspace, err_count)(stream)


def prepare_spec_verify(target_logits, draft_tokens, uniform, noise, draft_probs=None,
                        num_drafts=None, temperature=None, out_tokens=None, num_accepted=None,
                        workspace=None, err_count=None) -> Launch:
    """Validate and marshal a spec_verify call once; returns a reusable Launch."""
    _need_cuda(target_logits, "target_logits")
    if target_logits.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"target_logits must be bfloat16 or float32, got {target_logits.dtype}")
    _need_cuda(draft_tokens, "draft_tokens", torch.int32)
    _need_cuda(uniform, "uniform", torch.float32)
    _need_cuda(noise, "noise", torch.float32)
    _need_cuda(draft_probs, "draft_probs", torch.float32)
    if target_logits.dim() != 3 or draft_tokens.dim() != 2:
        raise ValueError("target_logits must be (batch, drafts + 1, vocab), draft_tokens "
                         "(batch, drafts)")
    (batch, drafts), vocab = draft_tokens.shape, target_logits.shape[2]
    if target_logits.shape[:2] != (batch, drafts + 1):
        raise ValueError("target_logits must have one position more than there are drafts")
    if uniform.shape != draft_tokens.shape:
        raise ValueError("uniform must have draft_tokens' shape")
    if noise.shape != (batch, vocab):
        raise ValueError("noise must be (batch, vocab)")
    if draft_probs is not None and draft_probs.shape != (batch, drafts, vocab):
        raise ValueError("draft_probs must be (batch, drafts, vocab)")
    for t, name in ((target_logits, "target_logits"), (noise, "noise"),
                    (draft_probs, "draft_probs")):
        if t is not None and vocab > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name} must have stride 1 along vocab")
    nd = _index_vector(num_drafts, "num_drafts", torch.int32, batch)
    temp = _index_vector(temperature, "temperature", torch.float32, batch)
    if out_tokens is None:
        out_tokens = torch.empty(batch, drafts + 1, dtype=torch.int32, device=draft_tokens.device)
    if num_accepted is None:
        num_accepted = torch.empty(batch, dtype=torch.int32, device=draft_tokens.device)
    _need_cuda(out_tokens, "out_tokens", torch.int32)
    if out_tokens.shape != (batch, drafts + 1) or not out_tokens.is_contiguous():
        raise ValueError("out_tokens must be a contiguous (batch, drafts + 1)")
    _index_vector(num_accepted, "num_accepted", torch.int32, batch)
    _need_cuda(err_count, "err_count", torch.int32)
    size = _lib.load().spec_verify_workspace(batch, drafts, vocab)
    scratch = _workspace(workspace, size, draft_tokens.device)
    pst = draft_probs.stride()[:2] if draft_probs is not None else (0, 0)
    call = (_ptr(target_logits), int(target_logits.dtype == torch.float32),
            *target_logits.stride()[:2], _ptr(draft_tokens), *draft_tokens.stride(),
            _ptr(draft_probs), *pst, _ptr(nd), _ptr(temp), _ptr(uniform), *uniform.stride(),
            _ptr(noise), noise.stride(0), _ptr(out_tokens), _ptr(num_accepted), batch, drafts,
            vocab, _ptr(scratch), scratch.numel(), _ptr(err_count))
    return ScratchLaunch("spec_verify", call, (out_tokens, num_accepted),
                         (target_logits, draft_tokens, uniform, noise, draft_probs, nd, temp,
                          out_tokens, num_accepted, scratch, err_count), scratch)
