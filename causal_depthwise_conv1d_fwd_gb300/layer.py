"""Python binding of include/ccv_layer.h: the operators a linear-attention layer
runs next to the causal convolution (gated delta rule, norms, draft
verification).  Argument marshalling only, as in :mod:`.api`.

A call with `stream` runs on that stream and allocates its workspace and what it
returns there; its inputs have to be ready on it.  The outputs may be used on the
caller's stream once that one waits for the given one."""
from __future__ import annotations

import struct
from typing import Optional, Tuple

import torch

from . import _lib
from .api import PAD_SLOT_ID, Launch, _check, _elsewhere

_ACTIVATIONS = {None: 0, "silu": 1, "swish": 1, "sigmoid": 2}
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_Tensor, _empty, _empty_like, _ONE = torch.Tensor, torch.empty, torch.empty_like, (1,)

# struct ccv_heads_view and struct ccv_gdr_args of include/ccv_layer.h.  A call
# passes them packed into bytes: building ctypes structures field by field costs
# more than the launch of a decode step.
_VIEW = struct.Struct("<Qqqqq")
_GDR = struct.Struct("<" + "Qqqqq" * 4 + "QQqqq" + "QQQqqqq" + "iiiiifii")

_FUNCTIONS = {}


def _call(name: str, args: tuple, device: int):
    """One call of an entry point on the tensors' device and that device's
    current stream."""
    fn = _FUNCTIONS.get(name)
    if fn is None:
        fn = _FUNCTIONS[name] = getattr(_lib.load(), name)
    if torch._C._cuda_getDevice() != device:
        with torch.cuda.device(device):
            return _call(name, args, device)
    _check(fn(*args, torch._C._cuda_getCurrentRawStream(device)), name)


def _made(tensors: tuple, given: tuple) -> tuple:
    """Those of a plan's tensors that it allocated: the ones not given to it."""
    return tuple(t for t, g in zip(tensors, given) if t is not g)


# The checks below run on every call of a decode step, so the common case is one
# expression per function and _need only finds out what to say.

def _need(dev: int, t: torch.Tensor, name: str, *dtypes):
    """t is a tensor of the call's CUDA device and of one of the types."""
    if not isinstance(t, _Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if dev >= 0 and t.get_device() != dev:
        raise ValueError(f"all tensors of a call must be on one device, got cuda:{dev} and "
                         f"{t.device} ({name})")
    return t


def _device(t) -> int:
    """The device index of a call's first tensor (-1: not a CUDA tensor)."""
    return t.get_device() if isinstance(t, _Tensor) else -1


def _vector(dev: int, t: Optional[torch.Tensor], name: str, dtype, length: int):
    """Pointer of a contiguous vector of at least `length` entries, or None."""
    if t is None:
        return None
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.get_device() != dev:
        _need(dev, t, name, dtype)
    if t.stride() != _ONE:
        raise ValueError(f"{name} must be a contiguous 1-D tensor")
    if t.numel() < length:
        raise ValueError(f"{name} has {t.shape[0]} entries, needs {length}")
    return t.data_ptr()


def _err(dev: int, t: Optional[torch.Tensor]):
    return None if t is None else _need(dev, t, "err_count", _I32).data_ptr()


def _workspace(dev: int, given: Optional[torch.Tensor], size: int, like: torch.Tensor):
    if given is None:
        return _empty(size, dtype=_U8, device=like.device)
    _need(dev, given, "workspace", _U8)
    if given.dim() != 1 or (given.shape[0] and given.stride(0) != 1):
        raise ValueError("workspace must be a contiguous 1-D tensor")
    return given


def _pack_gdr(q, k, v, g, beta, state, scale, qk_l2norm, a_log, dt_bias, pad_slot_id, out, mode):
    """Checks shared by gdr_fwd and gdr_update.  mode: "tokens" for (tokens,
    heads, dim) tensors, "rows" for (batch, heads, dim), "steps" for (batch,
    seqlen, heads, dim).  Returns (device, packed ccv_gdr_args, out, sizes)."""
    if (a_log is None) != (dt_bias is None):
        raise ValueError("a_log and dt_bias go together")
    dev = _device(v)
    dtype = _F32 if a_log is None else _BF16
    if not (dev >= 0 and v.dtype is _BF16 and isinstance(k, _Tensor) and k.dtype is _BF16
            and isinstance(q, _Tensor) and q.dtype is _BF16 and isinstance(g, _Tensor)
            and g.dtype is dtype and isinstance(beta, _Tensor) and beta.dtype is dtype
            and k.get_device() == q.get_device() == g.get_device() == beta.get_device() == dev):
        for t, name in ((v, "v"), (k, "k"), (q, "q")):
            _need(dev, t, name, _BF16)
        for t, name in ((g, "g"), (beta, "beta")):
            _need(dev, t, name, dtype)
    lead = 2 if mode == "steps" else 1
    vs, ks = v.shape, k.shape
    if len(vs) != lead + 2:
        raise ValueError(f"v must have {lead + 2} dimensions, got {len(vs)}")
    if q.shape != ks or ks[:lead] != vs[:lead] or len(ks) != lead + 2:
        raise ValueError("q and k must have the same shape, and v the same tokens")
    hv, dv = vs[lead:]
    hk, dk = ks[lead:]
    heads = vs[:-1]
    if g.shape != heads or beta.shape != heads:
        raise ValueError(f"g and beta must have shape {tuple(heads)}")
    gs = g.stride()
    if beta.stride() != gs:
        raise ValueError("g and beta must have the same strides")
    al = db = sp = lines = 0
    ss = (0, 0, 0, 0)
    if a_log is not None:
        al, db = _vector(dev, a_log, "a_log", _F32, hv), _vector(dev, dt_bias, "dt_bias", _F32, hv)
        if a_log.shape[0] != hv or dt_bias.shape[0] != hv:
            raise ValueError(f"a_log and dt_bias must have {hv} entries")
    if state is not None:
        if not isinstance(state, _Tensor) or state.dtype is not _F32 or state.get_device() != dev:
            _need(dev, state, "state", _F32)
        lines = state.shape[0]
        if state.shape != (lines, hv, dv, dk):
            raise ValueError("state must be (num_lines, num_v_heads, dim_v, dim_k)")
        ss, sp = state.stride(), state.data_ptr()
    if out is None:
        out = _empty_like(v)
    else:
        _need(dev, out, "out", _BF16)
        if out.shape != vs:
            raise ValueError("out must have v's shape")
    if scale is None:
        scale = dk ** -0.5 if dk else 0.0
    end = (al, db, sp, *ss, lines, hk, hv, dk, dv, scale, 1 if qk_l2norm else 0, pad_slot_id)
    pq, pk, pv, po, pg, pb = (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                              g.data_ptr(), beta.data_ptr())
    if mode == "tokens":
        packed = _GDR.pack(pq, 0, *q.stride(), pk, 0, *k.stride(), pv, 0, *v.stride(), po, 0,
                           *out.stride(), pg, pb, 0, *gs, *end)
    elif mode == "steps":
        packed = _GDR.pack(pq, *q.stride(), pk, *k.stride(), pv, *v.stride(), po, *out.stride(),
                           pg, pb, *gs, *end)
    else:
        (q0, q1, q2), (k0, k1, k2), (v0, v1, v2) = q.stride(), k.stride(), v.stride()
        o0, o1, o2 = out.stride()
        packed = _GDR.pack(pq, q0, 0, q1, q2, pk, k0, 0, k1, k2, pv, v0, 0, v1, v2, po, o0, 0, o1,
                           o2, pg, pb, gs[0], 0, gs[1], *end)
    return dev, packed, out, (hk, hv, dk, dv)


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
    if stream is not None:
        return _elsewhere(stream, v, gdr_fwd, q, k, v, g, beta, state, query_start_loc,
                          cache_indices, has_initial_state, scale, qk_l2norm, a_log, dt_bias,
                          pad_slot_id, out, workspace, err_count)
    dev, args, out, scratch, _ = _marshal_gdr_fwd(q, k, v, g, beta, state, query_start_loc,
                                                  cache_indices, has_initial_state, scale,
                                                  qk_l2norm, a_log, dt_bias, pad_slot_id, out,
                                                  workspace, err_count)
    _call("gdr_fwd", args, dev)
    return out


def prepare_gdr_fwd(q, k, v, g, beta, state, query_start_loc, cache_indices=None,
                    has_initial_state=None, scale=None, qk_l2norm=True, a_log=None, dt_bias=None,
                    pad_slot_id=PAD_SLOT_ID, out=None, workspace=None, err_count=None) -> Launch:
    """Validate and marshal a gdr_fwd call once; returns a reusable Launch."""
    _, args, result, scratch, keep = _marshal_gdr_fwd(q, k, v, g, beta, state, query_start_loc,
                                                      cache_indices, has_initial_state, scale,
                                                      qk_l2norm, a_log, dt_bias, pad_slot_id, out,
                                                      workspace, err_count)
    return Launch("gdr_fwd", args, result, keep, _made((result, scratch), (out, workspace)))


def _marshal_gdr_fwd(q, k, v, g, beta, state, query_start_loc, cache_indices, has_initial_state,
                     scale, qk_l2norm, a_log, dt_bias, pad_slot_id, out, workspace, err_count):
    dev, packed, out, sizes = _pack_gdr(q, k, v, g, beta, state, scale, qk_l2norm, a_log, dt_bias,
                                        pad_slot_id, out, "tokens")
    qsl = _vector(dev, query_start_loc, "query_start_loc", _I32, 1)
    if qsl is None:
        raise TypeError("query_start_loc must be a CUDA tensor")
    batch, total = query_start_loc.shape[0] - 1, v.shape[0]
    ci = _vector(dev, cache_indices, "cache_indices", _I32, batch)
    hi = has_initial_state
    if hi is not None:
        if hi.dtype not in (torch.bool, _U8):
            raise TypeError("has_initial_state must be bool or uint8")
        hi = _vector(dev, hi, "has_initial_state", hi.dtype, batch)
    size = _lib.load().gdr_fwd_workspace(total, batch, *sizes)
    scratch = _workspace(dev, workspace, size, v)
    args = (packed, qsl, batch, ci, hi, total, scratch.data_ptr(), scratch.shape[0],
            _err(dev, err_count))
    keep = (q, k, v, g, beta, state, query_start_loc, cache_indices, has_initial_state, a_log,
            dt_bias, out, scratch, err_count)
    return dev, args, out, scratch, keep


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
    if stream is not None:
        return _elsewhere(stream, v, gdr_update, q, k, v, g, beta, state, state_indices,
                          num_accepted_tokens, output_state_indices, scale, qk_l2norm, a_log,
                          dt_bias, pad_slot_id, out, err_count)
    dev, args, out, _ = _marshal_gdr_update(q, k, v, g, beta, state, state_indices,
                                            num_accepted_tokens, output_state_indices, scale,
                                            qk_l2norm, a_log, dt_bias, pad_slot_id, out, err_count)
    _call("gdr_update", args, dev)
    return out


def prepare_gdr_update(q, k, v, g, beta, state, state_indices=None, num_accepted_tokens=None,
                       output_state_indices=None, scale=None, qk_l2norm=True, a_log=None,
                       dt_bias=None, pad_slot_id=PAD_SLOT_ID, out=None, err_count=None) -> Launch:
    """Validate and marshal a gdr_update call once; returns a reusable Launch."""
    _, args, result, keep = _marshal_gdr_update(q, k, v, g, beta, state, state_indices,
                                                num_accepted_tokens, output_state_indices, scale,
                                                qk_l2norm, a_log, dt_bias, pad_slot_id, out,
                                                err_count)
    return Launch("gdr_update", args, result, keep, _made((result,), (out,)))


def _marshal_gdr_update(q, k, v, g, beta, state, state_indices, num_accepted_tokens,
                        output_state_indices, scale, qk_l2norm, a_log, dt_bias, pad_slot_id, out,
                        err_count):
    if state is None:
        raise TypeError("state must be a CUDA tensor")
    rows = v.dim() == 3
    dev, packed, out, _ = _pack_gdr(q, k, v, g, beta, state, scale, qk_l2norm, a_log, dt_bias,
                                    pad_slot_id, out, "rows" if rows else "steps")
    batch, seqlen = v.shape[0], 1 if rows else v.shape[1]
    oidx, ost, steps = output_state_indices, (0, 0), 0
    if oidx is not None:
        _need(dev, oidx, "output_state_indices", _I32)
        if oidx.dim() != 2 or oidx.shape[0] != batch:
            raise ValueError("output_state_indices must be (batch, steps)")
        oidx, ost, steps = oidx.data_ptr(), oidx.stride(), oidx.shape[1]
    args = (packed, _vector(dev, state_indices, "state_indices", _I32, batch),
            _vector(dev, num_accepted_tokens, "num_accepted_tokens", _I32, batch), oidx, *ost,
            steps, batch, seqlen, _err(dev, err_count))
    keep = (q, k, v, g, beta, state, state_indices, num_accepted_tokens, output_state_indices,
            a_log, dt_bias, out, err_count)
    return dev, args, out, keep


def gated_rms_norm(x: torch.Tensor, gate: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                   activation="silu", norm_before_gate: bool = True,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """RMS norm over the last dimension with a gate: norm(x) weight act(gate),
    or norm(x act(gate)) weight with norm_before_gate=False.  x, gate
    (tokens, heads, dim) or (tokens, dim) bf16; activation "silu", "sigmoid"
    or None.  Returns out."""
    if stream is not None:
        return _elsewhere(stream, x, gated_rms_norm, x, gate, weight, eps, activation,
                          norm_before_gate, out)
    dev, args, out, _ = _marshal_gated(x, gate, weight, eps, activation, norm_before_gate, out)
    _call("gated_rms_norm", args, dev)
    return out


def prepare_gated_rms_norm(x, gate, weight, eps=1e-6, activation="silu", norm_before_gate=True,
                           out=None) -> Launch:
    """Validate and marshal a gated_rms_norm call once; returns a reusable Launch."""
    _, args, result, keep = _marshal_gated(x, gate, weight, eps, activation, norm_before_gate, out)
    return Launch("gated_rms_norm", args, result, keep, _made((result,), (out,)))


def _marshal_gated(x, gate, weight, eps, activation, norm_before_gate, out):
    dev = _device(x)
    if not (dev >= 0 and x.dtype is _BF16 and isinstance(gate, _Tensor)
            and gate.dtype is _BF16 and gate.get_device() == dev):
        _need(dev, x, "x", _BF16)
        _need(dev, gate, "gate", _BF16)
    if activation not in _ACTIVATIONS:
        raise ValueError(f"unsupported activation: {activation!r}")
    shape = x.shape
    if len(shape) not in (2, 3) or gate.shape != shape:
        raise ValueError("x and gate must be (tokens, heads, dim) or (tokens, dim), one shape")
    if out is None:
        out = _empty_like(x)
    else:
        _need(dev, out, "out", _BF16)
        if out.shape != shape:
            raise ValueError("out must have x's shape")
    if weight is None:
        raise TypeError("weight must be a CUDA tensor")
    w = _norm_weight(dev, weight, "weight", shape[-1])
    xs, gs, os_ = x.stride(), gate.stride(), out.stride()
    if len(shape) == 2:
        xs, gs, os_ = ((s[0], 0, s[1]) for s in (xs, gs, os_))
        shape = (shape[0], 1, shape[1])
    args = (_VIEW.pack(x.data_ptr(), 0, *xs), _VIEW.pack(gate.data_ptr(), 0, *gs), w,
            _VIEW.pack(out.data_ptr(), 0, *os_), *shape, eps, _ACTIVATIONS[activation],
            1 if norm_before_gate else 0)
    return dev, args, out, (x, gate, weight, out)


def _norm_weight(dev: int, w: Optional[torch.Tensor], name: str, dim: int):
    if w is None:
        return None
    if not isinstance(w, _Tensor) or w.dtype is not _BF16 or w.get_device() != dev:
        _need(dev, w, name, _BF16)
    if w.shape != (dim,) or (dim > 1 and w.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {dim}")
    return w.data_ptr()


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
    if stream is not None:
        return _elsewhere(stream, x, residual_rms_norm, x, residual, weight, post_weight, gate,
                          scale, eps, weight_offset, out, residual_out)
    dev, args, result, _ = _marshal_residual(x, residual, weight, post_weight, gate, scale, eps,
                                             weight_offset, out, residual_out)
    _call("residual_rms_norm", args, dev)
    return result


def prepare_residual_rms_norm(x, residual, weight, post_weight=None, gate=None, scale=1.0,
                              eps=1e-6, weight_offset=0.0, out=None, residual_out=None) -> Launch:
    """Validate and marshal a residual_rms_norm call once; returns a reusable Launch."""
    _, args, result, keep = _marshal_residual(x, residual, weight, post_weight, gate, scale, eps,
                                              weight_offset, out, residual_out)
    return Launch("residual_rms_norm", args, result, keep, _made(result, (out, residual_out)))


def _marshal_residual(x, residual, weight, post_weight, gate, scale, eps, weight_offset, out,
                      residual_out):
    dev = _device(x)
    if not (dev >= 0 and x.dtype is _BF16 and isinstance(residual, _Tensor)
            and residual.dtype in (_BF16, _F32) and residual.get_device() == dev):
        _need(dev, x, "x", _BF16)
        _need(dev, residual, "residual", _BF16, _F32)
    shape, kind = x.shape, residual.dtype
    if len(shape) != 2 or residual.shape != shape:
        raise ValueError("x and residual must be (tokens, dim), one shape")
    tokens, dim = shape
    if weight is None:
        raise TypeError("weight must be a CUDA tensor")
    w, pw = (_norm_weight(dev, weight, "weight", dim),
             _norm_weight(dev, post_weight, "post_weight", dim))
    gp, gs = None, (0, 0)
    if gate is not None:
        _need(dev, gate, "gate", _BF16)
        if gate.shape not in ((dim,), (tokens, dim)):
            raise ValueError("gate must be (dim,) or (tokens, dim)")
        gp, gs = gate.data_ptr(), gate.stride() if gate.dim() == 2 else (0, gate.stride(0))
    if out is None:
        out = _empty_like(x)
    else:
        _need(dev, out, "out", _BF16)
    if residual_out is None:
        residual_out = _empty_like(residual)
    else:
        _need(dev, residual_out, "residual_out", kind)
    if out.shape != shape or residual_out.shape != shape:
        raise ValueError("out and residual_out must have x's shape")
    args = (x.data_ptr(), *x.stride(), residual.data_ptr(), *residual.stride(),
            1 if kind is _F32 else 0, w, pw, gp, *gs, out.data_ptr(), *out.stride(),
            residual_out.data_ptr(), *residual_out.stride(), tokens, dim, scale, eps,
            weight_offset)
    return (dev, args, (out, residual_out),
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
    if stream is not None:
        return _elsewhere(stream, target_logits, spec_verify, target_logits, draft_tokens, uniform,
                          noise, draft_probs, num_drafts, temperature, out_tokens, num_accepted,
                          workspace, err_count)
    dev, args, result, scratch, _ = _marshal_verify(target_logits, draft_tokens, uniform, noise,
                                                    draft_probs, num_drafts, temperature,
                                                    out_tokens, num_accepted, workspace, err_count)
    _call("spec_verify", args, dev)
    return result


def prepare_spec_verify(target_logits, draft_tokens, uniform, noise, draft_probs=None,
                        num_drafts=None, temperature=None, out_tokens=None, num_accepted=None,
                        workspace=None, err_count=None) -> Launch:
    """Validate and marshal a spec_verify call once; returns a reusable Launch."""
    _, args, result, scratch, keep = _marshal_verify(target_logits, draft_tokens, uniform, noise,
                                                     draft_probs, num_drafts, temperature,
                                                     out_tokens, num_accepted, workspace,
                                                     err_count)
    return Launch("spec_verify", args, result, keep,
                  _made((*result, scratch), (out_tokens, num_accepted, workspace)))


def _marshal_verify(target_logits, draft_tokens, uniform, noise, draft_probs, num_drafts,
                    temperature, out_tokens, num_accepted, workspace, err_count):
    dev = _device(target_logits)
    if not (dev >= 0 and target_logits.dtype in (_BF16, _F32)
            and isinstance(draft_tokens, _Tensor) and draft_tokens.dtype is _I32
            and isinstance(uniform, _Tensor) and uniform.dtype is _F32
            and isinstance(noise, _Tensor) and noise.dtype is _F32
            and draft_tokens.get_device() == uniform.get_device() == noise.get_device() == dev):
        _need(dev, target_logits, "target_logits", _BF16, _F32)
        _need(dev, draft_tokens, "draft_tokens", _I32)
        _need(dev, uniform, "uniform", _F32)
        _need(dev, noise, "noise", _F32)
    if target_logits.dim() != 3 or draft_tokens.dim() != 2:
        raise ValueError("target_logits must be (batch, drafts + 1, vocab), draft_tokens "
                         "(batch, drafts)")
    batch, drafts = draft_tokens.shape
    vocab = target_logits.shape[2]
    if target_logits.shape != (batch, drafts + 1, vocab):
        raise ValueError("target_logits must have one position more than there are drafts")
    if uniform.shape != (batch, drafts):
        raise ValueError("uniform must have draft_tokens' shape")
    if noise.shape != (batch, vocab):
        raise ValueError("noise must be (batch, vocab)")
    ts, ns = target_logits.stride(), noise.stride()
    pp, ps = None, (0, 0, 1)
    if draft_probs is not None:
        _need(dev, draft_probs, "draft_probs", _F32)
        if draft_probs.shape != (batch, drafts, vocab):
            raise ValueError("draft_probs must be (batch, drafts, vocab)")
        pp, ps = draft_probs.data_ptr(), draft_probs.stride()
    if vocab > 1 and not ts[2] == ns[1] == ps[2] == 1:
        raise ValueError("target_logits, noise and draft_probs must have stride 1 along vocab")
    nd = _vector(dev, num_drafts, "num_drafts", _I32, batch)
    temp = _vector(dev, temperature, "temperature", _F32, batch)
    device = noise.device
    if out_tokens is None:
        out_tokens = _empty((batch, drafts + 1), dtype=_I32, device=device)
    else:
        _need(dev, out_tokens, "out_tokens", _I32)
        if out_tokens.shape != (batch, drafts + 1) or not out_tokens.is_contiguous():
            raise ValueError("out_tokens must be a contiguous (batch, drafts + 1)")
    if num_accepted is None:
        num_accepted = _empty(batch, dtype=_I32, device=device)
    count = _vector(dev, num_accepted, "num_accepted", _I32, batch)
    size = _lib.load().spec_verify_workspace(batch, drafts, vocab)
    scratch = _workspace(dev, workspace, size, noise)
    args = (target_logits.data_ptr(), 1 if target_logits.dtype is _F32 else 0, ts[0], ts[1],
            draft_tokens.data_ptr(), *draft_tokens.stride(), pp, ps[0], ps[1], nd, temp,
            uniform.data_ptr(), *uniform.stride(), noise.data_ptr(), ns[0], out_tokens.data_ptr(),
            count, batch, drafts, vocab, scratch.data_ptr(), scratch.shape[0],
            _err(dev, err_count))
    keep = (target_logits, draft_tokens, uniform, noise, draft_probs, num_drafts, temperature,
            out_tokens, num_accepted, scratch, err_count)
    return dev, args, (out_tokens, num_accepted), scratch, keep
