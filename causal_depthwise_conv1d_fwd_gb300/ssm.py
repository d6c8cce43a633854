"""Python binding of include/ccv_ssm.h: the selective state space scan over
prompts and over the new tokens of each row.  Argument marshalling only, as in
:mod:`.layer`, whose words on streams hold here, too."""
from __future__ import annotations

import struct
from typing import Optional, Tuple

import torch

from . import _lib
from .api import PAD_SLOT_ID, Launch, _elsewhere
from .layer import (_BF16, _F32, _I32, _U8, _Tensor, _call, _device, _empty_like, _err, _made,
                    _need, _vector, _workspace)

# struct ccv_ssm_args of include/ccv_ssm.h, packed into bytes as in :mod:`.layer`.
_SSM = struct.Struct("<" + "Qqqqq" * 5 + "Qqqq" + "QQQ" + "Qqqqq" + "ff" + "i" * 9 + "4x")
_NO_LIMIT = (0.0, float("inf"))
_MAX = torch.finfo(torch.float32).max


def _pack_ssm(x, dt, A, B, C, state, D, z, dt_bias, dt_softplus, dt_limit, pad_slot_id, out, lead):
    """Checks shared by ssm_fwd and ssm_update; `lead` axes come before the
    heads.  Returns (device, packed ccv_ssm_args, out, sizes)."""
    dev = _device(x)
    if not (dev >= 0 and x.dtype is _BF16 and isinstance(B, _Tensor) and B.dtype is _BF16
            and isinstance(C, _Tensor) and C.dtype is _BF16 and isinstance(dt, _Tensor)
            and (dt.dtype is _BF16 or dt.dtype is _F32) and isinstance(A, _Tensor)
            and A.dtype is _F32 and B.get_device() == C.get_device() == dt.get_device()
            == A.get_device() == dev):
        for t, name in ((x, "x"), (B, "B"), (C, "C")):
            _need(dev, t, name, _BF16)
        _need(dev, dt, "dt", _BF16, _F32)
        _need(dev, A, "A", _F32)
    heads, xs = dt.shape, x.shape
    channels = len(xs) == lead + 1  # one channel a head, without an axis for it
    if len(heads) != lead + 1 or xs[:lead + 1] != heads or len(xs) > lead + 2:
        raise ValueError(f"x must be {tuple(heads)} with or without a head_dim axis, as dt; got {tuple(xs)}")
    h, p = heads[lead], 1 if channels else xs[-1]
    bs = B.shape
    if len(bs) != lead + 2 or bs != C.shape or bs[:lead] != xs[:lead]:
        raise ValueError("B and C must be (.., groups, dim_state), one shape, with x's tokens")
    g, n = bs[lead:]
    per_state = A.dim() == 2
    if A.shape != ((h, n) if per_state else (h,)) or not A.is_contiguous():
        raise ValueError(f"A must be a contiguous ({h},) or ({h}, {n})")
    dp, bp = _vector(dev, D, "D", _F32, h), _vector(dev, dt_bias, "dt_bias", _F32, h)
    if (D is not None and D.shape[0] != h) or (dt_bias is not None and dt_bias.shape[0] != h):
        raise ValueError(f"D and dt_bias must have {h} entries")
    if z is not None:
        if not isinstance(z, _Tensor) or z.dtype is not _BF16 or z.get_device() != dev:
            _need(dev, z, "z", _BF16)
        if z.shape != xs:
            raise ValueError("z must have x's shape")
    sp = lines = 0
    ss = (0, 0, 0, 0)
    if state is not None:
        if not isinstance(state, _Tensor) or state.dtype is not _F32 or state.get_device() != dev:
            _need(dev, state, "state", _F32)
        st = state.shape
        if len(st) < 3 or st[1:] != ((h, n) if channels else (h, p, n)):
            raise ValueError("state must be (num_lines, heads, head_dim, dim_state), without "
                             "head_dim where x has none")
        # an empty pool has no address, but is not none: any other one, which nothing reads
        lines, ss, sp = st[0], state.stride(), state.data_ptr() or x.data_ptr()
        if channels:
            ss = (ss[0], ss[1], 0, ss[2])
    if out is None:
        out = _empty_like(x)
    else:
        _need(dev, out, "out", _BF16)
        if out.shape != xs:
            raise ValueError("out must have x's shape")
    lo, hi = dt_limit
    if hi > _MAX:  # no limit, which fp32 has a value for
        hi = _NO_LIMIT[1]
    if lo < -_MAX:
        lo = -_NO_LIMIT[1]
    # row, token, head and dim strides: ssm_fwd's tokens are flat (no row), and a row of ssm_update
    # has one token, or as many as there are
    v, o, b, c, d = x.stride(), out.stride(), B.stride(), C.stride(), dt.stride()
    w = z.stride() if z is not None else v
    if lead == 1:
        v, w, o, b, c, d = ((t[0], *t) for t in (v, w, o, b, c, d))
    if channels:
        v, w, o = (*v, 0), (*w, 0), (*o, 0)
    packed = _SSM.pack(x.data_ptr(), *v, 0 if z is None else z.data_ptr(), *w, out.data_ptr(), *o,
                       B.data_ptr(), *b, C.data_ptr(), *c, dt.data_ptr(), *d, A.data_ptr(), dp or 0,
                       bp or 0, sp, *ss, lo, hi, 1 if dt.dtype is _F32 else 0,
                       1 if dt_softplus else 0, 1 if per_state else 0, lines, h, g, p, n,
                       pad_slot_id)
    return dev, packed, out, (h, g, p, n, 1 if per_state else 0)


def _mapped(t: torch.Tensor) -> bool:
    """Whether the chunked form reads a (tokens, heads, dim) tensor as it is (ssm_fwd_workspace)."""
    st = t.stride()
    return (st[2] == 1 and t.data_ptr() % 16 == 0 and st[0] > 0 and st[0] % 8 == 0
            and (t.shape[1] == 1 or (st[1] > 0 and st[1] % 8 == 0)))


def ssm_fwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
            state: Optional[torch.Tensor], query_start_loc: torch.Tensor,
            cache_indices: Optional[torch.Tensor] = None,
            has_initial_state: Optional[torch.Tensor] = None, D: Optional[torch.Tensor] = None,
            z: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
            dt_softplus: bool = True, dt_limit: Tuple[float, float] = _NO_LIMIT,
            pad_slot_id: int = PAD_SLOT_ID, out: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None, err_count: Optional[torch.Tensor] = None,
            stream=None) -> torch.Tensor:
    """Selective state space scan over varlen sequences (prefill), states updated in place.

    x is (total_tokens, heads, head_dim) bf16, or (total_tokens, channels) for
    layers whose channels each have their own step; dt is (total_tokens, heads
    or channels) bf16 or fp32, B and C are (total_tokens, groups, dim_state)
    bf16, any strides.  A is fp32 (heads,) or, a decay for every state, (heads,
    dim_state), contiguous; D and dt_bias are fp32 (heads,); z is a gate of x's
    shape.  state is (num_lines, heads, head_dim, dim_state) fp32, without
    head_dim where x has none.  Per token and head:

        d = clamp(softplus(dt + dt_bias), *dt_limit)
        S <- exp(d A) S + d x B^T,    out = (S C + D x) [silu(z)]

    Returns out.
    """
    if stream is not None:
        return _elsewhere(stream, x, ssm_fwd, x, dt, A, B, C, state, query_start_loc, cache_indices,
                          has_initial_state, D, z, dt_bias, dt_softplus, dt_limit, pad_slot_id, out,
                          workspace, err_count)
    dev, args, out, scratch, _ = _marshal_fwd(x, dt, A, B, C, state, query_start_loc, cache_indices,
                                              has_initial_state, D, z, dt_bias, dt_softplus,
                                              dt_limit, pad_slot_id, out, workspace, err_count)
    _call("ssm_fwd", args, dev)
    return out


def prepare_ssm_fwd(x, dt, A, B, C, state, query_start_loc, cache_indices=None,
                    has_initial_state=None, D=None, z=None, dt_bias=None, dt_softplus=True,
                    dt_limit=_NO_LIMIT, pad_slot_id=PAD_SLOT_ID, out=None, workspace=None,
                    err_count=None) -> Launch:
    """Validate and marshal an ssm_fwd call once; returns a reusable Launch."""
    _, args, result, scratch, keep = _marshal_fwd(x, dt, A, B, C, state, query_start_loc,
                                                  cache_indices, has_initial_state, D, z, dt_bias,
                                                  dt_softplus, dt_limit, pad_slot_id, out,
                                                  workspace, err_count)
    return Launch("ssm_fwd", args, result, keep, _made((result, scratch), (out, workspace)))


def _marshal_fwd(x, dt, A, B, C, state, query_start_loc, cache_indices, has_initial_state, D, z,
                 dt_bias, dt_softplus, dt_limit, pad_slot_id, out, workspace, err_count):
    dev, packed, out, sizes = _pack_ssm(x, dt, A, B, C, state, D, z, dt_bias, dt_softplus, dt_limit,
                                        pad_slot_id, out, 1)
    qsl = _vector(dev, query_start_loc, "query_start_loc", _I32, 1)
    if qsl is None:
        raise TypeError("query_start_loc must be a CUDA tensor")
    batch, total = query_start_loc.shape[0] - 1, x.shape[0]
    ci = _vector(dev, cache_indices, "cache_indices", _I32, batch)
    hi = has_initial_state
    if hi is not None:
        if hi.dtype not in (torch.bool, _U8):
            raise TypeError("has_initial_state must be bool or uint8")
        hi = _vector(dev, hi, "has_initial_state", hi.dtype, batch)
    copies = x.dim() == 2 or not (_mapped(x) and _mapped(B) and _mapped(C))
    size = _lib.load().ssm_fwd_workspace(total, batch, *sizes, 1 if copies else 0)
    scratch, sp, room = workspace, 0, 0
    if size or workspace is not None:
        scratch = _workspace(dev, workspace, size, x)
        sp, room = scratch.data_ptr(), scratch.shape[0]
    args = (packed, qsl, batch, ci, hi, total, sp, room, _err(dev, err_count))
    keep = (x, dt, A, B, C, state, query_start_loc, cache_indices, has_initial_state, D, z, dt_bias,
            out, scratch, err_count)
    return dev, args, out, scratch, keep


def ssm_update(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
               C: torch.Tensor, state: torch.Tensor, state_indices: Optional[torch.Tensor] = None,
               num_accepted_tokens: Optional[torch.Tensor] = None,
               output_state_indices: Optional[torch.Tensor] = None,
               D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
               dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True,
               dt_limit: Tuple[float, float] = _NO_LIMIT, pad_slot_id: int = PAD_SLOT_ID,
               out: Optional[torch.Tensor] = None, err_count: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """Selective state space scan over the new tokens of each row (decode, speculative verify).

    dt is (batch, heads) or, with several tokens a row, (batch, seqlen, heads);
    x, z, B and C have the axes of ssm_fwd after dt's first ones.  The row's
    state line state_indices[b] is updated in place; with output_state_indices
    (batch, steps >= seqlen) the state after token t goes to line [b, t]
    instead (-1: none), and with num_accepted_tokens the row starts from line
    [b, num_accepted_tokens[b] - 1].  Returns out with x's shape.
    """
    if stream is not None:
        return _elsewhere(stream, x, ssm_update, x, dt, A, B, C, state, state_indices,
                          num_accepted_tokens, output_state_indices, D, z, dt_bias, dt_softplus,
                          dt_limit, pad_slot_id, out, err_count)
    dev, args, out, _ = _marshal_update(x, dt, A, B, C, state, state_indices, num_accepted_tokens,
                                        output_state_indices, D, z, dt_bias, dt_softplus, dt_limit,
                                        pad_slot_id, out, err_count)
    _call("ssm_update", args, dev)
    return out


def prepare_ssm_update(x, dt, A, B, C, state, state_indices=None, num_accepted_tokens=None,
                       output_state_indices=None, D=None, z=None, dt_bias=None, dt_softplus=True,
                       dt_limit=_NO_LIMIT, pad_slot_id=PAD_SLOT_ID, out=None,
                       err_count=None) -> Launch:
    """Validate and marshal an ssm_update call once; returns a reusable Launch."""
    _, args, result, keep = _marshal_update(x, dt, A, B, C, state, state_indices,
                                            num_accepted_tokens, output_state_indices, D, z,
                                            dt_bias, dt_softplus, dt_limit, pad_slot_id, out,
                                            err_count)
    return Launch("ssm_update", args, result, keep, _made((result,), (out,)))


def _marshal_update(x, dt, A, B, C, state, state_indices, num_accepted_tokens,
                    output_state_indices, D, z, dt_bias, dt_softplus, dt_limit, pad_slot_id, out,
                    err_count):
    if state is None:
        raise TypeError("state must be a CUDA tensor")
    lead = dt.dim() - 1 if isinstance(dt, _Tensor) else 1
    if lead not in (1, 2):
        raise ValueError("dt must be (batch, heads) or (batch, seqlen, heads)")
    dev, packed, out, _ = _pack_ssm(x, dt, A, B, C, state, D, z, dt_bias, dt_softplus, dt_limit,
                                    pad_slot_id, out, lead)
    batch, seqlen = dt.shape[0], 1 if lead == 1 else dt.shape[1]
    oidx, ost, steps = output_state_indices, (0, 0), 0
    if oidx is not None:
        _need(dev, oidx, "output_state_indices", _I32)
        if oidx.dim() != 2 or oidx.shape[0] != batch:
            raise ValueError("output_state_indices must be (batch, steps)")
        oidx, ost, steps = oidx.data_ptr(), oidx.stride(), oidx.shape[1]
    args = (packed, _vector(dev, state_indices, "state_indices", _I32, batch),
            _vector(dev, num_accepted_tokens, "num_accepted_tokens", _I32, batch), oidx, *ost,
            steps, batch, seqlen, _err(dev, err_count))
    keep = (x, dt, A, B, C, state, state_indices, num_accepted_tokens, output_state_indices, D, z,
            dt_bias, out, err_count)
    return dev, args, out, keep
