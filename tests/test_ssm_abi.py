"""The C ABI and binding of include/ccv_ssm.h and include/ccv_logits.h on a host without a GPU: exports and refusals."""
from __future__ import annotations

import ctypes
import re
import subprocess

import pytest
import torch

from causal_depthwise_conv1d_fwd_gb300 import _lib, build

OK, NULLP, SIZE, ALIAS, STRIDE, CAP, ARG, DIM, HEADS, WORK = 0, -1, -3, -5, -6, -8, -9, -10, -11, -12
X, Z, O, B, C, T, S, A = (0x10000000 * i for i in range(1, 9))  # fake device addresses, far apart
IDX = 0x90000000
INF = float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.mark.parametrize("header,signatures,names", [
    (_lib.SSM_HEADER, _lib.SSM_SIGNATURES, {"ssm_fwd", "ssm_fwd_workspace", "ssm_update"}),
    (_lib.LOGITS_HEADER, _lib.LOGITS_SIGNATURES, {"logits_process"})])
def test_every_declared_function_is_exported(lib, header, signatures, names):
    assert names == set(_lib.declared_functions(header)) == set(signatures)
    out = subprocess.run(["nm", "-D", "--defined-only", build.LIB], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r" T (\w+)$", out, flags=re.M))


def test_packed_structures_match_the_header(lib):
    from causal_depthwise_conv1d_fwd_gb300 import logits, ssm

    assert ssm._SSM.size == ctypes.sizeof(_lib.SsmArgs) and logits._LOGITS.size == ctypes.sizeof(_lib.LogitsArgs)
    got = _lib.SsmArgs.from_buffer_copy(ssm._SSM.pack(*range(1, 38), 0.5, 0.75, *range(40, 49)))
    assert (got.x.data, got.z.stride_row, got.out.stride_tok, got.C.stride_dim, got.dt, got.dt_stride_head) == (1, 7, 13, 25, 26, 29)
    assert (got.A, got.D, got.dt_bias, got.state, got.s_stride_state) == (30, 31, 32, 33, 37)
    assert (got.dt_min, got.dt_max, got.dt_fp32, got.num_lines, got.dim_state, got.pad_slot_id) == (0.5, 0.75, 40, 43, 47, 48)
    got = _lib.LogitsArgs.from_buffer_copy(logits._LOGITS.pack(*range(1, 33)))
    assert (got.out, got.history, got.prompt_lengths, got.draft_tokens, got.presence, got.b_stride_b) == (4, 7, 11, 12, 17, 20)
    assert (got.mask, got.m_stride_pos, got.logits_fp32, got.vocab, got.pad_slot_id) == (21, 23, 24, 28, 32)


def ssm_args(**over):
    d = dict(x=(X, 512, 512, 64, 1), z=(Z, 512, 512, 64, 1), out=(O, 512, 512, 64, 1), B=(B, 256, 256, 128, 1), C=(C, 256, 256, 128, 1),
             dt=T, dr=8, dtok=8, dh=1, A=A, D=None, bias=None, state=S, sl=65536, sh=8192, sd=128, ss=1, lo=0.0, hi=INF, f32=0, soft=1,
             per=0, lines=8, heads=8, groups=2, dim=64, states=128, pad=-1)
    d.update(over)
    vals = list(d.values())
    return _lib.SsmArgs(*(_lib.HeadsView(*v) for v in vals[:5]), *vals[5:])


def fwd(lib, total=10, batch=2, qsl=IDX, hi_=None, ws=0xA0000000, wsb=1 << 50, **over):
    return lib.ssm_fwd(ctypes.byref(ssm_args(**over)), qsl, batch, None, hi_, total, ws, wsb, None, None)


def upd(lib, batch=2, seqlen=1, nacc=None, oidx=None, ost=(4, 1), steps=4, **over):
    return lib.ssm_update(ctypes.byref(ssm_args(**over)), None, nacc, oidx, *ost, steps, batch, seqlen, None, None)


@pytest.mark.parametrize("call", [fwd, upd])
def test_ssm_refusals(lib, call):
    assert call(lib, states=257) == DIM
    assert call(lib, dim=1025) == DIM
    assert call(lib, groups=3) == HEADS
    assert call(lib, groups=0) == HEADS
    assert call(lib, states=-1) == SIZE
    assert call(lib, lines=-1) == SIZE
    assert call(lib, batch=-1) == SIZE
    assert call(lib, heads=1 << 24, dim=1024) == SIZE
    assert call(lib, x=(X, 512, -512, 64, 1)) == STRIDE
    assert call(lib, sd=-128) == STRIDE
    assert call(lib, dtok=-1) == STRIDE
    for name in ("x", "out", "B", "C"):
        assert call(lib, **{name: (None, 512, 512, 64, 1)}) == NULLP
    assert call(lib, dt=None) == NULLP
    assert call(lib, A=None) == NULLP
    for name in ("x", "z", "B", "C"):
        assert call(lib, **{name: (O + 64, 512, 512, 64, 1)}) == ALIAS
    assert call(lib, dt=O) == ALIAS
    assert call(lib, A=O) == ALIAS
    assert call(lib, D=O + 4) == ALIAS
    assert call(lib, bias=O) == ALIAS
    assert call(lib, state=O - 4096) == ALIAS
    assert call(lib, batch=0) == OK
    assert call(lib, heads=0, groups=0) == OK
    assert call(lib, dim=0) == OK
    assert call(lib, states=0) == OK


@pytest.mark.parametrize("call", [fwd, upd])
def test_ssm_elements_that_share_places_are_refused(lib, call):
    """An expanded output or pool, and ones whose axes reach into one another."""
    assert call(lib, out=(O, 512, 512, 0, 1)) == STRIDE
    assert call(lib, out=(O, 511, 511, 64, 1)) == STRIDE
    assert call(lib, out=(O, 512, 512, 64, 0)) == STRIDE
    assert call(lib, out=(O, 512, 512, 63, 1)) == STRIDE
    assert call(lib, sl=0) == STRIDE
    assert call(lib, sl=65535) == STRIDE
    assert call(lib, sd=64) == STRIDE
    assert call(lib, ss=0) == STRIDE


def test_ssm_fwd_refusals(lib):
    assert fwd(lib, total=-1) == SIZE
    assert fwd(lib, total=(1 << 30) + 1) == SIZE
    assert fwd(lib, qsl=None) == NULLP
    assert fwd(lib, state=None, hi_=IDX) == ARG
    assert fwd(lib, total=0) == OK


def test_ssm_workspace(lib):
    """What ssm_fwd needs is refused when it is missing, too small or misaligned; sizes that it refuses need none."""
    for sizes in ((1 << 14, 4, 8, 2, 64, 128, 0), (1 << 14, 1, 2, 1, 64, 128, 0), (5000, 1, 512, 1, 1, 16, 1)):
        total, batch, heads, groups, dim, states, per = sizes
        need = lib.ssm_fwd_workspace(*sizes, 0)
        assert 0 <= need <= lib.ssm_fwd_workspace(*sizes, 1)
        if need:
            kw = dict(total=total, batch=batch, heads=heads, groups=groups, dim=dim, states=states, per=per)
            if dim == 1:  # (tokens, channels)
                v = (heads, heads, 1, 0)
                kw |= dict(x=(X, *v), z=(None, *v), out=(O, *v), B=(B, 16, 16, 16, 1), C=(C, 16, 16, 16, 1), dr=heads, dtok=heads,
                           sl=heads * 16, sh=16, sd=0)
            assert fwd(lib, wsb=need - 1, **kw) == WORK
            assert fwd(lib, ws=None, **kw) == WORK
            assert fwd(lib, ws=0xA0000008, **kw) == WORK
    for sizes in ((-1, 1, 8, 2, 64, 128, 0), (1 << 14, 1, 8, 3, 64, 128, 0), (1 << 14, 1, 8, 2, 64, 257, 0), (1 << 14, -1, 8, 2, 64, 128, 0),
                  (0, 1, 8, 2, 64, 128, 0), ((1 << 30) + 1, 1, 8, 2, 64, 128, 0), (1 << 14, 1, 0, 0, 64, 128, 0)):
        assert lib.ssm_fwd_workspace(*sizes, 1) == 0


def test_ssm_update_refusals(lib):
    assert upd(lib, seqlen=-1) == SIZE
    assert upd(lib, nacc=IDX) == ARG
    assert upd(lib, seqlen=5, oidx=IDX) == CAP
    assert upd(lib, oidx=IDX, ost=(-1, 1)) == STRIDE
    assert upd(lib, state=None) == NULLP
    assert upd(lib, seqlen=0) == OK


def process(lib, **over):
    d = dict(x=X, xb=3000, xp=1000, o=O, ob=3000, op=1000, h=B, hs=64, hi=None, hl=C, pl=None, d=None, db=2, dp=1, r=None, f=None, p=None,
             bi=None, b=None, bs=4, m=None, mb=96, mp=32, f32=0, of32=0, batch=2, n=3, vocab=1000, lines=4, size=64, biases=0, pad=-1)
    d.update(over)
    return lib.logits_process(ctypes.byref(_lib.LogitsArgs(*d.values())), None, None)


def test_logits_refusals(lib):
    assert process(lib, batch=-1) == SIZE
    assert process(lib, vocab=-1) == SIZE
    assert process(lib, vocab=(1 << 30) + 1) == SIZE
    assert process(lib, size=-1) == SIZE
    assert process(lib, biases=-1) == SIZE
    assert process(lib, xp=-1) == STRIDE
    assert process(lib, mb=-1) == STRIDE
    assert process(lib, x=None) == NULLP
    assert process(lib, o=None) == NULLP
    assert process(lib, hl=None) == NULLP
    assert process(lib, biases=4) == NULLP
    assert process(lib, o=X + 2) == ALIAS
    assert process(lib, o=X, op=1001) == ALIAS
    assert process(lib, o=X, of32=1) == ALIAS
    for name in ("h", "hl", "pl", "hi", "d", "r", "f", "p", "m"):
        assert process(lib, **{name: O + 16}) == ALIAS, name
    assert process(lib, bi=O, b=T, biases=4) == ALIAS
    assert process(lib, bi=T, b=O, biases=4) == ALIAS
    assert process(lib, batch=0) == OK
    assert process(lib, n=0) == OK
    assert process(lib, vocab=0) == OK
    assert lib.logits_process(None, None, None) == NULLP


def test_logits_rows_that_share_places_are_refused(lib):
    """An expanded output, or one whose rows reach into the next."""
    assert process(lib, ob=0) == STRIDE
    assert process(lib, op=0) == STRIDE
    assert process(lib, op=999) == STRIDE
    assert process(lib, ob=2999) == STRIDE
    assert process(lib, ob=1000, op=1999) == STRIDE
    assert process(lib, x=O, xb=0, ob=0) == STRIDE  # in place
    assert process(lib, ob=0, batch=1, vocab=0) == OK


def test_binding_refusals():
    """Shapes, types and devices, refused before any launch."""
    import causal_depthwise_conv1d_fwd_gb300 as ccv

    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(TypeError):
        ccv.ssm_fwd(bf(4, 2, 8), bf(4, 2), torch.zeros(2), bf(4, 1, 8), bf(4, 1, 8), None, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        ccv.ssm_update(bf(4, 2, 8), bf(4, 2), torch.zeros(2), bf(4, 1, 8), bf(4, 1, 8), torch.zeros(4, 2, 8, 8))
    with pytest.raises(TypeError):
        ccv.logits_process(torch.zeros(2, 8))


@pytest.mark.gpu
def test_binding_refusals_on_gpu_tensors():
    import causal_depthwise_conv1d_fwd_gb300 as ccv

    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    good = dict(x=bf(4, 2, 8), dt=bf(4, 2), A=f32(2), B=bf(4, 1, 16), C=bf(4, 1, 16), state=f32(4, 2, 8, 16))

    def refuse(kind, call, tail=(), **over):
        kw = {k: over.pop(k) for k in list(over) if k not in good}
        with pytest.raises(kind):
            call(*{**good, **over}.values(), *tail, **kw)

    for call, tail in ((ccv.ssm_fwd, (i32(2),)), (ccv.ssm_update, ())):
        refuse(ValueError, call, tail, x=bf(4, 3, 8))
        refuse(ValueError, call, tail, x=bf(4, 2, 8, 1))
        refuse(ValueError, call, tail, dt=bf(5, 2))
        refuse(TypeError, call, tail, dt=bf(4, 2).half())
        refuse(ValueError, call, tail, A=f32(3))
        refuse(ValueError, call, tail, A=f32(2, 8))
        refuse(ValueError, call, tail, A=f32(16, 2).t())
        refuse(TypeError, call, tail, A=bf(2))
        refuse(ValueError, call, tail, B=bf(4, 1, 15))
        refuse(ValueError, call, tail, B=bf(4, 16), C=bf(4, 16))
        refuse(ValueError, call, tail, state=f32(4, 2, 16))
        refuse(ValueError, call, tail, x=bf(4, 2))                     # channels: the state has no head_dim
        refuse(TypeError, call, tail, state=bf(4, 2, 8, 16))
        refuse(ValueError, call, tail, D=f32(3))
        refuse(ValueError, call, tail, dt_bias=f32(1))
        refuse(ValueError, call, tail, z=bf(4, 2, 7))
        refuse(TypeError, call, tail, z=f32(4, 2, 8))
        refuse(ccv.CcvError, call, tail, B=bf(4, 3, 16), C=bf(4, 3, 16))  # 2 heads, 3 groups
        refuse(ccv.CcvError, call, tail, out=good["x"])
        refuse(ValueError, call, tail, out=bf(4, 2, 9))
    refuse(ValueError, ccv.ssm_fwd, (i32(3), i32(1)))
    refuse(TypeError, ccv.ssm_fwd, (i32(2), None, f32(1)))
    refuse(TypeError, ccv.ssm_fwd, (None,))
    refuse(TypeError, ccv.ssm_update, state=None)
    refuse(ValueError, ccv.ssm_update, (i32(3),))
    refuse(ccv.CcvError, ccv.ssm_update, (None, i32(4)))
    refuse(ValueError, ccv.ssm_update, (None, None, i32(3, 1)))
    x = f32(2, 3, 40)

    def no(kind, *args, **kw):
        with pytest.raises(kind):
            ccv.logits_process(*args, **kw)

    no(ValueError, f32(40))
    no(TypeError, x.double())
    no(ValueError, f32(2, 40, 3).transpose(1, 2))
    no(ValueError, x, i32(2, 5))                                       # a history without its lengths
    no(ValueError, x, i32(2, 5), i32(1))
    no(ValueError, x, i32(1, 5), i32(1))
    no(ValueError, x, i32(5, 2).t(), i32(2))
    no(ValueError, x, i32(2, 5), i32(2), None, i32(1))
    no(TypeError, x, i32(2, 5).long(), i32(2))
    no(ValueError, x, draft_tokens=i32(2, 3))
    no(ValueError, x, repetition=f32(1))
    no(TypeError, x, frequency=bf(2))
    no(ValueError, x, bias=f32(2, 3))
    no(ValueError, x, bias=f32(2, 3), bias_ids=i32(2, 4))
    no(ValueError, x, bias=f32(2, 3), bias_ids=i32(2, 4)[:, :3])
    no(ValueError, x, mask=i32(2, 3, 1))
    no(ValueError, x, mask=i32(2, 2))
    no(ValueError, x, out=f32(2, 3, 41))
    no(TypeError, x, out=x.half())
    no(ccv.CcvError, x, out=x.view(torch.bfloat16)[..., :40])
