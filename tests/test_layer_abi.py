"""The C ABI and binding of include/ccv_layer.h on a host without a GPU: exports and refusals."""
from __future__ import annotations

import ctypes
import re
import subprocess

import pytest
import torch

from causal_depthwise_conv1d_fwd_gb300 import _lib, build

OK, NULLP, SIZE, ALIAS, STRIDE, CAP, ARG, DIM, HEADS, WORK = 0, -1, -3, -5, -6, -8, -9, -10, -11, -12
Q, K, V, O, G, B, S = (0x10000000 * i for i in range(1, 8))  # fake device addresses, far apart
IDX = 0x80000000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_every_declared_function_is_exported(lib):
    names = set(_lib.declared_functions(_lib.LAYER_HEADER))
    assert names == set(_lib.LAYER_SIGNATURES) == {"gdr_fwd", "gdr_fwd_workspace", "gdr_update", "gated_rms_norm",
                                                   "residual_rms_norm", "spec_verify", "spec_verify_workspace"}
    out = subprocess.run(["nm", "-D", "--defined-only", build.LIB], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r" T (\w+)$", out, flags=re.M))


def test_packed_structures_match_the_header(lib):
    """The binding packs the C structures itself: sizes and the order of the fields."""
    from causal_depthwise_conv1d_fwd_gb300 import layer

    assert layer._VIEW.size == ctypes.sizeof(_lib.HeadsView)
    assert layer._GDR.size == ctypes.sizeof(_lib.GdrArgs)
    numbers = list(range(1, 33)) + [0.5 if i == 5 else 40 + i for i in range(8)]
    got = _lib.GdrArgs.from_buffer_copy(layer._GDR.pack(*numbers))
    assert (got.q.data, got.k.stride_row, got.v.stride_tok, got.out.stride_dim) == (1, 7, 13, 20)
    assert (got.g, got.beta, got.gate_stride_head, got.a_log, got.state, got.s_stride_k) == (21, 22, 25, 26, 28, 32)
    assert (got.num_lines, got.dim_v, got.scale, got.qk_l2norm, got.pad_slot_id) == (40, 44, 0.5, 46, 47)


def test_status_strings(lib):
    for code in (DIM, HEADS, WORK):
        assert "unknown" not in _lib.status_string(code)


def gdr_args(**over):
    d = dict(q=(Q, 512, 256, 128, 1), k=(K, 512, 256, 128, 1), v=(V, 1024, 512, 128, 1), out=(O, 1024, 512, 128, 1),
             g=G, beta=B, gsr=4, gst=4, gsh=1, a_log=None, dt_bias=None, state=S, sl=65536, sh=16384, sv=128, sk=1,
             lines=8, hk=2, hv=4, dk=128, dv=128, scale=1.0, l2=1, pad=-1)
    d.update(over)
    vals = list(d.values())
    return _lib.GdrArgs(*(_lib.HeadsView(*x) for x in vals[:4]), *vals[4:])


def fwd(lib, total=10, batch=2, qsl=IDX, hi=None, ws=0x90000000, wsb=1 << 40, **over):
    return lib.gdr_fwd(ctypes.byref(gdr_args(**over)), qsl, batch, None, hi, total, ws, wsb, None, None)


def upd(lib, batch=2, seqlen=1, nacc=None, oidx=None, ost=(4, 1), steps=4, **over):
    return lib.gdr_update(ctypes.byref(gdr_args(**over)), None, nacc, oidx, *ost, steps, batch, seqlen, None, None)


@pytest.mark.parametrize("call", [fwd, upd])
def test_gdr_refusals(lib, call):
    assert call(lib, dk=257) == DIM
    assert call(lib, dv=1025) == DIM
    assert call(lib, hk=3) == HEADS
    assert call(lib, hk=0) == HEADS
    assert call(lib, dk=-1) == SIZE
    assert call(lib, lines=-1) == SIZE
    assert call(lib, batch=-1) == SIZE
    assert call(lib, q=(Q, 512, -256, 128, 1)) == STRIDE
    assert call(lib, sv=-128) == STRIDE
    assert call(lib, gst=-1) == STRIDE
    assert call(lib, q=(None, 512, 256, 128, 1)) == NULLP
    assert call(lib, g=None) == NULLP
    assert call(lib, a_log=IDX) == NULLP               # a_log and dt_bias go together
    assert call(lib, out=(V, 1024, 512, 128, 1)) == ALIAS
    assert call(lib, out=(Q + 64, 1024, 512, 128, 1)) == ALIAS
    assert call(lib, out=(G, 1024, 512, 128, 1)) == ALIAS
    assert call(lib, out=(S + 4096, 1024, 512, 128, 1)) == ALIAS
    assert call(lib, batch=0) == OK
    assert call(lib, hv=0, hk=0) == OK
    assert call(lib, dv=0) == OK


def test_gdr_fwd_refusals(lib):
    assert fwd(lib, total=-1) == SIZE
    assert fwd(lib, qsl=None) == NULLP
    assert fwd(lib, state=None, hi=IDX) == ARG
    assert fwd(lib, total=0) == OK
    need = lib.gdr_fwd_workspace(1 << 14, 4, 2, 4, 128, 128)
    assert need >= 0
    if need:
        assert fwd(lib, total=1 << 14, batch=4, wsb=need - 1) == WORK
        assert fwd(lib, total=1 << 14, batch=4, ws=None) == WORK
        assert fwd(lib, total=1 << 14, batch=4, ws=0x90000008) == WORK


def test_gdr_update_refusals(lib):
    assert upd(lib, seqlen=-1) == SIZE
    assert upd(lib, nacc=IDX) == ARG
    assert upd(lib, seqlen=5, oidx=IDX) == CAP
    assert upd(lib, oidx=IDX, ost=(-1, 1)) == STRIDE
    assert upd(lib, state=None) == NULLP
    assert upd(lib, seqlen=0) == OK


def gated(lib, x=(Q, 0, 512, 128, 1), z=(K, 0, 512, 128, 1), w=B, out=(O, 0, 512, 128, 1), tokens=4, heads=4, dim=128,
          act=1):
    x, z, out = (_lib.HeadsView(*v) for v in (x, z, out))
    return lib.gated_rms_norm(ctypes.byref(x), ctypes.byref(z), w, ctypes.byref(out), tokens, heads, dim, 1e-6, act, 1, None)


def test_gated_refusals(lib):
    assert gated(lib, dim=32769) == DIM
    assert gated(lib, tokens=-1) == SIZE
    assert gated(lib, act=3) == ARG
    assert gated(lib, x=(Q, 0, 512, -128, 1)) == STRIDE
    assert gated(lib, w=None) == NULLP
    assert gated(lib, out=(Q + 2, 0, 512, 128, 1)) == ALIAS
    assert gated(lib, out=(K, 0, 1024, 128, 1)) == ALIAS
    assert gated(lib, w=O + 256) == ALIAS
    assert gated(lib, tokens=0) == OK


def resid(lib, **over):
    d = dict(x=Q, xt=128, xd=1, r=K, rt=128, rd=1, f32=0, w=B, pw=None, g=None, gt=0, gd=1, out=O, ot=128, od=1, ro=V,
             rot=128, rod=1, tokens=4, dim=128, scale=1.0, eps=1e-6, off=0.0)
    d.update(over)
    return lib.residual_rms_norm(*d.values(), None)


def test_residual_refusals(lib):
    assert resid(lib, dim=40000) == DIM
    assert resid(lib, dim=-1) == SIZE
    assert resid(lib, rt=-128) == STRIDE
    assert resid(lib, r=None) == NULLP
    assert resid(lib, out=K) == ALIAS          # out over the residual
    assert resid(lib, ro=Q) == ALIAS
    assert resid(lib, out=V) == ALIAS          # both outputs in one place
    assert resid(lib, ro=K + 2) == ALIAS
    assert resid(lib, out=Q, ot=256) == ALIAS
    assert resid(lib, pw=O) == ALIAS
    assert resid(lib, g=V) == ALIAS
    assert resid(lib, tokens=0) == OK


def verify(lib, **over):
    d = dict(t=Q, f32=0, tb=4000, tp=1000, d=K, db=3, dp=1, p=None, pb=0, pp=0, nd=None, temp=None, u=V, ub=3, up=1, n=O,
             nb=1000, out=G, acc=B, batch=2, drafts=3, vocab=1000, ws=S, wsb=1 << 30, err=None, stream=None)
    d.update(over)
    return lib.spec_verify(*d.values())


def test_verify_refusals(lib):
    assert verify(lib, batch=-1) == SIZE
    assert verify(lib, vocab=0) == SIZE
    assert verify(lib, tp=-1) == STRIDE
    assert verify(lib, t=None) == NULLP
    assert verify(lib, d=None) == NULLP
    assert verify(lib, ws=None) == WORK
    assert verify(lib, ws=S + 4) == WORK
    assert verify(lib, wsb=lib.spec_verify_workspace(2, 3, 1000) - 1) == WORK
    assert verify(lib, out=K) == ALIAS
    assert verify(lib, acc=G + 4) == ALIAS
    assert verify(lib, batch=0) == OK


def test_binding_refusals():
    """Shapes, types and devices, refused before any launch."""
    import causal_depthwise_conv1d_fwd_gb300 as ccv

    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    starts = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        ccv.gdr_fwd(bf(4, 1, 8), bf(4, 1, 8), bf(4, 2, 8), torch.zeros(4, 2), torch.zeros(4, 2), None, starts)
    with pytest.raises(TypeError):
        ccv.gdr_update(bf(4, 1, 8), bf(4, 1, 8), bf(4, 2, 8), torch.zeros(4, 2), torch.zeros(4, 2), torch.zeros(4, 2, 8, 8))
    with pytest.raises(TypeError):
        ccv.gated_rms_norm(bf(4, 8), bf(4, 8), bf(8))
    with pytest.raises(TypeError):
        ccv.residual_rms_norm(bf(4, 8), bf(4, 8), bf(8))
    with pytest.raises(TypeError):
        ccv.spec_verify(torch.zeros(1, 2, 8), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1), torch.zeros(1, 8))


@pytest.mark.gpu
def test_binding_refusals_on_gpu_tensors():
    import causal_depthwise_conv1d_fwd_gb300 as ccv

    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    q, k, v, g, b, st = bf(4, 1, 8), bf(4, 1, 8), bf(4, 2, 8), f32(4, 2), f32(4, 2), f32(3, 2, 8, 8)

    def refuse(kind, call, *args, **kw):
        with pytest.raises(kind):
            call(*args, **kw)

    for call, tail in ((ccv.gdr_fwd, (i32(2),)), (ccv.gdr_update, ())):
        refuse(ValueError, call, bf(4, 1, 7), k, v, g, b, st, *tail)
        refuse(ValueError, call, q, k, bf(5, 2, 8), g, b, st, *tail)
        refuse(ValueError, call, q, k, v, f32(4, 1), f32(4, 1), st, *tail)
        refuse(TypeError, call, q, k, v, bf(4, 2), bf(4, 2), st, *tail)              # raw gates without a_log
        refuse(ValueError, call, q, k, v, g, f32(2, 4).t(), st, *tail)              # other strides
        refuse(ValueError, call, q, k, v, g, b, st, *tail, a_log=f32(2))
        refuse(ValueError, call, q, k, v, bf(4, 2), bf(4, 2), st, *tail, a_log=f32(1), dt_bias=f32(2))
        refuse(ValueError, call, q, k, v, g, b, f32(3, 2, 8, 9), *tail)
        refuse(TypeError, call, q, k, v, g, b, bf(3, 2, 8, 8), *tail)
        refuse(ccv.CcvError, call, bf(4, 3, 8), bf(4, 3, 8), v, g, b, st, *tail)     # 2 value heads, 3 key heads
        refuse(ccv.CcvError, call, q, k, v, g, b, st, *tail, out=v)
    refuse(ValueError, ccv.gdr_fwd, q, k, v, g, b, st, i32(3), i32(1))
    refuse(TypeError, ccv.gdr_fwd, q, k, v, g, b, st, i32(2), None, f32(1))
    refuse(TypeError, ccv.gdr_update, q, k, v, g, b, None)
    refuse(ValueError, ccv.gdr_update, q, k, v, g, b, st, i32(3))
    refuse(ccv.CcvError, ccv.gdr_update, q, k, v, g, b, st, None, i32(4))
    x, w = bf(4, 8), bf(8)
    refuse(ValueError, ccv.gated_rms_norm, x, bf(4, 7), w)
    refuse(ValueError, ccv.gated_rms_norm, x, x, bf(7))
    refuse(ValueError, ccv.gated_rms_norm, x, x, w, activation="relu")
    refuse(TypeError, ccv.gated_rms_norm, x, f32(4, 8), w)
    refuse(ValueError, ccv.residual_rms_norm, x, bf(5, 8), w)
    refuse(ValueError, ccv.residual_rms_norm, x, x, w, gate=bf(4))
    refuse(TypeError, ccv.residual_rms_norm, x, x, w, residual_out=f32(4, 8))
    refuse(ccv.CcvError, ccv.residual_rms_norm, x, bf(4, 8), w, residual_out=x)
    lg, t, u, n = f32(2, 3, 9), i32(2, 2), f32(2, 2), f32(2, 9)
    refuse(ValueError, ccv.spec_verify, f32(2, 2, 9), t, u, n)
    refuse(ValueError, ccv.spec_verify, lg, t, f32(2, 3), n)
    refuse(ValueError, ccv.spec_verify, lg, t, u, f32(2, 8))
    refuse(ValueError, ccv.spec_verify, lg, t, u, n, f32(2, 3, 9))
    refuse(ValueError, ccv.spec_verify, f32(2, 9, 3).transpose(1, 2), t, u, n)
    refuse(TypeError, ccv.spec_verify, lg, t.long(), u, n)
    refuse(ccv.CcvError, ccv.spec_verify, lg, t, u, n, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))


def test_size_limits(lib):
    assert verify(lib, vocab=(1 << 30) + 1, wsb=1 << 62) == SIZE
    args = _lib.GdrArgs()
    assert lib.gdr_fwd(ctypes.byref(args), Q, 1, None, None, (1 << 30) + 1, S, 1 << 62, None, None) == SIZE
