"""gated_rms_norm and residual_rms_norm against plain 64-bit forms.

Tolerances: a bf16 output is one rounding (at most 2^-9 of the value; 2^-8 is
allowed) of an fp32 value whose own error is a few units of 2^-23 of the terms
and a row sum's 2^-21 or less: 2^-20 of the magnitude covers both.  An fp32
residual has that second part alone.
"""
from __future__ import annotations

import pytest
import torch

import layer_ref as ref
from parity_util import SENTINEL, assert_bits

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
DIMS = [1, 7, 8, 64, 80, 128, 136, 250, 256, 264, 511, 512, 1000, 2048, 2056, 4096, 5001, 8192, 12288, 20000, 32768]


@pytest.fixture(scope="module")
def ccv():
    import causal_depthwise_conv1d_fwd_gb300 as module
    from causal_depthwise_conv1d_fwd_gb300 import build

    build.build()
    return module


def near(got, want, mag, what):
    rtol = 2.0 ** -8 if got.dtype == BF16 else 0.0
    ref.assert_within(got, want, rtol * want.abs() + 2.0 ** -20 * mag, what)


def randn(shape, g, std=1.0):
    return (std * torch.randn(shape, generator=g)).to(BF16)


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("before", [True, False])
def test_gated(ccv, dim, before):
    g = torch.Generator().manual_seed(dim)
    tokens, heads = (5, 3) if dim <= 4096 else (2, 1)
    x, z, w = randn((tokens, heads, dim), g), randn((tokens, heads, dim), g, 3.0), randn((dim,), g)
    for activation in ("silu", "sigmoid", None):
        got = ccv.gated_rms_norm(x.cuda(), z.cuda(), w.cuda(), 1e-6, activation, before)
        want = ref.gated_rms_norm(x, z, w, 1e-6, activation, before)
        near(got, want, want.abs(), f"{activation}")


@pytest.mark.parametrize("tokens", [1, 2, 9, 300])
def test_gated_layouts(ccv, tokens):
    """Heads inside wider rows, a dim axis that is not innermost, odd offsets, rank 2, in place."""
    g = torch.Generator().manual_seed(tokens)
    x, z, w = randn((tokens, 4, 128), g), randn((tokens, 4, 128), g), randn((128,), g)
    want = ref.gated_rms_norm(x, z, w, 1e-5, "silu", True)
    wide = torch.full((tokens, 4, 144), SENTINEL, dtype=torch.int16, device="cuda").view(BF16)
    out = wide[:, :, 8:136]
    ccv.gated_rms_norm(x.cuda(), z.cuda(), w.cuda(), 1e-5, out=out)
    near(out, want, want.abs(), "wide out")
    for edge in (wide[:, :, :8], wide[:, :, 136:]):
        assert_bits(edge, torch.full(edge.shape, SENTINEL, dtype=torch.int16).view(BF16), "around out")
    turned = x.cuda().permute(2, 1, 0).contiguous().permute(2, 1, 0)
    near(ccv.gated_rms_norm(turned, z.cuda(), w.cuda(), 1e-5), want, want.abs(), "turned")
    flat = torch.zeros(x.numel() + 1, dtype=BF16, device="cuda")
    flat[1:] = x.flatten().cuda()
    near(ccv.gated_rms_norm(flat[1:].view(x.shape), z.cuda(), w.cuda(), 1e-5), want, want.abs(), "odd offset")
    two = ccv.gated_rms_norm(x.flatten(0, 1).cuda(), z.flatten(0, 1).cuda(), w.cuda(), 1e-5)
    near(two, want.flatten(0, 1), want.abs().flatten(0, 1), "rank 2")
    for name in ("x", "gate"):
        a, b = x.cuda(), z.cuda()
        got = ccv.gated_rms_norm(a, b, w.cuda(), 1e-5, out=a if name == "x" else b)
        near(got, want, want.abs(), f"out is {name}")


def test_gated_extremes(ccv):
    g = torch.Generator().manual_seed(3)
    x, z, w = randn((6, 1, 128), g), randn((6, 1, 128), g), randn((128,), g)
    x[0] = 0                      # a row of zeros
    z[1] = -200.0                 # a closed gate
    z[2] = 200.0
    x[3] = x[3] * 1e12
    x[4] = x[4] * 1e-12           # eps decides
    for before in (True, False):
        got = ccv.gated_rms_norm(x.cuda(), z.cuda(), w.cuda(), 1e-6, "silu", before)
        want = ref.gated_rms_norm(x, z, w, 1e-6, "silu", before)
        near(got, want, want.abs() + 1e-30, f"{before}")
    x[5, 0, 9] = float("nan")
    got = ccv.gated_rms_norm(x.cuda(), z.cuda(), w.cuda())
    assert bool(got[5].isnan().all()) and not bool(got[:5].isnan().any())


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("res", [BF16, torch.float32])
def test_residual(ccv, dim, res):
    g = torch.Generator().manual_seed(dim + 1)
    tokens = 7 if dim <= 4096 else 2
    x, r = randn((tokens, dim), g), (2 * torch.randn(tokens, dim, generator=g)).to(res)
    w, pw = randn((dim,), g, 0.1), randn((dim,), g, 0.1)
    for post in (None, pw):
        for gate in (None, randn((dim,), g), randn((tokens, dim), g)):
            for scale, offset in ((1.0, 1.0), (-0.3, 0.0)):
                on = [None if t is None else t.cuda() for t in (post, gate)]
                out, h = ccv.residual_rms_norm(x.cuda(), r.cuda(), w.cuda(), *on, scale, 1e-6, offset)
                want, wh, mag = ref.residual_rms_norm(x, r, w, post, gate, scale, 1e-6, offset)
                near(h, wh, mag, "residual")
                rms = (wh.square().mean(-1, keepdim=True) + 1e-6).sqrt()
                near(out, want, (mag / rms) * (w.double() + offset).abs() + want.abs(), "out")


def test_residual_layouts(ccv):
    g = torch.Generator().manual_seed(9)
    x, r, w = randn((33, 256), g), randn((33, 256), g), randn((256,), g)
    want, wh, mag = ref.residual_rms_norm(x, r, w, None, None, 1.0, 1e-6, 0.0)
    a, b = x.cuda(), r.cuda()
    out, h = ccv.residual_rms_norm(a, b, w.cuda(), out=a, residual_out=b)
    assert out is a and h is b
    near(h, wh, mag, "in place residual")
    near(out, want, 4 * mag + want.abs(), "in place out")
    turned = x.cuda().t().contiguous().t()
    gate = randn((256, 33), g).t()  # strides (1, 33)
    want, wh, mag = ref.residual_rms_norm(x, r, w, None, gate, 1.0, 1e-6, 0.0)
    wide = torch.empty(33, 512, device="cuda", dtype=BF16)
    out, h = ccv.residual_rms_norm(turned, r.cuda(), w.cuda(), gate=gate.cuda(), residual_out=wide[:, 128:384])
    near(h, wh, mag, "strided residual")
    row = gate[:1].expand(33, 256)  # stride 0 along tokens
    want, wh, mag = ref.residual_rms_norm(x, r, w, None, row, 1.0, 1e-6, 0.0)
    _, h = ccv.residual_rms_norm(x.cuda(), r.cuda(), w.cuda(), gate=gate.cuda()[:1].expand(33, 256))
    near(h, wh, mag, "broadcast gate")


def test_norms_capture_and_streams(ccv):
    g = torch.Generator().manual_seed(10)
    x, z, r = (randn((40, 128), g).cuda() for _ in range(3))
    w = randn((128,), g).cuda()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    want = ccv.gated_rms_norm(x, z, w)
    want2, wanth = ccv.residual_rms_norm(want, r, w)
    a = ccv.gated_rms_norm(x, z, w, stream=stream)
    b, h = ccv.residual_rms_norm(a, r, w, stream=stream)
    stream.synchronize()
    torch.cuda.synchronize()
    for got, ref_ in ((a, want), (b, want2), (h, wanth)):
        assert_bits(got, ref_)
    p1 = ccv.prepare_gated_rms_norm(x, z, w)
    p2 = ccv.prepare_residual_rms_norm(p1.result, r, w)
    p1(), p2()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p1()
        p2()
    p2.result[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert_bits(p2.result[0], want2)


def test_norms_of_nothing(ccv):
    x = torch.empty(0, 4, 128, dtype=BF16, device="cuda")
    w = torch.ones(128, dtype=BF16, device="cuda")
    assert ccv.gated_rms_norm(x, x, w).shape == x.shape
    y = torch.empty(0, 128, dtype=BF16, device="cuda")
    out, h = ccv.residual_rms_norm(y, y, w)
    assert out.shape == h.shape == (0, 128)
