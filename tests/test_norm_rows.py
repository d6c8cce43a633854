"""Both norms on rows that go element by element: odd lengths, odd offsets and turned axes, around every change of the
lanes and elements that a row gets, and vector rows that keep one operand in registers.

Tolerances: a lane adds up to 32 squares and the lanes' sums meet in up to 10
steps: 42 roundings of 2^-24, which the root halves, less than 2^-19 of the
result; the few roundings around it are 2^-23 each and fit in the same.  A bf16
output adds its own rounding, at most 2^-9 of the value (2^-8 is allowed).
"""
from __future__ import annotations

import pytest
import torch

import layer_ref as ref
from parity_util import SENTINEL

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
LENGTHS = [2049, 2500, 4095, 4097, 5001, 8191, 8193, 12001, 16383, 16385, 32767]


@pytest.fixture(scope="module")
def ccv():
    import causal_depthwise_conv1d_fwd_gb300 as module
    from causal_depthwise_conv1d_fwd_gb300 import build

    build.build()
    return module


def near(got, want, mag, what):
    rtol = 2.0 ** -8 if got.dtype == BF16 else 0.0
    ref.assert_within(got, want, rtol * want.abs() + 2.0 ** -19 * mag, what)


def randn(shape, g, std=1.0):
    return (std * torch.randn(shape, generator=g)).to(BF16)


def place(t, layout):
    """t on the device: as it is, one element off, or with its last axis outermost."""
    t = t.cuda()
    if layout == "odd":
        flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.flatten()
        return flat[1:].view(t.shape)
    if layout == "turned":
        order = [t.dim() - 1, *range(t.dim() - 1)]
        return t.permute(order).contiguous().permute([*range(1, t.dim()), 0])
    return t


CASES = [(n, "plain") for n in LENGTHS] + [(n, layout) for n in (4096, 8192, 16384, 32768) for layout in ("odd", "turned")] + [
    (16392, "plain"), (32760, "plain")]


@pytest.mark.parametrize("dim,layout", CASES)
@pytest.mark.parametrize("before", [True, False])
def test_gated(ccv, dim, layout, before):
    g = torch.Generator().manual_seed(dim)
    x, z, w = randn((3, 2, dim), g), randn((3, 2, dim), g, 3.0), randn((dim,), g)
    for activation in ("silu", "sigmoid", None):
        want = ref.gated_rms_norm(x, z, w, 1e-6, activation, before)
        got = ccv.gated_rms_norm(place(x, layout), place(z, layout), w.cuda(), 1e-6, activation, before)
        near(got, want, want.abs(), f"{activation}")
    for name in ("x", "gate"):
        a, b = place(x, layout), place(z, layout)
        got = ccv.gated_rms_norm(a, b, w.cuda(), 1e-6, None, before, out=a if name == "x" else b)
        near(got, want, want.abs(), f"out is {name}")


@pytest.mark.parametrize("dim,layout", CASES)
@pytest.mark.parametrize("res", [BF16, torch.float32])
def test_residual(ccv, dim, layout, res):
    g = torch.Generator().manual_seed(dim + 1)
    x, r = randn((3, dim), g), (2 * torch.randn(3, dim, generator=g)).to(res)
    w, pw = randn((dim,), g, 0.1), randn((dim,), g, 0.1)
    for post in (None, pw):
        for gate in (None, randn((dim,), g), randn((3, dim), g)):
            on = [None if t is None else t.cuda() for t in (post, gate)]
            want, wh, mag = ref.residual_rms_norm(x, r, w, post, gate, -0.3, 1e-6, 1.0)
            rms = (wh.square().mean(-1, keepdim=True) + 1e-6).sqrt()
            out_mag = (mag / rms) * (w.double() + 1).abs() + want.abs()
            a, b = place(x, layout), place(r, layout)
            out, h = ccv.residual_rms_norm(a, b, w.cuda(), *on, -0.3, 1e-6, 1.0)
            near(h, wh, mag, "residual")
            near(out, want, out_mag, "out")
            ccv.residual_rms_norm(a, b, w.cuda(), *on, -0.3, 1e-6, 1.0, out=a, residual_out=b)
            near(b, wh, mag, "in place residual")
            near(a, want, out_mag, "in place out")


@pytest.mark.parametrize("dim", [2500, 16385, 32760])
def test_nothing_around_the_rows_is_written(ccv, dim):
    g = torch.Generator().manual_seed(dim)
    x, z, w = randn((4, dim), g), randn((4, dim), g), randn((dim,), g)

    def wide():
        return torch.full((4, dim + 16), SENTINEL, dtype=torch.int16, device="cuda").view(BF16)

    outs = [wide() for _ in range(3)]
    inner = [o[:, 8:dim + 8] for o in outs]
    ccv.gated_rms_norm(x.cuda(), z.cuda(), w.cuda(), out=inner[0])
    ccv.residual_rms_norm(x.cuda(), z.cuda(), w.cuda(), out=inner[1], residual_out=inner[2])
    for o in outs:
        bits = o.view(torch.int16)
        assert bool((bits[:, :8] == SENTINEL).all()) and bool((bits[:, dim + 8:] == SENTINEL).all())
        assert not bool((bits[:, 8:dim + 8] == SENTINEL).all())
