"""Calls on a stream that is given rather than current: what they allocate is theirs.

Memory that the caller's stream still uses must not become such a call's
workspace or output, and an output dropped early must not return to the caller's
stream while the call is running.  A pause on a stream holds its work back, so
each test's outcome is the same every time.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
PAUSE = 40_000_000  # cycles, some 20 ms


@pytest.fixture(scope="module")
def ccv():
    import causal_depthwise_conv1d_fwd_gb300 as module
    from causal_depthwise_conv1d_fwd_gb300 import build

    build.build()
    return module


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()


def heads(*shape, seed=0):
    return randn(*shape, seed=seed).to(BF16)


class Case:
    """call(**kw) makes the call, prepare() its plan; `spaces` are the sizes in bytes of what the call allocates."""

    def __init__(self, ccv, name):
        lib = __import__("causal_depthwise_conv1d_fwd_gb300._lib", fromlist=["load"]).load()
        t, hk, hv, d = 2000, 2, 4, 128
        q, k, v = heads(t, hk, d, seed=1), heads(t, hk, d, seed=2), heads(t, hv, d, seed=3)
        g, beta = -torch.rand(t, hv, device="cuda"), torch.rand(t, hv, device="cuda")
        pool = randn(2, hv, d, d, seed=4)
        starts = torch.tensor([0, 700, t], dtype=torch.int32, device="cuda")
        if name == "gdr_fwd":
            self.args = lambda: (q, k, v, g, beta, pool.clone(), starts)
            self.spaces = [lib.gdr_fwd_workspace(t, 2, hk, hv, d, d), 2 * t * hv * d]
        elif name == "gdr_update":
            rows = randn(t, hv, d, d, seed=5)
            self.args = lambda: (q, k, v, g, beta, rows.clone())
            self.spaces = [2 * t * hv * d]
        elif name == "gated_rms_norm":
            x, z, w = heads(t, 8, d, seed=6), heads(t, 8, d, seed=7), heads(d, seed=8)
            self.args = lambda: (x, z, w)
            self.spaces = [2 * t * 8 * d]
        elif name == "residual_rms_norm":
            x, r, w = heads(t, 1024, seed=9), randn(t, 1024, seed=10), heads(1024, seed=11)
            self.args = lambda: (x, r, w)
            self.spaces = [2 * t * 1024, 4 * t * 1024]
        else:
            b, n, vocab = 600, 2, 30000
            logits = randn(b, n + 1, vocab, seed=12)
            tokens = torch.randint(vocab, (b, n), device="cuda", dtype=torch.int32)
            u, noise = torch.rand(b, n, device="cuda"), torch.rand(b, vocab, device="cuda") + 0.01
            self.args = lambda: (logits, tokens, u, noise)
            self.spaces = [lib.spec_verify_workspace(b, n, vocab), 4 * b * (n + 1), 4 * b]
        self.fn, self.plan = getattr(ccv, name), getattr(ccv, "prepare_" + name)

    def call(self, args, **kw):
        return self.results(self.fn(*args, **kw), args)

    @staticmethod
    def results(got, args):
        """What the call returned, and the state that it updated."""
        got = got if isinstance(got, tuple) else (got,)
        return got + tuple(a for a in args if isinstance(a, torch.Tensor) and a.dim() == 4)


NAMES = ["gdr_fwd", "gdr_update", "gated_rms_norm", "residual_rms_norm", "spec_verify"]


def same(got, want):
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.int16) if a.dtype == BF16 else a, b.view(torch.int16) if b.dtype == BF16 else b)


def pattern(size):
    return torch.arange(size, device="cuda").to(torch.uint8)


@pytest.fixture(params=NAMES)
def case(request, ccv):
    return Case(ccv, request.param)


def pending_readers(sizes):
    """Tensors of these sizes whose only use, a copy, is still to run on the current stream when they are dropped."""
    torch.cuda.empty_cache()
    old = [pattern(n) for n in sizes if n]
    torch.cuda.synchronize()
    torch.cuda._sleep(PAUSE)
    return [t.clone() for t in old]


def test_no_memory_of_the_current_stream(case):
    want = case.call(case.args())
    args = case.args()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    copies = pending_readers(case.spaces)
    got = case.call(args, stream=stream)
    stream.synchronize()
    same(got, want)
    torch.cuda.synchronize()
    for c in copies:
        assert torch.equal(c, pattern(c.numel()))


def test_output_dropped_while_the_call_runs(case):
    args = case.args()
    stream = torch.cuda.Stream()
    case.call(case.args(), stream=stream)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(PAUSE)
    case.fn(*args, stream=stream)
    mine = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in case.spaces if n]
    torch.cuda.synchronize()
    for t in mine:
        assert bool((t == 7).all())


def test_output_dropped_while_the_caller_reads_it(case):
    """... and then the other stream allocates."""
    want = case.call(case.args())
    args = case.args()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = case.fn(*args, stream=stream)
    got = got if isinstance(got, tuple) else (got,)
    stream.synchronize()
    torch.cuda._sleep(PAUSE)
    copies = [t.clone() for t in got]
    del got
    with torch.cuda.stream(stream):
        for n in case.spaces:
            torch.full((max(n, 1),), 7, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    same(copies, want)


def test_calls_on_two_streams_at_once(case):
    """Different calls on the current stream and on another, neither waiting for the other, give what each gives alone."""
    want = case.call(case.args())
    streams = [torch.cuda.Stream() for _ in range(2)]
    argses = [case.args() for _ in range(12)]
    torch.cuda.synchronize()
    got = [case.call(a, **({} if i % 3 == 0 else {"stream": streams[i % 3 - 1]})) for i, a in enumerate(argses)]
    torch.cuda.synchronize()
    for x in got:
        same(x, want)


def test_raw_handles_and_the_default_stream(case):
    want = case.call(case.args())
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for given in (stream, stream.cuda_stream, torch.cuda.default_stream(), 0):
        got = case.call(case.args(), stream=given)
        torch.cuda.synchronize()
        same(got, want)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
