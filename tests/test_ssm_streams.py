"""ssm_fwd, ssm_update and logits_process on a stream that is given rather than current, and two graphs at once.

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


class Case:
    """call(**kw) makes the call; `spaces` are the sizes in bytes of what the call allocates."""

    def __init__(self, ccv, name):
        from causal_depthwise_conv1d_fwd_gb300 import _lib

        lib = _lib.load()
        bf = lambda *s, seed: randn(*s, seed=seed).to(BF16)  # noqa: E731
        starts = torch.tensor([0, 700, 4000], dtype=torch.int32, device="cuda")
        if name in ("ssm_fwd", "ssm_fwd_strided"):
            t, h, p, n = 4000, 4, 64, 128
            x, dt, b, c = bf(t, h, p, seed=1), bf(t, h, seed=2), bf(t, 1, n, seed=3), bf(t, 1, n, seed=4)
            strided = name != "ssm_fwd"
            if strided:  # (dim, tokens): copied into the workspace
                x = x.permute(1, 2, 0).contiguous().permute(2, 0, 1)
            a, pool = -torch.rand(h, device="cuda"), randn(2, h, p, n, seed=5)
            self.args = lambda: (x, dt, a, b, c, pool.clone(), starts)
            self.spaces = [lib.ssm_fwd_workspace(t, 2, h, 1, p, n, 0, strided), 2 * t * h * p]
        elif name == "ssm_fwd_channels":
            t, h, n = 4000, 200, 16
            x, dt, b, c = bf(t, h, seed=1), bf(t, h, seed=2), bf(t, 1, n, seed=3), bf(t, 1, n, seed=4)
            a, pool = -torch.rand(h, n, device="cuda"), randn(2, h, n, seed=5)
            self.args = lambda: (x, dt, a, b, c, pool.clone(), starts)
            self.spaces = [lib.ssm_fwd_workspace(t, 2, h, 1, 1, n, 1, 1), 2 * t * h]
        elif name == "ssm_update":
            t, h, p, n = 300, 4, 64, 128
            x, dt, b, c = bf(t, h, p, seed=1), bf(t, h, seed=2), bf(t, 1, n, seed=3), bf(t, 1, n, seed=4)
            a, pool = -torch.rand(h, device="cuda"), randn(t, h, p, n, seed=5)
            self.args = lambda: (x, dt, a, b, c, pool.clone())
            self.spaces = [2 * t * h * p]
        else:
            b, v = 40, 30000
            x = randn(b, 2, v, seed=1)
            ids = torch.randint(v, (b, 500), dtype=torch.int32, device="cuda")
            lengths = torch.full((b,), 400, dtype=torch.int32, device="cuda")
            self.args = lambda: (x, ids, lengths)
            self.spaces = [4 * b * 2 * v]
        self.name = name.split("_strided")[0].split("_channels")[0]
        self.fn, self.plan = getattr(ccv, self.name), getattr(ccv, "prepare_" + self.name)

    def call(self, args, **kw):
        return self.results(self.fn(*args, **kw), args)

    def results(self, got, args):
        """What the call returned, and the state that it updated."""
        return (got, args[5]) if self.name.startswith("ssm") else (got,)


@pytest.fixture(params=["ssm_fwd", "ssm_fwd_strided", "ssm_fwd_channels", "ssm_update", "logits_process"])
def case(request, ccv):
    return Case(ccv, request.param)


def same(got, want):
    for a, b in zip(got, want):
        assert torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def pattern(size):
    return torch.arange(size, device="cuda").to(torch.uint8)


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
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(PAUSE)
    out = case.call(args, stream=stream)[0]
    size = out.numel() * out.element_size()
    del out
    later = torch.zeros(size, dtype=torch.uint8, device="cuda")  # of the caller's stream
    torch.cuda.synchronize()
    assert not bool(later.any())


def test_plan_on_another_stream(case):
    want = case.call(case.args())
    args = case.args()
    plan = case.plan(*args)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = plan(stream)
    stream.synchronize()
    same(case.results(got, args), want)


def test_two_graphs_with_their_own_memory(case):
    """Two captured calls, replayed on two streams at once, give what one gives alone."""
    want = case.call(case.args())
    runs = []
    for _ in range(2):
        args = case.args()
        first = args[5].clone() if case.name.startswith("ssm") else None
        case.fn(*args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            if first is not None:
                args[5].copy_(first)
            out = case.fn(*args)
        runs.append((graph, out, args, first))  # the graph reads all of them
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(3):
        for stream, (graph, *_) in zip(streams, runs):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, args, _ in runs:
        same(case.results(out, args), want)
