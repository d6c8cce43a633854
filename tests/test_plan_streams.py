"""Plans that run on another stream than the one they were prepared on: what they allocated is handed over.

Memory that the preparing stream's queued work still uses must not be written by
a plan on another stream, and what a dropped plan owned must not return to the
preparing stream while the other one still runs it.  A pause on a stream holds
its work back, so each test's outcome is the same every time.
"""
from __future__ import annotations

import pytest
import torch

from causal_depthwise_conv1d_fwd_gb300 import workloads as wl
from test_layer_streams import NAMES, PAUSE, Case, ccv, pattern, pending_readers, same  # noqa: F401

pytestmark = pytest.mark.gpu


class ConvCase:
    def __init__(self, ccv):
        c = wl.varlen_prefill(31, [1200, 1, 800], 2048, has_init="all")
        self.args = lambda: tuple(t.cuda() if isinstance(t, torch.Tensor) else t for t in (
            c.x, c.weight, c.bias, c.conv_states, c.query_start_loc, c.cache_indices, c.has_initial_state))
        self.spaces, self.fn, self.plan = [2 * 2048 * 2001], ccv.ccv_fwd, ccv.prepare_ccv_fwd

    def call(self, args, **kw):
        return self.results(self.fn(*args, **kw), args)

    @staticmethod
    def results(got, args):
        return got, args[3]


@pytest.fixture(params=NAMES + ["ccv_fwd"])
def case(request, ccv):  # noqa: F811
    return ConvCase(ccv) if request.param == "ccv_fwd" else Case(ccv, request.param)


@pytest.fixture(params=["given", "current"])
def run(request):
    """Runs a plan on a stream that is given, or current."""
    def given(plan, stream):
        return plan(stream)

    def current(plan, stream):
        with torch.cuda.stream(stream):
            return plan()

    return given if request.param == "given" else current


def test_no_memory_that_is_still_read(case, run):
    want = case.call(case.args())
    args = case.args()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    copies = pending_readers(case.spaces)
    plan = case.plan(*args)
    got = case.results(run(plan, stream), args)
    stream.synchronize()
    same(got, want)
    torch.cuda.synchronize()
    for c in copies:
        assert torch.equal(c, pattern(c.numel()))


def test_plan_dropped_while_it_runs(case, run):
    args = case.args()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    plan = case.plan(*args)
    with torch.cuda.stream(stream):
        torch.cuda._sleep(PAUSE)
    run(plan, stream)
    del plan
    mine = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in case.spaces if n]
    torch.cuda.synchronize()
    for t in mine:
        assert bool((t == 7).all())


def test_later_calls_do_not_wait(case, run):
    """The hand-over happens once: after it a call does not wait for the preparing stream's work."""
    args = case.args()
    stream = torch.cuda.Stream()
    plan = case.plan(*args)
    run(plan, stream)
    torch.cuda.synchronize()
    torch.cuda._sleep(10 * PAUSE)
    home = torch.cuda.Event()
    home.record()
    run(plan, stream)
    stream.synchronize()
    assert not home.query()
    torch.cuda.synchronize()


def test_capture_on_another_stream(case, run):
    want = case.call(case.args())
    args = case.args()
    before = [t.clone() if isinstance(t, torch.Tensor) else t for t in args]
    plan = case.plan(*args)
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        plan()
    for _ in range(2):
        for t, b in zip(args, before):
            if isinstance(t, torch.Tensor):
                t.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        same(case.results(plan.result, args), want)
    got = case.results(run(plan, stream), args)  # and outside the graph, after it
    torch.cuda.synchronize()
    assert all(a.shape == b.shape for a, b in zip(got, want))


def test_plan_made_inside_a_capture(case):
    want = case.call(case.args())
    args = case.args()
    before = [t.clone() if isinstance(t, torch.Tensor) else t for t in args]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        plan = case.plan(*args)
        plan()
    for t, b in zip(args, before):
        if isinstance(t, torch.Tensor):
            t.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    same(case.results(plan.result, args), want)
