"""The convolution's calls that make their own output, on a stream that is given rather than current.

As in test_layer_streams: a pause on a stream holds its work back, so each
test's outcome is the same every time.
"""
from __future__ import annotations

import pytest
import torch

from causal_depthwise_conv1d_fwd_gb300 import workloads as wl
from test_layer_streams import PAUSE, ccv, pattern, pending_readers, same  # noqa: F401

pytestmark = pytest.mark.gpu


def on_gpu(kwargs):
    return {k: torch.empty_strided(v.shape, v.stride(), dtype=v.dtype, device="cuda").copy_(v)
            if isinstance(v, torch.Tensor) else v for k, v in kwargs.items()}


class Case:
    """call(args, **kw) returns the outputs; `spaces` are their sizes in bytes."""

    def __init__(self, ccv, name):
        self.fn = getattr(ccv, name)
        if name == "ccv_fwd":
            c = wl.varlen_prefill(31, [1200, 1, 800], 2048, has_init="all")
            self.args, out = (lambda: on_gpu(c.kwargs())), [2 * 2048 * 2001]
        elif name == "paged_sconv_fwd_streams":
            base, streams = wl.config_paged_streams()
            pools = {k: v for k, v in base.kwargs().items()
                     if k in ("cache", "positions", "block_table", "slot_mapping", "block_size", "activation", "use_residual")}

            def args():
                d = on_gpu(pools)
                d["seq_idx"], d["query_start"] = self.metadata(ccv, base)
                d["streams"] = [on_gpu({k: s[k] for k in ("x", "weight", "off_s", "ws")}) for s in streams]
                return d

            self.args, out = args, [2 * s["x"].numel() for s in streams]
        else:
            c = wl.config_paged()

            def args():
                d = on_gpu(c.kwargs())
                d.pop("seq_idx", None), d.pop("query_start", None)
                if name == "paged_sconv_fwd":
                    d["seq_idx"], d["query_start"] = self.metadata(ccv, c)
                else:
                    d.update(query_start_loc=c.query_start_loc.cuda(), num_reqs=len(c.req_lengths),
                             num_actual_tokens=c.num_actual_tokens)
                return d

            self.args, out = args, [2 * c.x.numel()]
        self.spaces = out

    @staticmethod
    def metadata(ccv, c):
        seq, qs = (torch.empty(c.T, dtype=torch.int32, device="cuda") for _ in range(2))
        ccv.paged_sconv_seq_metadata(c.query_start_loc.cuda(), len(c.req_lengths), c.num_actual_tokens, seq, qs, c.T)
        return seq, qs

    def call(self, args, **kw):
        got = self.fn(**args, **kw)
        return tuple(got) if isinstance(got, (tuple, list)) else (got,)


@pytest.fixture(params=["ccv_fwd", "paged_sconv_fwd", "paged_sconv_fwd_with_metadata", "paged_sconv_fwd_streams"])
def case(request, ccv):  # noqa: F811
    return Case(ccv, request.param)


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
    case.call(args, stream=stream)
    mine = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in case.spaces]
    torch.cuda.synchronize()
    for t in mine:
        assert bool((t == 7).all())


def test_output_dropped_while_the_caller_reads_it(case):
    want = case.call(case.args())
    args = case.args()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = case.call(args, stream=stream)
    stream.synchronize()
    torch.cuda._sleep(PAUSE)
    copies = [t.clone() for t in got]
    del got
    with torch.cuda.stream(stream):
        for n in case.spaces:
            torch.full((n,), 7, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    same(copies, want)


def test_given_outputs_are_used(case):
    """With an output given there is nothing to allocate: it is written on the given stream and returned."""
    want = case.call(case.args())
    args = case.args()
    if "streams" in args:
        outs = [torch.empty_like(s["x"]) for s in args["streams"]]
        for s, o in zip(args["streams"], outs):
            s["out"] = o
    else:
        outs = [torch.empty_strided(args["x"].shape, args["x"].stride(), dtype=args["x"].dtype, device="cuda")]
        args["out"] = outs[0]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = case.call(args, stream=stream)
    stream.synchronize()
    assert all(a is b for a, b in zip(got, outs))
    same(got, want)
