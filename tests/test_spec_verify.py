"""spec_verify against a row-by-row 64-bit form; its outputs are whole numbers and have to be equal."""
from __future__ import annotations

import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ccv():
    import causal_depthwise_conv1d_fwd_gb300 as module
    from causal_depthwise_conv1d_fwd_gb300 import build

    build.build()
    return module


def make(b, s, v, seed, dtype=torch.bfloat16, draft=True, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    logits = spread * torch.randn(b, s + 1, v, generator=g)
    probs = torch.softmax(logits[:, :s] + 0.5 * torch.randn(b, s, v, generator=g), -1)
    race = torch.empty(b, s, v).exponential_(generator=g)
    tokens = (probs / race).argmax(-1).to(torch.int32) if s else torch.empty(b, 0, dtype=torch.int32)
    return {"logits": logits.to(dtype), "tokens": tokens, "uniform": torch.rand(b, s, generator=g),
            "noise": torch.empty(b, v).exponential_(generator=g).clamp_min(1e-30), "probs": probs if draft else None}


def check(ccv, d, num_drafts=None, temperature=None, place=None, err_wanted=False, **more):
    want = ref.spec_verify(d["logits"], d["tokens"], d["uniform"], d["noise"], d["probs"], num_drafts, temperature)
    on = {n: None if t is None else t.cuda() for n, t in d.items()}
    if place is not None:
        on = {n: place(n, t) for n, t in on.items()}
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ccv.spec_verify(on["logits"], on["tokens"], on["uniform"], on["noise"], on["probs"],
                          None if num_drafts is None else num_drafts.cuda(),
                          None if temperature is None else temperature.cuda(), err_count=err, **more)
    assert torch.equal(got[1].cpu(), want[1]), (got[1].cpu(), want[1])
    assert torch.equal(got[0].cpu(), want[0]), (got[0].cpu() != want[0]).nonzero()
    assert (int(err) > 0) == err_wanted
    return got


@pytest.mark.parametrize("v", [1, 2, 7, 31, 33, 255, 1000, 4097, 32003, 70001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("draft", [True, False])
def test_vocabularies(ccv, v, dtype, draft):
    check(ccv, make(6, 3, v, v, dtype, draft))


@pytest.mark.parametrize("b,s", [(1, 1), (1, 8), (33, 2), (5, 0), (70, 5)])
def test_rows_and_drafts(ccv, b, s):
    check(ccv, make(b, s, 513, b + s))
    check(ccv, make(b, s, 513, b + s, draft=False))


@pytest.mark.parametrize("b,v,dtype", [(128, 40000, torch.bfloat16), (131, 39999, torch.bfloat16), (250, 20004, torch.float32),
                                       (700, 9001, torch.bfloat16)])
def test_many_rows(ccv, b, v, dtype):
    """More shares of the vocabulary than blocks fit on the card: a block of the draw goes round several times."""
    check(ccv, make(b, 1, v, b, dtype))


def test_ragged_and_padded(ccv):
    d = make(9, 4, 1001, 3)
    check(ccv, d, num_drafts=torch.tensor([4, 0, 1, 2, 3, -1, 4, -5, 2], dtype=torch.int32))
    check(ccv, d, num_drafts=torch.tensor([-1] * 9, dtype=torch.int32))


def test_temperatures(ccv):
    for dtype in (torch.bfloat16, torch.float32):
        d = make(8, 3, 2050, 4, dtype)
        t = torch.tensor([0.0, 1.0, 0.3, 2.5, 0.0, 0.7, 0.0, 1e-3])
        d["tokens"][0] = d["logits"][0, :3].float().argmax(-1)   # greedy drafts that hold
        d["tokens"][4, 0] = d["logits"][4, 0].float().argmax(-1)
        check(ccv, d, temperature=t)
        d["probs"] = None
        check(ccv, d, temperature=t)


def test_ties_go_to_the_lowest_index(ccv):
    d = make(4, 2, 3000, 5, draft=False)
    d["logits"][:] = 0
    d["logits"][:, :, 1700:1710] = 5.0
    d["noise"][:] = 0.5
    check(ccv, d, temperature=torch.tensor([0.0, 1.0, 0.0, 1.0]))


def test_all_kept_and_none_kept(ccv):
    d = make(4, 3, 777, 6)
    d["uniform"][:] = 0.0
    got = check(ccv, d)
    assert got[1].tolist() == [4] * 4
    d["uniform"][:] = 0.999999
    d["probs"][:] = 0
    d["probs"].scatter_(2, d["tokens"].long()[..., None], 1.0)
    got = check(ccv, d)
    assert got[1].tolist() == [1] * 4


def test_masked_logits(ccv):
    inf = float("inf")
    d = make(7, 2, 900, 7)
    d["logits"][0, :, 1:] = -inf             # one token left
    d["logits"][1, 0, :] = -inf              # nothing left at the first position
    d["logits"][2] = -inf                    # nothing left at all
    d["logits"][3, :, ::2] = float("nan")    # NaN is masked
    d["logits"][4, :, 5] = inf               # +inf takes everything
    d["logits"][5] = torch.finfo(torch.bfloat16).min
    d["logits"][6, :, :899] = torch.finfo(torch.bfloat16).min
    check(ccv, d)
    check(ccv, d, temperature=torch.zeros(7))
    d["probs"] = None
    check(ccv, d)


def test_residual_empty(ccv):
    """The draft's distribution is the target's: nothing is left above it, and a rejection has no token."""
    v = 64
    d = {"logits": torch.zeros(2, 2, v), "tokens": torch.tensor([[3], [4]], dtype=torch.int32),
         "uniform": torch.tensor([[0.5], [1.0]]), "noise": torch.ones(2, v), "probs": torch.full((2, 1, v), 1.0 / v)}
    got = check(ccv, d)
    assert got[0].tolist() == [[3, 0], [-1, -1]]


def test_tokens_outside_the_vocabulary(ccv):
    d = make(3, 2, 100, 9)
    d["uniform"][:] = 0
    d["tokens"][0, 0] = 100
    d["tokens"][1, 1] = -3
    check(ccv, d, err_wanted=True)
    d["probs"] = None
    check(ccv, d, err_wanted=True)


def test_strides_and_offsets(ccv):
    """Rows at odd offsets, rows inside wider ones, positions and rows in another order."""
    def place(name, t):
        if t is None:
            return t
        if name in ("logits", "probs", "noise"):
            wide = torch.full((*t.shape[:-1], t.shape[-1] + 3), 50.0, dtype=t.dtype, device=t.device)
            wide[..., 1:-2] = t
            return wide[..., 1:-2]
        return t.t().contiguous().t()

    for v in (1000, 1001):
        for dtype in (torch.bfloat16, torch.float32):
            check(ccv, make(5, 3, v, v, dtype), place=place)
    d = make(5, 3, 640, 11)
    check(ccv, d, place=lambda n, t: t.transpose(0, 1).contiguous().transpose(0, 1) if n in ("logits", "probs") else t)


def test_streams_graphs_and_repeats(ccv):
    d = make(6, 4, 40000, 12)
    want = check(ccv, d)
    on = {n: t.cuda() for n, t in d.items()}
    args = (on["logits"], on["tokens"], on["uniform"], on["noise"], on["probs"])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = ccv.spec_verify(*args, stream=stream)
    stream.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    plan = ccv.prepare_spec_verify(*args)
    plan()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan()
    for _ in range(3):
        for t in plan.result:
            t.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(plan.result[0], want[0]) and torch.equal(plan.result[1], want[1])


def test_calls_in_a_row(ccv):
    """The draw starts before the statistics end: with all inputs written just before each call and overwritten just
    after it, calls in a row give what they give one at a time."""
    cases = [make(40, 3, 70000, seed) for seed in (21, 22, 23)]
    wants = [check(ccv, d) for d in cases]
    on = [{n: t.cuda() for n, t in d.items()} for d in cases]
    now = {n: torch.zeros_like(t) for n, t in on[0].items()}
    space = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        got = []
        for d in on:
            for n, t in d.items():
                now[n].copy_(t)
            got.append(ccv.spec_verify(now["logits"], now["tokens"], now["uniform"], now["noise"], now["probs"], workspace=space))
            for t in now.values():
                t.zero_()
        for a, b in zip(got, wants):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_counts_feed_the_next_step(ccv):
    """The counts are gdr_update's num_accepted_tokens: a verify step of tokens [last, drafts] keeps `count` states."""
    b, s, v = 3, 3, 200
    d = make(b, s, v, 13)
    _, count = check(ccv, d)
    g = torch.Generator().manual_seed(14)
    mk = lambda *sh: torch.randn(*sh, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    q, k, val = mk(b, s + 1, 1, 64), mk(b, s + 1, 1, 64), mk(b, s + 1, 1, 64)
    gate = -torch.rand(b, s + 1, 1, generator=g).cuda()
    beta = torch.rand(b, s + 1, 1, generator=g).cuda()
    lines = torch.arange(b * (s + 1), dtype=torch.int32, device="cuda").reshape(b, s + 1)
    pool = torch.randn(b * (s + 1) + b, 1, 64, 64, generator=g).cuda()
    own = torch.arange(b, dtype=torch.int32, device="cuda") + b * (s + 1)
    after = pool.clone()
    ccv.gdr_update(q, k, val, gate, beta, after, own, output_state_indices=lines)
    new = [mk(b, 1, 1, 64) for _ in range(3)]
    step = [t[:, :1].contiguous() for t in (gate, beta)]
    direct = after.clone()
    out = ccv.gdr_update(*new, *step, direct, own, num_accepted_tokens=count, output_state_indices=lines)
    for r in range(b):
        one = after[lines[r, int(count[r]) - 1].long()][None].clone()
        o = ccv.gdr_update(*(t[r:r + 1] for t in new), *(t[r:r + 1] for t in step), one)
        assert torch.equal(o[0], out[r])
