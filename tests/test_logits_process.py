"""logits_process against a row-by-row 64-bit form: 32-bit sums of a few terms, rounded once to the output's type."""
from __future__ import annotations

import pytest
import torch

import ssm_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ccv():
    import causal_depthwise_conv1d_fwd_gb300 as module
    from causal_depthwise_conv1d_fwd_gb300 import build

    build.build()
    return module


def i32(*v):
    return torch.tensor(v, dtype=torch.int32)


def make(b, n, v, size, seed, kind=BF16, bias=0, mask=True):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=g)  # noqa: E731
    ids = lambda *s: (v * rand(*s) ** 3).to(torch.int32).clamp(max=v - 1)  # noqa: E731
    lengths = (1 + size * rand(b)).to(torch.int32).clamp(max=size)
    d = {"x": (3 * torch.randn(b, n, v, generator=g)).to(kind), "history": ids(b, size), "lengths": lengths,
         "prompts": (lengths * rand(b)).to(torch.int32), "drafts": ids(b, n - 1) if n > 1 else None,
         "repetition": 0.7 + rand(b), "frequency": rand(b) - 0.3, "presence": rand(b) - 0.5}
    if bias:
        d["bias_ids"], d["bias"] = ids(b, bias), torch.randn(b, bias, generator=g)
    if mask:
        words = torch.randint(-2 ** 31, 2 ** 31, (b, n, (v + 31) // 32), generator=g)
        d["mask"] = words.to(torch.int32)
    return d


NAMES = {"lengths": "history_lengths", "prompts": "prompt_lengths", "indices": "history_indices", "drafts": "draft_tokens"}


def call(ccv, d, **kw):
    on = {NAMES.get(k, k): None if t is None else t.cuda() for k, t in d.items() if k != "x"}
    return ccv.logits_process(kw.pop("logits") if "logits" in kw else d["x"].cuda(), **on, **kw)


def check(ccv, d, kind=None, err_wanted=False):
    """Out of place and, in the same type, in place; both give the same."""
    want, size = ref.logits(**d)
    kind = kind or d["x"].dtype
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    results = []
    for place in ([False, True] if kind is d["x"].dtype else [False]):
        logits = d["x"].cuda()
        out = logits if place else torch.full(logits.shape, float("nan"), dtype=kind, device="cuda")
        got = call(ccv, d, logits=logits, out=out, err_count=err)
        assert got is out
        results.append(got.cpu().double())
        if not place:
            assert torch.equal(logits.cpu().view(torch.uint8), d["x"].view(torch.uint8))
    got, told = results[0], ~want.isnan()
    assert torch.equal(got.isnan(), ~told)
    finite = want.isfinite()
    assert torch.equal(got[told & ~finite], want[told & ~finite])
    # half a step of the output's type, and a step of 2^-24 for each of up to 8 operations and of a bias list's sum
    step = 2.0 ** -8 if kind is BF16 else 2.0 ** -24
    bound = step * want.abs() + 2.0 ** -20 * size
    assert bool(((got - want).abs() <= bound)[finite].all()), float(((got - want).abs() / bound)[finite].max())
    if len(results) > 1:
        kept = torch.where(told, got, d["x"].double())
        assert torch.equal(results[1], kept)
    assert (int(err) > 0) == err_wanted
    return got


@pytest.mark.parametrize("v", [1, 2, 31, 32, 33, 1000, 4097, 8191, 8192, 8193, 32003])
@pytest.mark.parametrize("kind", [BF16, F32])
def test_vocabularies(ccv, v, kind):
    check(ccv, make(3, 3, v, 60, v, kind, bias=7))
    check(ccv, make(3, 1, v, 60, v, kind, mask=False))


@pytest.mark.parametrize("b,n,size", [(1, 1, 1), (1, 9, 5000), (70, 2, 33), (5, 4, 0), (300, 1, 17)])
def test_rows_positions_histories(ccv, b, n, size):
    check(ccv, make(b, n, 3001, size, b + n, bias=3))


def test_types(ccv):
    check(ccv, make(4, 2, 5000, 100, 1, BF16), kind=F32)
    check(ccv, make(4, 2, 5000, 100, 2, F32), kind=BF16)


@pytest.mark.parametrize("left_out", ["history", "prompts", "drafts", "repetition", "frequency", "presence", "bias", "mask"])
def test_each_argument_may_be_missing(ccv, left_out):
    d = make(4, 3, 3000, 50, 3, bias=5)
    for name in {"history": ("history", "lengths", "prompts"), "bias": ("bias", "bias_ids")}.get(left_out, (left_out,)):
        del d[name]
    check(ccv, d)


def test_nothing_to_do_copies(ccv):
    x = torch.randn(3, 2, 777).to(BF16).cuda()
    assert torch.equal(ccv.logits_process(x), x)
    assert torch.equal(ccv.logits_process(x[:, 0]), x[:, 0])
    y = x.clone()
    assert ccv.logits_process(y, out=y) is y and torch.equal(x, y)


def test_lines_and_padded_rows(ccv):
    d = make(6, 2, 2000, 40, 4, bias=4)
    d["indices"] = i32(5, -1, 0, 3, 3, -1)
    check(ccv, d)
    d["indices"] = i32(5, 6, 0, 3, -2, 1)
    check(ccv, d, err_wanted=True)


def test_tokens_outside_the_vocabulary(ccv):
    d = make(4, 3, 100, 40, 5, bias=4)
    d["history"][0, :3] = -1
    d["drafts"][1, 0] = -5
    d["bias_ids"][2, 1] = -1
    check(ccv, d)
    for name, at in (("history", (0, 0)), ("drafts", (1, 1)), ("bias_ids", (3, 2))):
        e = {k: t.clone() for k, t in d.items()}
        e[name][at] = 100
        check(ccv, e, err_wanted=True)
        e[name][at] = 2 ** 31 - 1
        check(ccv, e, err_wanted=True)


def test_lengths_outside_the_history(ccv):
    for name, value in (("lengths", 41), ("lengths", -1), ("prompts", 41), ("prompts", -3)):
        d = make(4, 1, 500, 40, 6)
        d[name][2] = value
        check(ccv, d, err_wanted=True)


def test_one_token_all_the_time(ccv):
    """Counts of thousands in one entry, the same id many times in the bias list, a draft that repeats."""
    d = make(2, 5, 900, 6000, 7, F32, bias=30)
    d["history"][:] = 17
    d["lengths"][:] = 6000
    d["drafts"][:] = 17
    d["bias_ids"][:] = 17
    check(ccv, d)


def test_masks(ccv):
    d = make(3, 2, 1000, 20, 8)
    d["mask"][0] = 0                         # nothing may follow
    d["mask"][1] = -1                        # everything
    got = check(ccv, d)
    assert bool((got[0] == -float("inf")).all()) and bool(got[1].isfinite().all())


def test_values_at_the_ends(ccv):
    """Infinities, NaN and the types' ends, in places that the mask leaves and in ones that it takes."""
    for kind in (BF16, F32):
        d = make(2, 1, 256, 30, 9, kind)
        del d["mask"]
        inf, top = float("inf"), torch.finfo(kind).max
        d["x"][:, :, 0:3] = torch.tensor([inf, -inf, -top])
        d["repetition"][:] = 1.0             # keeps the largest values in range
        d["presence"][:], d["frequency"][:] = 0.0, 0.0
        check(ccv, d)
        d["x"][0, 0, 7] = float("nan")
        got = call(ccv, d)
        assert bool(got[0, 0, 7].isnan()) and int(got.isnan().sum()) == 1
        d["mask"] = torch.zeros(2, 1, 8, dtype=torch.int32)
        assert bool((call(ccv, d) == -inf).all())
        logits = d["x"].cuda()
        assert bool((call(ccv, d, logits=logits, out=logits) == -inf).all())


def test_strides(ccv):
    """Rows at odd offsets, rows inside wider ones, positions and rows in another order, one mask for all positions."""
    d = make(5, 3, 3001, 50, 10, bias=6)
    want = call(ccv, d)

    def wide(t, extra=5, first=1):
        big = torch.zeros(*t.shape[:-1], t.shape[-1] + extra, dtype=t.dtype, device="cuda")
        big[..., first:first + t.shape[-1]] = t.cuda()
        return big[..., first:first + t.shape[-1]]

    x = wide(d["x"].transpose(0, 1).contiguous()).transpose(0, 1)
    e = {k: wide(t) if k in ("history", "bias", "bias_ids", "mask") else t.cuda() for k, t in d.items()}
    e["drafts"] = d["drafts"].t().contiguous().cuda().t()
    for first in range(9):
        out = wide(torch.zeros(5, 3, 3001, dtype=BF16), 9, first)
        assert torch.equal(call(ccv, e, logits=x, out=out), want)
    assert torch.equal(call(ccv, e, logits=x, out=x), want)
    d["mask"] = d["mask"][:, :1].expand(5, 3, -1)
    check(ccv, d)


def test_two_dimensions(ccv):
    d = make(4, 1, 2000, 30, 11)
    want = call(ccv, d)
    d["x"], d["mask"], d["drafts"] = d["x"][:, 0], d["mask"][:, 0], None
    assert torch.equal(call(ccv, d), want[:, 0])


def test_captured_and_replayed(ccv):
    d, e = make(6, 3, 20000, 500, 12), make(6, 3, 20000, 500, 13)
    want = [call(ccv, t) for t in (d, e)]
    on = {NAMES.get(k, k): t.cuda() for k, t in d.items()}
    logits = on.pop("x")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ccv.logits_process(logits, **on)
    for t, w in ((d, want[0]), (e, want[1])):
        logits.copy_(t["x"])
        for k, v in t.items():
            if k != "x":
                on[NAMES.get(k, k)].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


def test_drafts_are_verified_after_it(ccv):
    """Its output is what spec_verify reads: a masked draft is rejected, and no masked token is drawn."""
    b, n, v = 8, 3, 5000
    d = make(b, n, v, 60, 14)
    out = call(ccv, d)
    drafts = d["drafts"].cuda()
    noise = torch.empty(b, v, device="cuda").exponential_(generator=torch.Generator(device="cuda").manual_seed(1))
    tokens, count = ccv.spec_verify(out, drafts, torch.zeros(b, n - 1, device="cuda"), noise)
    for r in range(b):
        kept = int(count[r])
        for i in range(kept):
            token = int(tokens[r, i])
            assert (int(d["mask"][r, i, token // 32]) >> (token % 32)) & 1 == 1


@pytest.mark.parametrize("size", [12000, 13000, 40000])
def test_long_histories(ccv, size):
    """Histories around what a row's hash table takes in place, and far beyond; many different tokens, and few."""
    d = make(2, 2, 20000, size, 15, F32, mask=False)
    d["lengths"][:] = size
    d["history"][0] = torch.arange(size, dtype=torch.int32) % 20000
    check(ccv, d)


def test_dense_and_sparse_shares(ccv):
    """Every token of a share seen, and shares with one: both ways that a warp treats its vectors."""
    for kind in (BF16, F32):
        d = make(3, 2, 30000, 9000, 16, kind)
        d["lengths"][:] = 9000
        d["history"][0] = 8192 + torch.arange(9000, dtype=torch.int32) % 8192
        d["history"][1] = 77
        check(ccv, d)
        check(ccv, {**d, "x": d["x"]}, kind=BF16 if kind is F32 else F32)


def test_offsets_past_32_bits(ccv):
    d = make(2, 1, 5000, 30, 17)
    want = call(ccv, d)
    far = torch.empty(2 ** 31 + 2 ** 20, dtype=BF16, device="cuda").as_strided((2, 1, 5000), (2 ** 31 + 64, 5000, 1))
    far.copy_(d["x"])
    out = torch.empty(2 ** 31 + 2 ** 20, dtype=BF16, device="cuda").as_strided((2, 1, 5000), (2 ** 31 + 64, 5000, 1))
    assert torch.equal(call(ccv, d, logits=far, out=out), want)
    assert torch.equal(call(ccv, d, logits=far, out=far), want)


@pytest.mark.parametrize("b,n,size", [(1, 9, 5000), (2, 5, 900), (70, 3, 3000), (330, 3, 900), (200, 2, 5000)])
def test_positions_of_a_row_in_one_block_and_in_several(ccv, b, n, size):
    """Without a mask, so that in place a row's table serves all of its positions, or each position has one."""
    check(ccv, make(b, n, 2001, size, 7 * b + n, bias=3, mask=False))
