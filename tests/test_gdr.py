"""Gated delta rule: prefill and decode against the token-by-token recurrence in 64 bits."""
from __future__ import annotations

import pytest
import torch

import layer_ref as ref
from parity_util import SENTINEL, assert_bits

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ccv():
    import causal_depthwise_conv1d_fwd_gb300 as module
    from causal_depthwise_conv1d_fwd_gb300 import build

    build.build()
    return module


@pytest.fixture(params=["chunked", "recurrent", "segments1", "segments2"])
def path(request, monkeypatch):
    """The chunked form with sequences whole or cut into segments of 1 or 2 chunks, and the recurrent form."""
    cut = request.param.startswith("segments")
    monkeypatch.setenv("CCV_GDR_PATH", "chunked" if cut else request.param)
    monkeypatch.setenv("CCV_GDR_SEGMENT", request.param[-1] if cut else "0")
    return request.param


def silu_randn(shape, g):
    x = torch.randn(shape, generator=g)
    return (x * torch.sigmoid(x)).to(BF16)


def inputs(tokens, hk, hv, dk, dv, seed, raw=False):
    g = torch.Generator().manual_seed(seed)
    d = {"q": silu_randn((tokens, hk, dk), g), "k": silu_randn((tokens, hk, dk), g), "v": silu_randn((tokens, hv, dv), g)}
    if raw:
        d["g"] = torch.randn(tokens, hv, generator=g).to(BF16)
        d["beta"] = torch.randn(tokens, hv, generator=g).to(BF16)
        d["a_log"] = torch.log(1 + 15 * torch.rand(hv, generator=g))
        d["dt_bias"] = torch.randn(hv, generator=g) - 3
    else:
        d["g"] = -2.0 * torch.rand(tokens, hv, generator=g) ** 4
        d["beta"] = torch.rand(tokens, hv, generator=g)
    return d, g


def dev(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def split(d, s, e):
    g, beta = ref.gates(d["g"], d["beta"], d.get("a_log"), d.get("dt_bias"))
    return d["q"][s:e], d["k"][s:e], d["v"][s:e], g[s:e], beta[s:e]


def check_fwd(ccv, d, pool, lengths, lines=None, init=None, scale=None, l2=True, place=None, **more):
    """Runs gdr_fwd on copies and compares every sequence; returns (out, state)."""
    starts = [0]
    for n in lengths:
        starts.append(starts[-1] + n)
    total = d["v"].shape[0]
    dk = d["k"].shape[-1]
    dd = dev(d)
    if place is not None:
        for n in "qkv":
            dd[n] = place(dd[n])
    out = torch.empty(d["v"].shape, dtype=BF16, device="cuda")
    out.view(torch.int16).fill_(SENTINEL)
    if place is not None:
        out = place(out)
    state = pool.cuda().clone() if pool is not None else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(cache_indices=None if lines is None else torch.tensor(lines, dtype=torch.int32, device="cuda"),
              has_initial_state=None if init is None else torch.tensor(init, device="cuda"),
              a_log=dd.get("a_log"), dt_bias=dd.get("dt_bias"))
    got = ccv.gdr_fwd(dd["q"], dd["k"], dd["v"], dd["g"], dd["beta"], state,
                      torch.tensor(starts, dtype=torch.int32, device="cuda"), **kw, scale=scale, qk_l2norm=l2, out=out,
                      err_count=err, **more)
    torch.cuda.synchronize()
    assert got is out and int(err) == 0
    touched = torch.zeros(total, dtype=torch.bool)
    lines_seen = set()
    for i, n in enumerate(lengths):
        line = i if lines is None else lines[i]
        if line == -1 or n == 0:
            continue
        s, e = starts[i], starts[i + 1]
        touched[s:e] = True
        lines_seen.add(line)
        start = torch.zeros(d["v"].shape[1:] + (dk,), dtype=torch.float64)
        if pool is not None and init is not None and init[i]:
            start = pool[line].double()
        o, om, st, sm = ref.gdr_tokens(*split(d, s, e), start, dk ** -0.5 if scale is None else scale, l2)
        ref.assert_out(out[s:e], o, om, f"out of sequence {i}")
        if pool is not None:
            ref.assert_state(state[line], st, sm, f"state of sequence {i}")
    rest = out.cpu()[~touched]
    assert_bits(rest, torch.full(rest.shape, SENTINEL, dtype=torch.int16).view(BF16), "tokens of no sequence")
    if pool is not None:
        for line in range(pool.shape[0]):
            if line not in lines_seen:
                assert torch.equal(state[line].cpu(), pool[line]), f"line {line} was written"
    return out, state


DIMS = [(128, 128), (64, 64), (64, 128), (128, 64), (96, 80), (40, 130), (7, 5), (128, 256)]


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("hk,hv", [(1, 1), (2, 4), (1, 3)])
def test_fwd_dims_and_heads(ccv, path, dk, dv, hk, hv):
    lengths = [70, 1, 0, 129]
    d, g = inputs(sum(lengths), hk, hv, dk, dv, 1 + dk + hv)
    pool = 0.3 * torch.randn(6, hv, dv, dk, generator=g)
    check_fwd(ccv, d, pool, lengths, lines=[4, 0, 2, 5], init=[True, False, True, True])


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 127, 128, 129, 191, 192, 193, 320, 500])
def test_fwd_lengths(ccv, path, n):
    d, g = inputs(n, 1, 2, 128, 128, n, raw=n % 2 == 1)
    check_fwd(ccv, d, 0.3 * torch.randn(2, 2, 128, 128, generator=g), [n], lines=[1], init=[n % 3 != 0])


def test_fwd_many_sequences(ccv, path):
    """More sequences than a warp has lanes, some empty, some padded, lines in any order."""
    g = torch.Generator().manual_seed(5)
    lengths = [int(x) for x in torch.randint(0, 40, (83,), generator=g)]
    lengths[10] = 150
    lines = torch.randperm(90, generator=g)[:83].tolist()
    for i in (0, 40, 82):
        lines[i] = -1
    d, g = inputs(sum(lengths) + 9, 1, 2, 64, 64, 6, raw=True)
    for n in "qkv":  # what belongs to no sequence must not reach one
        at = 0
        for i, ln in enumerate(lengths):
            if lines[i] == -1:
                d[n][at:at + ln] = float("nan")
            at += ln
        d[n][at:] = float("nan")
    pool = 0.3 * torch.randn(90, 2, 64, 64, generator=g)
    check_fwd(ccv, d, pool, lengths, lines=lines, init=[i % 3 == 0 for i in range(83)])


def test_fwd_without_pool_or_indices(ccv, path):
    d, g = inputs(100, 1, 2, 128, 128, 8)
    check_fwd(ccv, d, None, [37, 63])
    check_fwd(ccv, d, 0.3 * torch.randn(2, 2, 128, 128, generator=g), [37, 63])


def test_fwd_nan_lines_without_initial_state(ccv, path):
    """A line without an initial state is not read, whatever it holds."""
    d, _ = inputs(70, 1, 1, 128, 128, 9)
    pool = torch.full((3, 1, 128, 128), float("nan"))
    starts = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    dd = dev(d)
    state = pool.cuda()
    out = ccv.gdr_fwd(dd["q"], dd["k"], dd["v"], dd["g"], dd["beta"], state, starts)
    zero = torch.zeros(1, 128, 128, dtype=torch.float64)
    o, om, st, sm = ref.gdr_tokens(*split(d, 0, 70), zero, 128 ** -0.5, True)
    ref.assert_out(out, o, om)
    ref.assert_state(state[0], st, sm)
    assert bool(state[1:].isnan().all())


@pytest.mark.parametrize("layout", ["channel_first", "interleaved", "odd_offset", "expanded_rows"])
def test_fwd_strides(ccv, path, layout):
    def place(t):
        if layout == "channel_first":      # tokens contiguous: the convolution's (dim, tokens) layout
            return t.permute(1, 2, 0).contiguous().permute(2, 0, 1)
        if layout == "interleaved":        # heads inside a wider row
            wide = torch.zeros(t.shape[0], t.shape[1] + 2, t.shape[2] + 8, dtype=t.dtype, device=t.device)
            wide[:, 1:-1, 8:] = t
            return wide[:, 1:-1, 8:]
        if layout == "odd_offset":         # 2-byte aligned only
            flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device=t.device)
            flat[1:] = t.flatten()
            return flat[1:].view(t.shape)
        return t.transpose(0, 1).contiguous().transpose(0, 1)

    d, g = inputs(150, 2, 4, 128, 128, 10)
    check_fwd(ccv, d, 0.3 * torch.randn(2, 4, 128, 128, generator=g), [81, 69], init=[True, True], place=place)


def test_fwd_state_strides(ccv, path):
    """A pool whose key axis is not the innermost."""
    d, g = inputs(100, 1, 2, 64, 64, 11)
    pool = 0.3 * torch.randn(2, 2, 64, 64, generator=g)
    dd = dev(d)
    starts = torch.tensor([0, 30, 100], dtype=torch.int32, device="cuda")
    init = torch.tensor([True, True], device="cuda")
    plain = pool.cuda().clone()
    a = ccv.gdr_fwd(dd["q"], dd["k"], dd["v"], dd["g"], dd["beta"], plain, starts, has_initial_state=init)
    turned = pool.cuda().transpose(2, 3).contiguous().transpose(2, 3)
    b = ccv.gdr_fwd(dd["q"], dd["k"], dd["v"], dd["g"], dd["beta"], turned, starts, has_initial_state=init)
    assert_bits(a, b)
    assert torch.equal(plain, turned)


@pytest.mark.parametrize("kind", ["reset", "deep", "tiny", "none", "mixed"])
def test_fwd_decays(ccv, path, kind):
    d, g = inputs(200, 1, 2, 128, 128, 12)
    if kind == "reset":                    # the state is cleared now and then
        d["g"][::50] = -torch.inf
        d["g"][130] = -3e38
    elif kind == "deep":                   # e^g underflows over a chunk
        d["g"] = -30.0 * torch.rand(200, 2, generator=g)
    elif kind == "tiny":
        d["g"] = -1e-6 * torch.rand(200, 2, generator=g)
    elif kind == "none":
        d["g"].zero_()
    else:
        d["g"][:, 0] = 0
        d["g"][:, 1] = -torch.inf
    check_fwd(ccv, d, 0.3 * torch.randn(1, 2, 128, 128, generator=g), [200], init=[True])


@pytest.mark.parametrize("kind", ["beta0", "beta2", "same_keys", "zero_keys", "zero_values", "zero_queries", "tiny_beta"])
def test_fwd_strengths_and_keys(ccv, path, kind):
    d, g = inputs(150, 1, 2, 128, 128, 13)
    if kind == "beta0":
        d["beta"][20:90] = 0
    elif kind == "beta2":
        d["beta"] = 2 * d["beta"]
    elif kind == "same_keys":
        d["k"][:] = d["k"][0]
    elif kind == "zero_keys":
        d["k"][10:80] = 0
    elif kind == "zero_values":
        d["v"].zero_()
    elif kind == "zero_queries":
        d["q"].zero_()
    else:
        d["beta"] = 1e-6 * d["beta"]
    init = kind != "tiny_beta"
    check_fwd(ccv, d, 0.3 * torch.randn(1, 2, 128, 128, generator=g), [150], init=[init])


@pytest.mark.parametrize("size", [1e-12, 1e-3, 1e4, 1e12])
def test_fwd_scales(ccv, path, size):
    """Values and states of any size, and rows of very different sizes: each row of the state is linear in its own."""
    d, g = inputs(180, 1, 1, 128, 128, 14)
    rows = torch.exp(4 * torch.randn(128, generator=g))
    d["v"] = (d["v"].float() * size * rows).to(BF16)
    pool = 0.3 * size * rows[:, None] * torch.randn(2, 1, 128, 128, generator=g)
    check_fwd(ccv, d, pool, [100, 80], init=[True, False])


@pytest.mark.parametrize("key_size", [0.02, 1.0, 40.0])
def test_fwd_keys_not_normalised(ccv, path, key_size):
    """qk_l2norm off: keys of any size with b |k|^2 <= 2."""
    d, g = inputs(150, 1, 2, 128, 128, 15)
    norm = d["k"].float().norm(dim=-1, keepdim=True)
    d["k"] = (d["k"].float() / norm * key_size).to(BF16)
    d["beta"] = d["beta"] / key_size ** 2
    check_fwd(ccv, d, 0.3 / key_size * torch.randn(1, 2, 128, 128, generator=g), [150], init=[True], l2=False, scale=0.7)


def test_fwd_growing_state(ccv, path):
    """Values that grow a thousandfold from chunk to chunk, then vanish."""
    d, g = inputs(640, 1, 1, 128, 128, 16)
    d["g"].zero_()
    steps = torch.tensor([1e-6, 1e-3, 1, 1e3, 1e6, 1e9, 1e3, 1, 0, 1e-3]).repeat_interleave(64)
    d["v"] = (d["v"].float() * steps[:, None, None]).to(BF16)
    check_fwd(ccv, d, torch.zeros(1, 1, 128, 128), [640])


def test_fwd_one_nan_row(ccv, path):
    """A NaN value makes its own row of the state NaN and no other."""
    d, _ = inputs(100, 1, 1, 128, 128, 17)
    clean = {k: v.clone() for k, v in d.items()}
    d["v"][40, 0, 77] = float("nan")
    starts = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    outs = []
    for x in (d, clean):
        dd, state = dev(x), torch.zeros(1, 1, 128, 128, device="cuda")
        outs.append((ccv.gdr_fwd(dd["q"], dd["k"], dd["v"], dd["g"], dd["beta"], state, starts), state))
    rows = torch.arange(128, device="cuda") != 77
    assert_bits(outs[0][0][:, :, rows], outs[1][0][:, :, rows])
    assert torch.equal(outs[0][1][:, :, rows], outs[1][1][:, :, rows])
    assert bool(outs[0][1][:, :, 77].isnan().all())


def test_fwd_bad_indices_are_counted(ccv, path):
    d, g = inputs(50, 1, 1, 64, 64, 18)
    dd = dev(d)
    pool = torch.randn(2, 1, 64, 64, generator=g).cuda()
    for starts, lines in (([0, 30, 20], [0, 1]), ([0, 30, 51], [0, 1]), ([0, 30, 50], [0, 2]), ([-1, 30, 50], [0, 1])):
        state, err = pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        ccv.gdr_fwd(dd["q"], dd["k"], dd["v"], dd["g"], dd["beta"], state,
                    torch.tensor(starts, dtype=torch.int32, device="cuda"),
                    torch.tensor(lines, dtype=torch.int32, device="cuda"), err_count=err)
        assert int(err) > 0
        bad = 0 if starts[0] < 0 else 1
        assert torch.equal(state[bad], pool[bad])
        assert not torch.equal(state[1 - bad], pool[1 - bad])


def test_fwd_other_stream_and_graph(ccv, path):
    d, g = inputs(200, 2, 4, 128, 128, 19, raw=True)
    pool = 0.3 * torch.randn(3, 4, 128, 128, generator=g)
    want, state = check_fwd(ccv, d, pool, [130, 0, 70], init=[True, True, True])
    dd = dev(d)
    starts = torch.tensor([0, 130, 130, 200], dtype=torch.int32, device="cuda")
    init = torch.tensor([True] * 3, device="cuda")
    got_state = pool.cuda().clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = ccv.gdr_fwd(dd["q"], dd["k"], dd["v"], dd["g"], dd["beta"], got_state, starts, None, init, a_log=dd["a_log"],
                      dt_bias=dd["dt_bias"], stream=stream)
    stream.synchronize()
    assert_bits(got, want)
    assert torch.equal(got_state, state)
    plan_state = pool.cuda().clone()
    plan = ccv.prepare_gdr_fwd(dd["q"], dd["k"], dd["v"], dd["g"], dd["beta"], plan_state, starts, None, init,
                               a_log=dd["a_log"], dt_bias=dd["dt_bias"])
    plan()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan()
    for _ in range(2):
        plan.result.zero_()
        plan_state.copy_(pool.cuda())
        graph.replay()
        torch.cuda.synchronize()
        assert_bits(plan.result, want)
        assert torch.equal(plan_state, state)


def test_fwd_is_deterministic(ccv, path):
    d, g = inputs(700, 2, 4, 128, 128, 20)
    pool = 0.3 * torch.randn(2, 4, 128, 128, generator=g).cuda()
    dd = dev(d)
    starts = torch.tensor([0, 333, 700], dtype=torch.int32, device="cuda")
    first = None
    for _ in range(5):
        state = pool.clone()
        out = ccv.gdr_fwd(dd["q"], dd["k"], dd["v"], dd["g"], dd["beta"], state, starts,
                          has_initial_state=torch.tensor([True, True], device="cuda"))
        if first is None:
            first = out, state
        assert_bits(out, first[0])
        assert torch.equal(state, first[1])


def test_fwd_cut_by_itself(ccv):
    """A long prompt with few heads, which the host cuts into segments without being told to."""
    d, g = inputs(2500, 1, 1, 128, 128, 22, raw=True)
    pool = 0.3 * torch.randn(3, 1, 128, 128, generator=g)
    check_fwd(ccv, d, pool, [2300, 0, 200], lines=[2, 1, 0], init=[True, True, False])


def test_fwd_split_is_continuation(ccv):
    """A prompt in two calls, the second from the first's state, is the prompt in one call (up to rounding)."""
    d, _ = inputs(300, 1, 2, 128, 128, 21)
    dd = dev(d)
    whole, parts = torch.zeros(1, 2, 128, 128, device="cuda"), torch.zeros(1, 2, 128, 128, device="cuda")

    def call(s, e, state, init):
        return ccv.gdr_fwd(*(dd[n][s:e] for n in ("q", "k", "v", "g", "beta")), state,
                           torch.tensor([0, e - s], dtype=torch.int32, device="cuda"),
                           has_initial_state=torch.tensor([init], device="cuda"))

    a = call(0, 300, whole, False)
    b = torch.cat([call(0, 111, parts, False), call(111, 300, parts, True)])
    zero = torch.zeros(2, 128, 128, dtype=torch.float64)
    o, om, st, sm = ref.gdr_tokens(*split(d, 0, 300), zero, 128 ** -0.5, True)
    for out, state in ((a, whole), (b, parts)):
        ref.assert_out(out, o, om)
        ref.assert_state(state[0], st, sm)


# ------------------------------------------------------------------ decode ----

def check_update(ccv, d, pool, b, t, lines=None, nacc=None, olines=None, place=None, scale=None, l2=True):
    """d holds (b * t, ...) tokens; compares every row and every line of the pool."""
    dk = d["k"].shape[-1]
    dd = dev(d)
    shaped = {n: dd[n].unflatten(0, (b, t)) if t > 1 else dd[n] for n in ("q", "k", "v", "g", "beta")}
    if place is not None:
        for n in "qkv":
            shaped[n] = place(shaped[n])
    out = torch.empty(shaped["v"].shape, dtype=BF16, device="cuda")
    out.view(torch.int16).fill_(SENTINEL)
    state = pool.cuda().clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    as_int = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got = ccv.gdr_update(shaped["q"], shaped["k"], shaped["v"], shaped["g"], shaped["beta"], state, as_int(lines),
                         as_int(nacc), as_int(olines), scale=scale, qk_l2norm=l2, a_log=dd.get("a_log"),
                         dt_bias=dd.get("dt_bias"), out=out, err_count=err)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.data_ptr() and got.shape == out.shape and int(err) == 0
    out = out.reshape(b, t, *d["v"].shape[1:])
    written = {}
    for r in range(b):
        line = r if lines is None else lines[r]
        if line == -1:
            rest = out[r].cpu()
            assert_bits(rest, torch.full(rest.shape, SENTINEL, dtype=torch.int16).view(BF16), "padded row")
            continue
        start = pool[olines[r][nacc[r] - 1] if nacc is not None else line].double()
        keep = []
        o, om, st, sm = ref.gdr_tokens(*split(d, r * t, (r + 1) * t), start,
                                       dk ** -0.5 if scale is None else scale, l2, keep)
        ref.assert_out(out[r], o, om, f"out of row {r}")
        if olines is None:
            written[line] = (st, sm)
        else:
            for i in range(t):
                if olines[r][i] >= 0:
                    written[olines[r][i]] = keep[i]
    for line in range(pool.shape[0]):
        if line in written:
            ref.assert_state(state[line], *written[line], f"line {line}")
        else:
            assert torch.equal(state[line].cpu(), pool[line]), f"line {line} was written"


@pytest.mark.parametrize("dk,dv", DIMS + [(256, 64), (200, 33), (1, 1)])
@pytest.mark.parametrize("raw", [False, True])
def test_update_dims(ccv, dk, dv, raw):
    d, g = inputs(5, 2, 4, dk, dv, dk + dv, raw=raw)
    check_update(ccv, d, torch.randn(7, 4, dv, dk, generator=g), 5, 1, lines=[6, -1, 0, 3, 2])


@pytest.mark.parametrize("b,hk,hv", [(1, 1, 1), (1, 16, 32), (3, 2, 2), (67, 1, 3)])
def test_update_rows(ccv, b, hk, hv):
    d, g = inputs(b, hk, hv, 128, 128, b + hv, raw=True)
    check_update(ccv, d, torch.randn(b, hv, 128, 128, generator=g), b, 1)


@pytest.mark.parametrize("t", [2, 4, 7])
@pytest.mark.parametrize("dk,dv", [(128, 128), (96, 80)])
def test_update_several_tokens(ccv, t, dk, dv):
    d, g = inputs(3 * t, 1, 2, dk, dv, t)
    check_update(ccv, d, torch.randn(4, 2, dv, dk, generator=g), 3, t, lines=[3, 0, 1])


@pytest.mark.parametrize("t", [1, 3, 5])
def test_update_speculative(ccv, t):
    """Per-step states and the start at the last kept token's state, over two rounds' worth of counts."""
    b = 4
    d, g = inputs(b * t, 2, 4, 128, 128, 30 + t, raw=True)
    pool = torch.randn(b * t + 5, 4, 128, 128, generator=g)
    olines = (torch.randperm(b * t, generator=g) + 5).reshape(b, t).tolist()
    lines = [0, 1, -1, 2]
    check_update(ccv, d, pool, b, t, lines=lines, olines=olines)
    nacc = torch.randint(1, t + 1, (b,), generator=g).tolist()
    check_update(ccv, d, pool, b, t, lines=lines, olines=olines, nacc=nacc)
    if t > 1:
        olines[0][1] = -1
        nacc[0] = 1
        check_update(ccv, d, pool, b, t, lines=lines, olines=olines, nacc=nacc)


def test_update_strides(ccv):
    d, g = inputs(6, 2, 4, 128, 128, 33)
    pool = torch.randn(6, 4, 128, 128, generator=g)

    def channel_first(x):
        return x.permute(1, 2, 0).contiguous().permute(2, 0, 1)

    def odd(x):
        flat = torch.zeros(x.numel() + 1, dtype=x.dtype, device=x.device)
        flat[1:] = x.flatten()
        return flat[1:].view(x.shape)

    for place in (channel_first, odd):
        check_update(ccv, d, pool, 6, 1, place=place)


def test_update_decays_and_norms(ccv):
    d, g = inputs(6, 1, 2, 128, 128, 34)
    d["g"][0] = -torch.inf
    d["g"][1] = -200
    d["g"][2] = 0
    d["beta"][3] = 0
    d["k"][4] = 0
    check_update(ccv, d, torch.randn(6, 2, 128, 128, generator=g), 6, 1)
    check_update(ccv, d, torch.randn(6, 2, 128, 128, generator=g), 6, 1, l2=False, scale=0.5)


def test_update_bad_indices_are_counted(ccv):
    d, g = inputs(4, 1, 1, 64, 64, 35)
    dd = dev(d)
    pool = torch.randn(4, 1, 64, 64, generator=g).cuda()
    sh = {n: dd[n].unflatten(0, (2, 2)) for n in ("q", "k", "v", "g", "beta")}
    ol = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")

    def call(**kw):
        state, err = pool.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        ccv.gdr_update(*sh.values(), state, err_count=err, **kw)
        return state, int(err)

    as_int = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    state, err = call(state_indices=as_int(4, 1))
    assert err > 0 and torch.equal(state[[0, 2, 3]], pool[[0, 2, 3]]) and not torch.equal(state[1], pool[1])
    state, err = call(state_indices=as_int(0, -7))
    assert err > 0 and torch.equal(state[1:], pool[1:])
    for bad in (0, 3, -1):
        state, err = call(output_state_indices=ol, num_accepted_tokens=as_int(bad, 1))
        assert err > 0 and torch.equal(state[:2], pool[:2]) and not torch.equal(state[2:], pool[2:])
    state, err = call(output_state_indices=torch.tensor([[0, 9], [2, 3]], dtype=torch.int32, device="cuda"),
                      num_accepted_tokens=as_int(1, 1))
    assert err > 0 and not torch.equal(state[0], pool[0]) and torch.equal(state[1], pool[1])


def test_update_matches_prefill(ccv):
    """A prompt token by token through gdr_update ends in gdr_fwd's state."""
    d, _ = inputs(40, 1, 2, 128, 128, 36)
    dd = dev(d)
    one, many = torch.zeros(1, 2, 128, 128, device="cuda"), torch.zeros(1, 2, 128, 128, device="cuda")
    a = ccv.gdr_fwd(*(dd[n] for n in ("q", "k", "v", "g", "beta")), one, torch.tensor([0, 40], dtype=torch.int32, device="cuda"))
    b = torch.cat([ccv.gdr_update(*(dd[n][t:t + 1] for n in ("q", "k", "v", "g", "beta")), many) for t in range(40)])
    zero = torch.zeros(2, 128, 128, dtype=torch.float64)
    o, om, st, sm = ref.gdr_tokens(*split(d, 0, 40), zero, 128 ** -0.5, True)
    for out, state in ((a, one), (b, many)):
        ref.assert_out(out, o, om)
        ref.assert_state(state[0], st, sm)


def test_update_past_32_bits(ccv):
    """State lines whose offsets pass 2^31 elements and q/k/v rows with wide strides."""
    lines = (1 << 31) // (2 * 128 * 128) + 3
    state = torch.empty(lines, 2, 128, 128, device="cuda")
    d, g = inputs(2, 1, 2, 128, 128, 37)
    start = torch.randn(2, 2, 128, 128, generator=g)
    idx = [lines - 1, 5]
    for i, line in enumerate(idx):
        state[line] = start[i].cuda()
    dd = dev(d)
    out = ccv.gdr_update(dd["q"], dd["k"], dd["v"], dd["g"], dd["beta"], state,
                         torch.tensor(idx, dtype=torch.int32, device="cuda"))
    for i, line in enumerate(idx):
        o, om, st, sm = ref.gdr_tokens(*split(d, i, i + 1), start[i].double(), 128 ** -0.5, True)
        ref.assert_out(out[i:i + 1], o, om)
        ref.assert_state(state[line], st, sm)


@pytest.mark.parametrize("heads", [(1, 2), (16, 32)])
def test_fwd_calls_in_a_row(ccv, path, heads):
    """Kernels start before the ones ahead of them end: calls that go on from each other's states, with one workspace and
    with inputs and indices written just before each, give the bits that they give one at a time."""
    hk, hv = heads
    d, g = inputs(700, hk, hv, 64, 64, 31)
    dd = dev(d)
    seed = torch.randn(4, hv, 64, 64, generator=g).cuda()
    starts = torch.tensor([0, 300, 300, 429, 700], dtype=torch.int32, device="cuda")
    lines = torch.tensor([2, 0, 3, 1], dtype=torch.int32, device="cuda")
    init = torch.tensor([True, True, False, True], device="cuda")
    space = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")

    def run(wait):
        state, outs = seed.clone(), []
        q, k, v = (torch.empty_like(dd[n]) for n in "qkv")
        qsl, idx, flags = torch.zeros_like(starts), torch.full_like(lines, -1), torch.zeros_like(init)
        for step in range(6):
            for to, of in ((q, dd["q"]), (k, dd["k"]), (v, dd["v"])):
                to.copy_(of.roll(step, 0))
            qsl.copy_(starts)
            idx.copy_(lines.roll(step))
            flags.copy_(init | (step % 2 == 1))
            outs.append(ccv.gdr_fwd(q, k, v, dd["g"], dd["beta"], state, qsl, idx, flags, workspace=space))
            if wait:
                torch.cuda.synchronize()
            for t in (q, k, v):
                t.fill_(float("nan"))
            qsl.zero_()
            idx.fill_(-1)
            if wait:
                torch.cuda.synchronize()
        return outs, state

    one_by_one = run(True)
    for _ in range(3):
        outs, state = run(False)
        assert torch.equal(state, one_by_one[1])
        for got, want in zip(outs, one_by_one[0]):
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))
