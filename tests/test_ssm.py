"""The selective state space scan, over prompts and over new tokens, against 64-bit forms with derived bounds."""
from __future__ import annotations

import os

import pytest
import torch

import ssm_ref as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
INF = float("inf")


@pytest.fixture(scope="module")
def ccv():
    import causal_depthwise_conv1d_fwd_gb300 as module
    from causal_depthwise_conv1d_fwd_gb300 import build

    build.build()
    return module


@pytest.fixture
def path(monkeypatch):
    """Forces a form of ssm_fwd, and the chunks of a segment."""
    def force(name, segment=None):
        monkeypatch.setenv("CCV_SSM_PATH", name)
        if segment is not None:
            monkeypatch.setenv("CCV_SSM_SEGMENT", str(segment))
    return force


def make(tokens, heads, dim, groups, states, seed, per_state=False, kind=BF16, gated=False, strong=False):
    """x (tokens, heads, dim), and the weights of a layer whose decays span the usual range (strong: up to e^-50 a token)."""
    g = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    a = -(1 + 15 * torch.rand(heads, generator=g)) * (20 if strong else 1)
    if per_state:
        a = -(1 + torch.arange(states)) * torch.exp(0.1 * normal(heads, states))
    bias = torch.log(torch.expm1(10 ** (-3 + 2 * torch.rand(heads, generator=g))))
    return {"x": normal(tokens, heads, dim).to(BF16), "dt": normal(tokens, heads).to(kind), "A": a,
            "B": normal(tokens, groups, states).to(BF16), "C": normal(tokens, groups, states).to(BF16), "D": normal(heads),
            "z": normal(tokens, heads, dim).to(BF16) if gated else None, "dt_bias": bias}


def pool(lines, heads, dim, states, seed):
    return torch.randn(lines, heads, dim, states, generator=torch.Generator().manual_seed(1000 + seed))


def cuda(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def check_fwd(ccv, t, lengths, init=None, lines=None, num_lines=None, seed=0, channels=False, state=True, err_wanted=False, **kw):
    """One call against the reference; returns (out, pool)."""
    h, p = t["x"].shape[1:]
    n = t["B"].shape[2]
    starts = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32)
    s = pool(num_lines or len(lengths), h, p, n, seed) if state else None
    want, bound, after, mag = ref.ssm_fwd(**t, state=s, starts=starts, lines=lines, init=init, **kw)
    on = cuda(t)
    got = None if s is None else s.cuda()
    if channels:
        on = {k: v[:, :, 0] if k in ("x", "z") and v is not None else v for k, v in on.items()}
        got = got[:, :, 0] if got is not None else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(on["x"].shape, float("nan"), dtype=BF16, device="cuda")
    given = {k: None if v is None else torch.tensor(v, device="cuda") if isinstance(v, list) else v.cuda()
             for k, v in (("cache_indices", lines), ("has_initial_state", init))}
    ccv.ssm_fwd(on["x"], on["dt"], on["A"], on["B"], on["C"], got, starts.cuda(), **given, D=on["D"], z=on["z"],
                dt_bias=on["dt_bias"], out=out, err_count=err, **kw)
    torch.cuda.synchronize()
    full = out.reshape(want.shape).cpu()
    told = ~want.isnan()
    assert torch.equal(full.isnan(), ~told)
    ref.assert_out(torch.where(told, full.double(), 0), want.nan_to_num(), bound)
    if s is not None:
        ref.assert_state(got.reshape(after.shape), after, mag)
    assert (int(err) > 0) == err_wanted
    return out, got


SHAPES = [(4, 64, 1, 128), (2, 64, 2, 128), (3, 64, 1, 64), (2, 128, 1, 128), (2, 80, 2, 96), (4, 32, 2, 16), (2, 33, 1, 100),
          (1, 1, 1, 1), (2, 200, 1, 7), (2, 64, 1, 256), (5, 8, 1, 37)]


@pytest.mark.parametrize("form", ["recurrent", "chunked"])
@pytest.mark.parametrize("heads,dim,groups,states", SHAPES)
def test_fwd_shapes(ccv, path, form, heads, dim, groups, states):
    path(form)
    lengths = [37, 1, 0, 64, 130, 300]
    t = make(sum(lengths), heads, dim, groups, states, heads + dim)
    check_fwd(ccv, t, lengths, init=[True, False, True, True, True, False])


@pytest.mark.parametrize("form", ["recurrent", "chunked"])
@pytest.mark.parametrize("lengths", [[1], [2], [63], [64], [65], [127], [128], [129], [255], [256], [257], [1, 1, 1, 1], [0, 5, 0],
                                     [128, 128], [511, 3, 640]])
def test_fwd_lengths(ccv, path, form, lengths):
    path(form)
    t = make(sum(lengths), 3, 64, 1, 128, sum(lengths), gated=True)
    check_fwd(ccv, t, lengths, init=[True] * len(lengths))


@pytest.mark.parametrize("form", ["recurrent", "chunked"])
def test_fwd_lines_and_padding(ccv, path, form):
    path(form)
    lengths = [100, 30, 200, 64]
    t = make(sum(lengths) + 9, 2, 64, 1, 128, 3)  # tokens past the last sequence stay as they are
    lines = torch.tensor([5, -1, 0, 3], dtype=torch.int32)
    check_fwd(ccv, t, lengths, init=[True, True, False, True], lines=lines, num_lines=7)
    check_fwd(ccv, t, lengths, init=None, lines=lines, num_lines=7)
    check_fwd(ccv, t, lengths, lines=None, state=False)


@pytest.mark.parametrize("form", ["recurrent", "chunked"])
@pytest.mark.parametrize("kw", [{"dt_softplus": False, "dt_limit": (0.001, 0.1)}, {"dt_limit": (0.01, 0.02)},
                                {"dt_softplus": False, "dt_limit": (0.0, 0.05)}])
def test_fwd_steps(ccv, path, form, kw):
    path(form)
    for kind in (BF16, torch.float32):
        t = make(150, 4, 64, 2, 128, 5, kind=kind)
        check_fwd(ccv, t, [150], init=[True], **kw)
    t["dt_bias"] = t["D"] = None
    check_fwd(ccv, t, [150], init=[True], **kw)


@pytest.mark.parametrize("form", ["recurrent", "chunked"])
def test_fwd_strong_decays(ccv, path, form):
    """Decays that leave nothing of a state within a token, and ones that leave it as it is."""
    path(form)
    t = make(300, 4, 64, 1, 128, 6, strong=True)
    t["dt_bias"] += 3
    check_fwd(ccv, t, [300], init=[True])
    t["A"][0], t["A"][1], t["A"][2] = 0.0, -1e4, -1e-6
    check_fwd(ccv, t, [299], init=[True])


@pytest.mark.parametrize("lengths", [[700], [5, 1300, 260], [128 * 6], [128 * 6 + 1]])
@pytest.mark.parametrize("segment", [0, 1, 2, 3])
def test_fwd_segments(ccv, path, lengths, segment):
    """Sequences cut into segments of a few chunks."""
    path("chunked", segment)
    t = make(sum(lengths), 3, 64, 1, 128, 7)
    check_fwd(ccv, t, lengths, init=[True] * len(lengths))


CHANNELS = [(32, 16), (100, 16), (1, 16), (257, 8), (64, 24), (33, 64), (40, 5), (16, 256), (7, 1), (640, 16)]


@pytest.mark.parametrize("form", ["recurrent", "scan"])
@pytest.mark.parametrize("channels,states", CHANNELS)
def test_fwd_channels(ccv, path, form, channels, states):
    path(form)
    lengths = [37, 1, 0, 64, 130, 3]
    t = make(sum(lengths), channels, 1, 1, states, channels, per_state=True, gated=channels % 2 == 0)
    check_fwd(ccv, t, lengths, init=[True, False, True, True, True, False], channels=True)


@pytest.mark.parametrize("form", ["recurrent", "scan"])
def test_fwd_channels_in_groups(ccv, path, form):
    """Several groups of B and C, one decay a channel, heads of several channels with decays a state."""
    path(form)
    lengths = [50, 200]
    check_fwd(ccv, make(250, 96, 1, 3, 16, 8, per_state=True, kind=torch.float32), lengths, init=[True, False], channels=True)
    check_fwd(ccv, make(250, 96, 1, 3, 16, 9), lengths, init=[True, False], channels=True)
    check_fwd(ccv, make(250, 6, 8, 2, 16, 10, per_state=True, gated=True), lengths, init=[True, False])


@pytest.mark.parametrize("segment", [1, 2, 5])
def test_fwd_channels_segments(ccv, path, segment):
    path("scan", segment)
    lengths = [700, 3, 0, 129]
    t = make(sum(lengths), 100, 1, 1, 16, 11, per_state=True, gated=True)
    check_fwd(ccv, t, lengths, init=[True, True, False, False], channels=True)


def strided(t, name):
    """The same values in another layout: channel-first, inside a wider tensor at an odd offset, or reversed axes."""
    if t.dim() < 2:
        return t
    if name == "channel_first":
        perm = list(range(1, t.dim())) + [0]
        return t.permute(perm).contiguous().permute([t.dim() - 1, *range(t.dim() - 1)])
    if name == "odd":
        wide = torch.zeros(*t.shape[:-1], t.shape[-1] + 3, dtype=t.dtype, device=t.device)
        wide[..., 1:1 + t.shape[-1]] = t
        return wide[..., 1:1 + t.shape[-1]]
    return t.transpose(1, -1).contiguous().transpose(1, -1)


@pytest.mark.parametrize("layout", ["channel_first", "odd", "swapped"])
@pytest.mark.parametrize("form", ["recurrent", "chunked", "scan"])
def test_fwd_strides(ccv, path, form, layout):
    path(form)
    per = form == "scan"
    h, p, n = (70, 1, 16) if per else (4, 64, 128)
    t = cuda(make(200, h, p, 1, n, 12, per_state=per, gated=True))
    starts = torch.tensor([0, 77, 200], dtype=torch.int32, device="cuda")
    init = torch.tensor([True, True], device="cuda")
    first = pool(2, h, p, n, 12).cuda()
    args = ("x", "dt", "A", "B", "C")
    a, b = first.clone(), strided(first.clone(), "odd")
    out = ccv.ssm_fwd(*(t[k] for k in args), a, starts, None, init, D=t["D"], z=t["z"], dt_bias=t["dt_bias"])
    o = {k: strided(v, layout) if k in ("x", "dt", "B", "C", "z") else v for k, v in t.items()}
    to = strided(torch.empty_like(t["x"]), layout)
    got = ccv.ssm_fwd(*(o[k] for k in args), b, starts, None, init, D=o["D"], z=o["z"], dt_bias=o["dt_bias"], out=to)
    torch.cuda.synchronize()
    # the order of a sum may differ: a bf16 step, and 2^-15 of the products' sizes (up to some 300 here); 2^-20 of the state
    assert ((got.double() - out.double()).abs() <= 2.0 ** -7 * out.double().abs() + 1e-2).all()
    assert float((b - a).norm()) <= 2.0 ** -20 * float(a.norm())


def update_case(b, steps, heads, dim, groups, states, seed, **kw):
    t = make(b * steps, heads, dim, groups, states, seed, **kw)
    return {k: v.unflatten(0, (b, steps)) if k in ("x", "dt", "B", "C", "z") and v is not None else v for k, v in t.items()}


def check_update(ccv, t, lines=None, out_lines=None, accepted=None, num_lines=None, flat=False, channels=False, seed=0, err_wanted=False):
    b, n, h, p = t["x"].shape
    ns = t["B"].shape[-1]
    s = pool(num_lines or b, h, p, ns, seed)
    d = ref.steps(t["dt"], t["dt_bias"], True, (0.0, INF))
    a = t["A"] if t["A"].dim() == 2 else t["A"][:, None]
    want = torch.full(t["x"].shape, float("nan"), dtype=torch.float64)
    bound = torch.zeros_like(want)
    after, mags = s.double().clone(), torch.zeros(s.shape, dtype=torch.float64)
    for r in range(b):
        line = r if lines is None else int(lines[r])
        if line == -1:
            continue
        source = line
        if accepted is not None:
            k = int(accepted[r])
            source = int(out_lines[r, k - 1]) if 1 <= k <= out_lines.shape[1] else -1
        if not (0 <= source < s.shape[0] and 0 <= line < s.shape[0]):
            continue
        keep = []
        z = None if t["z"] is None else t["z"][r]
        want[r], bound[r], last, mag = ref.ssm_tokens(t["x"][r], d[r], a, t["B"][r], t["C"][r], s[source].double(), t["D"], z, keep)
        if out_lines is None:
            after[line], mags[line] = last, mag
        else:
            for i in range(n):
                to = int(out_lines[r, i])
                if 0 <= to < s.shape[0]:
                    after[to], mags[to] = keep[i]
    on, got = cuda(t), s.cuda()
    out = torch.full(on["x"].shape, float("nan"), dtype=BF16, device="cuda")
    if channels:
        on = {k: v[..., 0] if k in ("x", "z") and v is not None else v for k, v in on.items()}
        got, out = got[:, :, 0], out[..., 0]
    if flat:
        on = {k: v[:, 0] if k in ("x", "dt", "B", "C", "z") and v is not None else v for k, v in on.items()}
        out = out[:, 0]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    place = lambda i: None if i is None else i.cuda()  # noqa: E731
    ccv.ssm_update(on["x"], on["dt"], on["A"], on["B"], on["C"], got, place(lines), place(accepted), place(out_lines), D=on["D"],
                   z=on["z"], dt_bias=on["dt_bias"], out=out, err_count=err)
    torch.cuda.synchronize()
    full, told = out.reshape(want.shape).cpu(), ~want.isnan()
    assert torch.equal(full.isnan(), ~told)
    ref.assert_out(torch.where(told, full.double(), 0), want.nan_to_num(), bound)
    ref.assert_state(got.reshape(after.shape), after, mags)
    assert (int(err) > 0) == err_wanted


@pytest.mark.parametrize("heads,dim,groups,states", SHAPES)
def test_update_shapes(ccv, heads, dim, groups, states):
    check_update(ccv, update_case(3, 1, heads, dim, groups, states, 20), flat=True)
    check_update(ccv, update_case(2, 3, heads, dim, groups, states, 21, gated=True))


@pytest.mark.parametrize("channels,states", CHANNELS)
def test_update_channels(ccv, channels, states):
    check_update(ccv, update_case(3, 1, channels, 1, 1, states, 22, per_state=True, gated=True), flat=True, channels=True)
    check_update(ccv, update_case(2, 2, channels, 1, 1, states, 23, per_state=True), channels=True)


def test_update_lines(ccv):
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    t = update_case(4, 1, 3, 64, 1, 128, 24)
    check_update(ccv, t, lines=i32(6, -1, 0, 2), num_lines=7, flat=True)
    check_update(ccv, t, lines=i32(6, 9, 0, 2), num_lines=7, flat=True, err_wanted=True)


def test_update_speculative(ccv):
    t = update_case(3, 4, 3, 64, 1, 128, 25)
    out_lines = torch.arange(1, 13, dtype=torch.int32).reshape(3, 4)
    accepted = torch.tensor([1, 4, 2], dtype=torch.int32)
    check_update(ccv, t, out_lines=out_lines, num_lines=13)
    check_update(ccv, t, out_lines=out_lines, accepted=accepted, num_lines=13)
    out_lines[1, 1] = -1
    check_update(ccv, t, out_lines=out_lines, accepted=accepted, num_lines=13)
    check_update(ccv, t, out_lines=out_lines, accepted=torch.tensor([0, 5, 2], dtype=torch.int32), num_lines=13, err_wanted=True)
    t = update_case(3, 4, 40, 1, 1, 16, 26, per_state=True, gated=True)
    check_update(ccv, t, out_lines=out_lines, accepted=accepted, num_lines=13, channels=True)


@pytest.mark.parametrize("per_state", [False, True])
def test_prompt_is_its_tokens_in_a_row(ccv, per_state):
    """ssm_fwd ends in the state that ssm_update reaches token by token, and a prompt in two parts in the same."""
    h, p, n = (48, 1, 16) if per_state else (4, 64, 128)
    t = cuda(make(400, h, p, 1, n, 27, per_state=per_state))
    one = torch.zeros(1, h, p, n, device="cuda")
    args = lambda s: (t["x"][s], t["dt"][s], t["A"], t["B"][s], t["C"][s])  # noqa: E731
    kw = {"D": t["D"], "dt_bias": t["dt_bias"]}
    outs = torch.cat([ccv.ssm_update(*args(slice(i, i + 1)), one, **kw) for i in range(400)])
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for cut in (400, 129, 1):
        state = torch.zeros_like(one)
        parts = [ccv.ssm_fwd(*args(slice(0, cut)), state, i32(0, cut), **kw)]
        if cut < 400:
            parts.append(ccv.ssm_fwd(*args(slice(cut, 400)), state, i32(0, 400 - cut), None, torch.tensor([True], device="cuda"), **kw))
        got = torch.cat(parts)
        assert float((state - one).norm()) <= 2.0 ** -16 * float(one.norm())
        assert float((got.float() - outs.float()).norm()) <= 2.0 ** -7 * float(outs.float().norm())


@pytest.mark.parametrize("form,per_state", [("recurrent", False), ("chunked", False), ("scan", True)])
@pytest.mark.parametrize("what", ["x", "B", "C", "dt"])
@pytest.mark.parametrize("value", [float("nan"), INF])
def test_not_finite_reaches_later_tokens_only(ccv, path, form, per_state, what, value):
    """Tokens before one that is not finite, other sequences, and (for x) other channels are as without it."""
    path(form)
    h, p, n = (40, 1, 16) if per_state else (2, 64, 128)
    t = make(450, h, p, 1, n, 28, per_state=per_state)
    starts = torch.tensor([0, 300, 450], dtype=torch.int32, device="cuda")

    def call(t):
        on = cuda(t)
        state = torch.zeros(2, h, p, n, device="cuda")
        out = ccv.ssm_fwd(*(on[k] for k in ("x", "dt", "A", "B", "C")), state, starts, D=on["D"], dt_bias=on["dt_bias"])
        return out, state

    out, state = call(t)
    at = 201
    if what == "dt":
        t["dt"][at, 1] = value
    elif what == "x":
        t["x"][at, 1, p // 2] = value
    else:
        t[what][at, 0, n // 2] = value
    got, after = call(t)
    same = lambda a, b: torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))  # noqa: E731
    assert same(got[:at], out[:at]) and same(got[300:], out[300:])
    assert torch.equal(after[1], state[1])
    if what in ("x", "dt"):
        assert same(got[:, 0], out[:, 0]) and torch.equal(after[0, 0], state[0, 0])
    touched = got[at, 1, p // 2] if what in ("x", "dt") else got[at].flatten()[0]
    assert not bool(touched.isfinite())
    if what == "x":
        assert not bool(after[0, 1, p // 2].isfinite().any())
        if p > 1:
            keep = [i for i in range(p) if i != p // 2]
            assert same(got[:, 1, keep], out[:, 1, keep]) and torch.equal(after[0, 1, keep], state[0, 1, keep])
    elif what == "C":
        assert same(got[at + 1:300], out[at + 1:300]) and torch.equal(after, state)
    elif what == "B":
        assert not bool(after[0, :, :, n // 2].isfinite().any())


@pytest.mark.parametrize("form", ["recurrent", "chunked"])
def test_bad_offsets_and_lines(ccv, path, form):
    path(form)
    t = cuda(make(300, 2, 64, 1, 128, 29))
    state = torch.zeros(2, 2, 64, 128, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda starts, lines: ccv.ssm_fwd(*(t[k] for k in ("x", "dt", "A", "B", "C")), state,  # noqa: E731
                                             torch.tensor(starts, dtype=torch.int32, device="cuda"),
                                             torch.tensor(lines, dtype=torch.int32, device="cuda"), err_count=err)
    for starts, lines in (([0, 301], [0]), ([-1, 200], [0]), ([200, 100], [0]), ([0, 200], [2]), ([0, 200], [-7])):
        before = int(err)
        call(starts, lines)
        assert int(err) > before, (starts, lines)
        assert not bool(state.any())
    call([0, 300], [-1])
    assert not bool(state.any())


def test_captured_and_replayed(ccv):
    """A prompt and a decode step in one graph, with new inputs in the same places."""
    for per_state in (False, True):
        h, p, n = (64, 1, 16) if per_state else (4, 64, 128)
        t, u = cuda(make(700, h, p, 1, n, 30, per_state=per_state)), cuda(make(700, h, p, 1, n, 31, per_state=per_state))
        starts = torch.tensor([0, 100, 700], dtype=torch.int32, device="cuda")
        state = torch.zeros(2, h, p, n, device="cuda")
        names = ("x", "dt", "A", "B", "C")
        at = lambda t: (t["x"][:2], t["dt"][:2], t["A"], t["B"][:2], t["C"][:2])  # noqa: E731

        def both(t):
            state.zero_()
            a = ccv.ssm_fwd(*(t[k] for k in names), state, starts, dt_bias=t["dt_bias"])
            return a, ccv.ssm_update(*at(t), state, dt_bias=t["dt_bias"])

        want = [(*(r.clone() for r in both(x)), state.clone()) for x in (t, u)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a, b = both(t)
        for x, w in ((t, want[0]), (u, want[1])):
            for k, v in x.items():
                if v is not None:
                    t[k].copy_(v)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(a, w[0]) and torch.equal(b, w[1]) and torch.equal(state, w[2])


def test_results_do_not_change_from_call_to_call(ccv):
    t = cuda(make(1500, 6, 64, 2, 128, 32))
    starts = torch.tensor([0, 1100, 1500], dtype=torch.int32, device="cuda")
    runs = []
    for _ in range(4):
        state = torch.zeros(2, 6, 64, 128, device="cuda")
        runs.append((ccv.ssm_fwd(*(t[k] for k in ("x", "dt", "A", "B", "C")), state, starts, D=t["D"], dt_bias=t["dt_bias"]), state))
    for out, state in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(state, runs[0][1])


def far(shape, stride0, dtype, seed):
    """(2, *shape) values, the second 2^31 and more elements after the first."""
    base = torch.empty(stride0 + 2 ** 20, dtype=dtype, device="cuda")
    inner = torch.empty(shape).stride()
    view = base.as_strided((2, *shape), (stride0, *inner))
    view.copy_(torch.randn(2, *shape, generator=torch.Generator().manual_seed(seed)))
    return view


def test_offsets_past_32_bits(ccv):
    """State lines and rows more than 2^31 elements apart."""
    for h, p, n, per in ((3, 64, 128, False), (70, 1, 16, True)):
        t = cuda(make(2, h, p, 1, n, 33, per_state=per))
        state = far((h, p, n), 2 ** 31 + 64, torch.float32, 34)
        x = far((h, p), 2 ** 31 + 64, BF16, 35)
        near, dense = state.clone(), x.contiguous()
        args = (t["dt"], t["A"], t["B"], t["C"])
        for call, tail in ((ccv.ssm_update, ()), (ccv.ssm_fwd, (torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), None,
                                                                torch.tensor([True, True], device="cuda")))):
            want = call(dense, *args, near, *tail)
            got = call(x, *args, state, *tail)
            assert torch.equal(got, want) and torch.equal(state, near)
        del state, x
        torch.cuda.empty_cache()


def test_one_chunk_of_many_sequences(ccv):
    """More sequences than a search looks at in one step, many of them empty, in segments and whole."""
    g = torch.Generator().manual_seed(36)
    lengths = [int(v) for v in torch.randint(0, 40, (300,), generator=g)]
    lengths[7] = 900
    for heads, dim, states, per in ((2, 64, 64, False), (40, 1, 16, True)):
        t = make(sum(lengths), heads, dim, 1, states, 37, per_state=per)
        check_fwd(ccv, t, lengths, init=[i % 3 == 0 for i in range(300)], channels=per)


@pytest.mark.parametrize("rows,channels,states", [(1100, 300, 16), (3100, 129, 7), (1601, 50, 100)])
def test_update_rows_that_share_rates(ccv, rows, channels, states):
    """A batch so large that a block takes several of its rows, among them skipped and refused ones."""
    t = update_case(rows, 1, channels, 1, 1, states, 38, per_state=True, gated=True)
    lines = torch.randperm(rows, generator=torch.Generator().manual_seed(39)).to(torch.int32)
    lines[::7], lines[5], lines[rows - 1] = -1, rows, -2
    check_update(ccv, t, lines=lines, flat=True, channels=True, err_wanted=True)


def test_fwd_sequences_that_share_rates(ccv, path):
    path("recurrent")
    lengths = [i % 4 for i in range(1300)]
    t = make(sum(lengths), 300, 1, 1, 16, 40, per_state=True)
    check_fwd(ccv, t, lengths, init=[i % 3 == 0 for i in range(1300)], channels=True)


@pytest.mark.parametrize("states", [32, 50, 100, 128, 130, 200])
@pytest.mark.parametrize("segment", [0, 1])
def test_fwd_channels_of_more_states(ccv, path, states, segment):
    """The token scan's tiles for every width of the state, whole and in segments, with decays a state and one decay a channel."""
    path("scan", segment)
    lengths = [300, 0, 17, 129]
    for channels, per in ((50, True), (35, False)):
        t = make(sum(lengths), channels, 1, 1, states, 41, per_state=per, gated=per)
        check_fwd(ccv, t, lengths, init=[True, True, False, True], channels=True)


@pytest.mark.parametrize("states", [20, 60, 129, 252])
@pytest.mark.parametrize("per_state", [False, True])
def test_update_of_more_states(ccv, states, per_state):
    check_update(ccv, update_case(3, 2, 5, 7, 1, states, 42, per_state=per_state, gated=True))
    check_update(ccv, update_case(2, 1, 4, 64, 2, states, 43, per_state=per_state), flat=True)
