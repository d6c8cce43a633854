"""Cases and plain forms of the linear-attention layer's operators: the gated delta rule (prefill and decode), the two
norms around it, and the verification of drafted tokens.

``run`` makes one pass: the plain form in elementary torch operations while ``own`` is false, the framework's call
otherwise.  ``exact`` computes the same outputs in 64 bits from each operator's definition, token by token.
"""
import math
import random

import torch

own = False

BF16 = torch.bfloat16
CHUNK = 64  # tokens per chunk of the plain chunked form
NORM_EPS = 1e-6


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # a tensor-parallel shard's share of a small batch of short prompts: latency counts
        {"name": "gdr_fwd_short_prompts", "op": "gdr_fwd", "lengths": "37,1,64,130", "hk": 4, "hv": 8, "dk": 128, "dv": 128,
         "raw_gates": True, "fresh": "some"},
        # one long odd-sized prompt on a shard: few rows, a long axis
        {"name": "gdr_fwd_one_long", "op": "gdr_fwd", "lengths": "11027", "hk": 8, "hv": 16, "dk": 128, "dv": 128,
         "raw_gates": True, "fresh": "all"},
        # a full prefill step over the convolution's 4 x 4096 tokens, dim 8192 = 16 + 16 key heads and 32 value heads of 128
        {"name": "gdr_fwd_4x4096", "op": "gdr_fwd", "lengths": "4096,4096,4096,4096", "hk": 16, "hv": 32, "dk": 128, "dv": 128,
         "raw_gates": True, "fresh": "none"},
        # one user's next token
        {"name": "gdr_update_one", "op": "gdr_update", "rows": 1, "steps": 1, "hk": 16, "hv": 32, "dk": 128, "dv": 128,
         "raw_gates": True},
        # a decode step of a full batch
        {"name": "gdr_update_256", "op": "gdr_update", "rows": 256, "steps": 1, "hk": 16, "hv": 32, "dk": 128, "dv": 128,
         "raw_gates": True},
        # speculative verify: four tokens a row, a state kept after each
        {"name": "gdr_update_spec_64x4", "op": "gdr_update", "rows": 64, "steps": 4, "hk": 16, "hv": 32, "dk": 128, "dv": 128,
         "raw_gates": True},
        # the gated norm of a decode step's heads
        {"name": "gated_norm_decode", "op": "gated_rms_norm", "tokens": 5, "heads": 32, "dim": 128, "before": True, "act": "silu"},
        # the gated norm of a prefill step's heads
        {"name": "gated_norm_16384", "op": "gated_rms_norm", "tokens": 16384, "heads": 32, "dim": 128, "before": True, "act": "silu"},
        # a decode step's residual add and norm
        {"name": "residual_norm_decode", "op": "residual_rms_norm", "tokens": 64, "dim": 2048, "post": False, "gate": "none",
         "res32": False},
        # a prefill step's: norm after the block, a gate for each channel, the residual kept in 32 bits
        {"name": "residual_norm_8191", "op": "residual_rms_norm", "tokens": 8191, "dim": 4096, "post": True, "gate": "channel",
         "res32": True},
        # three drafts from an n-gram table (no draft distribution), an odd vocabulary
        {"name": "verify_ngram", "op": "spec_verify", "rows": 4, "drafts": 3, "vocab": 32003, "dtype": "bf16", "draft": False,
         "ragged": True, "temperature": "mixed"},
        # a full batch's drafts with the drafting model's distributions
        {"name": "verify_64x4", "op": "spec_verify", "rows": 64, "drafts": 4, "vocab": 131072, "dtype": "bf16", "draft": True,
         "ragged": False, "temperature": "one"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gdr_fwd", "gdr_fwd", "gdr_update", "gdr_update", "gated_rms_norm", "residual_rms_norm", "spec_verify"])
    if op == "gdr_fwd":
        tokens, n = _log(rng, 40, 12000), _log(rng, 1, 24)
        cuts = sorted(rng.randrange(tokens + 1) for _ in range(n - 1))
        lengths = [b - a for a, b in zip([0] + cuts, cuts + [tokens])]
        hk = rng.choice([1, 2, 4, 8, 16])
        dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (96, 80)])
        return {"op": op, "lengths": ",".join(map(str, lengths)), "hk": hk, "hv": hk * rng.choice([1, 2]), "dk": dk, "dv": dv,
                "raw_gates": rng.random() < 0.5, "fresh": rng.choice(["all", "some", "none"])}
    if op == "gdr_update":
        hk = rng.choice([1, 2, 4, 8, 16])
        dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (96, 80)])
        steps = rng.choice([1, 1, 2, 3, 4, 5, 6])
        return {"op": op, "rows": _log(rng, 1, 256 // steps), "steps": steps, "hk": hk, "hv": hk * rng.choice([1, 2]),
                "dk": dk, "dv": dv, "raw_gates": rng.random() < 0.5}
    if op == "gated_rms_norm":
        tokens = _log(rng, 1, 16384)
        heads, dim = rng.choice([(4, 128), (8, 128), (16, 128), (32, 128), (16, 64), (5, 256), (1, 1000), (7, 80), (1, 4096)])
        return {"op": op, "tokens": tokens, "heads": heads, "dim": dim, "before": rng.random() < 0.7,
                "act": rng.choice(["silu", "silu", "sigmoid"])}
    if op == "residual_rms_norm":
        return {"op": op, "tokens": _log(rng, 1, 8191), "dim": rng.choice([256, 1000, 1536, 2048, 2500, 4096]),
                "post": rng.random() < 0.5, "gate": rng.choice(["none", "channel", "token"]), "res32": rng.random() < 0.5}
    return {"op": op, "rows": _log(rng, 1, 64), "drafts": rng.randint(1, 4), "vocab": _log(rng, 1000, 131072),
            "dtype": rng.choice(["bf16", "fp32"]), "draft": rng.random() < 0.6, "ragged": rng.random() < 0.5,
            "temperature": rng.choice(["one", "mixed"])}


# ----------------------------------------------------------------- inputs ----

def _mixed_qkv(n, case, g):
    """q, k, v as views of one convolution output (n, 2 hk dk + hv dv) after its SiLU."""
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    x = torch.randn(n, 2 * hk * dk + hv * dv, generator=g, device="cuda")
    x = (x / (1 + torch.exp(-x))).to(BF16)
    q = x[:, :hk * dk].unflatten(1, (hk, dk))
    k = x[:, hk * dk:2 * hk * dk].unflatten(1, (hk, dk))
    v = x[:, 2 * hk * dk:].unflatten(1, (hv, dv))
    return q, k, v


def _gates(n, case, g):
    """The projections' a and b with the layer's a_log and dt_bias, or the decay logarithm and the write strength themselves."""
    hv = case["hv"]
    a_log = torch.log(1 + 15 * torch.rand(hv, generator=g, device="cuda"))
    dt = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(hv, generator=g, device="cuda"))
    dt_bias = dt + torch.log(-torch.expm1(-dt))
    a = torch.randn(n, hv, generator=g, device="cuda").to(BF16)
    b = torch.randn(n, hv, generator=g, device="cuda").to(BF16)
    if case["raw_gates"]:
        return {"g": a, "beta": b, "a_log": a_log, "dt_bias": dt_bias}
    x = a.float() + dt_bias
    return {"g": -torch.exp(a_log) * torch.log1p(torch.exp(x)), "beta": 1 / (1 + torch.exp(-b.float())), "a_log": None, "dt_bias": None}


def _prepare_fwd(case, g, seed):
    lengths = [int(x) for x in case["lengths"].split(",")]
    n, total = len(lengths), sum(lengths)
    starts = [sum(lengths[:i]) for i in range(n + 1)]
    q, k, v = _mixed_qkv(total, case, g)
    lines = n + 3
    state = 0.2 * torch.randn(lines, case["hv"], case["dv"], case["dk"], generator=g, device="cuda")
    order = list(range(lines))
    random.Random(seed).shuffle(order)
    init = {"all": [False] * n, "none": [True] * n, "some": [i % 2 == 0 for i in range(n)]}[case["fresh"]]
    return {"q": q, "k": k, "v": v, **_gates(total, case, g), "state": state, "longest": max(lengths),
            "query_start_loc": torch.tensor(starts, dtype=torch.int32, device="cuda"),
            "cache_indices": torch.tensor(order[:n], dtype=torch.int32, device="cuda"),
            "has_initial_state": torch.tensor(init, device="cuda")}


def _prepare_update(case, g, seed):
    b, t = case["rows"], case["steps"]
    q, k, v = (x.unflatten(0, (b, t)) for x in _mixed_qkv(b * t, case, g))
    gates = {n: x.unflatten(0, (b, t)) if n in ("g", "beta") else x for n, x in _gates(b * t, case, g).items()}
    lines = b * t + 2
    state = 0.2 * torch.randn(lines, case["hv"], case["dv"], case["dk"], generator=g, device="cuda")
    order = list(range(lines))
    random.Random(seed).shuffle(order)
    out = {"q": q, "k": k, "v": v, **gates, "state": state}
    if t == 1:
        out["state_indices"] = torch.tensor(order[:b], dtype=torch.int32, device="cuda")
    else:
        out["output_state_indices"] = torch.tensor(order[:b * t], dtype=torch.int32, device="cuda").reshape(b, t)
        out["num_accepted_tokens"] = torch.randint(1, t + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
    return out


def _prepare_verify(case, g):
    b, s, vocab = case["rows"], case["drafts"], case["vocab"]
    logits = 3 * torch.randn(b, s + 1, vocab, generator=g, device="cuda")
    logits = logits.masked_fill(logits < -4, -math.inf)  # what a top-p filter leaves
    temperature = None
    if case["temperature"] == "mixed":
        temperature = 0.5 + torch.rand(b, generator=g, device="cuda")
        temperature[::3] = 0.0
    probs = torch.softmax(logits[:, :s] + 0.7 * torch.randn(b, s, vocab, generator=g, device="cuda"), -1)
    race = torch.empty(b, s, vocab, device="cuda").exponential_(generator=g)
    tokens = (probs / race).argmax(-1).to(torch.int32)
    del race
    drafts = torch.randint(0, s + 1, (b,), generator=g, device="cuda", dtype=torch.int32) if case["ragged"] else None
    return {"target_logits": logits.to(BF16 if case["dtype"] == "bf16" else torch.float32), "draft_tokens": tokens,
            "uniform": torch.rand(b, s, generator=g, device="cuda"), "temperature": temperature,
            "noise": torch.empty(b, vocab, device="cuda").exponential_(generator=g).clamp_min(1e-30),
            "draft_probs": probs if case["draft"] else None, "num_drafts": drafts}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "gdr_fwd":
        state = _prepare_fwd(case, g, seed)
    elif op == "gdr_update":
        state = _prepare_update(case, g, seed)
    elif op == "gated_rms_norm":
        shape = (case["tokens"], case["heads"], case["dim"])
        state = {"x": torch.randn(shape, generator=g, device="cuda").to(BF16),
                 "gate": torch.randn(shape, generator=g, device="cuda").to(BF16),
                 "weight": (1 + 0.1 * torch.randn(case["dim"], generator=g, device="cuda")).to(BF16),
                 "before": case["before"], "act": case["act"]}
    elif op == "residual_rms_norm":
        t, d = case["tokens"], case["dim"]
        state = {"x": torch.randn(t, d, generator=g, device="cuda").to(BF16),
                 "residual": (2 * torch.randn(t, d, generator=g, device="cuda")).to(torch.float32 if case["res32"] else BF16),
                 "weight": (0.1 * torch.randn(d, generator=g, device="cuda")).to(BF16),
                 "post_weight": (0.1 * torch.randn(d, generator=g, device="cuda")).to(BF16) if case["post"] else None,
                 "gate": None if case["gate"] == "none" else
                 torch.rand(*((d,) if case["gate"] == "channel" else (t, d)), generator=g, device="cuda").to(BF16),
                 "scale": 0.75}
    else:
        state = _prepare_verify(case, g)
    state["op"] = op
    return state


# ------------------------------------------------------------ plain forms ----

def _plain_gates(s):
    if s["a_log"] is None:
        return s["g"], s["beta"]
    x = s["g"].float() + s["dt_bias"]
    return -torch.exp(s["a_log"]) * torch.log1p(torch.exp(x)), 1 / (1 + torch.exp(-s["beta"].float()))


def _plain_qkv(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    q = q * torch.rsqrt((q * q).sum(-1, keepdim=True) + 1e-6) * q.shape[-1] ** -0.5
    k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    rep = v.shape[-2] // k.shape[-2]
    return q.repeat_interleave(rep, -2), k.repeat_interleave(rep, -2), v


def _plain_fwd(s):
    """The chunked form, all sequences padded to the longest: a loop over chunks carries the state."""
    q, k, v = _plain_qkv(s)
    g, beta = _plain_gates(s)
    start = s["query_start_loc"].long()
    n, total, c = start.numel() - 1, q.shape[0], CHUNK
    chunks = -(-s["longest"] // c)
    at = start[:-1, None] + torch.arange(chunks * c, device="cuda")
    real = at < start[1:, None]
    at = at.clamp(max=total - 1)

    def tiles(x):  # (tokens, heads, ...) -> (n, heads, chunks, c, ...), zeros past each sequence's end
        x = x[at] * real.reshape(real.shape + (1,) * (x.dim() - 1))
        return x.unflatten(1, (chunks, c)).movedim(3, 1)

    q, k, v, g, beta = tiles(q), tiles(k), tiles(v), tiles(g), tiles(beta)
    gsum = g.cumsum(-1)
    row = torch.arange(c, device="cuda")
    decay = torch.exp((gsum[..., :, None] - gsum[..., None, :]).masked_fill(row[:, None] < row, -math.inf))
    a = (k @ k.transpose(-1, -2) * decay * beta[..., None]).masked_fill(row[:, None] <= row, 0.0)
    inv = torch.eye(c, device="cuda").expand_as(a).clone()  # (I + a)^-1 by doubling its diagonal blocks
    half = 1
    while half < c:
        blocks = (c // (2 * half), 2 * half) * 2
        t, low = (x.reshape(x.shape[:-2] + blocks).diagonal(dim1=-4, dim2=-2).movedim(-1, -3) for x in (inv, a))
        done = t.clone()
        done[..., half:, :half] = -t[..., half:, half:] @ low[..., half:, :half] @ t[..., :half, :half]
        inv.reshape(a.shape[:-2] + blocks).diagonal(dim1=-4, dim2=-2).movedim(-1, -3).copy_(done)
        half *= 2
    u = inv @ (v * beta[..., None])
    w = inv @ (k * (beta * torch.exp(gsum))[..., None])
    p = q @ k.transpose(-1, -2) * decay
    qd = q * torch.exp(gsum)[..., None]
    kd = k * torch.exp(gsum[..., -1:] - gsum)[..., None]
    last = torch.exp(gsum[..., -1])[..., None, None]
    lines = s["cache_indices"].long()
    state = s["state"][lines] * s["has_initial_state"][:, None, None, None]
    outs = []
    for i in range(chunks):
        vn = u[:, :, i] - w[:, :, i] @ state.transpose(-1, -2)
        outs.append(qd[:, :, i] @ state.transpose(-1, -2) + p[:, :, i] @ vn)
        state = state * last[:, :, i] + vn.transpose(-1, -2) @ kd[:, :, i]
    s["state"][lines] = torch.where((start[1:] > start[:-1])[:, None, None, None], state, s["state"][lines])
    out = torch.stack(outs, 2).movedim(1, 3).flatten(1, 2)  # (n, chunks * c, heads, dv)
    return {"out": out[real].to(BF16), "state": s["state"]}


def _plain_update(s):
    q, k, v = _plain_qkv(s)
    g, beta = _plain_gates(s)
    spec = "output_state_indices" in s
    if spec:
        lines = s["output_state_indices"].long()
        read = lines.gather(1, s["num_accepted_tokens"].long()[:, None] - 1)[:, 0]
    else:
        read = s["state_indices"].long()
        lines = read[:, None]
    state, outs = s["state"][read], []
    for t in range(q.shape[1]):
        state = state * torch.exp(g[:, t])[..., None, None]
        d = beta[:, t, :, None] * (v[:, t] - (state * k[:, t, :, None, :]).sum(-1))
        state = state + d[..., None] * k[:, t, :, None, :]
        outs.append((state * q[:, t, :, None, :]).sum(-1))
        s["state"][lines[:, t]] = state
    return {"out": torch.stack(outs, 1).to(BF16), "state": s["state"]}


def _act(z, act):
    return z / (1 + torch.exp(-z)) if act == "silu" else 1 / (1 + torch.exp(-z))


def _rms(x):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + NORM_EPS)


def _plain_gated(s):
    x, z, w = s["x"].float(), _act(s["gate"].float(), s["act"]), s["weight"].float()
    return (_rms(x) * w * z if s["before"] else _rms(x * z) * w).to(BF16)


def _plain_residual(s):
    t = s["x"].float()
    if s["post_weight"] is not None:
        t = _rms(t) * (1 + s["post_weight"].float())
    if s["gate"] is not None:
        t = t * s["gate"].float()
    h = s["residual"].float() + s["scale"] * t
    return {"out": (_rms(h) * (1 + s["weight"].float())).to(BF16), "residual": h.to(s["residual"].dtype)}


def _first(x, best):
    """The lowest index at which x equals its row's largest value `best`."""
    v = x.shape[-1]
    return torch.where(x == best, torch.arange(v, device=x.device), v).amin(-1)


def _verify(s, kind):
    x, tokens = s["target_logits"].to(kind), s["draft_tokens"].long()
    (b, n), v = tokens.shape, x.shape[-1]
    drafts = s["num_drafts"].long() if s["num_drafts"] is not None else torch.full((b,), n, device=x.device)
    temp = s["temperature"].to(kind) if s["temperature"] is not None else torch.ones(b, device=x.device, dtype=kind)
    greedy = temp == 0
    best = x.amax(-1, keepdim=True)
    p = torch.exp((x - best) / torch.where(greedy, 1.0, temp)[:, None, None])
    p = p / p.sum(-1, keepdim=True)
    top = torch.arange(v, device=x.device) == _first(x, best)[..., None]
    p = torch.where(greedy[:, None, None], top.to(kind), p)
    px = p[:, :n].gather(2, tokens[..., None])[..., 0]
    qx = s["draft_probs"].gather(2, tokens[..., None])[..., 0].to(kind) if s["draft_probs"] is not None else torch.ones_like(px)
    at = torch.arange(n, device=x.device)
    kept = ((s["uniform"].to(kind) * qx < px) & (at < drafts[:, None])).long().cumprod(1).sum(1)
    rows = torch.arange(b, device=x.device)
    r = p[rows, kept]
    slot = kept.clamp(max=n - 1)
    if s["draft_probs"] is not None:
        q = s["draft_probs"][rows, slot].to(kind)
    else:
        q = (torch.arange(v, device=x.device) == tokens[rows, slot][:, None]).to(kind)
    r = torch.where(((kept < drafts) & ~greedy)[:, None], (r - q).clamp_min(0.0), r)
    score = torch.where(greedy[:, None], r, r / s["noise"].to(kind))
    best = score.amax(-1, keepdim=True)
    token = torch.where(best[:, 0] > 0, _first(score, best), -1)
    at = torch.arange(n + 1, device=x.device)
    kept = kept[:, None]
    padded = torch.nn.functional.pad(tokens, (0, 1))
    out = torch.where(at < kept, padded, torch.where(at == kept, token[:, None], -1))
    return {"tokens": out.to(torch.int32), "num_accepted": (kept[:, 0] + 1).to(torch.int32)}


# ------------------------------------------------------------------- runs ----

def _run_own(s):
    import causal_depthwise_conv1d_fwd_gb300 as ccv

    op = s["op"]
    if op == "gdr_fwd":
        out = ccv.gdr_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["query_start_loc"], s["cache_indices"],
                          s["has_initial_state"], a_log=s["a_log"], dt_bias=s["dt_bias"])
        return {"out": out, "state": s["state"]}
    if op == "gdr_update":
        out = ccv.gdr_update(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s.get("state_indices"),
                             num_accepted_tokens=s.get("num_accepted_tokens"),
                             output_state_indices=s.get("output_state_indices"), a_log=s["a_log"], dt_bias=s["dt_bias"])
        return {"out": out, "state": s["state"]}
    if op == "gated_rms_norm":
        return ccv.gated_rms_norm(s["x"], s["gate"], s["weight"], NORM_EPS, s["act"], s["before"])
    if op == "residual_rms_norm":
        out, residual = ccv.residual_rms_norm(s["x"], s["residual"], s["weight"], s["post_weight"], s["gate"], s["scale"],
                                              NORM_EPS, weight_offset=1.0)
        return {"out": out, "residual": residual}
    tokens, accepted = ccv.spec_verify(s["target_logits"], s["draft_tokens"], s["uniform"], s["noise"], s["draft_probs"],
                                       s["num_drafts"], s["temperature"])
    return {"tokens": tokens, "num_accepted": accepted}


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "gdr_fwd":
        return _plain_fwd(state)
    if op == "gdr_update":
        return _plain_update(state)
    if op == "gated_rms_norm":
        return _plain_gated(state)
    if op == "residual_rms_norm":
        return _plain_residual(state)
    return _verify(state, torch.float32)


def work(case):
    op = case["op"]
    if op in ("gdr_fwd", "gdr_update"):
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        gate = 4 if case["raw_gates"] else 8
        if op == "gdr_fwd":
            lengths = [int(x) for x in case["lengths"].split(",")]
            tokens = sum(lengths)
            read = {"all": 0, "none": sum(n > 0 for n in lengths),
                    "some": sum(n > 0 for n in lengths[::2])}[case["fresh"]]
            written = sum(n > 0 for n in lengths)
        else:
            tokens, read = case["rows"] * case["steps"], case["rows"]
            written = tokens
        return {"bytes": tokens * (2 * (2 * hk * dk + 2 * hv * dv) + gate * hv) + (read + written) * 4 * hv * dv * dk,
                "flops": tokens * hv * 6 * dk * dv}
    if op == "gated_rms_norm":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 6 * n + 2 * case["dim"], "flops": 8 * n}
    if op == "residual_rms_norm":
        n = case["tokens"] * case["dim"]
        return {"bytes": n * (4 + 2 * (4 if case["res32"] else 2) + (2 if case["gate"] == "token" else 0)) + 6 * case["dim"],
                "flops": 10 * n}
    size = 2 if case["dtype"] == "bf16" else 4
    rows = case["rows"]
    positions = (case["drafts"] / 2 if case["ragged"] else case["drafts"]) + 1
    return {"bytes": rows * case["vocab"] * (positions * size + 4 + (4 if case["draft"] else 0)),
            "flops": rows * case["vocab"] * (positions * 4 + 3)}


# ---------------------------------------------------------------- 64 bits ----

def _exact_gates(s):
    g, beta = s["g"].double(), s["beta"].double()
    if s["a_log"] is not None:
        g = -s["a_log"].double().exp() * torch.logaddexp(g + s["dt_bias"].double(), torch.zeros_like(g))
        beta = torch.sigmoid(beta)
    return g, beta


def _exact_step(state, q, k, v, g, beta):
    """One token of the recurrence for (rows, heads): the new state and the output."""
    rep = v.shape[1] // k.shape[1]
    q, k = (x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt() for x in (q, k))
    q, k = (q / math.sqrt(q.shape[-1])).repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    state = state * g.exp()[..., None, None]
    error = v - torch.matmul(state, k[..., None])[..., 0]
    state = state + (beta[..., None] * error)[..., None] * k[..., None, :]
    return state, torch.matmul(state, q[..., None])[..., 0]


def _exact_fwd(s):
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    g, beta = _exact_gates(s)
    starts = s["query_start_loc"].tolist()
    lines = s["cache_indices"].long()
    lengths = torch.tensor([b - a for a, b in zip(starts, starts[1:])], device="cuda")
    pool = s["state"].double()
    state = pool[lines] * s["has_initial_state"].double()[:, None, None, None]
    first = torch.tensor(starts[:-1], device="cuda")
    out = torch.zeros(v.shape, dtype=torch.float64, device="cuda")
    order = torch.argsort(lengths, descending=True)  # the sequences still running come first
    state, first, sizes = state[order], first[order], sorted((b - a for a, b in zip(starts, starts[1:])), reverse=True)
    live = sum(n > 0 for n in sizes)
    for t in range(s["longest"]):
        while live and sizes[live - 1] <= t:
            live -= 1
        at = first[:live] + t
        state[:live], out[at] = _exact_step(state[:live], q[at], k[at], v[at], g[at], beta[at])
    back = lines[order]
    some = sum(n > 0 for n in sizes)
    pool[back[:some]] = state[:some]
    return {"out": out, "state": pool}


def _exact_update(s):
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    g, beta = _exact_gates(s)
    pool = s["state"].double()
    if "output_state_indices" in s:
        lines = s["output_state_indices"].long()
        state = pool[lines[torch.arange(lines.shape[0], device="cuda"), s["num_accepted_tokens"].long() - 1]]
    else:
        lines = s["state_indices"].long()[:, None]
        state = pool[lines[:, 0]]
    out = torch.zeros(v.shape, dtype=torch.float64, device="cuda")
    for t in range(q.shape[1]):
        state, out[:, t] = _exact_step(state, q[:, t], k[:, t], v[:, t], g[:, t], beta[:, t])
        pool[lines[:, t]] = state
    return {"out": out, "state": pool}


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "gdr_fwd":
        return _exact_fwd(s)
    if op == "gdr_update":
        return _exact_update(s)
    if op == "gated_rms_norm":
        x, z, w = (s[n].double() for n in ("x", "gate", "weight"))
        z = torch.sigmoid(z) * (z if s["act"] == "silu" else 1.0)
        u = x if s["before"] else x * z
        y = u / (u.square().mean(-1, keepdim=True) + NORM_EPS).sqrt() * w
        return y * z if s["before"] else y
    if op == "residual_rms_norm":
        t = s["x"].double()
        if s["post_weight"] is not None:
            t = t / (t.square().mean(-1, keepdim=True) + NORM_EPS).sqrt() * (1 + s["post_weight"].double())
        h = s["residual"].double() + s["scale"] * (t if s["gate"] is None else t * s["gate"].double())
        return {"out": h / (h.square().mean(-1, keepdim=True) + NORM_EPS).sqrt() * (1 + s["weight"].double()), "residual": h}
    return None  # whole numbers only: nothing to round
