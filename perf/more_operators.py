"""Cases and plain forms of the selective state space layer's operators (the scan over prompts and over new tokens) and
of the adjustment of logits before tokens are chosen.

``run`` makes one pass: the plain form in elementary torch operations while ``own`` is false, the framework's call
otherwise.  ``exact`` computes the same outputs in 64 bits from each operator's definition, token by token.
"""
import math
import random

import torch

own = False

BF16 = torch.bfloat16
CHUNK = 64  # tokens per chunk of the plain chunked forms


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # a tensor-parallel shard's share of a small batch of short prompts, one decay a head: latency counts
        {"name": "ssm_fwd_short_prompts", "op": "ssm_fwd", "lengths": "37,1,64,130", "heads": 32, "dim": 64, "groups": 1,
         "states": 128, "per_state": False, "dt": "bf16", "gated": False, "fresh": "some"},
        # one long odd-sized prompt on a shard: few heads, a long axis
        {"name": "ssm_fwd_one_long", "op": "ssm_fwd", "lengths": "11027", "heads": 32, "dim": 64, "groups": 2,
         "states": 128, "per_state": False, "dt": "bf16", "gated": False, "fresh": "all"},
        # a full prefill step of 4 x 4096 tokens, inner size 8192 = 128 heads of 64
        {"name": "ssm_fwd_4x4096", "op": "ssm_fwd", "lengths": "4096,4096,4096,4096", "heads": 128, "dim": 64, "groups": 8,
         "states": 128, "per_state": False, "dt": "bf16", "gated": False, "fresh": "none"},
        # channels that each have a decay for every state, with the gate: a few prompts on a shard
        {"name": "ssm_fwd_channels_prompts", "op": "ssm_fwd", "lengths": "1009,37,300", "heads": 2048, "dim": 1, "groups": 1,
         "states": 16, "per_state": True, "dt": "bf16", "gated": True, "fresh": "some"},
        # the same over the convolution's 4 x 4096 tokens, dim 8192
        {"name": "ssm_fwd_channels_4x4096", "op": "ssm_fwd", "lengths": "4096,4096,4096,4096", "heads": 8192, "dim": 1,
         "groups": 1, "states": 16, "per_state": True, "dt": "bf16", "gated": True, "fresh": "none"},
        # one user's next token
        {"name": "ssm_update_one", "op": "ssm_update", "rows": 1, "steps": 1, "heads": 128, "dim": 64, "groups": 8,
         "states": 128, "per_state": False, "dt": "bf16", "gated": False},
        # a decode step of a full batch
        {"name": "ssm_update_256", "op": "ssm_update", "rows": 256, "steps": 1, "heads": 128, "dim": 64, "groups": 8,
         "states": 128, "per_state": False, "dt": "bf16", "gated": False},
        # speculative verify: four tokens a row, a state kept after each
        {"name": "ssm_update_spec_64x4", "op": "ssm_update", "rows": 64, "steps": 4, "heads": 128, "dim": 64, "groups": 8,
         "states": 128, "per_state": False, "dt": "bf16", "gated": False},
        # a decode step of the convolution's 256 rows of 8192 channels, a decay for every state
        {"name": "ssm_update_channels_256", "op": "ssm_update", "rows": 256, "steps": 1, "heads": 8192, "dim": 1, "groups": 1,
         "states": 16, "per_state": True, "dt": "bf16", "gated": True},
        # a few requests with penalties, a bias and a grammar, an odd vocabulary
        {"name": "logits_few", "op": "logits", "rows": 4, "drafts": 0, "vocab": 32003, "dtype": "bf16", "history": 900,
         "bias": 20, "mask": True, "in_place": False},
        # a full batch's speculative step: penalties that count the drafts before each position, and a grammar
        {"name": "logits_64x5", "op": "logits", "rows": 64, "drafts": 4, "vocab": 131072, "dtype": "bf16", "history": 4000,
         "bias": 0, "mask": True, "in_place": False},
        # penalties alone, on the logits where they are
        {"name": "logits_in_place_256", "op": "logits", "rows": 256, "drafts": 0, "vocab": 131072, "dtype": "fp32",
         "history": 4000, "bias": 0, "mask": False, "in_place": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lengths(rng, tokens, n):
    cuts = sorted(rng.randrange(tokens + 1) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [tokens]))


def draw(rng):
    op = rng.choice(["ssm_fwd", "ssm_fwd", "ssm_fwd", "ssm_update", "ssm_update", "logits", "logits"])
    if op == "ssm_fwd" and rng.random() < 0.5:
        groups = rng.choice([1, 1, 2, 4, 8])
        dim, states = rng.choice([(64, 128), (64, 128), (64, 64), (128, 128), (80, 96), (32, 16)])
        return {"op": op, "lengths": _lengths(rng, _log(rng, 40, 12000), _log(rng, 1, 24)),
                "heads": groups * rng.choice([1, 3, 4, 8, 16]), "dim": dim, "groups": groups, "states": states,
                "per_state": False, "dt": rng.choice(["bf16", "bf16", "fp32"]), "gated": rng.random() < 0.3,
                "fresh": rng.choice(["all", "some", "none"])}
    if op == "ssm_fwd":
        return {"op": op, "lengths": _lengths(rng, _log(rng, 40, 6000), _log(rng, 1, 6)),
                "heads": rng.choice([256, 1000, 1024, 1536, 2048, 2500, 4096]), "dim": 1, "groups": 1,
                "states": rng.choice([16, 16, 16, 8, 24]), "per_state": True, "dt": rng.choice(["bf16", "bf16", "fp32"]),
                "gated": rng.random() < 0.7, "fresh": rng.choice(["all", "some", "none"])}
    if op == "ssm_update":
        steps = rng.choice([1, 1, 2, 3, 4, 5, 6])
        case = {"op": op, "rows": _log(rng, 1, 256 // steps), "steps": steps, "dt": rng.choice(["bf16", "bf16", "fp32"]),
                "gated": rng.random() < 0.5}
        if rng.random() < 0.5:
            groups = rng.choice([1, 1, 2, 4, 8])
            dim, states = rng.choice([(64, 128), (64, 128), (64, 64), (128, 128), (80, 96), (32, 16)])
            return {**case, "heads": groups * rng.choice([1, 3, 4, 8, 16]), "dim": dim, "groups": groups, "states": states,
                    "per_state": False}
        return {**case, "heads": rng.choice([256, 1000, 2048, 2500, 4096, 8192]), "dim": 1, "groups": 1,
                "states": rng.choice([16, 16, 16, 8, 24]), "per_state": True}
    drafts = rng.choice([0, 0, 1, 2, 3, 4])
    return {"op": op, "rows": _log(rng, 1, 256 // (drafts + 1)), "drafts": drafts, "vocab": _log(rng, 1000, 131072),
            "dtype": rng.choice(["bf16", "fp32"]), "history": _log(rng, 4, 9000), "bias": rng.choice([0, 0, 1, 30, 300]),
            "mask": rng.random() < 0.5, "in_place": rng.random() < 0.4}


# ----------------------------------------------------------------- inputs ----

def _tokens(n, case, g):
    """What the projections and the convolution make for n tokens: x, B, C, dt and the gate; and the layer's weights."""
    h, p, gr, ns = (case[k] for k in ("heads", "dim", "groups", "states"))
    kind = BF16 if case["dt"] == "bf16" else torch.float32

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["per_state"]:
        x = normal(n, h)
        x = (x / (1 + torch.exp(-x))).to(BF16)
        bc = normal(n, 64 + 2 * ns).to(BF16)  # the projection to dt's low rank, B and C
        b, c = bc[:, None, 64:64 + ns], bc[:, None, 64 + ns:]
        a = -(1 + torch.arange(ns, device="cuda")) * torch.exp(0.1 * normal(h, ns))
    else:
        mixed = normal(n, h * p + 2 * gr * ns)  # the convolution's output after its SiLU
        mixed = (mixed / (1 + torch.exp(-mixed))).to(BF16)
        x = mixed[:, :h * p].unflatten(1, (h, p))
        b = mixed[:, h * p:h * p + gr * ns].unflatten(1, (gr, ns))
        c = mixed[:, h * p + gr * ns:].unflatten(1, (gr, ns))
        a = -(1 + 15 * torch.rand(h, generator=g, device="cuda"))
    step = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(h, generator=g, device="cuda"))
    return {"x": x, "B": b, "C": c, "A": a, "dt": normal(n, h).to(kind), "dt_bias": step + torch.log(-torch.expm1(-step)),
            "D": 1 + 0.1 * normal(h), "z": normal(*x.shape).to(BF16) if case["gated"] else None}


def _pool(lines, case, g):
    shape = (lines, case["heads"], case["states"]) if case["per_state"] else (lines, case["heads"], case["dim"], case["states"])
    return 0.2 * torch.randn(*shape, generator=g, device="cuda")


def _prepare_fwd(case, g, seed):
    lengths = [int(x) for x in case["lengths"].split(",")]
    n, total = len(lengths), sum(lengths)
    order = list(range(n + 3))
    random.Random(seed).shuffle(order)
    init = {"all": [False] * n, "none": [True] * n, "some": [i % 2 == 0 for i in range(n)]}[case["fresh"]]
    return {**_tokens(total, case, g), "state": _pool(n + 3, case, g), "longest": max(lengths),
            "query_start_loc": torch.tensor([sum(lengths[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda"),
            "cache_indices": torch.tensor(order[:n], dtype=torch.int32, device="cuda"),
            "has_initial_state": torch.tensor(init, device="cuda")}


def _prepare_update(case, g, seed):
    b, t = case["rows"], case["steps"]
    out = {k: x.unflatten(0, (b, t)) if k in ("x", "B", "C", "dt", "z") and x is not None else x
           for k, x in _tokens(b * t, case, g).items()}
    lines = b * t + 2
    order = list(range(lines))
    random.Random(seed).shuffle(order)
    out["state"] = _pool(lines, case, g)
    if t == 1:
        out["state_indices"] = torch.tensor(order[:b], dtype=torch.int32, device="cuda")
    else:
        out["output_state_indices"] = torch.tensor(order[:b * t], dtype=torch.int32, device="cuda").reshape(b, t)
        out["num_accepted_tokens"] = torch.randint(1, t + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
    return out


def _prepare_logits(case, g, seed):
    b, n, v, size = case["rows"], case["drafts"] + 1, case["vocab"], case["history"]
    kind = BF16 if case["dtype"] == "bf16" else torch.float32

    def ids(*shape):  # text repeats itself: a few tokens come often
        u = torch.rand(*shape, generator=g, device="cuda")
        return (v * u * u * u * u).to(torch.int32).clamp(max=v - 1)

    rng = random.Random(seed)
    total = [rng.randint(max(1, size // 2), size) for _ in range(b)]
    order = list(range(b + 2))
    rng.shuffle(order)
    lengths = torch.zeros(b + 2, dtype=torch.int32)
    lengths[torch.tensor(order[:b])] = torch.tensor(total, dtype=torch.int32)
    prompt = (lengths * torch.rand(b + 2, generator=torch.Generator().manual_seed(seed))).to(torch.int32)
    mask = None
    if case["mask"]:  # a grammar that leaves a quarter of the tokens
        mask = torch.randint(-2 ** 31, 2 ** 31, (2, b, n, -(-v // 32)), generator=g, device="cuda").to(torch.int32)
        mask = mask[0] & mask[1]
    bias = case["bias"]
    return {"logits": (3 * torch.randn(b, n, v, generator=g, device="cuda")).to(kind), "history": ids(b + 2, size),
            "history_indices": torch.tensor(order[:b], dtype=torch.int32, device="cuda"),
            "prompt_lengths": prompt.cuda(), "history_lengths": lengths.cuda(),
            "draft_tokens": ids(b, n - 1) if n > 1 else None,
            "repetition": 1 + 0.5 * torch.rand(b, generator=g, device="cuda"),
            "frequency": 0.3 * torch.rand(b, generator=g, device="cuda"),
            "presence": torch.rand(b, generator=g, device="cuda") - 0.3,
            "bias_ids": torch.argsort(torch.rand(b, v, generator=g, device="cuda"), -1)[:, :bias].to(torch.int32) if bias else None,
            "bias": 5 * torch.randn(b, bias, generator=g, device="cuda") if bias else None,
            "mask": mask, "in_place": case["in_place"]}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = {"ssm_fwd": _prepare_fwd, "ssm_update": _prepare_update, "logits": _prepare_logits}[case["op"]]
    return {**make(case, g, seed), "op": case["op"]}


# ------------------------------------------------------------ plain forms ----

def _plain_dt(s):
    dt = s["dt"].float() + s["dt_bias"]
    return torch.where(dt > 20.0, dt, torch.log1p(torch.exp(dt.clamp(max=20.0))))


def _finish(y, s):
    """The outputs of the recurrence y (.., heads, dim) with D x and the gate."""
    x = s["x"].float().reshape(y.shape)
    y = y + s["D"][:, None] * x
    if s["z"] is not None:
        z = s["z"].float().reshape(y.shape)
        y = y * (z / (1 + torch.exp(-z)))
    return y.to(BF16).reshape(s["x"].shape)


def _chunk_heads(x, dt, logs, b, c):
    """Chunks on their own, one decay a head, by products: outputs from a zero state, what a first state adds to each
    token's output (the rows that multiply it), the chunk's own final state, and the decay of the whole chunk.
    x (n, chunks, c, heads, dim); dt, logs (n, chunks, c, heads); b, c (n, chunks, c, groups, states)."""
    size, groups = x.shape[2], b.shape[3]
    sums = logs.double().cumsum(2)
    row = torch.arange(size, device="cuda")
    diff = (sums[:, :, :, None] - sums[:, :, None]).float().masked_fill((row[:, None] < row)[:, :, None], -math.inf)
    cb = torch.einsum("nkigs,nkjgs->nkgij", c, b).repeat_interleave(x.shape[3] // groups, 2)
    m = cb * torch.exp(diff).permute(0, 1, 4, 2, 3) * dt.transpose(2, 3)[:, :, :, None]
    xt = x.transpose(2, 3)
    y = m @ xt
    tail = dt * torch.exp((sums[:, :, -1:] - sums).float())
    xg = (x * tail[..., None]).unflatten(3, (groups, -1))
    own_state = torch.einsum("nkjgrp,nkjgs->nkgrps", xg, b).flatten(2, 3)
    return y.transpose(2, 3), torch.exp(sums.float()), own_state, torch.exp(sums[:, :, -1].float())[..., None, None]


def _chunk_states(x, dt, a, b):
    """The states after every token of chunks on their own, a decay for every state: b_t summed with decays by doubling
    the distance.  Returns them and the decays since the chunk's start, (n, chunks, c, channels, states)."""
    size = x.shape[2]
    decay = torch.exp(dt[..., None] * a)
    state = (dt * x)[..., None] * b
    step = 1
    while step < size:
        state[:, :, step:] = state[:, :, step:] + decay[:, :, step:] * state[:, :, :-step]
        decay[:, :, step:] = decay[:, :, step:] * decay[:, :, :-step]
        step *= 2
    return state, decay


def _plain_fwd(s):
    """All sequences padded to the longest; a loop over chunks carries the state."""
    start = s["query_start_loc"].long()
    n, total, size = start.numel() - 1, s["x"].shape[0], CHUNK
    chunks = -(-s["longest"] // size)
    at = start[:-1, None] + torch.arange(chunks * size, device="cuda")
    real = at < start[1:, None]
    at = at.clamp(max=total - 1)

    def tiles(x):  # (tokens, ...) -> (n, chunks, c, ...), zeros past each sequence's end
        return (x[at] * real.reshape(real.shape + (1,) * (x.dim() - 1))).unflatten(1, (chunks, size))

    x, dt, b, c = tiles(s["x"].float()), tiles(_plain_dt(s)), tiles(s["B"].float()), tiles(s["C"].float())
    lines = s["cache_indices"].long()
    keep = s["has_initial_state"].float()
    state = s["state"][lines] * keep.reshape(-1, *(1,) * (s["state"].dim() - 1))
    firsts = []
    if s["A"].dim() == 1:
        y, rows, own_state, last = _chunk_heads(x, dt, dt * s["A"], b, c)
        for k in range(chunks):
            firsts.append(state)
            state = last[:, k] * state + own_state[:, k]
        first = torch.stack(firsts, 1).unflatten(2, (b.shape[3], -1))
        y = y + torch.einsum("nkigs,nkgrps->nkigrp", c, first).flatten(3, 4) * rows[..., None]
    else:
        states, decay = _chunk_states(x, dt, s["A"], b)
        for k in range(chunks):
            firsts.append(state)
            state = decay[:, k, -1] * state + states[:, k, -1]
        states += decay * torch.stack(firsts, 1)[:, :, None]
        y = (states @ c.transpose(3, 4))
    s["state"][lines] = torch.where((start[1:] > start[:-1]).reshape(-1, *(1,) * (state.dim() - 1)), state, s["state"][lines])
    return {"out": _finish(y.flatten(1, 2)[real], s), "state": s["state"]}


def _plain_update(s):
    spec = "output_state_indices" in s
    if spec:
        lines = s["output_state_indices"].long()
        read = lines.gather(1, s["num_accepted_tokens"].long()[:, None] - 1)[:, 0]
    else:
        read = s["state_indices"].long()
        lines = read[:, None]
    dt = _plain_dt(s)
    heads = s["dt"].shape[-1]
    pool = s["state"].reshape(s["state"].shape[0], heads, -1, s["state"].shape[-1])
    a = s["A"].reshape(heads, 1, -1)
    x = s["x"].float().reshape(*s["dt"].shape, -1)
    rep = heads // s["B"].shape[2]
    b, c = (s[k].float().repeat_interleave(rep, 2) for k in ("B", "C"))
    state, outs = pool[read], []
    for t in range(x.shape[1]):
        step = dt[:, t, :, None, None]
        state = state * torch.exp(step * a) + step * x[:, t, :, :, None] * b[:, t, :, None]
        outs.append((state * c[:, t, :, None]).sum(-1))
        pool[lines[:, t]] = state
    return {"out": _finish(torch.stack(outs, 1), s), "state": s["state"]}


def _plain_logits(s):
    x = s["logits"].float()
    b, n, v = x.shape
    line = s["history_indices"].long()
    ids, length, prompt = s["history"][line].long(), s["history_lengths"][line], s["prompt_lengths"][line]
    at = torch.arange(ids.shape[1], device="cuda")
    told = at < length[:, None]
    said = told & (at >= prompt[:, None])
    seen = torch.zeros(b, v, device="cuda").scatter_add_(1, ids, told.float())
    count = torch.zeros(b, v, device="cuda").scatter_add_(1, ids, said.float())
    seen, count = seen[:, None].repeat(1, n, 1), count[:, None].repeat(1, n, 1)
    if n > 1:  # position i follows drafts 0 .. i - 1
        drafts = s["draft_tokens"].long()
        after = torch.arange(n, device="cuda")[:, None] > torch.arange(n - 1, device="cuda")
        where = drafts[:, None].expand(b, n, n - 1)
        one = after.float().expand(b, n, n - 1)
        seen.scatter_add_(2, where, one)
        count.scatter_add_(2, where, one)
    r = s["repetition"][:, None, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / r, x * r), x)
    x = x - s["frequency"][:, None, None] * count - s["presence"][:, None, None] * (count > 0)
    if s["bias_ids"] is not None:
        x = x + torch.zeros(b, v, device="cuda").scatter_add_(1, s["bias_ids"].long(), s["bias"])[:, None]
    if s["mask"] is not None:
        bits = (s["mask"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        x = x.masked_fill(bits.flatten(2)[..., :v] == 0, -math.inf)
    if s["in_place"]:
        s["logits"].copy_(x)
        return s["logits"]
    return x.to(s["logits"].dtype)


# ------------------------------------------------------------------- runs ----

def _run_own(s):
    import causal_depthwise_conv1d_fwd_gb300 as ccv

    if s["op"] == "ssm_fwd":
        out = ccv.ssm_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], s["query_start_loc"], s["cache_indices"],
                          s["has_initial_state"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
        return {"out": out, "state": s["state"]}
    if s["op"] == "ssm_update":
        out = ccv.ssm_update(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], s.get("state_indices"),
                             num_accepted_tokens=s.get("num_accepted_tokens"),
                             output_state_indices=s.get("output_state_indices"), D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
        return {"out": out, "state": s["state"]}
    return ccv.logits_process(s["logits"], s["history"], s["history_lengths"], s["prompt_lengths"], s["history_indices"],
                              draft_tokens=s["draft_tokens"], repetition=s["repetition"], frequency=s["frequency"],
                              presence=s["presence"], bias_ids=s["bias_ids"], bias=s["bias"], mask=s["mask"],
                              out=s["logits"] if s["in_place"] else None)


def run(state):
    if own:
        return _run_own(state)
    return {"ssm_fwd": _plain_fwd, "ssm_update": _plain_update, "logits": _plain_logits}[state["op"]](state)


def work(case):
    if case["op"] == "logits":
        b, n, v = case["rows"], case["drafts"] + 1, case["vocab"]
        size = 2 if case["dtype"] == "bf16" else 4
        told = 3 * case["history"] / 4
        touched = min(v, told + case["drafts"] + case["bias"])
        mask = v / 8 if case["mask"] else 0
        # in place, a logit that nothing changes is neither read nor written, and a masked one only written
        if not case["in_place"]:
            per = n * (2 * v * size + mask)
        else:
            per = n * (2 * touched * size + mask + (0.75 * v * size if case["mask"] else 0))
        return {"bytes": b * (per + 4 * told + 8 * case["bias"] + 12), "flops": b * n * touched * 6}
    h, p, gr, ns = (case[k] for k in ("heads", "dim", "groups", "states"))
    token = 2 * (2 * h * p + 2 * gr * ns) + (2 if case["dt"] == "bf16" else 4) * h + (2 * h * p if case["gated"] else 0)
    weights = 4 * h * (2 + (ns if case["per_state"] else 1))
    if case["op"] == "ssm_fwd":
        lengths = [int(x) for x in case["lengths"].split(",")]
        tokens = sum(lengths)
        read = {"all": 0, "none": sum(n > 0 for n in lengths), "some": sum(n > 0 for n in lengths[::2])}[case["fresh"]]
        written = sum(n > 0 for n in lengths)
    else:
        tokens, read = case["rows"] * case["steps"], case["rows"]
        written = tokens
    return {"bytes": tokens * token + weights + (read + written) * 4 * h * p * ns, "flops": tokens * h * p * ns * 5}


# ---------------------------------------------------------------- 64 bits ----

def _exact_step(state, x, dt, a, b, c):
    """One token of the recurrence: state (rows, heads, dim, states), x (rows, heads, dim), dt (rows, heads), a (heads, 1,
    states or 1), b and c (rows, groups, states)."""
    rep = x.shape[1] // b.shape[1]
    b, c = b.repeat_interleave(rep, 1), c.repeat_interleave(rep, 1)
    state = torch.exp(dt[..., None, None] * a) * state + (dt[..., None] * x)[..., None] * b[:, :, None]
    return state, torch.matmul(state, c[..., None])[..., 0]


def _exact_ssm(s):
    heads = s["dt"].shape[-1]
    x, z = (None if t is None else t.double().reshape(*s["dt"].shape, -1) for t in (s["x"], s["z"]))
    dt = torch.logaddexp(s["dt"].double() + s["dt_bias"].double(), torch.zeros(1, dtype=torch.float64, device="cuda"))
    a, b, c = s["A"].double().reshape(heads, 1, -1), s["B"].double(), s["C"].double()
    pool = s["state"].double().reshape(s["state"].shape[0], heads, -1, s["state"].shape[-1])
    out = torch.zeros_like(x)
    if s["op"] == "ssm_fwd":
        starts, lines = s["query_start_loc"].tolist(), s["cache_indices"].long()
        sizes = [e - f for f, e in zip(starts, starts[1:])]
        order = sorted(range(len(sizes)), key=lambda i: -sizes[i])  # the sequences still running come first
        pick = torch.tensor(order, device="cuda")
        first = torch.tensor([starts[i] for i in order], device="cuda")
        state = pool[lines[pick]] * s["has_initial_state"][pick].double()[:, None, None, None]
        live = sum(n > 0 for n in sizes)
        some = live
        for t in range(s["longest"]):
            while live and sizes[order[live - 1]] <= t:
                live -= 1
            at = first[:live] + t
            state[:live], out[at] = _exact_step(state[:live], x[at], dt[at], a, b[at], c[at])
        pool[lines[pick[:some]]] = state[:some]
    else:
        if "output_state_indices" in s:
            lines = s["output_state_indices"].long()
            state = pool[lines[torch.arange(lines.shape[0], device="cuda"), s["num_accepted_tokens"].long() - 1]]
        else:
            lines = s["state_indices"].long()[:, None]
            state = pool[lines[:, 0]]
        for t in range(x.shape[1]):
            state, out[:, t] = _exact_step(state, x[:, t], dt[:, t], a, b[:, t], c[:, t])
            pool[lines[:, t]] = state
    out = out + s["D"].double()[:, None] * x
    if z is not None:
        out = out * z * torch.sigmoid(z)
    return {"out": out.reshape(s["x"].shape), "state": pool.reshape(s["state"].shape)}


def _exact_logits(s):
    x = s["logits"].double()
    b, n, v = x.shape
    for r in range(b):
        line = int(s["history_indices"][r])
        told, prompt = int(s["history_lengths"][line]), int(s["prompt_lengths"][line])
        ids = s["history"][line, :told].long()
        seen, count = torch.bincount(ids, minlength=v) > 0, torch.bincount(ids[prompt:], minlength=v)
        for i in range(n):
            if i > 0:
                token = int(s["draft_tokens"][r, i - 1])
                seen[token] = True
                count[token] += 1
            y, rep = x[r, i], s["repetition"][r].double()
            y = torch.where(seen, torch.where(y > 0, y / rep, y * rep), y)
            y = y - s["frequency"][r].double() * count - s["presence"][r].double() * (count > 0)
            if s["bias_ids"] is not None:
                y[s["bias_ids"][r].long()] += s["bias"][r].double()
            if s["mask"] is not None:
                words = s["mask"][r, i].long()
                at = torch.arange(v, device="cuda")
                y = torch.where((words[at // 32] >> (at % 32)) & 1 == 1, y, -math.inf)
            x[r, i] = y
    return x


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_logits(s) if s["op"] == "logits" else _exact_ssm(s)
