"""The state-space layer's operators and the token log probabilities, as cases to be measured.

Each case is one call a user makes: the short causal convolution and the selective scan over
prompts and over single tokens, the residual's addition with the root-mean-square norm in front of
such a layer, and the log probabilities, entropy and top alternatives behind a model's logits.

``prepare`` makes a case's inputs, ``run`` makes the call (``own``: the library's; else the same
formulas in elementary torch operations, 32 bits inside, rounded once at the end), ``exact``
evaluates the definition in 64 bits, ``work`` counts the bytes and operations of the definition.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
E4M3_MAX = 448.0


def listed():
    return [
        # one stream's next token through one layer: nothing but latency
        {"name": "conv step b1", "op": "conv_step", "dtype": "bf16", "sequences": 1,
         "channels": 2048, "width": 4, "pool": 4},
        # a batch of long and short prompts, packed without padding, some of them continued
        {"name": "conv ragged 12288", "op": "conv", "dtype": "bf16", "sequences": 24,
         "tokens": 12288, "ragged": True, "channels": 4096, "width": 4, "resume": True, "pool": 40},
        # windows of equal length at the LSTM stack's own widths and step count, in fp32
        {"name": "conv windows b32 t589", "op": "conv", "dtype": "f32", "sequences": 32,
         "tokens": 32 * 589, "ragged": False, "channels": 256, "width": 3, "resume": False,
         "pool": 32},
        # one window at the LSTM stack's own widths, in fp32
        {"name": "scan window t589", "op": "scan", "dtype": "f32", "sequences": 1, "tokens": 589,
         "ragged": False, "channels": 256, "state": 16, "groups": 1, "gate": True,
         "resume": False, "pool": 1},
        # one prompt of a single user: few channels, a long axis
        {"name": "scan prompt 4096", "op": "scan", "dtype": "bf16", "sequences": 1,
         "tokens": 4096, "ragged": False, "channels": 2048, "state": 16, "groups": 1,
         "gate": True, "resume": False, "pool": 4},
        # a packed batch of unequal prompts of a larger layer, some of them continued: throughput
        {"name": "scan ragged 12288", "op": "scan", "dtype": "bf16", "sequences": 24,
         "tokens": 12288, "ragged": True, "channels": 4096, "state": 16, "groups": 1,
         "gate": True, "resume": True, "pool": 40},
        # the next token of one stream
        {"name": "scan step b1", "op": "scan_step", "dtype": "bf16", "sequences": 1,
         "channels": 2048, "state": 16, "groups": 1, "gate": True, "pool": 4},
        # the next token of a full serving batch, its states scattered over a pool
        {"name": "scan step b256", "op": "scan_step", "dtype": "bf16", "sequences": 256,
         "channels": 4096, "state": 16, "groups": 1, "gate": True, "pool": 300},
        # a decode batch's activations before a projection in 8 bits
        {"name": "norm 16x2048 e4m3 row", "op": "norm", "dtype": "bf16", "out": "e4m3",
         "rows": 16, "cols": 2048, "group": 0, "residual": True},
        # a prompt batch's activations before a projection in 8 bits with a scale per 128 columns
        {"name": "norm 12288x4096 e4m3 128", "op": "norm", "dtype": "bf16", "out": "e4m3",
         "rows": 12288, "cols": 4096, "group": 128, "residual": True},
        # every frame of a batch of windows over the dense heads' seven classes
        {"name": "logprobs 18848x7", "op": "logprobs", "dtype": "f32", "rows": 32 * 589,
         "vocab": 7, "top": 3},
        # a decode batch over a text vocabulary of odd size
        {"name": "logprobs 64x100003", "op": "logprobs", "dtype": "bf16", "rows": 64,
         "vocab": 100003, "top": 20},
    ]


def _spread(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def _sized(rng, low, high):
    """A size over the range's logarithm: a power of two, or 5/4 or 7/4 of one; one time in three
    an odd number, or eight times one."""
    if rng.random() < 0.34:
        eight = rng.choice([1, 8]) if high >= 8 * low else 1
        return eight * (2 * _spread(rng, -(-low // (2 * eight)), (high // eight - 1) // 2) + 1)
    quarter = _spread(rng, -(-low // 4), high // 7)
    return (1 << (quarter.bit_length() - 1)) * rng.choice([4, 5, 7])


def draw(rng):
    op = rng.choice(["conv", "conv_step", "scan", "scan", "scan_step", "norm", "logprobs"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op in ("conv", "conv_step", "scan", "scan_step"):
        case["channels"] = _sized(rng, 32, 4096)
        if op.endswith("step"):
            case["sequences"] = _spread(rng, 1, 256)
        else:
            most = 12288 * 4096 // case["channels"] // (1 if case["dtype"] != "f32" else 2)
            case["tokens"] = _spread(rng, 1, min(most, 12288))
            case["sequences"] = _spread(rng, 1, min(64, case["tokens"]))
            case["ragged"] = rng.random() < 0.6
            if not case["ragged"]:
                case["tokens"] = max(1, case["tokens"] // case["sequences"]) * case["sequences"]
            case["resume"] = rng.random() < 0.5
        case["pool"] = case["sequences"] + rng.randrange(0, 16)
    if op.startswith("conv"):
        case["width"] = rng.choice([2, 3, 4, 4])
    if op.startswith("scan"):
        case["state"] = rng.choice([4, 8, 13, 16, 16, 16])
        if op == "scan_step" and rng.random() < 0.3:
            case["state"] = 64
            case["sequences"] = min(case["sequences"], 64)
        case["groups"] = rng.choice([1, 1, 2]) if case["channels"] % 2 == 0 else 1
        case["gate"] = rng.random() < 0.8
    if op == "norm":
        case["cols"] = _sized(rng, 32, 8192)
        case["rows"] = _spread(rng, 1, 12288 * 4096 // case["cols"] // 2 if case["cols"] > 2048 else 12288)
        case["out"] = rng.choice(["e4m3", "e4m3", case["dtype"]])
        case["group"] = rng.choice([0, 128, 64]) if case["out"] == "e4m3" else 0
        case["residual"] = rng.random() < 0.8
    if op == "logprobs":
        case["vocab"] = _sized(rng, 7, 128000)
        case["rows"] = _spread(rng, 1, max(1, min(18848, 64 * 128000 // case["vocab"])))
        case["top"] = min(case["vocab"], rng.choice([0, 1, 5, 20]))
    return case


# ---------------------------------------------------------------------------------------------
# Inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bounds(case, seed):
    """Where each sequence starts, and where the last one ends."""
    s, t = case["sequences"], case["tokens"]
    if not case["ragged"]:
        return [k * (t // s) for k in range(s + 1)]
    # lengths spread over a factor of about thirty, as prompts' lengths are
    host = torch.Generator().manual_seed(seed + 17)
    share = torch.exp(3.4 * torch.rand(s, generator=host, dtype=torch.float64))
    cut = torch.floor(torch.cumsum(share, 0) / share.sum() * t).long().tolist()
    cut[-1] = t
    return [0] + cut


def prepare(case, seed):
    g, op, dt = _gen(seed), case["op"], DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    st = {"case": case, "op": op}
    if op == "norm":
        st["x"] = normal(case["rows"], case["cols"], dtype=dt)
        st["residual"] = normal(case["rows"], case["cols"], scale=4.0, dtype=dt) if case["residual"] else None
        st["weight"] = 0.5 + uniform(case["cols"])
        st["eps"] = 1e-5
        return st
    if op == "logprobs":
        logits = normal(case["rows"], case["vocab"], scale=3.0)
        # words that a decoder forbids come as the lowest value
        logits.masked_fill_(uniform(case["rows"], case["vocab"]) < 0.01, -math.inf)
        logits[:, 0] = 0.0
        st["logits"] = logits.to(dt)
        st["tokens"] = (uniform(case["rows"]) * case["vocab"]).long().clamp_(max=case["vocab"] - 1)
        st["tokens"][::3] = 0
        return st
    step = op.endswith("step")
    d, s = case["channels"], case["sequences"]
    tokens = s if step else case["tokens"]
    # the input and the gate are halves of one projection's output
    xz = normal(tokens, 2 * d, dtype=dt)
    st["x"], st["z"] = xz[:, :d], xz[:, d:]
    st["slots"] = torch.randperm(case["pool"], generator=g, device="cuda")[:s].int()
    st["resume"] = st["offsets"] = None
    st["sequences"] = s
    if not step:
        bounds = _bounds(case, seed)
        st["bounds"] = bounds
        if case["ragged"]:
            st["offsets"] = torch.tensor(bounds, dtype=torch.int32, device="cuda")
        if case["resume"]:
            st["resume"] = (uniform(s) < 0.5).int()
    if op.startswith("conv"):
        w = case["width"]
        st["w"] = normal(d, w, scale=0.5)
        st["bias"] = normal(d, scale=0.1)
        st["state"] = normal(case["pool"], w - 1, d, dtype=dt)
        return st
    n, groups = case["state"], case["groups"]
    st["x"] = torch.nn.functional.silu(st["x"])
    # the step sizes before their bias and softplus, then B and C, from one narrow projection
    st["dt"] = normal(tokens, d, scale=0.5, dtype=dt)
    rank = (d + 15) // 16
    dbc = normal(tokens, rank + 2 * groups * n, dtype=dt)
    st["b"] = dbc[:, rank:rank + groups * n]
    st["c"] = dbc[:, rank + groups * n:]
    st["a"] = -torch.arange(1, n + 1, device="cuda", dtype=torch.float32) * torch.exp(normal(d, n, scale=0.2))
    target = torch.exp(math.log(1e-3) + uniform(d) * math.log(100.0))
    st["dt_bias"] = target + torch.log(-torch.expm1(-target))
    st["skip"] = torch.ones(d, device="cuda") + normal(d, scale=0.1)
    st["state"] = normal(case["pool"], d, n, scale=0.5)
    if not case["gate"]:
        st["z"] = None
    return st


# ---------------------------------------------------------------------------------------------
# One pass


def run(st):
    return RUN[st["op"]][own](st)


def _conv_own(st):
    from bidirectional_lstm_stack_gb300 import binding
    y = binding.lstm_causal_conv(st["x"], st["w"], st["bias"], silu=True, sequences=st["sequences"],
                                 offsets=st["offsets"], state=st["state"], slots=st["slots"],
                                 resume=st["resume"])
    return {"y": y, "state": st["state"]}


def _conv_step_own(st):
    from bidirectional_lstm_stack_gb300 import binding
    y = binding.lstm_causal_conv_step(st["x"], st["w"], st["bias"], st["state"], silu=True,
                                      slots=st["slots"])
    return {"y": y, "state": st["state"]}


def _scan_own(st):
    from bidirectional_lstm_stack_gb300 import binding
    y = binding.lstm_selective_scan(st["x"], st["dt"], st["a"], st["b"], st["c"], skip=st["skip"],
                                    z=st["z"], dt_bias=st["dt_bias"], softplus=True,
                                    groups=st["case"]["groups"], sequences=st["sequences"],
                                    offsets=st["offsets"], state=st["state"], slots=st["slots"],
                                    resume=st["resume"])
    return {"y": y, "state": st["state"]}


def _scan_step_own(st):
    from bidirectional_lstm_stack_gb300 import binding
    y = binding.lstm_selective_scan_step(st["x"], st["dt"], st["a"], st["b"], st["c"], st["state"],
                                         skip=st["skip"], z=st["z"], dt_bias=st["dt_bias"],
                                         softplus=True, groups=st["case"]["groups"],
                                         slots=st["slots"])
    return {"y": y, "state": st["state"]}


def _norm_own(st):
    from bidirectional_lstm_stack_gb300 import binding
    case = st["case"]
    y, scales, residual = binding.lstm_residual_rms_norm(
        st["x"], st["weight"], st["eps"], residual=st["residual"],
        quantize=case["out"] == "e4m3", group=case["group"])
    return {"y": y, "scales": scales, "residual": residual}


def _logprobs_own(st):
    from bidirectional_lstm_stack_gb300 import binding
    logp, entropy, top_logp, top_ids = binding.lstm_token_logprobs(st["logits"], st["tokens"],
                                                                   top=st["case"]["top"])
    return {"logp": logp, "entropy": entropy, "top_logp": top_logp, "top_ids": top_ids}


def _token_starts(st, tokens):
    """For every token the number of its sequence, and where that sequence starts."""
    dev = st["x"].device
    if st["offsets"] is None:
        seq = torch.arange(tokens, device=dev) // (tokens // st["sequences"])
        return seq, seq * (tokens // st["sequences"])
    at = st["offsets"].long()
    seq = torch.searchsorted(at, torch.arange(tokens, device=dev), right=True) - 1
    return seq, at[seq]


def _old_state(st, rows):
    old = st["state"][rows].float()
    if st["resume"] is None:
        return torch.zeros_like(old)
    return torch.where((st["resume"] != 0).reshape(-1, *[1] * (old.dim() - 1)), old, torch.zeros_like(old))


def _conv_plain(st):
    x, w = st["x"], st["w"]
    tokens, width = x.shape[0], w.shape[1]
    rows = st["slots"].long()
    old = _old_state(st, rows)
    seq, start = _token_starts(st, tokens)
    # one table: every token, then every sequence's width - 1 tokens before its first
    table = torch.cat([x.float(), old.reshape(-1, x.shape[1])])
    at = torch.arange(tokens, device=x.device)[:, None] + torch.arange(1 - width, 1, device=x.device)
    before = at - start[:, None]
    at = torch.where(before >= 0, at, tokens + seq[:, None] * (width - 1) + (width - 1) + before)
    y = (table[at] * w.t()).sum(1) + st["bias"]
    y = y * torch.sigmoid(y)
    if st["offsets"] is None:
        ends = torch.arange(1, len(rows) + 1, device=x.device) * (tokens // st["sequences"])
        starts = ends - tokens // st["sequences"]
    else:
        starts, ends = st["offsets"][:-1].long(), st["offsets"][1:].long()
    at = ends[:, None] + torch.arange(1 - width, 0, device=x.device)
    before = at - starts[:, None]
    number = torch.arange(len(rows), device=x.device)[:, None]
    at = torch.where(before >= 0, at, tokens + number * (width - 1) + (width - 1) + before)
    st["state"][rows] = table[at].to(st["state"].dtype)
    return {"y": y.to(x.dtype), "state": st["state"]}


def _conv_step_plain(st):
    x, rows = st["x"], st["slots"].long()
    window = torch.cat([st["state"][rows].float(), x.float()[:, None]], 1)
    y = (window * st["w"].t()).sum(1) + st["bias"]
    y = y * torch.sigmoid(y)
    st["state"][rows] = window[:, 1:].to(st["state"].dtype)
    return {"y": y.to(x.dtype), "state": st["state"]}


def _softplus(v):
    return torch.clamp(v, min=0.0) + torch.log1p(torch.exp(-v.abs()))


def _scan_terms(st):
    """The step sizes, the states' decay and what each token adds, [tokens, channels(, state)]."""
    x, groups, n = st["x"].float(), st["case"]["groups"], st["a"].shape[1]
    tokens, d = x.shape
    dt = _softplus(st["dt"].float() + st["dt_bias"])
    decay = torch.exp(dt[:, :, None] * st["a"])
    b = st["b"].float().reshape(tokens, groups, 1, n)
    add = (dt * x).reshape(tokens, groups, d // groups, 1) * b
    return x, decay, add.reshape(tokens, d, n)


def _scan_out(st, x, h):
    groups, n = st["case"]["groups"], st["a"].shape[1]
    tokens, d = x.shape
    c = st["c"].float().reshape(tokens, groups, 1, n)
    y = (h.reshape(tokens, groups, d // groups, n) * c).sum(-1).reshape(tokens, d) + st["skip"] * x
    if st["z"] is not None:
        z = st["z"].float()
        y = y * z * torch.sigmoid(z)
    return y.to(st["x"].dtype)


def _scan_plain(st):
    x, decay, add = _scan_terms(st)
    tokens, rows = x.shape[0], st["slots"].long()
    old = _old_state(st, rows)
    seq, start = _token_starts(st, tokens)
    first = (torch.arange(tokens, device=x.device) == start).nonzero()[:, 0]
    add[first] += decay[first] * old[seq[first]]
    decay[first] = 0.0
    # h[t] = decay[t] h[t-1] + add[t], each turn joining spans of twice the length
    reach = 1
    longest = max(b - a for a, b in zip(st["bounds"], st["bounds"][1:]))
    while reach < longest:
        more = torch.zeros_like(add)
        more[reach:] = decay[reach:] * add[:-reach]
        add = add + more
        joined = torch.zeros_like(decay)
        joined[reach:] = decay[reach:] * decay[:-reach]
        decay = joined
        reach *= 2
    y = _scan_out(st, x, add)
    if st["offsets"] is None:
        ends = torch.arange(1, len(rows) + 1, device=x.device) * (tokens // st["sequences"])
        empty = torch.zeros(len(rows), dtype=torch.bool, device=x.device)
    else:
        ends = st["offsets"][1:].long()
        empty = ends == st["offsets"][:-1]
    st["state"][rows] = torch.where(empty[:, None, None], old, add[(ends - 1).clamp(min=0)])
    return {"y": y, "state": st["state"]}


def _scan_step_plain(st):
    x, decay, add = _scan_terms(st)
    rows = st["slots"].long()
    h = decay * st["state"][rows] + add
    st["state"][rows] = h
    return {"y": _scan_out(st, x, h), "state": st["state"]}


def _norm_plain(st):
    case = st["case"]
    v = st["x"].float()
    residual = None
    if st["residual"] is not None:
        v = v + st["residual"].float()
        residual = v.to(st["x"].dtype)
    y = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + st["eps"]) * st["weight"]
    if case["out"] != "e4m3":
        return {"y": y.to(st["x"].dtype), "scales": None, "residual": residual}
    rows, cols = v.shape
    group = case["group"] or cols
    wide = torch.zeros(rows, -(-cols // group) * group, device=v.device)
    wide[:, :cols] = y
    wide = wide.reshape(rows, -1, group)
    top = wide.abs().amax(-1, keepdim=True)
    scales = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    q = (wide / scales).clamp(-E4M3_MAX, E4M3_MAX).reshape(rows, -1)[:, :cols]
    return {"y": q.to(torch.float8_e4m3fn), "scales": scales[..., 0], "residual": residual}


def _logprobs_plain(st):
    logits, top = st["logits"].float(), st["case"]["top"]
    v = logits - logits.amax(-1, keepdim=True)
    e = torch.exp(v)
    total = e.sum(-1, keepdim=True)
    logp = v - torch.log(total)
    p = e / total
    entropy = -(p * torch.where(p > 0, logp, torch.zeros_like(logp))).sum(-1)
    given = logp.gather(1, st["tokens"][:, None])[:, 0]
    if not top:
        return {"logp": given, "entropy": entropy, "top_logp": None, "top_ids": None}
    # a stable sort: equal values stay in their order, the lowest index first
    ids = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :top].contiguous()
    return {"logp": given, "entropy": entropy, "top_logp": logp.gather(1, ids), "top_ids": ids}


RUN = {
    "conv": (_conv_plain, _conv_own),
    "conv_step": (_conv_step_plain, _conv_step_own),
    "scan": (_scan_plain, _scan_own),
    "scan_step": (_scan_step_plain, _scan_step_own),
    "norm": (_norm_plain, _norm_own),
    "logprobs": (_logprobs_plain, _logprobs_own),
}


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    for key, v in st.items():
        if torch.is_tensor(v) and v.is_floating_point():
            st[key] = v.double()
    op = case["op"]
    if op == "norm":
        v = st["x"] if st["residual"] is None else st["x"] + st["residual"]
        y = v / torch.sqrt((v * v).sum(-1, keepdim=True) / case["cols"] + st["eps"]) * st["weight"]
        out = {"y": y, "scales": None, "residual": None if st["residual"] is None else v}
        if case["out"] == "e4m3":
            group = case["group"] or case["cols"]
            parts = [y[:, k:k + group] for k in range(0, case["cols"], group)]
            tops = [p.abs().max(-1).values / E4M3_MAX for p in parts]
            out["y"] = torch.cat([p / t[:, None] for p, t in zip(parts, tops)], 1)
            out["scales"] = torch.stack(tops, 1)
        return out
    if op == "logprobs":
        logits, top = st["logits"], case["top"]
        logp = logits - torch.logsumexp(logits, -1, keepdim=True)
        rows = torch.arange(case["rows"], device="cuda")
        best = logp.sort(-1, descending=True).values[:, :top].contiguous() if top else None
        return {"logp": logp[rows, st["tokens"]], "entropy": torch.special.entr(logp.exp()).sum(-1),
                "top_logp": best, "top_ids": None}
    if op.startswith("conv"):
        return _conv_exact(case, st)
    return _scan_exact(case, st)


def _spans(case, st):
    """(sequence, first token, end, whether it goes on from its state)."""
    if case["op"].endswith("step"):
        return [(k, k, k + 1, True) for k in range(case["sequences"])]
    goes_on = [False] * case["sequences"] if st["resume"] is None else st["resume"].bool().tolist()
    return [(k, a, b, goes_on[k]) for k, (a, b) in enumerate(zip(st["bounds"], st["bounds"][1:]))]


def _conv_exact(case, st):
    x, w, width = st["x"], st["w"], case["width"]
    y, slots = torch.zeros(x.shape, dtype=torch.float64, device="cuda"), st["slots"].tolist()
    for k, a, b, goes_on in _spans(case, st):
        past = st["state"][slots[k]] if goes_on else torch.zeros_like(st["state"][slots[k]])
        line = torch.cat([past, x[a:b]])
        for tap in range(width):
            y[a:b] += line[tap:tap + b - a] * w[:, tap]
        st["state"][slots[k]] = line[len(line) - (width - 1):]
    y += st["bias"]
    return {"y": y / (1 + torch.exp(-y)), "state": st["state"]}


def _scan_exact(case, st):
    d, n, groups = case["channels"], case["state"], case["groups"]
    dt = torch.logaddexp(st["dt"] + st["dt_bias"], torch.zeros((), dtype=torch.float64, device="cuda"))
    of_group = torch.arange(d, device="cuda") // (d // groups)
    b = st["b"].reshape(-1, groups, n)
    c = st["c"].reshape(-1, groups, n)
    y = torch.zeros(st["x"].shape, dtype=torch.float64, device="cuda")
    spans = _spans(case, st)
    if sum(e - a for _, a, e, _ in spans) * d * n > 1 << 32:
        return None
    # all sequences side by side, the longest first, one token of each at a time
    spans.sort(key=lambda s: s[1] - s[2])
    slots = st["slots"].long()[[s[0] for s in spans]]
    h = st["state"][slots] * torch.tensor([float(s[3]) for s in spans], device="cuda")[:, None, None]
    lengths = [s[2] - s[1] for s in spans]
    starts = torch.tensor([s[1] for s in spans], device="cuda")
    live = len(spans)
    for t in range(lengths[0]):
        while lengths[live - 1] <= t:
            live -= 1
        at = starts[:live] + t
        h[:live] = (h[:live] * torch.exp(dt[at, :, None] * st["a"])
                    + (dt[at] * st["x"][at])[:, :, None] * b[at][:, of_group])
        y[at] = (h[:live] * c[at][:, of_group]).sum(-1)
    y += st["skip"] * st["x"]
    if st["z"] is not None:
        y = y * st["z"] / (1 + torch.exp(-st["z"]))
    st["state"][slots] = h
    return {"y": y, "state": st["state"]}


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    op, size = case["op"], BYTES[case["dtype"]]
    if op == "norm":
        cells = case["rows"] * case["cols"]
        groups = -(-case["cols"] // (case["group"] or case["cols"]))
        moved = cells * size * (3 if case["residual"] else 1) + cells * BYTES[case["out"]]
        moved += 4 * case["cols"] + (4 * case["rows"] * groups if case["out"] == "e4m3" else 0)
        return {"bytes": moved, "flops": 6 * cells}
    if op == "logprobs":
        cells = case["rows"] * case["vocab"]
        return {"bytes": cells * size + case["rows"] * (16 + 12 * case["top"]), "flops": 5 * cells}
    s, d = case["sequences"], case["channels"]
    tokens = s if op.endswith("step") else case["tokens"]
    reads = s if op.endswith("step") else s // 2 if case["resume"] else 0
    if op.startswith("conv"):
        w = case["width"]
        moved = 2 * tokens * d * size + (reads + s) * (w - 1) * d * size + 4 * d * (w + 1)
        return {"bytes": moved, "flops": tokens * d * (2 * w + 5)}
    n = case["state"]
    moved = tokens * d * size * (4 if case["gate"] else 3) + 2 * tokens * n * case["groups"] * size
    moved += (reads + s) * d * n * 4 + 4 * d * (n + 2)
    # per state: the decay's product and exponential, the update's two products and sum, the output's
    return {"bytes": moved, "flops": tokens * d * (n * 7 + 15)}
