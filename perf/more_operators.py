"""Linear attention with a decay for each head and the dense products around it, as cases to be
measured.

Each case is one call a user makes: linear attention over packed prompts and over single tokens,
and a matrix product with bias, activation and residual in its epilogue, as it stands in front of
and behind such a layer.

``prepare`` makes a case's inputs, ``run`` makes the call (``own``: the library's; else the same
formulas in elementary torch operations, 32 bits inside, rounded once at the end), ``exact``
evaluates the definition in 64 bits, ``work`` counts the bytes and operations of the definition.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
CHUNK = 64


def listed():
    return [
        # windows of equal length at the LSTM stack's own step count, in fp32
        {"name": "attention windows b32 t589", "op": "attention", "dtype": "f32", "sequences": 32,
         "tokens": 32 * 589, "ragged": False, "heads": 4, "q_heads": 4, "k_heads": 4, "v_heads": 4,
         "keys": 32, "values": 64, "each_token": False, "resume": False, "pool": 32},
        # one prompt of a single user: few heads, a long axis
        {"name": "attention prompt 4096", "op": "attention", "dtype": "bf16", "sequences": 1,
         "tokens": 4096, "ragged": False, "heads": 16, "q_heads": 16, "k_heads": 16, "v_heads": 16,
         "keys": 128, "values": 128, "each_token": False, "resume": False, "pool": 4},
        # a packed batch of unequal prompts, some of them continued: queries and keys shared by
        # groups of heads, a decay for each token and head, as state-space layers have them
        {"name": "attention ragged 12288", "op": "attention", "dtype": "bf16", "sequences": 24,
         "tokens": 12288, "ragged": True, "heads": 32, "q_heads": 2, "k_heads": 2, "v_heads": 32,
         "keys": 64, "values": 64, "each_token": True, "resume": True, "pool": 40},
        # long documents, keys and values shared by groups of heads: throughput
        {"name": "attention long 4x16384", "op": "attention", "dtype": "bf16", "sequences": 4,
         "tokens": 4 * 16384, "ragged": False, "heads": 16, "q_heads": 16, "k_heads": 4,
         "v_heads": 4, "keys": 128, "values": 128, "each_token": False, "resume": False, "pool": 4},
        # the next token of one stream
        {"name": "attention step b1", "op": "attention_step", "dtype": "bf16", "sequences": 1,
         "heads": 16, "q_heads": 16, "k_heads": 16, "v_heads": 16, "keys": 128, "values": 128,
         "each_token": False, "pool": 4},
        # the next token of a full serving batch, its states scattered over a pool
        {"name": "attention step b256", "op": "attention_step", "dtype": "bf16", "sequences": 256,
         "heads": 16, "q_heads": 16, "k_heads": 16, "v_heads": 16, "keys": 128, "values": 128,
         "each_token": True, "pool": 300},
        # one stream's next token through a layer's last product, onto its residual
        {"name": "dense 1x4096x4096", "op": "dense", "dtype": "bf16", "rows": 1, "in": 4096,
         "out": 4096, "bias": False, "activation": None, "residual": True},
        # a decode batch through a layer's widening product
        {"name": "dense 64x4096x16384 silu", "op": "dense", "dtype": "f16", "rows": 64, "in": 4096,
         "out": 16384, "bias": False, "activation": "silu", "residual": False},
        # every frame of a batch of windows from the LSTM stack's output width, in fp32
        {"name": "dense 18848x256x512 gelu", "op": "dense", "dtype": "f32", "rows": 32 * 589,
         "in": 256, "out": 512, "bias": True, "activation": "gelu", "residual": False},
        # sizes that no tile and no vector divides
        {"name": "dense 1001x777x1003 relu", "op": "dense", "dtype": "f16", "rows": 1001, "in": 777,
         "out": 1003, "bias": True, "activation": "relu", "residual": True},
        # a prompt batch through a layer's widening product
        {"name": "dense 2048x2048x8192 gelu_tanh", "op": "dense", "dtype": "bf16", "rows": 2048,
         "in": 2048, "out": 8192, "bias": True, "activation": "gelu_tanh", "residual": False},
        # a large prompt batch onto its residual: throughput
        {"name": "dense 12288x4096x4096", "op": "dense", "dtype": "bf16", "rows": 12288, "in": 4096,
         "out": 4096, "bias": True, "activation": None, "residual": True},
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
    op = rng.choice(["attention", "attention", "attention_step", "dense", "dense"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op == "dense":
        case["in"] = _sized(rng, 16, 8192)
        case["out"] = _sized(rng, 16, 16384)
        most = 12288 * 4096 * 4096 // (case["in"] * case["out"]) // (1 if case["dtype"] != "f32" else 16)
        case["rows"] = _spread(rng, 1, max(1, min(18848, most)))
        case["bias"] = rng.random() < 0.6
        case["activation"] = rng.choice([None, None, "relu", "gelu", "gelu_tanh", "silu"])
        case["residual"] = rng.random() < 0.5
        return case
    heads = case["heads"] = rng.choice([1, 2, 3, 4, 8, 12, 16, 32])
    shared = [h for h in (1, 2, 4, heads, heads, heads) if heads % h == 0]
    case["q_heads"] = rng.choice([heads, heads, rng.choice(shared)])
    case["k_heads"], case["v_heads"] = rng.choice(shared), rng.choice(shared)
    case["keys"] = _sized(rng, 16, 128)
    case["values"] = _sized(rng, 16, 256)
    case["each_token"] = rng.random() < 0.5
    cells = heads * case["keys"] * case["values"]
    if op == "attention_step":
        case["sequences"] = _spread(rng, 1, max(1, min(256, 256 * 16 * 128 * 128 // cells)))
    else:
        most = 4 * 16384 * 16 * 128 * 128 // 4 // cells // (1 if case["dtype"] != "f32" else 2)
        case["tokens"] = _spread(rng, 1, max(1, min(most, 32768)))
        case["sequences"] = _spread(rng, 1, min(64, case["tokens"]))
        case["ragged"] = rng.random() < 0.6
        if not case["ragged"]:
            case["tokens"] = max(1, case["tokens"] // case["sequences"]) * case["sequences"]
        case["resume"] = rng.random() < 0.5
    case["pool"] = case["sequences"] + rng.randrange(0, 16)
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
    if op == "dense":
        st["x"] = normal(case["rows"], case["in"], dtype=dt)
        st["w"] = normal(case["out"], case["in"], scale=case["in"] ** -0.5, dtype=dt)
        st["bias"] = normal(case["out"], scale=0.1) if case["bias"] else None
        st["residual"] = normal(case["rows"], case["out"], dtype=dt) if case["residual"] else None
        return st
    step = op.endswith("step")
    s, heads, keys, values = case["sequences"], case["heads"], case["keys"], case["values"]
    tokens = s if step else case["tokens"]
    # queries, keys and values are columns of one projection's output
    wide = [case["q_heads"] * keys, case["k_heads"] * keys, case["v_heads"] * values]
    q, k, v = normal(tokens, sum(wide), dtype=dt).split(wide, 1)
    st["q"] = q.unflatten(1, (case["q_heads"], keys))
    st["k"] = k.unflatten(1, (case["k_heads"], keys))
    st["v"] = v.unflatten(1, (case["v_heads"], values))
    st["scale"] = keys ** -0.5
    if case["each_token"]:
        # step sizes between 0.001 and 0.1 times a rate of each head
        rate = 1.0 + 15.0 * uniform(heads)
        st["log_decay"] = -rate * torch.exp(math.log(1e-3) + uniform(tokens, heads) * math.log(100.0))
    else:
        # memories of 32 to 256 tokens
        st["log_decay"] = torch.log1p(-torch.exp2(-torch.linspace(5.0, 8.0, heads, device="cuda")))
    st["slots"] = torch.randperm(case["pool"], generator=g, device="cuda")[:s].int()
    st["state"] = normal(case["pool"], heads, keys, values)
    st["sequences"] = s
    st["resume"] = st["offsets"] = None
    if not step:
        st["bounds"] = _bounds(case, seed)
        if case["ragged"]:
            st["offsets"] = torch.tensor(st["bounds"], dtype=torch.int32, device="cuda")
        if case["resume"]:
            st["resume"] = (uniform(s) < 0.5).int()
    return st


# ---------------------------------------------------------------------------------------------
# One pass


def run(st):
    return RUN[st["op"]][own](st)


def _attention_own(st):
    from bidirectional_lstm_stack_gb300 import binding
    y = binding.lstm_linear_attention(st["q"], st["k"], st["v"], st["log_decay"], scale=st["scale"],
                                      sequences=st["sequences"], offsets=st["offsets"],
                                      state=st["state"], slots=st["slots"], resume=st["resume"])
    return {"y": y, "state": st["state"]}


def _attention_step_own(st):
    from bidirectional_lstm_stack_gb300 import binding
    y = binding.lstm_linear_attention_step(st["q"], st["k"], st["v"], st["log_decay"], st["state"],
                                           scale=st["scale"], slots=st["slots"])
    return {"y": y, "state": st["state"]}


def _dense_own(st):
    from bidirectional_lstm_stack_gb300 import binding
    return {"y": binding.lstm_dense(st["x"], st["w"], st["bias"], activation=st["case"]["activation"],
                                    residual=st["residual"])}


def _of_heads(t, heads):
    """[..., some heads, width] with each of them repeated for the heads that share it."""
    return t.repeat_interleave(heads // t.shape[-2], -2)


def _attention_plain(st):
    heads, dev = st["case"]["heads"], st["q"].device
    tokens, rows = st["q"].shape[0], st["slots"].long()
    bounds = torch.tensor(st["bounds"], device=dev)
    lengths = bounds[1:] - bounds[:-1]
    old = st["state"][rows]
    if st["resume"] is None:
        old = torch.zeros_like(old)
    else:
        old = torch.where((st["resume"] != 0)[:, None, None, None], old, torch.zeros_like(old))
    # every sequence in chunks of its own
    counts = (lengths + CHUNK - 1) // CHUNK
    last = torch.cumsum(counts, 0)
    chunks = sum(-(-(b - a) // CHUNK) for a, b in zip(st["bounds"], st["bounds"][1:]))
    seq = torch.searchsorted(last, torch.arange(chunks, device=dev), right=True)
    number = torch.arange(chunks, device=dev) - (last - counts)[seq]
    at = (bounds[seq] + number * CHUNK)[:, None] + torch.arange(CHUNK, device=dev)
    there = at < bounds[seq + 1][:, None]
    at = at.clamp(max=tokens - 1)
    gone = torch.zeros((), device=dev)
    q, k, v = (torch.where(there[..., None, None], _of_heads(st[n][at].float(), heads), gone)
               for n in ("q", "k", "v"))
    decay = st["log_decay"].double()
    decay = decay[at] if decay.dim() == 2 else decay.expand(chunks, CHUNK, heads)
    fall = torch.cumsum(torch.where(there[..., None], decay, gone.double()), 1)
    # within a chunk: every query with the keys up to its own
    q, k, v = q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2)
    fall = fall.transpose(1, 2)
    upto = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    between = torch.where(upto, fall[..., :, None] - fall[..., None, :], -math.inf)
    y = ((q @ k.transpose(-1, -2)) * torch.exp(between).float()) @ v
    # what a chunk adds to the state and what it leaves of the one before, joined in spans of
    # twice the length each turn
    add = (k * torch.exp(fall[..., -1:] - fall).float()[..., None]).transpose(-1, -2) @ v
    left = torch.exp(fall[..., -1])[..., None, None].float()
    first = (number == 0).nonzero()[:, 0]
    add[first] += left[first] * old[seq[first]]
    left[first] = 0.0
    reach, longest = 1, max(-(-(b - a) // CHUNK) for a, b in zip(st["bounds"], st["bounds"][1:]))
    while reach < longest:
        more = torch.zeros_like(add)
        more[reach:] = left[reach:] * add[:-reach]
        joined = torch.zeros_like(left)
        joined[reach:] = left[reach:] * left[:-reach]
        add, left = add + more, joined
        reach *= 2
    before = torch.roll(add, 1, 0)
    before[first] = old[seq[first]]
    y = y + (q @ before) * torch.exp(fall).float()[..., None]
    out = torch.zeros(tokens, heads, v.shape[-1], device=dev)
    out[at[there]] = y.transpose(1, 2)[there] * st["scale"]
    st["state"][rows] = torch.where((counts == 0)[:, None, None, None], old,
                                    add[(last - 1).clamp(min=0)])
    return {"y": out.to(st["q"].dtype), "state": st["state"]}


def _attention_step_plain(st):
    heads, rows = st["case"]["heads"], st["slots"].long()
    q, k, v = (_of_heads(st[n].float(), heads) for n in ("q", "k", "v"))
    left = torch.exp(st["log_decay"])
    s = st["state"][rows] * left[..., None, None] + k[..., :, None] * v[..., None, :]
    y = (q[..., :, None] * s).sum(-2) * st["scale"]
    st["state"][rows] = s
    return {"y": y.to(st["q"].dtype), "state": st["state"]}


def _dense_plain(st):
    y = st["x"].float() @ st["w"].float().t()
    if st["bias"] is not None:
        y = y + st["bias"]
    kind = st["case"]["activation"]
    if kind == "relu":
        y = y.clamp(min=0.0)
    elif kind == "silu":
        y = y * torch.sigmoid(y)
    elif kind == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    elif kind == "gelu_tanh":
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return {"y": y.to(st["x"].dtype)}


RUN = {
    "attention": (_attention_plain, _attention_own),
    "attention_step": (_attention_step_plain, _attention_step_own),
    "dense": (_dense_plain, _dense_own),
}


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    for key, v in st.items():
        if torch.is_tensor(v) and v.is_floating_point():
            st[key] = v.double()
    if case["op"] == "dense":
        if case["rows"] * case["in"] * case["out"] > 1 << 42:
            return None
        y = torch.einsum("rk,nk->rn", st["x"], st["w"])
        if case["bias"]:
            y += st["bias"]
        gate = {None: lambda t: torch.ones_like(t), "relu": lambda t: (t > 0).double(),
                "silu": lambda t: 1 / (1 + torch.exp(-t)),
                "gelu": lambda t: torch.special.ndtr(t),
                # (1 + tanh z) / 2 is the logistic function of 2 z
                "gelu_tanh": lambda t: 1 / (1 + torch.exp(-2 * math.sqrt(2 / math.pi)
                                                          * (t + 0.044715 * t ** 3)))}
        y = y * gate[case["activation"]](y)
        return {"y": y + st["residual"] if case["residual"] else y}
    return _attention_exact(case, st)


def _attention_exact(case, st):
    heads, s = case["heads"], case["sequences"]
    step = case["op"].endswith("step")
    bounds = list(range(s + 1)) if step else st["bounds"]
    goes_on = [step] * s if st["resume"] is None else st["resume"].bool().tolist()
    spans = [(n, a, b) for n, (a, b) in enumerate(zip(bounds, bounds[1:]))]
    # all sequences side by side, the longest first, one token of each at a time
    spans.sort(key=lambda p: p[1] - p[2])
    lengths = [b - a for _, a, b in spans]
    if lengths[0] * s * heads * case["keys"] * case["values"] > 1 << 36 or lengths[0] > 1 << 16:
        return None
    slots = st["slots"].long()[[p[0] for p in spans]]
    h = st["state"][slots] * torch.tensor([float(goes_on[p[0]]) for p in spans],
                                          device="cuda")[:, None, None, None]
    starts = torch.tensor([p[1] for p in spans], device="cuda")
    of = {n: torch.arange(heads, device="cuda") // (heads // case[n + "_heads"]) for n in "qkv"}
    left = torch.exp(st["log_decay"])
    y = torch.zeros(st["q"].shape[0], heads, case["values"], dtype=torch.float64, device="cuda")
    live = len(spans)
    for t in range(lengths[0]):
        while lengths[live - 1] <= t:
            live -= 1
        at = starts[:live] + t
        now = left[at] if left.dim() == 2 else left
        h[:live] *= now[..., None, None]
        h[:live] += st["k"][at][:, of["k"], :, None] * st["v"][at][:, of["v"], None, :]
        y[at] = torch.einsum("shk,shkv->shv", st["q"][at][:, of["q"]], h[:live])
    st["state"][slots] = h
    return {"y": y * st["scale"], "state": st["state"]}


# ---------------------------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    op, size = case["op"], BYTES[case["dtype"]]
    if op == "dense":
        rows, k, n = case["rows"], case["in"], case["out"]
        moved = size * (rows * k + n * k + rows * n * (2 if case["residual"] else 1))
        return {"bytes": moved + (4 * n if case["bias"] else 0), "flops": 2 * rows * k * n}
    s, heads, keys, values = case["sequences"], case["heads"], case["keys"], case["values"]
    step = op.endswith("step")
    tokens = s if step else case["tokens"]
    reads = s if step else s // 2 if case["resume"] else 0
    width = (case["q_heads"] + case["k_heads"]) * keys + (case["v_heads"] + heads) * values
    moved = tokens * width * size + (reads + s) * heads * keys * values * 4
    moved += 4 * heads * (tokens if case["each_token"] else 1)
    # per cell of the state: the decay, the product of key and value, the query's
    return {"bytes": moved, "flops": tokens * heads * keys * values * 5}
