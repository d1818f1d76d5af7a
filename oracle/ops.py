"""Float64 definitions of the state-space layer's operators and of the token
log probabilities, written as sequential numpy loops (tests only).

The recurrences also return a bound of what fp32 arithmetic may lose on the
way: every product, sum and function value is off by a few units of 2^-24, and
the bound is carried through the same recurrence, so that it grows and decays
as the errors do.
"""
import numpy as np

U32 = 2.0 ** -24  # fp32's unit roundoff


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))


def spans(tokens, sequences, offsets):
    if offsets is None:
        n = tokens // sequences
        return [(s * n, (s + 1) * n) for s in range(sequences)]
    return [(int(offsets[s]), int(offsets[s + 1])) for s in range(sequences)]


def slot_of(s, state, slots):
    if state is None:
        return None
    k = s if slots is None else int(slots[s])
    return k if 0 <= k < len(state) else None


def causal_conv(x, w, bias, act, spans_, state=None, slots=None, resume=None, step=False):
    """(y, new state, bound of y's fp32 error); float64 arrays."""
    width = w.shape[1]
    y, bound = np.zeros_like(x), np.zeros_like(x)
    new = None if state is None else state.copy()
    for s, (a, b) in enumerate(spans_):
        k = slot_of(s, state, slots)
        goes_on = k is not None and (step or (resume is not None and resume[s] != 0))
        past = state[k] if goes_on else np.zeros((width - 1, x.shape[1]))
        line = np.concatenate([past, x[a:b]])
        v = np.zeros((b - a, x.shape[1])) if bias is None else np.tile(bias, (b - a, 1))
        size = np.abs(v)
        for j in range(width):
            v += line[j:j + b - a] * w[:, j]
            size += np.abs(line[j:j + b - a] * w[:, j])
        off = (width + 2) * U32 * size
        if act:
            # |silu'| < 1.1; e^-v is off by |v| ulps and a few more, the quotient by two
            y[a:b] = silu(v)
            bound[a:b] = 1.1 * off + np.abs(y[a:b]) * (8 + 2 * np.abs(v)) * U32
        else:
            y[a:b], bound[a:b] = v, off
        if k is not None:
            new[k] = line[len(line) - (width - 1):]
    return y, new, bound


def selective_scan(u, dt, a, b, c, skip, z, dt_bias, softplus, groups, spans_, state=None,
                   slots=None, resume=None, step=False):
    """(y, new state, bound of y's fp32 error, bound of the states')."""
    tokens, d = u.shape
    n = a.shape[1]
    of = np.arange(d) // (d // groups)
    b, c = b.reshape(tokens, groups, n), c.reshape(tokens, groups, n)
    y, bound = np.zeros_like(u), np.zeros_like(u)
    new = None if state is None else state.copy()
    new_bound = None if state is None else np.zeros_like(state)
    for s, (t0, t1) in enumerate(spans_):
        k = slot_of(s, state, slots)
        goes_on = k is not None and (step or (resume is not None and resume[s] != 0))
        h = state[k].copy() if goes_on else np.zeros((d, n))
        size, off = np.abs(h), np.zeros((d, n))
        for t in range(t0, t1):
            v = dt[t] + (0.0 if dt_bias is None else dt_bias)
            # the sum's rounding moves v by U32 |v|, and log(1 + e^v) by no more
            # relatively; its own evaluation adds a few ulps
            s_t = np.logaddexp(v, 0.0) if softplus else v
            s_off = (8 + 2 * np.abs(v)) * U32
            arg = s_t[:, None] * a
            decay = np.exp(arg)
            # the exponent's relative error is s's and three roundings', and
            # the exponential is good to a few ulps; twice that, as a state may
            # be carried over a span in one product of decays instead of many
            decay_off = 2 * (np.abs(arg) * (s_off[:, None] + 3 * U32) + 4 * U32)
            add = (s_t * u[t])[:, None] * b[t][of]
            off = decay * off + (decay_off + 2 * U32) * decay * size \
                + (s_off[:, None] + 4 * U32) * np.abs(add)
            h = decay * h + add
            size = decay * size + np.abs(add)
            ct = c[t][of]
            out = (h * ct).sum(1)
            o = (off * np.abs(ct)).sum(1) + (n + 2) * U32 * (size * np.abs(ct)).sum(1)
            if skip is not None:
                out = out + skip * u[t]
                o = o + 2 * U32 * (np.abs(skip * u[t]) + np.abs(out))
            if z is not None:
                g = silu(z[t])
                o = o * np.abs(g) + np.abs(out * g) * (8 + 2 * np.abs(z[t])) * U32
                out = out * g
            y[t], bound[t] = out, o
        if k is not None:
            new[k], new_bound[k] = h, off
    return y, new, bound, new_bound


def residual_rms_norm(x, residual, weight, eps):
    """(n, v): the norm and the sum it is taken of."""
    v = x if residual is None else x + residual
    return v / np.sqrt((v * v).mean(1, keepdims=True) + eps) * weight, v


def group_scales(n, group):
    """The e4m3 scale of every group of columns (0: of every row)."""
    group = group or n.shape[1]
    top = np.stack([np.abs(n[:, k:k + group]).max(1) for k in range(0, n.shape[1], group)], 1)
    return np.where(top > 0, np.maximum(top / 448.0, 2.0 ** -126), 1.0)


def token_logprobs(logits, tokens, top):
    """(logp, entropy, top ids, top logp, bound of logp's and entropy's fp32 error)."""
    rows, vocab = logits.shape
    out_logp, out_h = np.zeros(rows), np.zeros(rows)
    ids, ids_logp = np.zeros((rows, top), np.int64), np.zeros((rows, top))
    bound = np.zeros((rows, 2))
    for r in range(rows):
        x = logits[r]
        # stable, so equal logits (zeros of either sign among them) stay in
        # order; NaN first
        order = np.argsort(np.where(np.isnan(x), -np.inf, -x), kind="stable")
        first = order[np.isnan(x[order])]
        order = np.concatenate([first, order[~np.isnan(x[order])]])
        m = x.max()
        if np.isnan(m) or m == np.inf:
            l, h = np.full(vocab, np.nan), np.nan
        elif m == -np.inf:
            l, h = np.full(vocab, -np.inf), 0.0
        else:
            d = x - m
            p = np.exp(d)
            l = d - np.log(p.sum())
            p = p / p.sum()
            h = -(p[p > 0] * l[p > 0]).sum()
            # every term e^d is off by (|d| + 4) ulps; the sums run over at
            # most 64 terms a lane and some 20 joins
            spread = (p[p > 0] * -d[p > 0]).sum()
            bound[r, 0] = (spread + 128) * U32
            bound[r, 1] = bound[r, 0] + ((p[p > 0] * d[p > 0] ** 2).sum() + 128 * spread + 2 * abs(h)) * U32
        out_h[r] = h
        if tokens is not None:
            t = int(tokens[r])
            out_logp[r] = 0.0 if t < 0 else np.nan if t >= vocab else l[t]
        ids[r], ids_logp[r] = order[:top], l[order[:top]]
    return out_logp, out_h, ids, ids_logp, bound
