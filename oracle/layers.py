"""Float64 definitions of linear attention and the dense product, written as
sequential numpy loops (tests only), with bounds of what the kernels' arithmetic
may lose.

Attention: `size` carries the sum of the terms' absolute values through the same
recurrence as the state; a term's relative error times it bounds the state's
error.  A term k v e^c is off by its weight's rounding to three parts of bf16 (24 bits) and
its product's smallest parts, by the exponential, and by sums: at most 64
terms of a span are summed in fp32 before they join the state, once a span.  An
output also takes the state or q.k rounded to two (16-bit types) or three
(fp32) parts of bf16.
"""
import math

import numpy as np

from .ops import U32, slot_of

PARTS = {"bf16": 2.0 ** -15, "f16": 2.0 ** -15, "f32": 2.0 ** -22}
WEIGHT = 2.0 ** -22
SUMS = 400  # roundings or truncations of a span's sums and of the exponential


def linear_attention(q, k, v, log_decay, scale, spans_, dtype, state=None, slots=None, resume=None,
                     step=False):
    """(y, new state, bound of y's error before its rounding, bound of the state's);
    q [tokens, q_heads, keys] and so on, float64."""
    heads = log_decay.shape[-1]
    of = [np.arange(heads) // (heads // m.shape[1]) for m in (q, k, v)]
    y = np.zeros((q.shape[0], heads, v.shape[2]))
    y_bound = np.zeros_like(y)
    new = None if state is None else state.copy()
    new_bound = None if state is None else np.zeros_like(state)
    with np.errstate(invalid="ignore", over="ignore"):
        for n, (a, b) in enumerate(spans_):
            slot = slot_of(n, state, slots)
            goes_on = slot is not None and (step or (resume is not None and resume[n] != 0))
            s = state[slot].copy() if goes_on else np.zeros((heads, q.shape[2], v.shape[2]))
            size = np.abs(s)
            for t in range(a, b):
                left = np.exp(log_decay[t] if log_decay.ndim == 2 else log_decay)[:, None, None]
                add = k[t, of[1], :, None] * v[t, of[2], None, :]
                s = left * s + add
                size = left * size + np.abs(add)
                sums = (SUMS + 8 * ((t - a) // 64 + 1)) * U32
                term = sums if step else WEIGHT + sums
                mine = q[t, of[0]]
                y[t] = scale * np.einsum("hk,hkv->hv", mine, s)
                y_bound[t] = (abs(scale) * (term + (0 if step else PARTS[dtype]) + 2 * sums)
                              * np.einsum("hk,hkv->hv", np.abs(mine), size))
            if slot is not None:
                new[slot] = s
                if b > a:
                    new_bound[slot] = term * size
    return y, new, y_bound, new_bound


def _erf(v):
    return np.vectorize(math.erf)(v)


def activate(kind, v):
    with np.errstate(over="ignore"):
        if kind == "relu":
            return np.maximum(v, 0.0)
        if kind == "gelu":
            return 0.5 * v * (1.0 + _erf(v / math.sqrt(2.0)))
        if kind == "gelu_tanh":
            return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
        if kind == "silu":
            return v / (1.0 + np.exp(-v))
    return v


def dense(x, w, bias, activation, residual):
    """(y, bound of its error before the last rounding)."""
    v = x @ w.T
    size = np.abs(x) @ np.abs(w).T
    if bias is not None:
        v, size = v + bias, size + np.abs(bias)
    # products keep 22 bits at least; every sum is off by an ulp (2 U32) of a partial sum
    off = (2.0 ** -22 + (2 * x.shape[1] + 16) * U32) * size
    y = activate(activation, v)
    # the activations' slopes are below 1.13; their factor of v is off by a few ulps of 1
    bound = 1.13 * off + (32 * U32 * np.abs(v) if activation not in (None, "relu") else 0.0)
    if residual is not None:
        y = y + residual
        bound = bound + U32 * np.abs(y)
    return y, bound
