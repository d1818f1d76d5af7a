"""include/lstm_layers.h without a GPU: every declared symbol is exported and
bound, and bad arguments are refused before CUDA is touched."""
import inspect
import os
import re

import pytest
import torch

from bidirectional_lstm_stack_gb300 import binding
from bidirectional_lstm_stack_gb300 import build as build_mod

HEADER = os.path.join(build_mod.INCLUDE, "lstm_layers.h")
INVALID, LENGTH, OVERFLOW = (binding.LSTM_E_INVALID, binding.LSTM_E_LENGTH,
                             binding.LSTM_E_OVERFLOW)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return binding.load()


def test_every_declared_symbol_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(lstm_[a-z0-9_]+)\s*\(", text))
    assert {"lstm_linear_attention", "lstm_linear_attention_step", "lstm_dense"} <= names
    for n in names:
        assert hasattr(lib, n)
        assert n.startswith("lstm_test_") or callable(getattr(binding, n))


def _attention(lib, step=False, q=64, q_stride=64, q_head=16, q_heads=4, k=64, k_stride=64, k_head=16,
               k_heads=4, v=64, v_stride=32, v_head=8, v_heads=4, decay=64, decay_stride=0, dtype=0,
               tokens=4, heads=4, keys=16, values=8, sequences=1, state=None, slots=0, y=64, y_stride=32):
    a = (q, q_stride, q_head, q_heads, k, k_stride, k_head, k_heads, v, v_stride, v_head, v_heads, decay,
         decay_stride, 1.0, dtype)
    if step:
        return lib.lstm_linear_attention_step(*a, tokens, heads, keys, values, state, slots, None, y,
                                              y_stride, None)
    return lib.lstm_linear_attention(*a, tokens, heads, keys, values, sequences, None, state, slots, None,
                                     None, y, y_stride, None, 0, None)


BAD = [dict(q=None), dict(k=None), dict(v=None), dict(y=None), dict(decay=None), dict(dtype=3),
       dict(dtype=-1), dict(tokens=-1), dict(heads=0), dict(heads=40000), dict(keys=0),
       dict(keys=129), dict(values=0), dict(values=257), dict(q_heads=3), dict(k_heads=0), dict(v_heads=8),
       dict(q_stride=15), dict(k_stride=0), dict(v_stride=7), dict(y_stride=31), dict(q_head=15),
       dict(k_head=0), dict(v_head=-8), dict(decay_stride=3), dict(q=66), dict(k=65), dict(v=63), dict(y=66),
       dict(decay=66), dict(state=66, slots=4), dict(state=64, slots=-1)]


@pytest.mark.parametrize("bad", BAD + [dict(sequences=0), dict(sequences=-1)])
def test_attention_refuses(lib, bad):
    assert _attention(lib, **bad) == INVALID
    assert "lstm_linear_attention" in binding.lstm_stack_last_error()


@pytest.mark.parametrize("bad", BAD + [dict(state=None)])
def test_attention_step_refuses(lib, bad):
    assert _attention(lib, step=True, **{"state": 64, "slots": 4, **bad}) == INVALID
    assert "lstm_linear_attention_step" in binding.lstm_stack_last_error()


def test_attention_lengths(lib):
    assert _attention(lib, tokens=5, sequences=2) == LENGTH
    assert _attention(lib, tokens=0x7fffff80) == OVERFLOW
    assert _attention(lib, step=True, tokens=(1 << 30) + 1, state=64, slots=4) == OVERFLOW


def _dense(lib, x=64, x_stride=16, w=64, w_stride=16, bias=None, activation=0, residual=None,
           residual_stride=0, dtype=0, rows=4, n_in=16, n_out=8, y=64, y_stride=8):
    return lib.lstm_dense(x, x_stride, w, w_stride, bias, activation, residual, residual_stride, dtype,
                          rows, n_in, n_out, y, y_stride, None, 0, None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(w=None), dict(y=None), dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(n_in=0),
    dict(n_out=0), dict(activation=5), dict(activation=-1), dict(x_stride=15), dict(w_stride=15),
    dict(y_stride=7), dict(x=66), dict(w=66), dict(y=66), dict(bias=66),
    dict(residual=64, residual_stride=7), dict(residual=66, residual_stride=8)])
def test_dense_refuses(lib, bad):
    assert _dense(lib, **bad) == INVALID
    assert "lstm_dense" in binding.lstm_stack_last_error()


def test_dense_overflow(lib):
    for size in ("rows", "n_in", "n_out"):
        assert _dense(lib, **{size: (1 << 29) + 1}) == OVERFLOW


def test_sizes_that_are_refused_need_no_workspace(lib):
    assert lib.lstm_dense_workspace(64, 16, 64, 16, 0, 1 << 29, 16, 8) > 0
    for sizes in (((1 << 29) + 1, 16, 8), (4, (1 << 29) + 1, 8), (4, 16, (1 << 29) + 1), (4, 0, 8), (4, 16, -1),
                  (-4, 16, 8)):
        assert lib.lstm_dense_workspace(64, 16, 64, 16, 0, *sizes) == 0
    most = 0x7fffff00
    assert binding.lstm_linear_attention_workspace(most, 1, 64, 64, 1, True) > 0
    for sizes in ((most + 1, 1, 64, 64, 1), (1 << 20, 0, 64, 64, 1), (1 << 20, 1, 129, 64, 1),
                  (1 << 20, 1, 64, 257, 1), (1 << 20, 1, 64, 64, -1), (-5, 1, 64, 64, 1)):
        assert binding.lstm_linear_attention_workspace(*sizes, True) == 0


# ---- the binding ---------------------------------------------------------------------------------
def _calls(m):
    z = torch.zeros
    return [lambda: binding.lstm_linear_attention(m, m, m, z(2)),
            lambda: binding.lstm_linear_attention_step(m, m, m, z(2), z(4, 2, 8, 8)),
            lambda: binding.lstm_dense(m, z(8, 8))]


@pytest.mark.parametrize("function", range(3))
@pytest.mark.parametrize("bad,error", [(torch.zeros(4, 2, 8), ValueError), (torch.zeros(2, 8), ValueError),
                                       (torch.zeros(8), ValueError), (torch.zeros(()), ValueError),
                                       (None, TypeError), ([[0.0]], TypeError)])
def test_host_tensors_and_others_are_refused(function, bad, error):
    with pytest.raises(error):
        _calls(bad)[function]()


@pytest.mark.parametrize("function", range(3))
def test_tensors_that_require_a_gradient_are_refused(function):
    m = torch.zeros(*((4, 2, 8) if function < 2 else (4, 8)), requires_grad=True)
    with pytest.raises(ValueError, match="requires a gradient"):
        _calls(m)[function]()
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):
        _calls(m)[function]()


def test_names_and_defaults():
    for name in ("lstm_linear_attention", "lstm_linear_attention_step", "lstm_dense"):
        f = getattr(binding, name)
        assert "stream" in inspect.signature(f).parameters and f.__doc__
        with pytest.raises(TypeError):
            f()


def test_an_unknown_activation_is_refused():
    with pytest.raises(ValueError, match="swish"):
        binding.lstm_dense(torch.zeros(2, 2), torch.zeros(2, 2), activation="swish")


@pytest.mark.gpu
def test_arguments_that_are_wrong_beside_good_ones():
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)
    q, k, v, d = z(6, 4, 16), z(6, 2, 16), z(6, 4, 8), z(4)
    att, step, dense = (binding.lstm_linear_attention, binding.lstm_linear_attention_step,
                        binding.lstm_dense)
    state = z(6, 4, 16, 8)
    x, w = z(6, 16), z(8, 16)
    for call, error in [(lambda: att(q, k[:5], v, d), ValueError), (lambda: att(q, z(6, 2, 8), v, d), ValueError),
                        (lambda: att(q, k, v.half(), d), ValueError), (lambda: att(q, k, v.cpu(), d), ValueError),
                        (lambda: att(q, k, v, d.half()), ValueError), (lambda: att(q, k, v, z(5, 4)), ValueError),
                        (lambda: att(q, k, v, z(3)), binding.LSTMError), (lambda: att(q, k, v, None), TypeError),
                        (lambda: att(q, k, v, z(6, 4, 1)), ValueError),
                        (lambda: att(q, k, v, d, scale=None), TypeError),
                        (lambda: att(q, k, v, d, scale="1"), TypeError),
                        (lambda: att(q, k, v, d, state=z(4, 16, 8)), ValueError),
                        (lambda: att(q, k, v, d, state=state.half()), ValueError),
                        (lambda: att(q, k, v, d, slots=z(1, dtype=torch.int32)), ValueError),
                        (lambda: att(q, k, v, d, y=z(6, 4, 16)), ValueError),
                        (lambda: att(q, k, v, d, y=z(4, 6, 8).transpose(0, 1)), ValueError),
                        (lambda: att(z(6, 16, 4).transpose(1, 2), k, v, d), ValueError),
                        (lambda: att(q, k, v, d, sequences=4), binding.LSTMError),
                        (lambda: step(q, k, v, d, None), binding.LSTMError),
                        (lambda: step(q, k, v, d, state[:5]), ValueError),
                        (lambda: step(q, k, v, d, state.transpose(2, 3)), ValueError),
                        (lambda: dense(x, w[:, :8]), ValueError), (lambda: dense(x, w.half()), ValueError),
                        (lambda: dense(x, None), TypeError), (lambda: dense(x, w, z(7)), ValueError),
                        (lambda: dense(x, w, z(8).half()), ValueError),
                        (lambda: dense(x, w, residual=z(6, 16)), ValueError),
                        (lambda: dense(x, w, y=z(6, 8).half()), ValueError),
                        (lambda: dense(x, z(16, 8).t()), ValueError), (lambda: dense(x.double(), w), ValueError)]:
        with pytest.raises(error):
            call()
    att(q, k, v, d, state=state)
    step(q, k, v, d, state)
    dense(x, w)
