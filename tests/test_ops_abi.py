"""include/lstm_ops.h without a GPU: every declared symbol is exported and
bound, and bad arguments are refused before CUDA is touched."""
import os
import re

import pytest

from bidirectional_lstm_stack_gb300 import binding
from bidirectional_lstm_stack_gb300 import build as build_mod

HEADER = os.path.join(build_mod.INCLUDE, "lstm_ops.h")
INVALID, LENGTH = binding.LSTM_E_INVALID, binding.LSTM_E_LENGTH


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return binding.load()


def test_every_declared_symbol_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(lstm_[a-z0-9_]+)\s*\(", text))
    assert names == {"lstm_causal_conv", "lstm_causal_conv_step", "lstm_selective_scan",
                     "lstm_selective_scan_step", "lstm_selective_scan_workspace", "lstm_residual_rms_norm", "lstm_token_logprobs",
                     "lstm_test_scan_step_timeout"}
    for n in names:
        assert hasattr(lib, n)
        assert n.startswith("lstm_test_") or callable(getattr(binding, n))


def _conv(lib, x=64, x_stride=16, dtype=0, tokens=4, channels=16, width=4, w=64, sequences=1,
          offsets=None, state=None, state_slots=0, y=64, y_stride=16):
    return lib.lstm_causal_conv(x, x_stride, dtype, tokens, channels, width, w, None, 1, sequences,
                                offsets, state, state_slots, None, None, y, y_stride, None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(y=None), dict(w=None), dict(dtype=3), dict(dtype=-1), dict(tokens=-1),
    dict(sequences=-1), dict(sequences=0), dict(channels=0), dict(width=1), dict(width=5),
    dict(x_stride=15), dict(y_stride=0), dict(x=66), dict(state=64, state_slots=-1),
    dict(state=66, state_slots=1)])
def test_conv_refuses(lib, bad):
    assert _conv(lib, **bad) == INVALID
    assert "lstm_causal_conv" in binding.lstm_stack_last_error()


def test_prompts_of_equal_length_divide_the_tokens(lib):
    assert _conv(lib, tokens=5, sequences=2) == LENGTH
    assert "5 tokens" in binding.lstm_stack_last_error()


def _scan(lib, u=64, dt=64, a=64, b=64, c=64, z=None, z_stride=0, b_stride=8, u_stride=16, dtype=0,
          tokens=4, channels=16, states=8, groups=1, sequences=1, state=None, slots=0, y=64):
    return lib.lstm_selective_scan(u, u_stride, dt, 16, a, b, b_stride, c, 8, None, z, z_stride,
                                   None, 1, dtype, tokens, channels, states, groups, sequences,
                                   None, state, slots, None, None, y, 16, None, 0, None)


@pytest.mark.parametrize("bad", [
    dict(u=None), dict(dt=None), dict(a=None), dict(b=None), dict(c=None), dict(y=None),
    dict(dtype=3), dict(tokens=-1), dict(channels=0), dict(states=0), dict(states=129),
    dict(groups=0), dict(groups=3), dict(groups=2), dict(u_stride=8), dict(b_stride=7),
    dict(z=64, z_stride=3), dict(u=65), dict(sequences=-2), dict(state=64, slots=-1)])
def test_scan_refuses(lib, bad):
    assert _scan(lib, **bad) == INVALID
    assert "lstm_selective_scan" in binding.lstm_stack_last_error()


def test_steps_need_a_state(lib):
    assert lib.lstm_causal_conv_step(64, 16, 0, 1, 16, 4, 64, None, 1, None, 0, None, 64, 16,
                                     None) == INVALID
    assert lib.lstm_selective_scan_step(64, 16, 64, 16, 64, 64, 8, 64, 8, None, None, 0, None, 1, 0,
                                        1, 16, 8, 1, None, 0, None, 64, 16, None) == INVALID
    assert "state is null" in binding.lstm_stack_last_error()


def _norm(lib, x=64, res=None, dtype=0, weight=64, eps=1e-6, rows=2, cols=16, out=None, y=64,
          y_dtype=0, scales=None, group=0, stride=16):
    return lib.lstm_residual_rms_norm(x, stride, res, 16, dtype, weight, eps, rows, cols, out, 16, y,
                                      16, y_dtype, scales, group, None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(y=None), dict(weight=None), dict(dtype=3), dict(y_dtype=1), dict(rows=-1),
    dict(cols=0), dict(cols=32769), dict(eps=-1.0), dict(res=64), dict(out=64), dict(stride=4),
    dict(y_dtype=3), dict(y_dtype=3, scales=64, group=16), dict(y_dtype=3, scales=66)])
def test_norm_refuses(lib, bad):
    assert _norm(lib, **bad) == INVALID
    assert "lstm_residual_rms_norm" in binding.lstm_stack_last_error()


def test_norm_of_no_rows(lib):
    assert _norm(lib, x=None, y=None, rows=0) == binding.LSTM_OK


def _logprobs(lib, logits=64, stride=100, dtype=0, rows=2, vocab=100, tokens=None, logp=None, top=0,
              top_logp=None, top_ids=None):
    return lib.lstm_token_logprobs(logits, stride, dtype, rows, vocab, tokens, logp, None, top,
                                   top_logp, top_ids, None)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(dtype=3), dict(rows=-1), dict(vocab=0), dict(stride=99), dict(top=-1),
    dict(top=33), dict(vocab=5, top=6), dict(top=1), dict(top=1, top_logp=64), dict(tokens=64),
    dict(logp=64), dict(logits=66)])
def test_logprobs_refuses(lib, bad):
    assert _logprobs(lib, **bad) == INVALID
    assert "lstm_token_logprobs" in binding.lstm_stack_last_error()


def test_logprobs_sizes(lib):
    assert _logprobs(lib, vocab=(1 << 30) + 1, stride=1 << 31) == binding.LSTM_E_OVERFLOW
    assert _logprobs(lib, logits=None, rows=0) == binding.LSTM_OK


def test_very_many_tokens(lib):
    assert _conv(lib, tokens=0x7fffffff) == binding.LSTM_E_OVERFLOW
    assert _scan(lib, tokens=0x7fffffff) == binding.LSTM_E_OVERFLOW


def _conv_step(lib, sequences):
    return lib.lstm_causal_conv_step(64, 16, 0, sequences, 16, 4, 64, None, 1, 64, 8, None, 64, 16,
                                     None)


def _scan_step(lib, sequences):
    return lib.lstm_selective_scan_step(64, 16, 64, 16, 64, 64, 8, 64, 8, None, None, 0, None, 1, 0,
                                        sequences, 16, 8, 1, 64, 8, None, 64, 16, None)


MOST = 1 << 30


@pytest.mark.parametrize("call", [
    lambda lib, n: _conv(lib, tokens=n, sequences=n),
    lambda lib, n: _conv(lib, tokens=4, sequences=n, offsets=64),
    lambda lib, n: _scan(lib, tokens=n, sequences=n), _conv_step, _scan_step],
    ids=["conv", "conv with offsets", "scan", "conv step", "scan step"])
def test_very_many_sequences(lib, call):
    """Sequence numbers are added up and stepped over in 32 bits: beyond 2^30 the search for a
    tile's sequence would go negative and not end, next to 2^31 a step's rows would."""
    for n in (MOST + 1, 0x7fffffff):
        assert call(lib, n) == binding.LSTM_E_OVERFLOW
        assert f"{n} sequences" in binding.lstm_stack_last_error()
    assert call(lib, MOST) != binding.LSTM_E_OVERFLOW  # (made-up pointers: refused for those)
    assert call(lib, -1) == INVALID


def test_workspace_of_sizes_that_are_refused(lib):
    assert binding.lstm_selective_scan_workspace(MOST + 1, 64, 16, 1, MOST + 1, False) == 0


@pytest.mark.parametrize("channels,groups,states", [
    (MOST + 1, 1, 8), (0x7fffffff, 1, 16), (MOST, MOST // 4, 8), (1 << 28, 1 << 28, 16)])
def test_very_wide_scans(lib, channels, groups, states):
    """Channels a block beyond the last, and places in a row of b, are counted in 32 bits."""
    big = 1 << 40
    prompt = lib.lstm_selective_scan(64, big, 64, big, 64, 64, big, 64, big, None, None, 0, None, 1, 0,
                                     4, channels, states, groups, 1, None, None, 0, None, None, 64,
                                     big, None, 0, None)
    assert prompt == binding.LSTM_E_OVERFLOW
    step = lib.lstm_selective_scan_step(64, big, 64, big, 64, 64, big, 64, big, None, None, 0, None, 1,
                                        0, 4, channels, states, groups, 64, 8, None, 64, big, None)
    assert step == binding.LSTM_E_OVERFLOW
    assert f"{channels} channels" in binding.lstm_stack_last_error()


def test_timeout_hook_refuses_limits_above_two_seconds(lib):
    assert lib.lstm_test_scan_step_timeout(1, 2000001, 0) == INVALID
