"""The short causal convolution over packed prompts and over single tokens
against its float64 definition: types, widths, channel counts with and without
16-byte rows, lengths from zero on, states and slots, and refusals."""
import numpy as np
import pytest
import torch

from bidirectional_lstm_stack_gb300 import binding
from oracle import ops as oracle
from ops_util import DTYPES, assert_close, at_element, f64, gen, normal, slice_of

pytestmark = pytest.mark.gpu


def _check(dtype, channels, width, lengths, *, bias=True, act=True, slots=None, pool=None,
           resume=None, strided=False, uniform=False, seed=1):
    g = gen(seed)
    tokens, sequences = sum(lengths), len(lengths)
    x = normal(g, tokens, channels, dtype=DTYPES[dtype])
    if strided:
        x = slice_of(x, 3, 2)
    w = normal(g, channels, width, scale=0.5)
    b = normal(g, channels, scale=0.3) if bias else None
    state = None if pool is None else normal(g, pool, width - 1, channels, dtype=DTYPES[dtype])
    offsets = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    dev = lambda a: None if a is None else torch.tensor(a, dtype=torch.int32, device="cuda")
    before = f64(state)
    y = binding.lstm_causal_conv(x, w, b, silu=act, sequences=sequences,
                                 offsets=None if uniform else dev(offsets), state=state,
                                 slots=dev(slots), resume=dev(resume))
    ref, new, bound = oracle.causal_conv(f64(x), f64(w), f64(b), act,
                                         oracle.spans(tokens, sequences, offsets), before, slots,
                                         resume)
    assert_close(y, ref, bound, dtype, "y")
    if state is not None:
        np.testing.assert_array_equal(f64(state), new)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("channels", [1, 7, 8, 60, 256, 1029, 2048])
def test_one_prompt(dtype, channels):
    _check(dtype, channels, 4, [37])


@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("length", [0, 1, 2, 3, 15, 16, 17, 33, 257])
def test_lengths_and_widths_with_state(width, length):
    _check("bf16", 64, width, [length], pool=1, resume=[1])
    _check("f32", 33, width, [length], pool=1, resume=[0])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("channels", [24, 25])
def test_packed_prompts(dtype, channels):
    lengths = [5, 0, 1, 16, 40, 2, 0, 3, 100, 31]
    _check(dtype, channels, 4, lengths, pool=12, slots=[3, 0, 11, 7, 5, 1, 2, 9, 8, 10],
           resume=[1, 1, 1, 0, 1, 0, 0, 1, 1, 0])


def test_slots_outside_the_pool_have_no_state():
    _check("bf16", 40, 4, [5, 6, 7], pool=3, slots=[-1, 1, 3], resume=[1, 1, 1])


def test_equal_lengths_without_offsets():
    _check("f16", 256, 3, [21] * 6, uniform=True, pool=6, resume=[0, 1, 0, 1, 1, 1])


def test_rows_of_wider_matrices():
    _check("bf16", 64, 4, [19, 30], strided=True, pool=2, resume=[1, 1])


def test_without_bias_and_activation():
    _check("f32", 16, 4, [50], bias=False, act=False)


def test_wide_range_of_values():
    g = gen(5)
    x = normal(g, 64, 32, scale=100.0)
    w = normal(g, 32, 4, scale=3.0)
    y = binding.lstm_causal_conv(x, w)
    ref, _, bound = oracle.causal_conv(f64(x), f64(w), None, True, [(0, 64)])
    # e^-v leaves fp32's range for v < -88: the quotient is 0 there, as
    # v / (1 + e^-v) is below 1e-36
    assert_close(y, ref, bound + 1e-36, "f32")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("channels,width", [(1, 4), (15, 2), (64, 3), (2048, 4)])
@pytest.mark.parametrize("sequences", [1, 5])
def test_step(dtype, channels, width, sequences):
    g = gen(3)
    x = normal(g, sequences, channels, dtype=DTYPES[dtype])
    w, b = normal(g, channels, width), normal(g, channels)
    state = normal(g, 7, width - 1, channels, dtype=DTYPES[dtype])
    slots = [6, -1, 2, 7, 0][:sequences]
    before = f64(state)
    y = binding.lstm_causal_conv_step(x, w, b, state,
                                      slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    ref, new, bound = oracle.causal_conv(f64(x), f64(w), f64(b), True,
                                         [(s, s + 1) for s in range(sequences)], before, slots,
                                         step=True)
    assert_close(y, ref, bound, dtype)
    np.testing.assert_array_equal(f64(state), new)


def test_prompt_then_steps_equal_one_prompt():
    g = gen(9)
    x = normal(g, 23, 48, dtype=torch.bfloat16)
    w, b = normal(g, 48, 4), normal(g, 48)
    whole = binding.lstm_causal_conv(x, w, b)
    state = torch.zeros(1, 3, 48, dtype=torch.bfloat16, device="cuda")
    parts = [binding.lstm_causal_conv(x[:2], w, b, state=state)]
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    parts.append(binding.lstm_causal_conv(x[2:20], w, b, state=state, resume=one))
    parts += [binding.lstm_causal_conv_step(x[t:t + 1], w, b, state) for t in range(20, 23)]
    assert torch.equal(torch.cat(parts), whole)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("channels", [60, 62, 63])
@pytest.mark.parametrize("offset", [0, 1, 2, 4])
@pytest.mark.parametrize("width", [2, 3, 4])
def test_rows_of_every_alignment(dtype, channels, offset, width):
    """Columns of a wider matrix as input and as output, tokens and steps."""
    g = gen(channels + offset)
    wide = normal(g, 45, 136, dtype=DTYPES[dtype])
    out = torch.zeros(45, 136, device="cuda", dtype=DTYPES[dtype])
    x, y = wide[:, offset:offset + channels], out[:, 68 + offset:68 + offset + channels]
    w, b = normal(g, channels, width, scale=0.5), normal(g, channels, scale=0.3)
    state = normal(g, 45, width - 1, channels, dtype=DTYPES[dtype])
    before = f64(state)
    binding.lstm_causal_conv(x, w, b, y=y, state=state, resume=torch.ones(1, dtype=torch.int32,
                                                                          device="cuda"))
    ref, new, bound = oracle.causal_conv(f64(x), f64(w), f64(b), True, [(0, 45)], before, None, [1])
    assert_close(y, ref, bound, dtype, "y")
    np.testing.assert_array_equal(f64(state), new)
    rest = out.clone()
    rest[:, 68 + offset:68 + offset + channels] = 0
    assert not rest.any()
    before = f64(state)
    binding.lstm_causal_conv_step(x, w, b, state, y=y)
    ref, new, bound = oracle.causal_conv(f64(x), f64(w), f64(b), True,
                                         [(i, i + 1) for i in range(45)], before, None, [1] * 45)
    assert_close(y, ref, bound, dtype, "y of the step")
    np.testing.assert_array_equal(f64(state), new)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("offset", [0, 1, 2, 3])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("channels", [64, 62, 63])
def test_weights_at_any_element(dtype, offset, width, channels):
    """Weights and bias that are views into a larger buffer of parameters."""
    g = gen(channels + offset)
    x = normal(g, 45, channels, dtype=DTYPES[dtype])
    w = at_element(normal(g, channels, width, scale=0.5), offset)
    b = at_element(normal(g, channels, scale=0.3), (offset + 1) % 4)
    assert w.data_ptr() % 16 == 4 * offset
    y = binding.lstm_causal_conv(x, w, b)
    ref, _, bound = oracle.causal_conv(f64(x), f64(w), f64(b), True, [(0, 45)])
    assert_close(y, ref, bound, dtype, "y")
    state = at_element(normal(g, 45, width - 1, channels, dtype=DTYPES[dtype]), offset)
    before = f64(state)
    y = binding.lstm_causal_conv_step(x, w, b, state)
    ref, new, bound = oracle.causal_conv(f64(x), f64(w), f64(b), True,
                                         [(i, i + 1) for i in range(45)], before, None, [1] * 45)
    assert_close(y, ref, bound, dtype, "y of the step")
    np.testing.assert_array_equal(f64(state), new)


# all lengths from nothing to several runs of 32 tokens, on both sides of multiples of 4, 12, 16 and 32
LENGTHS = [1, 0, 2, 3, 4, 5, 11, 12, 13, 15, 16, 17, 0, 31, 32, 33, 47, 48, 49, 63, 64, 65, 100]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("channels,tokens,width", [
    (4096, 2100, 4), (4094, 2100, 4), (4095, 1100, 4), (2048, 4100, 3),   # runs of 32 tokens
    (4096, 740, 4), (4094, 740, 4), (4095, 740, 4), (2048, 1100, 2)])     # runs of 16
def test_long_runs(dtype, channels, tokens, width):
    """From 2^19 vectors of channels on a thread works on 16 tokens, from 2^21 on 32, its rows
    on their way through a ring; with four, two and one channels a thread."""
    lengths = LENGTHS + [tokens - sum(LENGTHS)]
    n = len(lengths)
    assert lengths[-1] > 0
    _check(dtype, channels, width, lengths, pool=n + 2, slots=[(5 * k + 3) % (n + 2) for k in range(n)],
           resume=[k % 3 != 1 for k in range(n)])


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_long_runs_of_equal_prompts(dtype):
    _check(dtype, 4096, 4, [70] * 31, uniform=True, pool=31, resume=[k % 2 for k in range(31)])
    _check(dtype, 2048, 4, [1031], uniform=True, strided=True, act=False, bias=False)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("channels", [32, 30, 31])
@pytest.mark.parametrize("act", [False, True])
def test_infinities_and_nan_stay_where_the_definition_has_them(dtype, channels, act):
    g = gen(11)
    x = normal(g, 40, channels, dtype=DTYPES[dtype])
    x[7, 3], x[20, 4], x[39, 5], x[0, 29] = (float(v) for v in ("inf", "-inf", "nan", "inf"))
    w, state = normal(g, channels, 4), normal(g, 1, 3, channels, dtype=DTYPES[dtype])
    before = f64(state)
    y = binding.lstm_causal_conv(x, w, silu=act, state=state)
    with np.errstate(invalid="ignore"):
        ref, new, bound = oracle.causal_conv(f64(x), f64(w), None, act, [(0, 40)], before)
    np.testing.assert_array_equal(f64(state), new)
    odd = ~np.isfinite(ref)
    assert odd.any()
    np.testing.assert_array_equal(f64(y)[odd], ref[odd])
    assert_close(torch.where(torch.from_numpy(odd), torch.zeros(()), y.cpu().float()),
                 np.where(odd, 0.0, ref), np.where(odd, 0.0, bound), dtype)


def test_on_another_stream():
    g = gen(2)
    x, w = normal(g, 300, 128), normal(g, 128, 4)
    ref = binding.lstm_causal_conv(x, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        y = binding.lstm_causal_conv(x, w, stream=stream)
        s.synchronize()
        assert torch.equal(y, ref)


def test_refusals():
    x = torch.zeros(12, 16, device="cuda")
    w = torch.zeros(16, 4, device="cuda")
    state = torch.zeros(2, 3, 16, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")

    def code(fn):
        with pytest.raises(binding.LSTMError) as e:
            fn()
        return e.value.code

    assert code(lambda: binding.lstm_causal_conv(x, torch.zeros(16, 5, device="cuda"))) == binding.LSTM_E_INVALID
    assert code(lambda: binding.lstm_causal_conv(x, torch.zeros(16, 1, device="cuda"))) == binding.LSTM_E_INVALID
    assert code(lambda: binding.lstm_causal_conv(x, w, sequences=5)) == binding.LSTM_E_LENGTH
    for bad in (
            lambda: binding.lstm_causal_conv(x.double(), w),
            lambda: binding.lstm_causal_conv(x, w.half()),
            lambda: binding.lstm_causal_conv(x, w[:8]),
            lambda: binding.lstm_causal_conv(x, w.cpu()),
            lambda: binding.lstm_causal_conv(x.t(), torch.zeros(12, 4, device="cuda")),
            lambda: binding.lstm_causal_conv(x, w, y=torch.zeros(12, 15, device="cuda")),
            lambda: binding.lstm_causal_conv(x, w, y=torch.zeros(12, 16, device="cuda").half()),
            lambda: binding.lstm_causal_conv(x, w, state=state[:, :2]),
            lambda: binding.lstm_causal_conv(x, w, state=state.half()),
            lambda: binding.lstm_causal_conv(x, w, slots=i32(0)),
            lambda: binding.lstm_causal_conv(x, w, sequences=3, state=state),
            lambda: binding.lstm_causal_conv(x, w, offsets=i32(0, 12).long()),
            lambda: binding.lstm_causal_conv(x, w, offsets=i32(0, 12), sequences=2),
            lambda: binding.lstm_causal_conv_step(x, w, None, state)):
        with pytest.raises(ValueError):
            bad()


def test_offsets_outside_the_rows_are_clamped():
    g = gen(4)
    x, w = normal(g, 20, 16), normal(g, 16, 4)
    y = torch.full_like(x, float("nan"))
    binding.lstm_causal_conv(x, w, offsets=torch.tensor([-5, 8, 400], dtype=torch.int32, device="cuda"), y=y)
    ref, _, bound = oracle.causal_conv(f64(x), f64(w), None, True, [(0, 8), (8, 20)])
    assert_close(y, ref, bound, "f32")
