"""The selective scan over packed prompts and over single tokens against its
float64 definition: types, numbers of channels, states and groups, lengths from
zero to long ones, states and slots, strides, and refusals."""
import numpy as np
import pytest
import torch

from bidirectional_lstm_stack_gb300 import binding
from oracle import ops as oracle
from ops_util import DTYPES, assert_close, at_element, f64, gen, normal, slice_of, uniform

pytestmark = pytest.mark.gpu


def _i32(a):
    return None if a is None else torch.tensor(a, dtype=torch.int32, device="cuda")


def _inputs(dtype, tokens, channels, states, groups=1, strided=False, seed=1, scale=0.5):
    g = gen(seed)
    t = DTYPES[dtype]
    xz = normal(g, tokens, 2 * channels, dtype=t)
    dbc = normal(g, tokens, 3 + 2 * groups * states, dtype=t)
    v = {"u": xz[:, :channels], "z": xz[:, channels:],
         "dt": normal(g, tokens, channels, scale=scale, dtype=t),
         "b": dbc[:, 3:3 + groups * states], "c": dbc[:, 3 + groups * states:],
         "a": -torch.exp(normal(g, channels, states)), "skip": normal(g, channels),
         "dt_bias": normal(g, channels) - 2.0}
    if not strided:
        v = {k: t.contiguous() for k, t in v.items()}
    return v


def _check(dtype, lengths, channels, states=16, *, groups=1, pool=None, slots=None, resume=None,
           strided=False, uniform_=False, softplus=True, without=(), seed=1, y=None, scale=0.5):
    tokens, sequences = sum(lengths), len(lengths)
    v = _inputs(dtype, tokens, channels, states, groups, strided, seed, scale)
    for k in without:
        v[k] = None
    if not softplus:
        v["dt"], v["dt_bias"] = v["dt"].abs() * 0.2, None
    state = None if pool is None else normal(gen(seed + 1), pool, channels, states)
    before = f64(state)
    offsets = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    got = binding.lstm_selective_scan(
        v["u"], v["dt"], v["a"], v["b"], v["c"], skip=v["skip"], z=v["z"], dt_bias=v["dt_bias"],
        softplus=softplus, groups=groups, sequences=sequences,
        offsets=None if uniform_ else _i32(offsets), state=state, slots=_i32(slots),
        resume=_i32(resume), y=y)
    ref, new, bound, new_bound = oracle.selective_scan(
        f64(v["u"]), f64(v["dt"]), f64(v["a"]), f64(v["b"]), f64(v["c"]), f64(v["skip"]),
        f64(v["z"]), f64(v["dt_bias"]), softplus, groups, oracle.spans(tokens, sequences, offsets),
        before, slots, resume)
    assert_close(got, ref, bound, dtype, "y")
    if state is not None:
        assert_close(state, new, new_bound, "f32", "state")
        return state


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("channels", [1, 5, 32, 64, 130, 256])
def test_one_prompt(dtype, channels):
    _check(dtype, [41], channels)


@pytest.mark.parametrize("states", [1, 3, 4, 8, 13, 16, 17, 32, 33, 64, 65, 100, 128])
def test_numbers_of_states(states):
    _check("bf16", [30], 40, states, pool=1, resume=[1])
    _check("f32", [9, 11], 6, states, pool=2, resume=[1, 0])


@pytest.mark.parametrize("length", [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300])
def test_lengths(length):
    _check("bf16", [length], 64, pool=1, resume=[1])
    _check("f32", [length], 33, pool=1, resume=[0])


def test_only_empty_prompts():
    # states that are not gone on from become zeros, the others stay
    n = 400
    state = normal(gen(1), n, 64, 16)
    before = state.clone()
    resume = torch.arange(n, device="cuda").int() % 2
    v = _inputs("bf16", 1, 64, 16)
    y = binding.lstm_selective_scan(v["u"][:0], v["dt"][:0], v["a"], v["b"][:0], v["c"][:0],
                                    offsets=_i32([0] * (n + 1)), state=state, resume=resume)
    assert y.shape == (0, 64)
    assert torch.equal(state[1::2], before[1::2]) and (state[::2] == 0).all()
    conv = normal(gen(2), n, 3, 64)
    kept = conv.clone()
    binding.lstm_causal_conv(torch.empty(0, 64, device="cuda"), torch.ones(64, 4, device="cuda"),
                             offsets=_i32([0] * (n + 1)), state=conv, resume=resume)
    assert torch.equal(conv[1::2], kept[1::2]) and (conv[::2] == 0).all()


def test_very_many_prompts_in_one_piece():
    """2^21 prompts of 128 blocks of channels: more than 2^31 states a thread of one block, which
    only prompts in several spans are limited to."""
    n, channels = 1 << 21, 16384
    state = torch.full((2, channels, 16), 7.0, device="cuda")
    slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    slots[0], slots[n - 1] = 1, 0
    empty = torch.zeros(0, channels, device="cuda")
    bc = torch.zeros(0, 16, device="cuda")
    y = binding.lstm_selective_scan(empty, empty, -torch.ones(channels, 16, device="cuda"), bc, bc,
                                    offsets=torch.zeros(n + 1, dtype=torch.int32, device="cuda"),
                                    state=state, slots=slots)
    assert y.shape == (0, channels) and not state.any()


@pytest.mark.parametrize("length", [589, 1000, 2500])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_prompts(dtype, length):
    _check(dtype, [length], 24, pool=1, resume=[1])


@pytest.mark.parametrize("lengths,channels,states,equal", [
    ([600], 4096, 16, True), ([24] * 32, 2048, 16, True), ([150] * 4, 1024, 16, True),
    ([90, 7, 300, 0, 41, 200, 1, 64, 128, 33] * 2, 1024, 16, False),
    ([33, 700, 2, 90, 400], 500, 16, False), ([260] * 2, 1024, 64, True),
    ([20, 300, 45] * 6, 640, 64, False), ([500, 64, 1], 1026, 8, False),
    ([40] * 20, 1024, 4, True), ([170, 80], 259, 5, False), ([33, 65, 129], 2048, 32, False)])
def test_large_layers(lengths, channels, states, equal):
    """Sizes on both sides of where the work is divided otherwise."""
    n = len(lengths)
    _check("bf16", lengths, channels, states, uniform_=equal, pool=n + 1,
           slots=[(3 * k + 1) % (n + 1) if (n + 1) % 3 else n - k for k in range(n)],
           resume=[k % 3 != 0 for k in range(n)])


@pytest.mark.parametrize("dtype,channels,states,copies", [
    ("bf16", 4096, 16, 2), ("f32", 4100, 16, 2), ("f16", 4095, 13, 2), ("bf16", 2048, 16, 4),
    ("bf16", 1030, 8, 2), ("f16", 515, 64, 2), ("bf16", 512, 128, 2), ("f32", 512, 32, 4),
    ("bf16", 4096, 4, 2), ("bf16", 2049, 5, 2)])
def test_unequal_prompts_in_order_and_whole(dtype, channels, states, copies):
    """Prompts that are put in order, but not divided: the workspace holds their order alone."""
    lengths = [0, 1, 2, 7, 8, 9, 15, 16, 17, 33, 64, 120] * copies
    n = len(lengths)
    size = binding.lstm_selective_scan_workspace(sum(lengths), channels, states, 1, n, False)
    assert size == 8 * (n + 1), size
    _check(dtype, lengths, channels, states, pool=n + 3, slots=[(7 * k + 2) % (n + 3) for k in range(n)],
           resume=[k % 3 != 2 for k in range(n)])


def test_large_layers_in_fp32():
    _check("f32", [100, 350, 20], 1024, pool=3, resume=[1, 0, 1])
    _check("f32", [130, 1, 257], 771, pool=3, resume=[1, 1, 1])


def test_long_memory():
    # step sizes so small that the first token still counts at the last
    _check("f32", [1500], 8, scale=0.01, pool=1, resume=[1])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("channels", [48, 50])
def test_packed_prompts(dtype, channels):
    _check(dtype, [70, 0, 1, 16, 200, 2, 0, 33], channels, pool=9, slots=[3, 0, 8, 7, 5, 1, 2, 6],
           resume=[1, 1, 1, 0, 1, 0, 0, 1], strided=True)


def test_many_short_prompts():
    _check("bf16", [3, 1, 4, 1, 5, 9, 2, 6] * 12, 64, pool=96, resume=[0, 1, 1] * 32)


def test_slots_outside_the_pool_have_no_state():
    _check("bf16", [25, 26, 27], 40, pool=3, slots=[-1, 1, 3], resume=[1, 1, 1])


def test_equal_lengths_without_offsets():
    _check("f16", [50] * 6, 96, uniform_=True, pool=6, resume=[0, 1, 0, 1, 1, 1])


@pytest.mark.parametrize("groups,channels", [(2, 64), (4, 20), (3, 99), (8, 512)])
def test_groups(groups, channels):
    _check("bf16", [37, 20], channels, groups=groups, pool=2, resume=[1, 1])


@pytest.mark.parametrize("without", [("z",), ("skip",), ("dt_bias",), ("z", "skip", "dt_bias")])
def test_without_optional_arguments(without):
    _check("f32", [45], 64, without=without)


def test_step_sizes_as_given():
    _check("bf16", [45], 64, softplus=False, pool=1, resume=[1])


def test_step_sizes_far_from_zero():
    # softplus of large, and of very negative, arguments
    _check("f32", [40], 32, scale=20.0)


def _check_infinities(dtype, channels, states, tokens, step, skip, least=-8.0, at=(5, 9), gated=False):
    """An infinite input of two channels against the definition: b and c positive, so that the
    infinities of its states add up to one.  Everything else stays finite."""
    v = _inputs(dtype, tokens, channels, states)
    v["u"][at[0], 3 % channels], v["u"][at[1], 17 % channels] = float("inf"), float("-inf")
    v["a"].clamp_(min=least)
    v["b"].abs_()
    v["c"].abs_()
    v["skip"] = v["skip"].abs() + 0.1 if skip else None
    v["z"] = v["z"].abs() + 0.1 if gated else None
    state = normal(gen(3), tokens if step else 1, channels, states)
    before = f64(state)
    call = binding.lstm_selective_scan_step if step else binding.lstm_selective_scan
    first = [v[k] for k in ("u", "dt", "a", "b", "c")] + ([state] if step else [])
    y = call(*first, skip=v["skip"], z=v["z"], **({} if step else {"state": state}))
    with np.errstate(invalid="ignore", over="ignore"):
        ref, new, bound, new_bound = oracle.selective_scan(
            *(f64(v[k]) for k in ("u", "dt", "a", "b", "c", "skip", "z")), None, True, 1,
            [(t, t + 1) for t in range(tokens)] if step else [(0, tokens)], before, step=step)
    assert np.isposinf(ref).any() and np.isneginf(ref).any() and not np.isnan(ref).any()
    for got, expected, off, t in ((y, ref, bound, dtype), (state, new, new_bound, "f32")):
        finite = np.isfinite(expected)
        np.testing.assert_array_equal(f64(got)[~finite], expected[~finite])
        assert_close(torch.where(torch.from_numpy(finite), got.cpu(), torch.zeros_like(got).cpu()),
                     np.where(finite, expected, 0.0), np.where(finite, off, 0.0), t)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("channels,states", [(40, 4), (40, 16), (40, 128)])
@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("skip", [False, True])
def test_an_infinite_input_stays_an_infinity(dtype, channels, states, step, skip):
    _check_infinities(dtype, channels, states, 24, step, skip)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("states", [1, 2, 3, 5, 7, 9, 13, 17, 24, 33, 48, 65, 100])
@pytest.mark.parametrize("channels", [40, 33])
@pytest.mark.parametrize("step", [False, True])
def test_an_infinite_input_beside_unused_places(dtype, channels, states, step):
    """States that do not fill the lanes' places."""
    _check_infinities(dtype, channels, states, 24, step, True)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("states", [4, 13, 16, 64])
def test_an_infinite_input_in_a_long_prompt(dtype, states):
    """Decays so fast that a span's product of them is 0, while no token's is."""
    assert binding.lstm_selective_scan_workspace(600, 24, states, 1, 1, True) > 0  # (in spans)
    _check_infinities(dtype, 24, states, 600, False, True, least=-30.0, at=(40, 300))


def test_an_infinite_state_in_a_long_prompt():
    v = _inputs("f32", 600, 24, 16)
    v["a"] = -torch.linspace(1, 40, 16, device="cuda").repeat(24, 1)
    state = torch.zeros(1, 24, 16, device="cuda")
    state[0, 5, 1], state[0, 6, 15] = float("inf"), float("-inf")
    binding.lstm_selective_scan(v["u"], v["dt"], v["a"], v["b"], v["c"], state=state,
                                resume=_i32([1]))
    assert state[0, 5, 1] == float("inf") and state[0, 6, 15] == float("-inf")
    assert int(torch.isfinite(state).sum()) == 24 * 16 - 2


@pytest.mark.parametrize("states", [13, 33])
def test_infinite_step_sizes(states):
    v = _inputs("f32", 30, 20, states)
    v["dt"][6, 3] = float("inf")
    v["b"].abs_()
    v["c"].abs_()
    v["u"].abs_()
    y = binding.lstm_selective_scan(v["u"], v["dt"], v["a"], v["b"], v["c"])
    # the states become infinities and, without a step size of that kind, stay so
    assert torch.isposinf(y[6:, 3]).all() and torch.isfinite(y[:6]).all()
    assert torch.isfinite(y[:, :3]).all() and torch.isfinite(y[:, 4:]).all()


@pytest.mark.parametrize("skip", [False, True])
def test_an_infinite_input_in_a_large_batch_of_steps(skip):
    _check_infinities("bf16", 128, 16, 300, True, skip, gated=True)


def test_other_rows_are_left_alone():
    y = torch.full((20, 33), 7.0, device="cuda")
    v = _inputs("f32", 20, 33, 16)
    binding.lstm_selective_scan(v["u"], v["dt"], v["a"], v["b"], v["c"], y=y,
                                offsets=_i32([2, 9, 15]))
    got = f64(y)
    assert (got[:2] == 7).all() and (got[15:] == 7).all() and not (got[2:15] == 7).any()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("channels,states,groups", [(1, 16, 1), (40, 13, 1), (64, 16, 2),
                                                    (2048, 16, 1), (30, 64, 3), (8, 128, 1),
                                                    (16, 4, 1), (16, 8, 1), (9, 32, 1), (5, 2, 1)])
@pytest.mark.parametrize("sequences", [1, 5])
def test_step(dtype, channels, states, groups, sequences):
    v = _inputs(dtype, sequences, channels, states, groups, strided=True)
    state = normal(gen(8), 7, channels, states)
    slots = [6, -1, 2, 7, 0][:sequences]
    before = f64(state)
    y = binding.lstm_selective_scan_step(v["u"], v["dt"], v["a"], v["b"], v["c"], state,
                                         skip=v["skip"], z=v["z"], dt_bias=v["dt_bias"],
                                         groups=groups, slots=_i32(slots))
    ref, new, bound, new_bound = oracle.selective_scan(
        f64(v["u"]), f64(v["dt"]), f64(v["a"]), f64(v["b"]), f64(v["c"]), f64(v["skip"]),
        f64(v["z"]), f64(v["dt_bias"]), True, groups, [(s, s + 1) for s in range(sequences)],
        before, slots, step=True)
    assert_close(y, ref, bound, dtype, "y")
    assert_close(state, new, new_bound, "f32", "state")


@pytest.mark.parametrize("dtype,sequences,channels,states,groups", [
    ("bf16", 300, 96, 16, 1), ("bf16", 300, 500, 16, 1), ("f32", 70, 1300, 16, 1),
    ("f16", 2000, 130, 4, 1), ("bf16", 700, 200, 8, 1), ("bf16", 300, 130, 32, 1),
    ("bf16", 90, 256, 64, 4), ("f32", 40, 256, 128, 1), ("bf16", 600, 256, 16, 2),
    ("bf16", 600, 130, 16, 2), ("bf16", 700, 129, 13, 1), ("bf16", 9000, 8, 16, 1)])
def test_step_of_a_large_batch(dtype, sequences, channels, states, groups):
    v = _inputs(dtype, sequences, channels, states, groups, strided=True)
    state = normal(gen(8), sequences + 10, channels, states)
    slots = torch.randperm(sequences + 10, generator=torch.Generator().manual_seed(1))[:sequences].int()
    slots[5::17] = -1
    before = f64(state)
    y = binding.lstm_selective_scan_step(v["u"], v["dt"], v["a"], v["b"], v["c"], state,
                                         skip=v["skip"], z=v["z"], dt_bias=v["dt_bias"],
                                         groups=groups, slots=slots.cuda())
    ref, new, bound, new_bound = oracle.selective_scan(
        f64(v["u"]), f64(v["dt"]), f64(v["a"]), f64(v["b"]), f64(v["c"]), f64(v["skip"]),
        f64(v["z"]), f64(v["dt_bias"]), True, groups, [(s, s + 1) for s in range(sequences)],
        before, slots.tolist(), step=True)
    assert binding.lstm_fault_status() == 0
    assert_close(y, ref, bound, dtype, "y")
    assert_close(state, new, new_bound, "f32", "state")


@pytest.mark.parametrize("offset", [0, 1, 2, 3])
@pytest.mark.parametrize("dtype,sequences,channels,states", [
    ("bf16", 300, 128, 16), ("f32", 4, 64, 16), ("f16", 5, 33, 8), ("bf16", 20, 40, 13)])
def test_weights_and_states_at_any_element(offset, dtype, sequences, channels, states):
    """Views into larger buffers: prompts of one token each, and steps."""
    v = _inputs(dtype, sequences, channels, states)
    for k, shift in (("a", 0), ("skip", 1), ("dt_bias", 2)):
        v[k] = at_element(v[k], (offset + shift) % 4)
    start = normal(gen(8), sequences, channels, states)
    for what in ("prompts", "step"):
        state = at_element(start, offset)
        assert state.data_ptr() % 16 == 4 * offset
        first = [v[k] for k in ("u", "dt", "a", "b", "c")]
        more = {k: v[k] for k in ("skip", "z", "dt_bias")}
        if what == "step":
            y = binding.lstm_selective_scan_step(*first, state, **more)
        else:
            y = binding.lstm_selective_scan(*first, state=state, sequences=sequences,
                                            resume=torch.ones(sequences, device="cuda").int(), **more)
        ref, new, bound, new_bound = oracle.selective_scan(
            *(f64(v[k]) for k in ("u", "dt", "a", "b", "c", "skip", "z", "dt_bias")), True, 1,
            [(s, s + 1) for s in range(sequences)], f64(start), step=True)
        assert_close(y, ref, bound, dtype, what)
        assert_close(state, new, new_bound, "f32", what + "'s state")


def test_a_step_whose_states_do_not_arrive_is_reported():
    lib = binding.load()
    v = _inputs("bf16", 300, 128, 16)
    state = normal(gen(8), 300, 128, 16)
    before = state.clone()
    call = lambda: binding.lstm_selective_scan_step(v["u"], v["dt"], v["a"], v["b"], v["c"], state)
    try:
        assert lib.lstm_test_scan_step_timeout(1, 1000, 0) == 0
        call()
        assert binding.lstm_fault_status() == 1 << 6
        assert torch.equal(state, before)
    finally:
        assert lib.lstm_test_scan_step_timeout(0, 0, 0) == 0
    # the context stays usable
    y = call()
    ref, new, bound, new_bound = oracle.selective_scan(
        f64(v["u"]), f64(v["dt"]), f64(v["a"]), f64(v["b"]), f64(v["c"]), None, None, None, True, 1,
        [(s, s + 1) for s in range(300)], f64(before), step=True)
    assert binding.lstm_fault_status() == 0
    assert_close(y, ref, bound, "bf16")
    assert_close(state, new, new_bound, "f32")


def test_launch_failures_are_reported():
    lib = binding.load()
    v = _inputs("bf16", 400, 64, 16)
    call = lambda: binding.lstm_selective_scan(v["u"], v["dt"], v["a"], v["b"], v["c"])
    ref = call()
    try:
        for skip in range(3):  # two passes and what carries the states between them
            lib.lstm_test_fail_launches(skip, 1)
            with pytest.raises(binding.LSTMError) as e:
                call()
            assert e.value.code == binding.LSTM_E_CUDA
    finally:
        lib.lstm_test_fail_launches(0, 0)
    assert torch.equal(call(), ref)


def test_a_workspace_that_is_too_short_is_refused():
    lib = binding.load()
    size = binding.lstm_selective_scan_workspace(400, 64, 16, 1, 1, True)
    assert size > 0
    z = torch.zeros(400 * 64, device="cuda")
    at, s = z.data_ptr(), torch.cuda.current_stream().cuda_stream
    call = lambda w, n: lib.lstm_selective_scan(
        at, 64, at, 64, at, at, 16, at, 16, None, None, 0, None, 1, 0, 400, 64, 16, 1, 1, None, None,
        0, None, None, at, 64, w, n, s)
    assert call(None, 0) == binding.LSTM_E_INVALID
    assert call(at, size - 1) == binding.LSTM_E_LENGTH
    assert call(at + 4, size) == binding.LSTM_E_INVALID


def test_prompt_in_parts_and_steps_goes_on_from_its_state():
    v = _inputs("f32", 90, 48, 16)
    call = lambda a, b, **k: binding.lstm_selective_scan(
        v["u"][a:b], v["dt"][a:b], v["a"], v["b"][a:b], v["c"][a:b], skip=v["skip"], z=v["z"][a:b],
        dt_bias=v["dt_bias"], **k)
    state, last = torch.empty(1, 48, 16, device="cuda"), torch.empty(1, 48, 16, device="cuda")
    whole = call(0, 90, state=last)
    one = _i32([1])
    parts = [call(0, 33, state=state), call(33, 80, state=state, resume=one)]
    for t in range(80, 90):
        parts.append(binding.lstm_selective_scan_step(
            v["u"][t:t + 1], v["dt"][t:t + 1], v["a"], v["b"][t:t + 1], v["c"][t:t + 1], state,
            skip=v["skip"], z=v["z"][t:t + 1], dt_bias=v["dt_bias"]))
    ref, new, bound, new_bound = oracle.selective_scan(
        *(f64(v[k]) for k in ("u", "dt", "a", "b", "c", "skip", "z", "dt_bias")), True, 1,
        [(0, 90)], np.zeros((1, 48, 16)))
    for got, s in ((whole, last), (torch.cat(parts), state)):
        assert_close(got, ref, bound, "f32")
        assert_close(s, new, new_bound, "f32")


def test_the_same_bits_every_time_and_on_another_stream():
    v = _inputs("bf16", 700, 64, 16)
    call = lambda **k: binding.lstm_selective_scan(v["u"], v["dt"], v["a"], v["b"], v["c"],
                                                   skip=v["skip"], z=v["z"], **k)
    ref = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (None, s, s.cuda_stream):
        y = call(stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(y, ref)


def test_in_a_graph():
    v = _inputs("bf16", 200, 64, 16)
    state = torch.zeros(1, 64, 16, device="cuda")
    y = torch.empty_like(v["u"])
    call = lambda: binding.lstm_selective_scan(v["u"], v["dt"], v["a"], v["b"], v["c"], state=state,
                                               resume=one, y=y)
    one = _i32([1])
    call()
    first, after = y.clone(), state.clone()
    call()
    second, twice = y.clone(), state.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    state.zero_()
    graph.replay()
    assert torch.equal(y, first) and torch.equal(state, after)
    graph.replay()
    assert torch.equal(y, second) and torch.equal(state, twice)


def test_refusals():
    v = _inputs("f32", 12, 16, 8)

    def run(**k):
        first = [k.pop(n, v[n]) for n in ("u", "dt", "a", "b", "c")]
        return binding.lstm_selective_scan(*first, **k)

    z = lambda *s: torch.zeros(*s, device="cuda")
    with pytest.raises(binding.LSTMError) as e:
        run(a=z(16, 129), b=z(12, 129), c=z(12, 129))
    assert e.value.code == binding.LSTM_E_INVALID
    with pytest.raises(binding.LSTMError) as e:
        run(groups=3, b=z(12, 24), c=z(12, 24))
    assert e.value.code == binding.LSTM_E_INVALID
    with pytest.raises(binding.LSTMError) as e:
        run(sequences=5)
    assert e.value.code == binding.LSTM_E_LENGTH
    for bad in (dict(u=v["u"].half()), dict(dt=z(12, 15)), dict(dt=z(11, 16)), dict(a=z(15, 8)),
                dict(a=z(16, 8).double()), dict(b=z(12, 9)), dict(c=v["c"].bfloat16()),
                dict(z=z(12, 17)), dict(skip=z(17)), dict(dt_bias=z(16).half()),
                dict(groups=2), dict(state=z(1, 16, 9)), dict(state=z(1, 16, 8).half()),
                dict(state=z(1, 16, 8), sequences=2), dict(slots=_i32([0])),
                dict(state=z(1, 16, 8), slots=_i32([0, 1])), dict(offsets=_i32([0, 12]).long()),
                dict(y=z(12, 15)), dict(a=z(16, 8).cpu())):
        with pytest.raises(ValueError):
            run(**bad)
    with pytest.raises(ValueError):
        binding.lstm_selective_scan_step(v["u"], v["dt"], v["a"], v["b"], v["c"], z(2, 16, 8))
