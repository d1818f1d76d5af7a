"""Linear attention with a decay for each head over packed prompts and over single
tokens against its float64 definition: types, heads and who shares them, sizes,
lengths from zero to long ones, decays from none to forgetting, states and slots,
strides, values that are not finite, streams and graphs, and refusals."""
import numpy as np
import pytest
import torch

from bidirectional_lstm_stack_gb300 import binding
from oracle import layers as oracle
from oracle.ops import spans
from ops_util import DTYPES, assert_close, at_element, f64, gen, normal, uniform

pytestmark = pytest.mark.gpu


def _i32(a):
    return None if a is None else torch.tensor(a, dtype=torch.int32, device="cuda")


def _decays(g, kind, tokens, heads):
    shape = (tokens, heads) if kind.startswith("each") else (heads,)
    d = -torch.exp(normal(g, *shape) - 3.0)
    if kind.endswith("none"):
        d = torch.zeros(shape, device="cuda")
    if kind.endswith("strong"):
        d = -30.0 * uniform(g, *shape)
    if kind.endswith("forget"):
        d[uniform(g, *shape) < 0.1] = -float("inf")
    if kind.endswith("grow"):
        d = 0.01 * uniform(g, *shape)
    return d


def _inputs(dtype, tokens, heads, keys, values, shared=(1, 1, 1), layout="dense", seed=1):
    g, t = gen(seed), DTYPES[dtype]
    own = [heads // s for s in shared]
    widths = [own[0] * keys, own[1] * keys, own[2] * values]
    if layout == "dense":
        m = [normal(g, tokens, w, dtype=t) for w in widths]
    else:  # columns of one wide matrix, which begins and ends with NaN
        pad = {"slices": 8, "odd": 1}[layout]
        wide = torch.full((tokens, sum(widths) + 2 * pad), float("nan"), dtype=t, device="cuda")
        wide[:, pad:-pad] = normal(g, tokens, sum(widths), dtype=t)
        m = wide[:, pad:-pad].split(widths, 1)
    return [x.unflatten(1, (n, -1)) for x, n in zip(m, own)]


def _check(dtype, lengths, heads=2, keys=64, values=64, *, shared=(1, 1, 1), layout="dense",
           decay="each", pool=None, slots=None, resume=None, equal=False, seed=1, scale=0.125, y=None,
           step=False):
    tokens, sequences = sum(lengths), len(lengths)
    q, k, v = _inputs(dtype, tokens, heads, keys, values, shared, layout, seed)
    g = gen(seed + 1)
    d = _decays(g, decay, tokens, heads)
    state = None if pool is None else normal(g, pool, heads, keys, values)
    before = f64(state)
    offsets = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    if step:
        got = binding.lstm_linear_attention_step(q, k, v, d, state, scale=scale, slots=_i32(slots),
                                                 y=y)
    else:
        got = binding.lstm_linear_attention(
            q, k, v, d, scale=scale, sequences=sequences, offsets=None if equal else _i32(offsets),
            state=state, slots=_i32(slots), resume=_i32(resume), y=y)
    assert got.dtype == DTYPES[dtype] and got.shape == (tokens, heads, values)
    ref, new, bound, new_bound = oracle.linear_attention(
        f64(q), f64(k), f64(v), f64(d), scale, spans(tokens, sequences, offsets), dtype, before,
        slots, resume, step)
    assert_close(got, ref, bound, dtype, "y")
    # the bound adds up every rounding at its worst; they point all ways, and each of the three of
    # an output is a half step of bf16 at most.  In fp32 a head's e^g, rounded to 2^-24 of itself,
    # is off to the same side at every token: 2^-24 times the length
    if ref.size >= 4096:
        off = np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)
        assert off <= {"bf16": 3 * 2.0 ** -8, "f16": 2.0 ** -11 + 2.0 ** -14,
                       "f32": 2.0 ** -20 + max(lengths) * 2.0 ** -24}[dtype]
    if state is not None:
        assert_close(state, new, new_bound, "f32", "state")
    return got, state


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("length", [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 300])
def test_lengths(dtype, length):
    _check(dtype, [length], pool=1, resume=[1])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("keys,values", [(1, 1), (3, 5), (8, 16), (16, 8), (17, 33), (32, 64), (64, 32),
                                         (65, 64), (64, 65), (96, 80), (100, 130), (128, 128),
                                         (128, 256), (127, 255), (2, 256), (128, 1)])
def test_sizes(dtype, keys, values):
    _check(dtype, [70, 9], 2, keys, values, pool=2, resume=[1, 0])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("decay", ["none", "each", "strong", "each strong", "forget", "each forget",
                                   "grow", "each grow", "each none"])
def test_decays(dtype, decay):
    _check(dtype, [200, 65], 3, 32, 48, decay=decay, pool=2, resume=[1, 1])


@pytest.mark.parametrize("heads,shared", [(1, (1, 1, 1)), (4, (1, 4, 4)), (4, (4, 4, 1)), (6, (3, 2, 1)),
                                          (6, (1, 6, 2)), (12, (12, 12, 12))])
def test_heads_that_share(heads, shared):
    for dtype in DTYPES:
        _check(dtype, [67], heads, 32, 32, shared=shared, pool=1, resume=[1])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("layout", ["slices", "odd"])
@pytest.mark.parametrize("keys,values", [(64, 64), (40, 24), (33, 31), (128, 128)])
def test_columns_of_wider_rows(dtype, layout, keys, values):
    _check(dtype, [66, 3], 2, keys, values, layout=layout, pool=2, resume=[1, 0])


def test_any_strides_between_heads_and_tokens():
    g = gen(3)
    # [heads, tokens, keys] and interleaved q, k, v of each head
    q = normal(g, 3, 80, 32, dtype=torch.bfloat16).transpose(0, 1)
    kv = normal(g, 80, 3, 96, dtype=torch.bfloat16)
    k, v = kv[..., :32], kv[..., 32:]
    d = _decays(g, "each", 80, 3)
    one = binding.lstm_linear_attention(q, k, v, d)
    assert torch.equal(binding.lstm_linear_attention_step(q, k, v, d, torch.zeros(80, 3, 32, 64).cuda()),
                       binding.lstm_linear_attention_step(q.contiguous(), k.contiguous(), v.contiguous(), d,
                                                          torch.zeros(80, 3, 32, 64).cuda()))
    two = binding.lstm_linear_attention(q.contiguous(), k.contiguous(), v.contiguous(), d)
    assert torch.equal(one, two)
    # a decay that is a column slice, and one row for all
    wide = torch.full((80, 7), float("nan"), device="cuda")
    wide[:, 2:5] = d
    assert torch.equal(binding.lstm_linear_attention(q.contiguous(), k, v, wide[:, 2:5]), one)
    row = d[0].clone()
    assert torch.equal(binding.lstm_linear_attention(q.contiguous(), k, v, row),
                       binding.lstm_linear_attention(q.contiguous(), k, v, row.expand(80, 3)))
    # outputs into columns of wider rows, the others left as they were
    wide = torch.full((80, 3 * 64 + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    y = wide[:, 2:2 + 192].unflatten(1, (3, 64))
    assert binding.lstm_linear_attention(q.contiguous(), k, v, d, y=y) is y
    assert torch.equal(y, one) and (wide[:, :2] == 7).all() and (wide[:, -3:] == 7).all()


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_packed_prompts_and_their_slots(dtype):
    lengths = [5, 0, 130, 64, 1, 0, 77]
    _, state = _check(dtype, lengths, 3, 32, 32, pool=9, slots=[8, 0, 3, 5, 1, 7, -1],
                      resume=[1, 0, 0, 1, 1, 1, 1])
    _check(dtype, lengths, 3, 32, 32, pool=9, slots=[8, 0, 3, 9, 1, 7, 2])
    _check(dtype, lengths, 3, 32, 32)


def test_prompts_of_equal_length():
    _check("bf16", [100] * 5, equal=True, pool=5)
    _check("f32", [100] * 5, equal=True, pool=6, slots=[5, 4, 3, 2, 0], resume=[1, 0, 1, 0, 1])


def test_tokens_behind_the_last_sequence_stay():
    q, k, v = _inputs("bf16", 100, 2, 32, 32)
    y = torch.full((100, 2, 32), 3.0, dtype=torch.bfloat16, device="cuda")
    binding.lstm_linear_attention(q, k, v, torch.zeros(2, device="cuda"),
                                  offsets=_i32([4, 40, 70]), y=y)
    assert (y[:4] == 3).all() and (y[70:] == 3).all() and (y[4:70] != 3).any()


def test_prompts_in_pieces_are_prompts_in_one():
    q, k, v = _inputs("f32", 300, 2, 64, 64)
    d = _decays(gen(5), "each", 300, 2)
    whole = torch.zeros(1, 2, 64, 64, device="cuda")
    y = binding.lstm_linear_attention(q, k, v, d, state=whole)
    state, parts = torch.zeros_like(whole), []
    for a, b in [(0, 1), (1, 130), (130, 131), (131, 300)]:
        if b - a == 1:
            parts.append(binding.lstm_linear_attention_step(q[a:b], k[a:b], v[a:b], d[a:b], state))
        else:
            parts.append(binding.lstm_linear_attention(q[a:b], k[a:b], v[a:b], d[a:b], state=state,
                                                       resume=_i32([1])))
    for got, ref in ((torch.cat(parts), y), (state, whole)):
        assert (got - ref).norm() <= 2.0 ** -19 * ref.norm()


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_long_prompts(dtype):
    # few heads: the long axis is split
    _check(dtype, [3000], 1, 64, 64, pool=1, resume=[1])
    _check(dtype, [1500, 20, 900], 2, 32, 48, pool=3, resume=[1, 1, 0], decay="each none")
    _check(dtype, [2048] * 2, 1, 128, 128, equal=True, pool=2, decay="head", resume=[0, 1])


def test_many_short_prompts():
    lengths = [(i * 7) % 5 for i in range(700)]
    _check("bf16", lengths, 1, 16, 16, pool=700, resume=[i % 2 for i in range(700)])


# ---- values that are not finite -----------------------------------------------------------------
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("what", ["q", "k", "v"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_tokens_before_one_that_is_not_finite_are_as_without(dtype, what, bad):
    lengths, heads = [70, 100, 30], 2
    tokens = sum(lengths)
    m = dict(zip("qkv", _inputs(dtype, tokens, heads, 32, 48)))
    d = _decays(gen(2), "each", tokens, heads)
    offsets = _i32([0, 70, 170, 200])

    def call():
        state = torch.zeros(3, heads, 32, 48, device="cuda")
        y = binding.lstm_linear_attention(m["q"], m["k"], m["v"], d, offsets=offsets, state=state)
        return y, state

    y, state = call()
    sizes = binding.lstm_linear_attention(m["q"].abs(), m["k"].abs(), m["v"].abs(), d, offsets=offsets)
    at = 70 + 41
    m[what][at, 1, 7] = bad
    y2, state2 = call()
    if what == "v":
        # its column's sums over the 64 tokens around are made in another order, which moves them
        # by 64 ulps (2^-23) of the terms' sizes at most, and then one rounding to the type
        off = (y2[70:at, 1, 7].double() - y[70:at, 1, 7].double()).abs()
        assert (off <= 2.0 ** -17 * sizes[70:at, 1, 7].double()
                + torch.finfo(y.dtype).eps * y[70:at, 1, 7].double().abs()).all()
        y2[70:at, 1, 7] = y[70:at, 1, 7]
    assert torch.equal(y2[:at], y[:at]) and torch.equal(y2[170:], y[170:])
    assert torch.equal(y2[:, 0], y[:, 0])
    assert torch.equal(state2[[0, 2]], state[[0, 2]]) and torch.equal(state2[1, 0], state[1, 0])
    if what == "q":
        assert not y2[at, 1].isfinite().any()
        assert torch.equal(y2[at + 1:], y[at + 1:]) and torch.equal(state2, state)
    if what == "k":
        assert not y2[at:170, 1].isfinite().any() and not state2[1, 1, 7].isfinite().any()
    if what == "v":
        assert not y2[at:170, 1, 7].isfinite().any()
        others = [c for c in range(48) if c != 7]
        assert torch.equal(y2[..., others], y[..., others])
        assert torch.equal(state2[..., others], state[..., others])
        assert not state2[1, 1, :, 7].isfinite().any()


def test_a_decay_that_is_not_a_number():
    q, k, v = _inputs("bf16", 150, 2, 32, 32)
    d = _decays(gen(2), "each", 150, 2)
    y = binding.lstm_linear_attention(q, k, v, d)
    d[100, 1] = float("nan")
    y2 = binding.lstm_linear_attention(q, k, v, d)
    assert torch.equal(y2[:100], y[:100]) and torch.equal(y2[:, 0], y[:, 0])
    assert not y2[100:, 1].isfinite().any()


def test_unused_slots_and_other_rows_may_hold_anything():
    q, k, v = _inputs("bf16", 90, 2, 32, 32)
    d = _decays(gen(2), "head", 90, 2)
    state = torch.full((4, 2, 32, 32), float("nan"), device="cuda")
    y = binding.lstm_linear_attention(q, k, v, d, state=state, slots=_i32([2]))
    assert y.isfinite().all() and state[2].isfinite().all() and state[[0, 1, 3]].isnan().all()


# ---- single tokens ------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("keys,values", [(1, 1), (3, 5), (16, 16), (33, 20), (64, 64), (100, 130),
                                         (128, 128), (128, 256), (7, 255), (128, 4), (1, 256)])
def test_step_sizes(dtype, keys, values):
    _check(dtype, [1] * 3, 2, keys, values, pool=3, step=True)


@pytest.mark.parametrize("sequences", [1, 2, 7, 64, 200])
def test_steps_of_batches(sequences):
    slots = torch.randperm(sequences + 5, generator=torch.Generator().manual_seed(1)).tolist()[:sequences]
    for dtype, decay, shared in (("bf16", "head", (1, 1, 1)), ("f32", "each forget", (4, 4, 1)),
                                 ("f16", "each", (2, 1, 4))):
        _check(dtype, [1] * sequences, 4, 32, 64, shared=shared, decay=decay, pool=sequences + 5,
               slots=slots, layout="odd" if dtype == "f16" else "slices", step=True)


def test_steps_without_a_slot_start_from_zeros():
    _check("bf16", [1] * 4, pool=4, slots=[-1, 3, 4, 0], step=True)


def test_states_at_any_element():
    for dtype in ("bf16", "f32"):
        q, k, v = _inputs(dtype, 66, 2, 32, 32)
        d = _decays(gen(2), "each", 66, 2)
        s0 = normal(gen(4), 1, 2, 32, 32)
        for call in ("prompt", "step"):
            out = []
            for offset in (0, 1, 2, 4):
                state = at_element(s0, offset)
                if call == "prompt":
                    y = binding.lstm_linear_attention(q, k, v, d, state=state, resume=_i32([1]))
                else:
                    y = binding.lstm_linear_attention_step(q[:1], k[:1], v[:1], d[:1], state)
                out.append((y, state.clone()))
            for y, state in out[1:]:
                # (another vector width joins a column's sums in another order)
                assert (y.float() - out[0][0].float()).norm() <= 2.0 ** -8 * y.float().norm()
                assert torch.allclose(state, out[0][1], rtol=1e-6, atol=1e-6)


# ---- streams, graphs, repeats ---------------------------------------------------------------------
def test_the_same_call_gives_the_same_bits():
    q, k, v = _inputs("bf16", 3000, 2, 64, 64)
    d = _decays(gen(2), "each", 3000, 2)
    outs = [binding.lstm_linear_attention(q, k, v, d) for _ in range(3)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_other_streams_and_calls_at_once():
    streams = [torch.cuda.Stream() for _ in range(2)]
    inputs = [(_inputs("bf16", 2000, 2, 64, 64, seed=s), _decays(gen(s), "each", 2000, 2))
              for s in (1, 2)]
    alone = [binding.lstm_linear_attention(*m, d) for m, d in inputs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [binding.lstm_linear_attention(*m, d, stream=s) for (m, d), s in zip(inputs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, got))


def test_a_captured_call_reads_what_is_there_when_it_is_replayed():
    q, k, v = _inputs("bf16", 600, 2, 64, 64)
    d = _decays(gen(2), "each", 600, 2)
    offsets, slots, resume = _i32([0, 250, 600]), _i32([1, 0]), _i32([1, 1])
    state = torch.zeros(2, 2, 64, 64, device="cuda")
    y = torch.empty(600, 2, 64, dtype=torch.bfloat16, device="cuda")
    y1 = torch.empty(2, 2, 64, dtype=torch.bfloat16, device="cuda")

    def both():
        binding.lstm_linear_attention(q, k, v, d, offsets=offsets, state=state, slots=slots,
                                      resume=resume, y=y)
        binding.lstm_linear_attention_step(q[:2], k[:2], v[:2], d[:2], state, slots=slots, y=y1)

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    g = gen(9)
    for bounds in ([0, 250, 600], [0, 590, 600], [0, 0, 64]):
        q.copy_(normal(g, 600, 2, 64))
        offsets.copy_(_i32(bounds))
        state.copy_(normal(g, 2, 2, 64, 64))
        start = state.clone()
        graph.replay()
        replayed = y[:bounds[-1]].clone(), y1.clone(), state.clone()
        state.copy_(start)
        both()
        assert all(torch.equal(a, b) for a, b in zip(replayed, (y[:bounds[-1]], y1, state)))


def test_calls_under_inference_mode_and_versions():
    q, k, v = _inputs("bf16", 10, 2, 16, 16)
    state = torch.zeros(1, 2, 16, 16, device="cuda")
    version = state._version
    binding.lstm_linear_attention(q, k, v, torch.zeros(2, device="cuda"), state=state)
    assert state._version > version
    with torch.inference_mode():
        binding.lstm_linear_attention_step(q[:1], k[:1], v[:1], torch.zeros(2, device="cuda"),
                                           torch.zeros(1, 2, 16, 16, device="cuda"))


def test_launch_failures_are_errors():
    q, k, v = _inputs("bf16", 10, 2, 16, 16)
    d, state = torch.zeros(2, device="cuda"), torch.zeros(10, 2, 16, 16, device="cuda")
    lib = binding.load()
    for call in (lambda: binding.lstm_linear_attention(q, k, v, d),
                 lambda: binding.lstm_linear_attention_step(q, k, v, d, state)):
        assert lib.lstm_test_fail_launches(0, 1) == 0
        with pytest.raises(binding.LSTMError):
            call()
        call()


def test_a_wait_that_runs_out_sets_the_fault_word_and_the_next_call_works():
    lib = binding.load()
    for dtype, keys in (("bf16", 64), ("f32", 128)):
        q, k, v = _inputs(dtype, 300, 2, keys, 64)
        d = _decays(gen(2), "each", 300, 2)
        ref = binding.lstm_linear_attention(q, k, v, d)
        assert binding.lstm_fault_status() == 0
        try:
            assert lib.lstm_test_attention_timeout(1, 1000, 0) == 0
            binding.lstm_linear_attention(q, k, v, d)
            torch.cuda.synchronize()
        finally:
            assert lib.lstm_test_attention_timeout(0, 0, 0) == 0
        assert binding.lstm_fault_status() != 0
        assert torch.equal(binding.lstm_linear_attention(q, k, v, d), ref)
        torch.cuda.synchronize()
        assert binding.lstm_fault_status() == 0


# ---- sequences cut into spans, rows copied in boxes ---------------------------------------------
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("keys,values", [(128, 130), (33, 200), (64, 64)])
def test_spans_of_unequal_sequences(dtype, keys, values):
    _check(dtype, [1, 1400, 0, 63, 2100, 64], 2, keys, values, shared=(1, 2, 1), pool=7,
           slots=[3, 0, 6, 5, -1, 1], resume=[1, 1, 0, 1, 0, 1], layout="slices")


@pytest.mark.parametrize("decay", ["head", "each strong", "each forget", "each none", "each grow"])
def test_spans_and_their_decays(decay):
    for dtype in ("bf16", "f32"):
        _check(dtype, [1300], 2, 48, 64, decay=decay, pool=2, slots=[1], resume=[1])


def test_spans_start_from_the_slot_that_the_last_one_writes():
    # (the same slot is read by the first span and written by the last)
    q, k, v = _inputs("f32", 4000, 2, 64, 64)
    d = _decays(gen(5), "each", 4000, 2)
    state = normal(gen(6), 3, 2, 64, 64)
    start = state.clone()
    ys = [binding.lstm_linear_attention(q, k, v, d, state=state.copy_(start), slots=_i32([1]),
                                        resume=_i32([1])).clone() for _ in range(5)]
    assert all(torch.equal(y, ys[0]) for y in ys[1:])
    assert torch.equal(state[[0, 2]], start[[0, 2]])


@pytest.mark.parametrize("tokens", [130, 3000])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_rows_around_a_sequence_may_hold_anything(tokens, what):
    q, k, v = _inputs("bf16", tokens + 100, 2, 64, 64)
    d = _decays(gen(2), "each", tokens + 100, 2)
    offsets = _i32([50, 50 + tokens - 17])
    states = []
    for m in (None, what):
        if m is not None:
            for x in (q, k, v, d):
                x[:50] = m
                x[50 + tokens - 17:] = m
        state = torch.zeros(1, 2, 64, 64, device="cuda")
        y = torch.full((tokens + 100, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        binding.lstm_linear_attention(q, k, v, d, offsets=offsets, state=state, y=y)
        states.append((y, state))
    assert torch.equal(states[0][0], states[1][0]) and torch.equal(states[0][1], states[1][1])


def test_a_value_that_is_not_finite_far_into_a_cut_sequence():
    q, k, v = _inputs("bf16", 3000, 2, 64, 64)
    d = _decays(gen(2), "each", 3000, 2)
    state = torch.zeros(1, 2, 64, 64, device="cuda")
    y = binding.lstm_linear_attention(q, k, v, d)
    v[1777, 1, 7] = float("inf")
    y2 = binding.lstm_linear_attention(q, k, v, d, state=state)
    assert torch.equal(y2[:1777], y[:1777]) and torch.equal(y2[:, 0], y[:, 0])
    others = [c for c in range(64) if c != 7]
    assert torch.equal(y2[..., others], y[..., others])
    assert not y2[1777:, 1, 7].isfinite().any() and not state[0, 1, :, 7].isfinite().any()


def test_a_workspace_that_is_short_or_missing_is_refused():
    lib = binding.load()
    q, k, v = _inputs("bf16", 4000, 1, 64, 64)
    d, y = torch.zeros(1, device="cuda"), torch.empty(4000, 64, dtype=torch.bfloat16, device="cuda")
    need = binding.lstm_linear_attention_workspace(4000, 1, 64, 64, 1, True)
    assert need > 0
    space = torch.empty(need, dtype=torch.uint8, device="cuda")

    def call(at, size):
        return lib.lstm_linear_attention(
            q.data_ptr(), 64, 64, 1, k.data_ptr(), 64, 64, 1, v.data_ptr(), 64, 64, 1, d.data_ptr(), 0,
            1.0, binding.LSTM_BF16, 4000, 1, 64, 64, 1, None, None, 0, None, None, y.data_ptr(), 64, at,
            size, None)

    assert call(None, need) == binding.LSTM_E_INVALID
    assert call(space.data_ptr(), need - 1) == binding.LSTM_E_LENGTH
    assert call(space.data_ptr(), need) == 0
    torch.cuda.synchronize()
    assert torch.equal(y.view(4000, 1, 64), binding.lstm_linear_attention(q, k, v, d))


def test_a_captured_call_in_spans_reads_what_is_there_when_it_is_replayed():
    q, k, v = _inputs("bf16", 4000, 2, 64, 64)
    d = _decays(gen(2), "each", 4000, 2)
    offsets, slots, resume = _i32([0, 1500, 4000]), _i32([1, 0]), _i32([1, 1])
    state = torch.zeros(2, 2, 64, 64, device="cuda")
    y = torch.empty(4000, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert binding.lstm_linear_attention_workspace(4000, 2, 64, 64, 2, False) > 0

    def call():
        binding.lstm_linear_attention(q, k, v, d, offsets=offsets, state=state, slots=slots,
                                      resume=resume, y=y)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    g = gen(9)
    for bounds, again in (([0, 1500, 4000], [1, 1]), ([0, 3990, 4000], [0, 1]), ([7, 7, 3000], [1, 0])):
        q.copy_(normal(g, 4000, 2, 64))
        offsets.copy_(_i32(bounds))
        resume.copy_(_i32(again))
        state.copy_(normal(g, 2, 2, 64, 64))
        start = state.clone()
        graph.replay()
        replayed = y[bounds[0]:bounds[-1]].clone(), state.clone()
        state.copy_(start)
        call()
        assert torch.equal(replayed[0], y[bounds[0]:bounds[-1]]) and torch.equal(replayed[1], state)


@pytest.mark.parametrize("count", [2, 63, 64, 65, 200])
def test_unequal_sequences_in_any_order(count):
    # (up to 64 of them each block puts in order, the longest first; equal ones keep theirs)
    lengths = [(i * 37) % 90 if i % 3 else 50 for i in range(count)]
    _check("bf16", lengths, 16, 16, 16, pool=count, resume=[i % 2 for i in range(count)])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("again", [0, 1])
@pytest.mark.parametrize("first,lengths", [
    (1000, [2500]),        # a cut sequence behind rows of several spans' length
    (3000, [100]),         # a sequence of one span there
    (1700, [0, 900, 40]),
])
def test_rows_before_the_first_sequence_of_a_call_in_spans(dtype, again, first, lengths):
    # the same sequences at the front of as many tokens are cut the same way: the same bits
    tokens, n = 4000, len(lengths)
    total = sum(lengths)
    assert binding.lstm_linear_attention_workspace(tokens, 2, 64, 64, n, False) > 0
    m = [*_inputs(dtype, total, 2, 64, 64), _decays(gen(2), "each", total, 2)]
    start = normal(gen(3), n + 1, 2, 64, 64)
    out = []
    for begin in (0, first):
        parts = []
        for x in m:
            rows = torch.full((tokens, *x.shape[1:]), float("nan"), dtype=x.dtype, device="cuda")
            rows[begin:begin + total] = x
            parts.append(rows)
        y = torch.full((tokens, 2, 64), 3.0, dtype=DTYPES[dtype], device="cuda")
        state = start.clone()
        binding.lstm_linear_attention(*parts, state=state, resume=_i32([again] * n), y=y,
                                      offsets=_i32(np.cumsum([begin] + lengths)))
        assert (y[:begin] == 3).all() and (y[begin + total:] == 3).all()
        out.append((y[begin:begin + total], state))
    assert out[0][0].isfinite().all() and out[0][1].isfinite().all()
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    assert torch.equal(out[1][1][n:], start[n:])


def test_products_of_fp32_numbers_keep_their_bits():
    # Sequences of one token, one key and one value: y is (q k) v and the state k v.  Of a product of
    # three parts each 2^-24 is left out, and its last sum is cut off below 2^-23 of itself: 1.5 x 2^-23
    # and a little for each product.
    g = gen(2)
    n = 300
    q, k, v = (1.0 + uniform(g, n, 1, 1) for _ in range(3))
    for m in (q, k, v):
        m[:4, 0, 0] = torch.tensor([1.0078124, 1.0039062, 1.9960936, 1.00390612], device="cuda")
    state = torch.zeros(n, 1, 1, 1, device="cuda")
    y = binding.lstm_linear_attention(q, k, v, torch.zeros(1, device="cuda"), sequences=n, state=state)
    for got, ref, off in ((y, f64(q) * f64(k) * f64(v), 2.0 ** -21), (state[..., 0], f64(k) * f64(v), 2.0 ** -22)):
        assert (np.abs(f64(got) - ref) <= off * ref).all(), np.max(np.abs(f64(got) / ref - 1))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("keys,values", [(64, 64), (128, 128), (40, 200)])
@pytest.mark.parametrize("lengths", [[64], [300, 17], [3000]])
def test_states_keep_their_bits(dtype, keys, values, lengths):
    # Of the norm: a weight's exponential is off by 2^-22, and the decays between chunks, of e^-3 and
    # less, add a twentieth to that; the tensor cores' sums are cut off below 2^-23 of themselves at
    # the four blocks of 16 tokens that make a chunk's, 2^-21; the sum with the state is rounded once
    # (2^-24), and a product loses 2^-24: below 2^-20.  (Two parts of w v instead of three would
    # leave 2^-17 of a term.)
    tokens, n = sum(lengths), len(lengths)
    q, k, v = _inputs(dtype, tokens, 2, keys, values)
    d = torch.full((tokens, 2), -0.05, device="cuda") * (0.9 + 0.2 * uniform(gen(4), tokens, 2))
    state = torch.zeros(n, 2, keys, values, device="cuda")
    offsets = np.concatenate([[0], np.cumsum(lengths)])
    binding.lstm_linear_attention(q, k, v, d, offsets=_i32(offsets), state=state)
    k, v, d = (x.double() for x in (k, v, d))
    for s in range(n):
        a, b = offsets[s], offsets[s + 1]
        w = torch.exp(d[a:b].flip(0).cumsum(0).flip(0) - d[a:b])
        ref = torch.einsum("th,thk,thv->hkv", w, k[a:b], v[a:b])
        assert (state[s].double() - ref).norm() <= 2.0 ** -20 * ref.norm()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("keys,values", [(64, 64), (128, 128), (40, 200)])
@pytest.mark.parametrize("lengths", [[200], [1000, 300]])
def test_outputs_of_16_bits_are_off_by_their_own_rounding(dtype, keys, values, lengths):
    # P and S are rounded to two parts of bf16, 2^-17 of themselves, and to either side: of the norm
    # some 2^-16, for which 2^-12 leaves room, where one part each would add 2^-10.  The rounding's own
    # norm is known from these outputs' to a few hundredths.
    tokens = sum(lengths)
    q, k, v = _inputs(dtype, tokens, 2, keys, values)
    d = _decays(gen(4), "each", tokens, 2)
    state = normal(gen(5), len(lengths), 2, keys, values)
    start = f64(state)
    offsets = np.concatenate([[0], np.cumsum(lengths)])
    got = f64(binding.lstm_linear_attention(q, k, v, d, offsets=_i32(offsets), state=state,
                                            resume=_i32([1] * len(lengths)), scale=0.125))
    ref = oracle.linear_attention(f64(q), f64(k), f64(v), f64(d), 0.125,
                                  spans(tokens, len(lengths), offsets), dtype, start, None,
                                  [1] * len(lengths))[0]
    rounding = np.linalg.norm(f64(torch.tensor(ref).to(DTYPES[dtype])) - ref)
    assert np.linalg.norm(got - ref) <= 1.05 * rounding + 2.0 ** -12 * np.linalg.norm(ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("count", [3, 126, 127, 128, 129])
def test_as_many_unequal_sequences_as_blocks_put_in_order(dtype, count):
    # (no spans: there are blocks enough; some are equal, some empty)
    lengths = [(i * 53) % 70 if i % 4 else 33 for i in range(count)]
    assert binding.lstm_linear_attention_workspace(sum(lengths), 208, 8, 8, count, False) == 0
    _check(dtype, lengths, 208 if count < 100 else 6, 8, 8, pool=count, resume=[i % 2 for i in range(count)])


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_states_next_to_the_largest_number(dtype):
    # 3.4e38 is beyond bf16's largest number; a query of 2^-14 brings it back
    state = torch.full((1, 1, 16, 16), 3.4e38, device="cuda")
    q, k, v = (torch.zeros(3, 1, 16, dtype=DTYPES[dtype], device="cuda") for _ in range(3))
    q[:, :, 5] = 2.0 ** -14
    y = binding.lstm_linear_attention(q, k, v, torch.zeros(1, device="cuda"), state=state, resume=_i32([1]),
                                      scale=2.0 ** -100)
    assert (state == 3.4e38).all()
    # (no number of these types is near the type's end: the scale brings it to 2^14)
    ref = float(torch.tensor(3.4e38).double()) * 2.0 ** -114
    off = 2.0 ** -15 + torch.finfo(DTYPES[dtype]).eps / 2
    assert ((y.double() - ref).abs() <= off * ref).all()


def _far(rows, *sizes, dtype):
    """[rows, *sizes] whose last rows lie beyond 2^31 elements."""
    stride = (1 << 31) // rows + 1024
    stride -= stride % 8
    at = torch.empty(rows * stride, dtype=dtype, device="cuda").as_strided(
        (rows, *sizes), (stride, *([sizes[1], 1] if len(sizes) > 1 else [1])))
    assert (rows - 1) * stride > 1 << 31
    return at


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_beyond_32_bits_of_elements(dtype):
    tokens, t = 70001, DTYPES[dtype]
    m = _inputs(dtype, tokens, 2, 16, 24)
    d = _decays(gen(2), "each", tokens, 2)
    offsets = _i32([0, 1000, 35000, tokens])
    ref = binding.lstm_linear_attention(*m, d, offsets=offsets)
    y = _far(tokens, 2, 24, dtype=t)
    assert torch.equal(binding.lstm_linear_attention(*m, d, offsets=offsets, y=y), ref)
    del y
    far = [_far(tokens, *x.shape[1:], dtype=t).copy_(x) for x in m[:2]]
    assert torch.equal(binding.lstm_linear_attention(*far, m[2], d, offsets=offsets), ref)
