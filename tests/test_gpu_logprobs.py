"""Token log probabilities, entropy and top alternatives against the float64
definition: row lengths on both sides of every split, types, alignments, ties,
masked logits, rows with nothing left, NaN and infinities, and refusals."""
import numpy as np
import pytest
import torch

from bidirectional_lstm_stack_gb300 import binding
from oracle import ops as oracle
from ops_util import DTYPES, assert_close, f64, gen, normal, slice_of, uniform

pytestmark = pytest.mark.gpu


def _check(logits, tokens, top):
    logp, h, top_logp, top_ids = binding.lstm_token_logprobs(logits, tokens, top=top)
    ref, ref_h, ids, ids_logp, bound = oracle.token_logprobs(
        f64(logits), None if tokens is None else tokens.cpu().numpy(), top)
    # l = d - ln s: d's rounding and the difference's
    own = lambda v: np.where(np.isfinite(v), 3 * oracle.U32 * (np.abs(v) + 16), 0.0)
    if tokens is not None:
        assert_close(logp, ref, bound[:, 0] + own(ref), "f32", "logp")
    assert_close(h, ref_h, bound[:, 1], "f32", "entropy")
    if top:
        np.testing.assert_array_equal(top_ids.cpu().numpy(), ids)
        assert_close(top_logp, ids_logp, bound[:, :1] + own(ids_logp), "f32", "top")


def _tokens(g, rows, vocab):
    return (uniform(g, rows) * vocab).long().clamp_(max=vocab - 1)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 31, 32, 33, 100, 257, 512, 513, 2048, 2049, 4096, 4097, 5000, 16384,
                                   50021])
def test_row_lengths(dtype, vocab):
    g = gen(vocab)
    logits = normal(g, 5, vocab, scale=3.0, dtype=DTYPES[dtype])
    _check(logits, _tokens(g, 5, vocab), min(vocab, 20))


@pytest.mark.parametrize("rows,vocab", [(1, 131072), (2, 100003), (700, 40000)])
def test_long_rows(rows, vocab):
    g = gen(rows)
    logits = normal(g, rows, vocab, scale=2.0, dtype=torch.bfloat16)
    got = binding.lstm_token_logprobs(logits, _tokens(g, rows, vocab), top=32)
    take = slice(0, 4)
    ref, h, ids, ids_logp, bound = oracle.token_logprobs(
        f64(logits[take]), _tokens(gen(0), rows, vocab)[take].cpu().numpy() * 0, 32)
    np.testing.assert_array_equal(got[3][take].cpu().numpy(), ids)
    assert_close(got[2][take], ids_logp, bound[:, :1] + 3 * oracle.U32 * (np.abs(ids_logp) + 16), "f32")
    assert_close(got[1][take], h, bound[:, 1], "f32")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,vocab", [(1, 131072), (2, 100003), (70, 40000), (5, 300007), (160, 20000)])
@pytest.mark.parametrize("top", [0, 32])
def test_all_outputs_of_long_rows(dtype, rows, vocab, top):
    """Rows shared by one to eight blocks, tokens in the part of each."""
    g = gen(vocab)
    logits = normal(g, rows, vocab, scale=2.0, dtype=DTYPES[dtype])
    for part in range(8 if rows <= 2 else 1):
        tokens = (_tokens(g, rows, vocab) + part * vocab // 8) % vocab
        tokens[0] = [0, vocab - 1, vocab // 2, vocab // 8][part % 4]
        _check(logits, tokens, top)


@pytest.mark.parametrize("rows", [1, 33, 2000])
def test_many_rows_of_few_classes(rows):
    g = gen(rows)
    _check(normal(g, rows, 7, scale=4.0), _tokens(g, rows, 7), 3)


def test_as_many_rows_as_there_can_be():
    rows = (1 << 31) - 1
    logits = torch.zeros(rows, 1, device="cuda", dtype=torch.bfloat16)
    entropy = torch.full((rows,), 7.0, device="cuda")
    st = binding.load().lstm_token_logprobs(logits.data_ptr(), 1, binding.LSTM_BF16, rows, 1, None,
                                            None, entropy.data_ptr(), 0, None, None,
                                            torch.cuda.current_stream().cuda_stream)
    assert st == binding.LSTM_OK, binding.lstm_stack_last_error()
    assert not entropy.any()


@pytest.mark.parametrize("top", [0, 1, 2, 31, 32])
@pytest.mark.parametrize("vocab", [32, 1000, 30000])
def test_numbers_of_alternatives(top, vocab):
    g = gen(top)
    _check(normal(g, 3, vocab, dtype=torch.float16), _tokens(g, 3, vocab), top)


@pytest.mark.parametrize("vocab", [8, 20, 500, 9001, 70000])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "two values", "signed zeros"])
def test_ties_and_orders(vocab, kind):
    n = torch.arange(vocab, device="cuda", dtype=torch.float32)
    row = {"equal": torch.full_like(n, 1.5), "rising": n * 0.25, "falling": -n * 0.25,
           "two values": (n % 3 == 1).float(), "signed zeros": torch.where(n % 2 == 0, 0.0, -0.0)}[kind]
    _check(torch.stack([row, row - 3]), torch.tensor([0, vocab - 1], device="cuda"), min(vocab, 25))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("vocab", [7, 30, 300, 40000])
def test_masks(dtype, vocab):
    g = gen(vocab)
    low = torch.finfo(DTYPES[dtype]).min
    logits = normal(g, 8, vocab, dtype=DTYPES[dtype])
    logits[0] = float("-inf")                     # nothing left
    logits[1] = low                               # everything at the type's lowest value
    logits[2, :-1] = float("-inf")                # one left
    logits[3, 1:] = low
    logits[4, ::2] = float("-inf")
    logits[5, vocab // 2] = float("nan")
    logits[6, vocab // 3] = float("inf")
    logits[7, 0] = torch.finfo(DTYPES[dtype]).max
    _check(logits, _tokens(g, 8, vocab), min(vocab, 6))


def test_lowest_value_beside_larger_ones_of_its_size():
    # differences that leave fp32's range, and ones near its end
    row = torch.full((2, 5000), -3.4e38, device="cuda")
    row[0, 17] = -1e35
    row[1, 4000] = 3e38
    _check(row, torch.tensor([17, 4000], device="cuda"), 3)


def test_tokens_outside_the_row():
    g = gen(1)
    logits = normal(g, 4, 50)
    logp = binding.lstm_token_logprobs(logits, torch.tensor([-1, 49, 50, -100], device="cuda"))[0]
    got = f64(logp)
    assert got[0] == 0 and got[3] == 0 and np.isnan(got[2]) and np.isfinite(got[1])


@pytest.mark.parametrize("pad", [1, 2, 3, 8])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_any_alignment(pad, dtype):
    g = gen(pad)
    logits = slice_of(normal(g, 6, 3001, dtype=DTYPES[dtype]), pad, 5)
    _check(logits, _tokens(g, 6, 3001), 10)


def test_parts_that_are_not_asked_for():
    logits = normal(gen(2), 4, 500)
    full = binding.lstm_token_logprobs(logits, torch.zeros(4, dtype=torch.int64, device="cuda"), top=5)
    assert binding.lstm_token_logprobs(logits, entropy=False) == (None, None, None, None)
    part = binding.lstm_token_logprobs(logits, entropy=False, top=5)
    assert part[0] is None and part[1] is None
    assert torch.equal(part[2], full[2]) and torch.equal(part[3], full[3])


def test_no_rows():
    out = binding.lstm_token_logprobs(torch.zeros(0, 9, device="cuda"), top=2)
    assert out[1].shape == (0,) and out[3].shape == (0, 2)


def test_the_same_bits_every_time():
    logits = normal(gen(3), 3, 60000, dtype=torch.bfloat16)
    a = binding.lstm_token_logprobs(logits, torch.zeros(3, dtype=torch.int64, device="cuda"), top=32)
    for _ in range(3):
        b = binding.lstm_token_logprobs(logits, torch.zeros(3, dtype=torch.int64, device="cuda"), top=32)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_behind_the_heads():
    # log-probabilities are logits too: the classes' own come back
    g = gen(7)
    logp = torch.log_softmax(normal(g, 600, 7, scale=2.0), -1)
    got, h, top_logp, ids = binding.lstm_token_logprobs(logp, logp.argmax(-1), top=7)
    assert torch.equal(ids[:, 0], logp.argmax(-1))
    torch.testing.assert_close(top_logp.exp().sum(1), torch.ones(600, device="cuda"), rtol=1e-5, atol=0)
    torch.testing.assert_close(got, logp.amax(-1), rtol=1e-5, atol=1e-6)


def test_very_many_alternatives_are_refused_before_memory_is_asked_for():
    with pytest.raises(binding.LSTMError) as e:
        binding.lstm_token_logprobs(torch.zeros(64, 100, device="cuda"), top=(1 << 31) - 1)
    assert e.value.code == binding.LSTM_E_INVALID


def test_refusals():
    x = torch.zeros(4, 10, device="cuda")
    run = binding.lstm_token_logprobs
    for top in (-1, 11, 33):
        with pytest.raises(binding.LSTMError) as e:
            run(x if top != 33 else torch.zeros(4, 100, device="cuda"), top=top)
        assert e.value.code == binding.LSTM_E_INVALID
    for bad in (lambda: run(x, torch.zeros(4, dtype=torch.int32, device="cuda")),
                lambda: run(x, torch.zeros(5, dtype=torch.int64, device="cuda")),
                lambda: run(x.double()), lambda: run(x.t().contiguous().t())):
        with pytest.raises(ValueError):
            bad()
