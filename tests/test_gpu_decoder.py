"""The state-space decoder example: the operators together.  Tokens decoded one
at a time from the states, prompts continued from them, and prompts packed
beside others give what one pass over the whole sequence gives."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
from state_space_decoder import Decoder, Sizes  # noqa: E402

pytestmark = pytest.mark.gpu


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _close(a, b):
    # bf16 activations are rounded at the same places either way; what differs
    # is the order of fp32 sums (a split or a whole scan, matrix products of
    # other heights), which now and then moves a rounding, of 2^-8, and an 8-bit
    # one, of 2^-4, in some of the 4 layers' 256 columns
    assert a.shape == b.shape
    assert torch.isfinite(a).all()
    rel = (a.float() - b.float()).norm() / b.float().norm()
    assert rel < 2.0 ** -5, float(rel)


@pytest.fixture(scope="module")
def decoder():
    return Decoder(slots=9)


def _tokens(n, seed=1, vocab=Sizes.vocab):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(vocab, (n,), generator=g, device="cuda")


def test_steps_equal_the_whole_prompt(decoder):
    t = _tokens(40)
    whole = decoder.prompts(t, _i32(0, 40), _i32(2))
    parts = [decoder.prompts(t[:25], _i32(0, 25), _i32(4))]
    parts += [decoder.step(t[k:k + 1], _i32(4)) for k in range(25, 40)]
    _close(torch.cat(parts), whole)


def test_continued_prompts_equal_whole_ones(decoder):
    t = _tokens(600, seed=2)
    whole = decoder.prompts(t, _i32(0, 600), _i32(1))
    a = decoder.prompts(t[:333], _i32(0, 333), _i32(3))
    b = decoder.prompts(t[333:], _i32(0, 267), _i32(3), resume=_i32(1))
    _close(torch.cat([a, b]), whole)


def test_packed_prompts_equal_single_ones(decoder):
    lengths = [70, 1, 200, 33]
    t = _tokens(sum(lengths), seed=3)
    ends = [0, 70, 71, 271, 304]
    packed = decoder.prompts(t, _i32(*ends), _i32(0, 8, 5, 6))
    alone = [decoder.prompts(t[a:b], _i32(0, b - a), _i32(7)) for a, b in zip(ends, ends[1:])]
    _close(packed, torch.cat(alone))


def test_generation_is_reproducible_and_ranks(decoder):
    t = _tokens(60, seed=4)
    args = (t, _i32(0, 10, 60), _i32(6, 2), 5)
    one = decoder.generate(*args)
    two = decoder.generate(*args)
    for a, b in zip(one, two):
        assert torch.equal(a, b)
    tokens, logp, entropy, alternatives = one
    assert tokens.shape == (5, 2) and alternatives.shape == (5, 2, 5)
    assert torch.equal(tokens, alternatives[:, :, 0])
    assert (logp <= 0).all() and (entropy >= 0).all()
