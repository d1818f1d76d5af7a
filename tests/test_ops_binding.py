"""What binding.py's functions of include/lstm_ops.h refuse before the library
is called, and how they take their arguments."""
import inspect
import sys
import threading

import pytest
import torch

from bidirectional_lstm_stack_gb300 import binding
from bidirectional_lstm_stack_gb300 import build as build_mod


@pytest.fixture(scope="module", autouse=True)
def built():
    build_mod.build()


def _calls(m):
    """Each function with m as the matrix that gives the call its sizes."""
    v = torch.zeros(8)
    return [lambda: binding.lstm_causal_conv(m, torch.zeros(8, 4)),
            lambda: binding.lstm_causal_conv_step(m, torch.zeros(8, 4), None, torch.zeros(2, 3, 8)),
            lambda: binding.lstm_selective_scan(m, m, torch.zeros(8, 16), m, m),
            lambda: binding.lstm_selective_scan_step(m, m, torch.zeros(8, 16), m, m,
                                                     torch.zeros(2, 8, 16)),
            lambda: binding.lstm_residual_rms_norm(m, v, 1e-5),
            lambda: binding.lstm_token_logprobs(m)]


@pytest.mark.parametrize("function", range(6))
@pytest.mark.parametrize("bad,error", [(torch.zeros(2, 8), ValueError), (torch.zeros(8), ValueError),
                                       (torch.zeros(()), ValueError), (None, TypeError),
                                       ([[0.0]], TypeError), (torch.zeros(1, 2, 8), ValueError)])
def test_a_matrix_on_the_host_or_no_matrix_is_refused(function, bad, error):
    with pytest.raises(error):
        _calls(bad)[function]()


def test_names_and_defaults():
    for name in ("lstm_causal_conv", "lstm_causal_conv_step", "lstm_selective_scan",
                 "lstm_selective_scan_step", "lstm_residual_rms_norm", "lstm_token_logprobs"):
        f = getattr(binding, name)
        assert "stream" in inspect.signature(f).parameters and f.__doc__
        with pytest.raises(TypeError):
            f()


def test_a_module_that_is_not_built_is_missing(monkeypatch):
    monkeypatch.setattr(binding, "_ops", None)
    monkeypatch.delattr(sys.modules["bidirectional_lstm_stack_gb300"], "_native", raising=False)
    monkeypatch.setitem(sys.modules, "bidirectional_lstm_stack_gb300._native", None)
    with pytest.raises(binding.LibraryMissing):
        binding.lstm_token_logprobs(torch.zeros(2, 8))


@pytest.mark.parametrize("function", range(6))
def test_a_matrix_that_requires_a_gradient_is_refused(function):
    m = torch.zeros(2, 8, requires_grad=True)
    with pytest.raises(ValueError, match="requires a gradient"):
        _calls(m)[function]()
    with pytest.raises(ValueError, match="requires a gradient"):  # of a graph's inner tensors too
        _calls(m * 2)[function]()
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):  # (nothing else is wrong)
        _calls(m)[function]()


@pytest.mark.gpu
def test_any_tensor_that_requires_a_gradient_is_refused():
    ones = lambda *s: torch.ones(*s, device="cuda")
    x, n = ones(2, 8), 4
    calls = [
        (binding.lstm_causal_conv, [x, ones(8, 4)],
         dict(bias=ones(8), state=ones(2, 3, 8), sequences=2, y=ones(2, 8))),
        (binding.lstm_causal_conv_step, [x, ones(8, 4), ones(8), ones(2, 3, 8)], dict(y=ones(2, 8))),
        (binding.lstm_selective_scan, [x, x, -ones(8, n), ones(2, n), ones(2, n)],
         dict(skip=ones(8), z=x, dt_bias=ones(8), state=ones(2, 8, n), sequences=2, y=ones(2, 8))),
        (binding.lstm_selective_scan_step, [x, x, -ones(8, n), ones(2, n), ones(2, n), ones(2, 8, n)],
         dict(skip=ones(8), z=x, dt_bias=ones(8), y=ones(2, 8))),
        (binding.lstm_residual_rms_norm, [x, ones(8), 1e-5],
         dict(residual=x, residual_out=ones(2, 8), y=ones(2, 8))),
        (binding.lstm_residual_rms_norm, [x, ones(8), 1e-5], dict(quantize=True, scales=ones(2, 1))),
        (binding.lstm_token_logprobs, [x], {})]
    for call, args, more in calls:
        expected = call(*[a.clone() if torch.is_tensor(a) else a for a in args],
                        **{k: v.clone() if torch.is_tensor(v) else v for k, v in more.items()})
        for k, v in list(enumerate(args)) + list(more.items()):
            if not torch.is_tensor(v):
                continue
            other_args, other = list(args), dict(more)
            (other_args if isinstance(k, int) else other)[k] = v.clone().requires_grad_()
            with pytest.raises(ValueError, match="requires a gradient"):
                call(*other_args, **other)
        with torch.no_grad():
            got = call(*[a.clone().requires_grad_() if torch.is_tensor(a) else a for a in args],
                       **{k: v.clone() if torch.is_tensor(v) else v for k, v in more.items()})
        first = lambda r: r if torch.is_tensor(r) else r[0] if r[0] is not None else r[1]
        assert torch.equal(first(got).float(), first(expected).float())


@pytest.mark.gpu
def test_arguments_that_are_wrong_beside_a_good_matrix():
    x, w, v = torch.zeros(4, 8).cuda(), torch.zeros(8, 4).cuda(), torch.ones(8).cuda()
    conv, norm, logp = (binding.lstm_causal_conv, binding.lstm_residual_rms_norm,
                        binding.lstm_token_logprobs)
    for call, error in [(lambda: conv(x, None), TypeError),
                        (lambda: conv(x, torch.tensor(1.0).cuda()), ValueError),
                        (lambda: conv(x, w.cpu()), ValueError),
                        (lambda: conv(x, w, bias=[0.0] * 8), TypeError),
                        (lambda: conv(x, w, sequences="1"), TypeError),
                        (lambda: conv(x, w, sequences=1 << 40), ValueError),
                        (lambda: conv(x, w, stream="0"), AttributeError),
                        (lambda: conv(x, w, state=torch.tensor(0.0).cuda()), ValueError),
                        (lambda: conv(x, w, offsets=torch.zeros(0, dtype=torch.int32).cuda()),
                         binding.LSTMError),
                        (lambda: conv(x.double(), w), ValueError),
                        (lambda: conv(x, w, y=torch.zeros(4, 8)), ValueError),
                        (lambda: norm(x, v, None), TypeError),
                        (lambda: norm(x, v, "1"), TypeError),
                        (lambda: norm(x, v, 1e-5, group=1 << 40, quantize=True), ValueError),
                        (lambda: norm(x, v, 1e-5, residual=x.half()), ValueError),
                        (lambda: logp(x, torch.zeros(4).cuda()), ValueError),
                        (lambda: logp(x, top=1 << 40), ValueError)]:
        with pytest.raises(error):
            call()
    y, scales, out = norm(x, v, 1)
    assert scales is None and out is None and y.shape == x.shape
    assert all(t is None for t in logp(x, entropy=False)[2:])


@pytest.mark.gpu
def test_given_outputs_are_what_is_returned():
    x, w, v = torch.randn(4, 8).cuda(), torch.randn(8, 4).cuda(), torch.ones(8).cuda()
    y = torch.empty_like(x)
    got = binding.lstm_causal_conv(x, w, y=y)
    assert got.data_ptr() == y.data_ptr() and torch.equal(y, binding.lstm_causal_conv(x, w))
    r = torch.randn(4, 8).cuda()
    expected = r + x
    assert binding.lstm_residual_rms_norm(x, v, 1e-5, residual=r,
                                          residual_out=r)[2].data_ptr() == r.data_ptr()
    assert torch.equal(r, expected)


def _overwriting_calls():
    ones = lambda *s: torch.ones(*s, device="cuda")
    x, n = ones(2, 8), 4
    scan = (x, x, -ones(8, n), ones(2, n), ones(2, n))
    y, state, scan_state = ones(2, 8), ones(2, 3, 8), ones(2, 8, n)
    residual, scales, q = ones(2, 8), ones(2, 1), ones(2, 8).to(torch.float8_e4m3fn)
    return [(lambda: binding.lstm_causal_conv(x, ones(8, 4), state=state, sequences=2, y=y), (state, y)),
            (lambda: binding.lstm_causal_conv_step(x, ones(8, 4), None, state, y=y), (state, y)),
            (lambda: binding.lstm_selective_scan(*scan, state=scan_state, sequences=2, y=y),
             (scan_state, y)),
            (lambda: binding.lstm_selective_scan_step(*scan, scan_state, y=y), (scan_state, y)),
            (lambda: binding.lstm_residual_rms_norm(x, ones(8), 1e-5, residual=residual,
                                                    residual_out=residual, y=y), (residual, y)),
            (lambda: binding.lstm_residual_rms_norm(x, ones(8), 1e-5, quantize=True, y=q,
                                                    scales=scales), (q, scales))], x


@pytest.mark.gpu
def test_overwritten_tensors_count_it():
    """What autograd checks tensors that it has saved by."""
    calls, x = _overwriting_calls()
    for call, tensors in calls:
        before = [t._version for t in tensors]
        call()
        assert all(t._version > b for t, b in zip(tensors, before)) and x._version == 0
    w = torch.ones(2, 8, device="cuda", requires_grad=True)
    y = torch.ones(2, 8, device="cuda")
    loss = (w * y).sum()  # saves y
    binding.lstm_causal_conv(x, torch.ones(8, 4, device="cuda"), y=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.gpu
def test_tensors_of_inference_mode():
    with torch.inference_mode():
        for call, _ in _overwriting_calls()[0]:
            call()
        inside = _overwriting_calls()[0]
    for call, _ in inside:
        call()


@pytest.mark.gpu
def test_calls_of_two_threads():
    x, w = torch.randn(256, 64).cuda(), torch.randn(64, 4).cuda()
    expected = binding.lstm_causal_conv(x, w)
    torch.cuda.synchronize()
    wrong = []

    def work():
        stream = torch.cuda.Stream()
        for _ in range(200):
            y = binding.lstm_causal_conv(x, w, stream=stream)
        stream.synchronize()
        if not torch.equal(y, expected):
            wrong.append(y)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.gpu
def test_outputs_do_not_leak():
    x, w = torch.randn(256, 64).cuda(), torch.randn(64, 4).cuda()
    v = torch.ones(64).cuda()

    def work():
        binding.lstm_causal_conv(x, w)
        binding.lstm_residual_rms_norm(x, v, 1e-5, residual=x, quantize=True)
        binding.lstm_token_logprobs(x, top=3)
        with pytest.raises(binding.LSTMError):
            binding.lstm_causal_conv(x, w, sequences=3)  # (256 rows are no three equal prompts)

    work()
    before = torch.cuda.memory_allocated()
    refs = sys.getrefcount(x), sys.getrefcount(None)
    for _ in range(50):
        work()
    assert torch.cuda.memory_allocated() == before
    assert sys.getrefcount(x) == refs[0] and abs(sys.getrefcount(None) - refs[1]) < 50
