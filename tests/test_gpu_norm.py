"""Residual addition and RMS norm, in the input's type and in 8 bits, against
the float64 definition."""
import numpy as np
import pytest
import torch

from bidirectional_lstm_stack_gb300 import binding
from oracle import ops as oracle
from ops_util import DTYPES, ROUND, assert_close, at_element, f64, gen, normal, slice_of, uniform

pytestmark = pytest.mark.gpu

# the mean of squares is summed in lanes, warps and a block (at most 32 terms
# in a row, then ten joins), and the square root, two products and the
# residual's sum add a few roundings more
NORM = 64 * oracle.U32


def _inputs(dtype, rows, cols, residual, strided=False, seed=1):
    g = gen(seed)
    x = normal(g, rows, cols, dtype=DTYPES[dtype])
    res = normal(g, rows, cols, scale=3.0, dtype=DTYPES[dtype]) if residual else None
    if strided:
        x, res = slice_of(x, 1, 4), None if res is None else slice_of(res, 8, 8)
    return x, res, 0.5 + uniform(g, cols)


def _check(dtype, rows, cols, residual=True, quantize=False, group=0, strided=False, eps=1e-5):
    x, res, weight = _inputs(dtype, rows, cols, residual, strided)
    y, scales, v = binding.lstm_residual_rms_norm(x, weight, eps, residual=res, quantize=quantize,
                                                  group=group)
    ref, ref_v = oracle.residual_rms_norm(f64(x), f64(res), f64(weight), eps)
    # x + residual cancels: the norm's error is relative to what was added
    size = np.abs(f64(x)) + (0 if res is None else np.abs(f64(res)))
    bound = NORM * np.abs(ref) + oracle.U32 * size * np.abs(f64(weight)) / np.sqrt(
        (ref_v ** 2).mean(1, keepdims=True) + eps)
    if residual:
        assert_close(v, ref_v, oracle.U32 * np.abs(ref_v), dtype, "residual")
    else:
        assert v is None
    if not quantize:
        assert scales is None
        assert_close(y, ref, bound, dtype, "y")
        return
    assert y.dtype == torch.float8_e4m3fn
    s_ref = oracle.group_scales(ref, group)
    np.testing.assert_allclose(f64(scales), s_ref, rtol=2 * NORM, atol=0)
    wide = np.repeat(f64(scales), group or cols, axis=1)[:, :cols]
    got = f64(y.float()) * wide
    # 3 mantissa bits: half a unit is 2^-4 of the value, 2^-10 below the least normal
    tol = np.abs(ref) * 2.0 ** -4 + wide * 2.0 ** -10 + 2 * bound
    assert (np.abs(got - ref) <= tol).all()
    # the largest of every group uses the whole range
    tops = np.stack([np.abs(f64(y.float()))[:, k:k + (group or cols)].max(1)
                     for k in range(0, cols, group or cols)], 1)
    assert (tops == 448.0).all()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("cols", [1, 2, 33, 60, 256, 1000, 1029, 2048, 4104, 8192])
def test_norm(dtype, cols):
    _check(dtype, 5, cols)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("cols", [16384, 16385, 32768])
def test_wide_rows(dtype, cols):
    _check(dtype, 2, cols)
    _check(dtype, 2, cols, quantize=True, group=128)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("cols", [1, 40, 128, 200, 1111, 4096])
def test_eight_bits(dtype, group, cols):
    _check(dtype, 7, cols, quantize=True, group=group)


@pytest.mark.parametrize("rows", [1, 3, 500])
def test_rows(rows):
    _check("bf16", rows, 512, quantize=True, group=128)
    _check("f32", rows, 100, residual=False)


@pytest.mark.parametrize("quantize", [False, True])
def test_rows_of_wider_matrices(quantize):
    _check("bf16", 9, 256, strided=True, quantize=quantize)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("offset", [1, 2, 3, 4])
@pytest.mark.parametrize("quantize", [False, True])
def test_weights_at_any_element(dtype, offset, quantize):
    x, res, weight = _inputs(dtype, 5, 264, True)
    at = at_element(weight, offset)
    assert at.data_ptr() % 16 == 4 * offset % 16
    run = lambda w: binding.lstm_residual_rms_norm(x, w, 1e-5, residual=res, quantize=quantize, group=64)
    y, scales, v = run(at)
    ref, ref_v = oracle.residual_rms_norm(f64(x), f64(res), f64(weight), 1e-5)
    size = (np.abs(f64(x)) + np.abs(f64(res))) * np.abs(f64(weight)) / np.sqrt(
        (ref_v ** 2).mean(1, keepdims=True) + 1e-5)
    bound = NORM * np.abs(ref) + oracle.U32 * size
    assert torch.equal(v, run(weight)[2])
    if not quantize:
        assert_close(y, ref, bound, dtype, "y")
        return
    wide = np.repeat(f64(scales), 64, axis=1)[:, :264]
    got = f64(y.float()) * wide
    assert (np.abs(got - ref) <= np.abs(ref) * 2.0 ** -4 + wide * 2.0 ** -10 + 2 * bound).all()


def test_residual_in_place():
    x, res, weight = _inputs("bf16", 6, 264, True)
    y1, _, v1 = binding.lstm_residual_rms_norm(x, weight, 1e-6, residual=res)
    y2, _, v2 = binding.lstm_residual_rms_norm(x, weight, 1e-6, residual=res, residual_out=res)
    assert v2 is res
    assert torch.equal(v1, v2) and torch.equal(y1, y2)


def test_zero_rows_and_zero_values():
    weight = torch.ones(256, device="cuda")
    y, scales, _ = binding.lstm_residual_rms_norm(torch.zeros(0, 256, device="cuda"), weight, 1e-6,
                                                  quantize=True, group=64)
    assert y.shape == (0, 256) and scales.shape == (0, 4)
    x = torch.zeros(2, 256, device="cuda")
    x[1, 70] = 5.0
    y, scales, _ = binding.lstm_residual_rms_norm(x, weight, 1e-6, quantize=True, group=64)
    assert (f64(y.float())[0] == 0).all() and f64(y.float())[1, 70] == 448.0
    # groups without a value keep the scale 1
    np.testing.assert_array_equal(f64(scales)[0], 1.0)
    np.testing.assert_array_equal(f64(scales)[1, [0, 2, 3]], 1.0)
    y, _, _ = binding.lstm_residual_rms_norm(torch.zeros(1, 256, device="cuda"), weight, 1e-6)
    assert (y == 0).all()


def _e4m3(v):
    """fp32 values rounded to the nearest e4m3 value (on the host)."""
    return torch.from_numpy(v).to(torch.float8_e4m3fn).float().numpy()


@pytest.mark.parametrize("cols", [32, 60, 512, 1111, 4096, 16384, 20001])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("size", [1.0, 1e-36, 1e-30, 1e12, 1e30])
def test_eight_bits_are_the_quotients_own(cols, group, size):
    """Scales and 8-bit values bit for bit: fp32's quotients of the norm that the same kernel
    gives for fp32 output.  The residual's sizes make the norm's sizes differ widely in a row."""
    g = gen(cols)
    x = normal(g, 40, cols) * torch.exp2(-12 * uniform(g, 40, cols))
    weight = (0.5 + uniform(g, cols)) * size
    x[3] = 0.0
    x[4, ::2] = 0.0
    x[5] = torch.where(x[5] < 0, -1.0, 1.0)
    n = binding.lstm_residual_rms_norm(x, weight, 1e-5)[0].cpu().numpy()
    y, scales, _ = binding.lstm_residual_rms_norm(x, weight, 1e-5, quantize=True, group=group)
    step = group or cols
    top = np.stack([np.abs(n[:, k:k + step]).max(1) for k in range(0, cols, step)], 1)
    expected = np.where(top > 0, np.maximum(top / np.float32(448), np.float32(2.0 ** -126)),
                        np.float32(1))
    assert expected.dtype == np.float32
    np.testing.assert_array_equal(scales.cpu().numpy(), expected)
    wide = np.repeat(expected, step, 1)[:, :cols]
    np.testing.assert_array_equal(y.float().cpu().numpy(), _e4m3(n / wide))


@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("cols", [256, 255])
def test_eight_bits_of_an_infinite_norm(cols, group):
    weight = torch.ones(cols, device="cuda")
    weight[40] = float("inf")
    y, scales, _ = binding.lstm_residual_rms_norm(torch.ones(2, cols, device="cuda"), weight, 1e-6,
                                                  quantize=True, group=group)
    y, scales = f64(y.float()), f64(scales)
    # beside it in its group: a quotient by an infinity
    ours = np.arange(cols) // (group or cols) == 40 // (group or cols)
    assert np.isinf(scales[:, 40 // (group or cols)]).all() and np.isfinite(scales).sum() == scales.size - 2
    assert np.isnan(y[:, 40]).all() and int(np.isnan(y).sum()) == 2
    y[:, 40] = 0.0
    assert (y[:, ours] == 0.0).all() and (y[:, ~ours] == 448.0).all()


def test_tiny_and_huge_values():
    weight = torch.ones(64, device="cuda")
    # the mean of squares underflows to zero: eps alone divides
    x = torch.full((1, 64), 1e-30, device="cuda")
    y, scales, _ = binding.lstm_residual_rms_norm(x, weight, 1e-6, quantize=True)
    got = f64(y.float()) * f64(scales)
    np.testing.assert_allclose(got, 1e-30 / np.sqrt(1e-6), rtol=2.0 ** -4)
    x = torch.full((1, 64), 1e15, device="cuda")
    y, _, _ = binding.lstm_residual_rms_norm(x, weight, 1e-6)
    np.testing.assert_allclose(f64(y), 1.0, rtol=NORM)


def test_rows_of_infinities_and_zeros_beside_them():
    x = torch.ones(4, 300, device="cuda")
    x[1, 7], x[2] = float("inf"), 0.0
    y = f64(binding.lstm_residual_rms_norm(x, torch.ones(300, device="cuda"), 0.0)[0])
    assert np.isnan(y[1, 7]) and (np.delete(y[1], 7) == 0).all()  # v / infinity
    assert np.isnan(y[2]).all()  # 0 / 0
    np.testing.assert_allclose(y[[0, 3]], 1.0, rtol=NORM)


def test_not_a_number_stays_in_its_row():
    x = torch.ones(3, 128, device="cuda")
    x[1, 5] = float("nan")
    y, scales, _ = binding.lstm_residual_rms_norm(x, torch.ones(128, device="cuda"), 1e-6,
                                                  quantize=True, group=32)
    nan = torch.isnan(y.float())
    assert nan[1].all() and not nan[0].any() and not nan[2].any()


def test_refusals():
    x = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    run = binding.lstm_residual_rms_norm
    for bad in (dict(quantize=True, group=48), dict(quantize=True, group=-1)):
        with pytest.raises(binding.LSTMError) as e:
            run(x, w, 1e-6, **bad)
        assert e.value.code == binding.LSTM_E_INVALID
    for eps in (-1.0, float("nan")):
        with pytest.raises(binding.LSTMError) as e:
            run(x, w, eps)
        assert e.value.code == binding.LSTM_E_INVALID
    with pytest.raises(binding.LSTMError):
        run(torch.zeros(1, 32769, device="cuda"), torch.ones(32769, device="cuda"), 1e-6)
    for bad in (lambda: run(x, w[:32], 1e-6), lambda: run(x, w.half(), 1e-6),
                lambda: run(x.double(), w, 1e-6), lambda: run(x, w, 1e-6, residual=x.half()),
                lambda: run(x, w, 1e-6, residual=x[:2]), lambda: run(x, w, 1e-6, residual_out=x),
                lambda: run(x, w, 1e-6, y=x.half()),
                lambda: run(x, w, 1e-6, quantize=True, y=torch.empty_like(x)),
                lambda: run(x, w, 1e-6, quantize=True, scales=torch.empty(4, 2, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
