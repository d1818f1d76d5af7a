"""The dense product against its float64 definition: types, sizes that no tile
divides, activations, residuals, strides and alignment, values that are not
finite, streams and graphs."""
import math

import numpy as np
import pytest
import torch

from bidirectional_lstm_stack_gb300 import binding
from oracle import layers as oracle
from ops_util import DTYPES, assert_close, at_element, f64, gen, normal, slice_of

pytestmark = pytest.mark.gpu


def _check(dtype, rows, n_in, n_out, *, bias=True, activation=None, residual=True, layout="dense",
           seed=1, in_place=False):
    g, t = gen(seed), DTYPES[dtype]
    x = normal(g, rows, n_in, dtype=t)
    w = normal(g, n_out, n_in, scale=n_in ** -0.5, dtype=t)
    b = normal(g, n_out) if bias else None
    r = normal(g, rows, n_out, dtype=t) if residual else None
    if layout != "dense":
        pad = {"slices": 8, "odd": 3}[layout]
        x, w = slice_of(x, pad, pad), slice_of(w, pad, pad)
        r = None if r is None else slice_of(r, pad, pad)
    y = None
    if layout != "dense":
        y = slice_of(torch.zeros(rows, n_out, dtype=t, device="cuda"), pad, pad)
    ref, bound = oracle.dense(f64(x), f64(w), f64(b), activation, f64(r))
    if in_place:
        y = r
    got = binding.lstm_dense(x, w, b, activation=activation, residual=r, y=y)
    assert y is None or got is y
    assert_close(got, ref, bound, dtype, f"{dtype} {rows}x{n_in}x{n_out}")
    return got


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows", [0, 1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200,
                                  257, 600])
def test_rows(dtype, rows):
    _check(dtype, rows, 96, 136)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows", [1, 5, 40, 130])
@pytest.mark.parametrize("n_in,n_out", [(1, 1), (1, 300), (7, 5), (64, 64), (63, 65), (65, 127), (129, 257),
                                        (777, 1003), (256, 1024), (1000, 8), (2048, 24)])
def test_sizes(dtype, rows, n_in, n_out):
    _check(dtype, rows, n_in, n_out, bias=n_in != 64, residual=n_out != 65)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows", [3, 150])
@pytest.mark.parametrize("activation", [None, "relu", "gelu", "gelu_tanh", "silu"])
def test_activations(dtype, rows, activation):
    for bias, residual in ((False, False), (True, False), (False, True), (True, True)):
        _check(dtype, rows, 80, 72, activation=activation, bias=bias, residual=residual)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("layout", ["slices", "odd"])
@pytest.mark.parametrize("rows,n_in,n_out", [(1, 64, 64), (40, 100, 90), (150, 128, 256), (300, 33, 31)])
def test_columns_of_wider_rows(dtype, layout, rows, n_in, n_out):
    _check(dtype, rows, n_in, n_out, layout=layout)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_the_residual_in_place(dtype):
    for rows, layout in ((1, "dense"), (17, "odd"), (300, "dense"), (300, "slices")):
        _check(dtype, rows, 200, 264, in_place=True, layout=layout, activation="silu")


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_weights_and_biases_at_any_element(dtype):
    g = gen(3)
    x, w, b = (normal(g, 70, 64, dtype=DTYPES[dtype]), normal(g, 96, 64, dtype=DTYPES[dtype]),
               normal(g, 96))
    ref = binding.lstm_dense(x, w, b)
    for offset in (1, 2, 3, 4, 5):
        for m in (dict(x=at_element(x, offset)), dict(w=at_element(w, offset)),
                  dict(b=at_element(b, offset))):
            m = {"x": x, "w": w, "b": b, **m}
            assert torch.equal(binding.lstm_dense(m["x"], m["w"], m["b"]), ref)


def test_larger_products():
    _check("bf16", 1100, 1024, 1536)
    _check("f16", 1030, 520, 2050, activation="gelu")
    _check("f32", 700, 600, 900, activation="gelu_tanh")
    _check("bf16", 1, 4096, 2048)
    _check("bf16", 33, 4100, 1000)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows", [5, 200])
def test_values_that_are_not_finite_stay_in_their_rows_and_columns(dtype, rows):
    g, t = gen(1), DTYPES[dtype]
    x, w = normal(g, rows, 100, dtype=t), normal(g, 150, 100, dtype=t)
    y = binding.lstm_dense(x, w)
    x[3, 40], w[70, 99], w[90, 0] = float("inf"), float("nan"), float("-inf")
    got = binding.lstm_dense(x, w)
    assert not got[3].isfinite().any() and not got[:, [70, 90]].isfinite().any()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[3] = False
    keep[:, [70, 90]] = False
    assert torch.equal(got[keep], y[keep])
    # of the residual and the bias too, and nothing is hidden by an activation
    r, b = torch.zeros(rows, 150, dtype=t, device="cuda"), torch.zeros(150, device="cuda")
    r[0, 5], b[6] = float("nan"), float("nan")
    for activation in (None, "relu", "gelu", "gelu_tanh", "silu"):
        got = binding.lstm_dense(x, w, b, activation=activation, residual=r)
        assert got[0, 5].isnan() and got[:, 6].isnan().all() and got[:, 70].isnan().all()


@pytest.mark.parametrize("activation", ["relu", "gelu", "gelu_tanh", "silu"])
def test_activations_far_out(activation):
    v = torch.tensor([-1e30, -200.0, -90.0, -20.0, -0.0, 0.0, 20.0, 90.0, 1e30], device="cuda")
    got = binding.lstm_dense(v[:, None], torch.ones(1, 1, device="cuda"), activation=activation)[:, 0]
    ref = oracle.activate(activation, f64(v))
    # below -12 the functions' factor is the difference of numbers next to 1
    assert np.allclose(f64(got), ref, rtol=2.0 ** -20, atol=1e-5)


def test_large_and_small_fp32_numbers():
    x = torch.tensor([[3.4e38, 0.0], [0.0, 1e-30], [1.0, 2.0 ** -23]], device="cuda")
    w = torch.tensor([[1.0, 1.0], [0.5, 1.0]], device="cuda")
    got = binding.lstm_dense(x, w)
    assert torch.equal(got, x @ w.t())


def test_the_same_call_gives_the_same_bits():
    for rows in (1, 20, 700):
        g = gen(1)
        x, w = normal(g, rows, 2048, dtype=torch.bfloat16), normal(g, 512, 2048, dtype=torch.bfloat16)
        y = binding.lstm_dense(x, w)
        for _ in range(3):
            assert torch.equal(binding.lstm_dense(x, w), y)


def test_other_streams_and_calls_at_once():
    streams = [torch.cuda.Stream() for _ in range(2)]
    for dtype, offset in ((torch.bfloat16, 0), (torch.float32, 0), (torch.float16, 1)):
        m = [(at_element(normal(gen(s), 300, 640, dtype=dtype), offset), normal(gen(s), 500, 640, dtype=dtype))
             for s in (1, 2)]
        alone = [binding.lstm_dense(x, w) for x, w in m]
        torch.cuda.synchronize()
        for _ in range(5):
            got = [binding.lstm_dense(x, w, stream=s) for (x, w), s in zip(m, streams)]
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(alone, got))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows", [1, 30, 300])
def test_a_captured_call_reads_what_is_there_when_it_is_replayed(dtype, rows):
    g, t = gen(1), DTYPES[dtype]
    x, w = normal(g, rows, 512, dtype=t), normal(g, 384, 512, dtype=t)
    y = torch.empty(rows, 384, dtype=t, device="cuda")
    binding.lstm_dense(x, w, y=y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.lstm_dense(x, w, y=y)
    for _ in range(2):
        x.copy_(normal(g, rows, 512))
        w.copy_(normal(g, 384, 512))
        graph.replay()
        assert torch.equal(y, binding.lstm_dense(x, w))


def test_launch_failures_are_errors():
    lib = binding.load()
    x, w = torch.zeros(5, 8, device="cuda"), torch.zeros(8, 8, device="cuda")
    assert lib.lstm_test_fail_launches(0, 1) == 0
    with pytest.raises(binding.LSTMError):
        binding.lstm_dense(x, w)
    binding.lstm_dense(x, w)


@pytest.mark.parametrize("rows", [4, 70, 400])
def test_a_wait_that_runs_out_sets_the_fault_word_and_the_next_call_works(rows):
    lib = binding.load()
    x, w = normal(gen(1), rows, 1024, dtype=torch.bfloat16), normal(gen(2), 256, 1024, dtype=torch.bfloat16)
    ref = binding.lstm_dense(x, w)
    assert binding.lstm_fault_status() == 0
    try:
        assert lib.lstm_test_dense_timeout(1, 1000, 0) == 0
        binding.lstm_dense(x, w)
        torch.cuda.synchronize()
    finally:
        assert lib.lstm_test_dense_timeout(0, 0, 0) == 0
    assert binding.lstm_fault_status() != 0
    assert torch.equal(binding.lstm_dense(x, w), ref)
    torch.cuda.synchronize()
    assert binding.lstm_fault_status() == 0


# ---- the ways a product is cut up -----------------------------------------------------------------
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,n_in,n_out", [
    (5000, 100, 520),    # pairs of SMs, a tile of 256 x 256 each
    (4865, 72, 515),     # the same, the last tile a row and three columns wide
    (2000, 136, 1000),   # tiles of one SM
    (130, 1500, 200),    # parts of K, joined in a cluster
    (40, 2100, 300),     # few rows, parts of K
])
def test_tiles(dtype, rows, n_in, n_out):
    _check(dtype, rows, n_in, n_out, activation="silu")
    _check(dtype, rows, n_in, n_out, bias=False, layout="odd")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows", [1, 2, 3])
@pytest.mark.parametrize("n_in,n_out", [(1, 1), (31, 5), (256, 3), (257, 64), (4096, 130), (5000, 7)])
def test_a_row_or_a_few(dtype, rows, n_in, n_out):
    for layout in ("dense", "slices", "odd"):
        _check(dtype, rows, n_in, n_out, activation="gelu", layout=layout)


def test_pairs_give_the_same_bits_each_time_and_in_place():
    g = gen(4)
    x, w = normal(g, 5000, 256, dtype=torch.bfloat16), normal(g, 1024, 256, dtype=torch.bfloat16)
    r = normal(g, 5000, 1024, dtype=torch.bfloat16)
    ref = binding.lstm_dense(x, w, residual=r)
    for _ in range(5):
        y = r.clone()
        assert binding.lstm_dense(x, w, residual=y, y=y) is y
        assert torch.equal(y, ref)


@pytest.mark.parametrize("rows", [2, 5000])
def test_values_that_are_not_finite_stay_in_their_rows_and_columns(rows):
    g = gen(5)
    x, w = normal(g, rows, 200, dtype=torch.bfloat16), normal(g, 600, 200, dtype=torch.bfloat16)
    ref = binding.lstm_dense(x, w)
    x[1, 7], w[300, 3] = float("nan"), float("inf")
    y = binding.lstm_dense(x, w)
    assert not y[1].isfinite().any() and not y[:, 300].isfinite().any()
    rows_ok = [r for r in range(rows) if r != 1]
    cols_ok = [c for c in range(600) if c != 300]
    assert torch.equal(y[rows_ok][:, cols_ok], ref[rows_ok][:, cols_ok])


def test_a_wait_of_a_pair_that_runs_out_sets_the_fault_word_and_the_next_call_works():
    lib = binding.load()
    x, w = normal(gen(1), 5000, 512, dtype=torch.bfloat16), normal(gen(2), 512, 512, dtype=torch.bfloat16)
    ref = binding.lstm_dense(x, w)
    assert binding.lstm_fault_status() == 0
    try:
        assert lib.lstm_test_dense_timeout(1, 1000, 0) == 0
        binding.lstm_dense(x, w)
        torch.cuda.synchronize()
    finally:
        assert lib.lstm_test_dense_timeout(0, 0, 0) == 0
    assert binding.lstm_fault_status() != 0
    assert torch.equal(binding.lstm_dense(x, w), ref)
    torch.cuda.synchronize()
    assert binding.lstm_fault_status() == 0


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows", [1, 4, 70, 400])
def test_gelu_keeps_its_relative_accuracy_far_out(dtype, rows):
    # The factor Phi(v) is off by: its fit (2^-24), ten roundings of sums that are 2.4 times what
    # they sum up to at most (2^-24 each, the first ones damped: 4 in all), the reciprocal (2^-23),
    # the exponential (2^-22), three products (2^-24 each): below 2^-20 of itself.  (v is one
    # operand of the type, the other is 1: the product is exact.)  For 16-bit results the fit is off by
    # 4.7e-6, and the exponent a^2 / 2, up to 78 at 12.5, is rounded twice on its way to the
    # exponential: 78 x 2^-24 and as much again at most; together below 2^-16.
    top = 12.5 if dtype != "f16" else 4.0  # (results below are subnormal)
    v = torch.linspace(-top, top, 64 * rows, device="cuda").view(rows, 64).to(DTYPES[dtype])
    got = f64(binding.lstm_dense(v, torch.eye(64, dtype=DTYPES[dtype], device="cuda"), activation="gelu"))
    x = f64(v)
    ref = x * 0.5 * np.vectorize(math.erfc)(-x / math.sqrt(2.0))
    rel = 2.0 ** (-20 if dtype == "f32" else -16) + torch.finfo(DTYPES[dtype]).eps / 2
    least = 2.0 ** -25 if dtype == "f16" else 0.0
    assert (np.abs(got - ref) <= rel * (1 + 2.0 ** -7) * np.abs(ref) + least).all(), np.max(
        np.abs(got - ref) / (np.abs(ref) + 1e-300))


@pytest.mark.parametrize("rows", [1, 4, 70, 400])
def test_products_of_fp32_numbers_keep_their_bits(rows):
    # Of a product of three parts each, 2^-24 is left out; sums are cut off below 2^-23 of
    # themselves, and those before the last are 2^-7 of it: 1.5 x 2^-23 and a little.
    g = gen(2)
    x, w = (1.0 + torch.rand(n, generator=g, device="cuda") for n in (rows, 96))
    x[0] = w[0] = 1.0078124  # (all ones behind the first eight bits)
    w[1] = 1.9960936
    x, w = (m * torch.exp2(torch.randint(-50, 50, m.shape, generator=g, device="cuda")) for m in (x, w))
    got = f64(binding.lstm_dense(x[:, None], w[:, None]))
    ref = np.outer(f64(x), f64(w))
    assert (np.abs(got - ref) <= 2.0 ** -22 * ref).all(), np.max(np.abs(got / ref - 1))


@pytest.mark.parametrize("rows", [1, 8, 70, 400])
def test_fp32_numbers_next_to_the_largest_and_the_smallest(rows):
    # as above, and a number's parts end at 2^-133: what lies below half of that is lost
    values = [3.4028234e38, -3.4e38, 3.39e38, 1e-30, 2.0 ** -110 * 1.2345678, 1.2345678e-36, -1.2345678e-38,
              1e-40]
    x = torch.zeros(rows, 2, device="cuda")
    x[:, 0] = torch.tensor((values * 50)[:rows])
    w = torch.zeros(5, 2, device="cuda")
    w[:, 0] = torch.tensor([1.0, -0.5, 0.33333334, 0.99999994, 1.2345678e-7])
    for a, b in ((x, w), (torch.cat([w] * 80)[:max(rows, 4)], x[:8])):
        got, ref = f64(binding.lstm_dense(a, b)), f64(a) @ f64(b).T
        assert (np.abs(got - ref) <= 2.0 ** -22 * np.abs(ref) + 2.0 ** -133).all()


@pytest.mark.parametrize("rows", [1, 5, 70, 400])
def test_infinities_of_fp32_give_what_one_product_gives(rows):
    inf = float("inf")
    values = torch.tensor([inf, -inf, 1.0, -2.0, 0.1, 1e30, -1e-30, 0.0], device="cuda")
    x, w = torch.zeros(rows, 100, device="cuda"), torch.zeros(8, 100, device="cuda")
    x[:, 0], w[:, 0] = values.repeat(50)[:rows], values
    got = binding.lstm_dense(x, w)
    ref = x[:, :1] * w[:, 0]
    far = ref.abs() == inf
    assert torch.equal(got.isnan(), ref.isnan()) and torch.equal(got[far], ref[far])
    # beside finite products, and two infinities that cancel
    x, w = normal(gen(1), rows, 100), normal(gen(2), 8, 100)
    x[0, 40] = inf
    got = binding.lstm_dense(x, w)
    assert torch.equal(got[0], torch.copysign(torch.full_like(w[:, 40], inf), w[:, 40]))
    assert got[1:].isfinite().all()
    x[0, 41] = torch.copysign(torch.tensor(inf), -w[0, 40] * w[0, 41])
    assert binding.lstm_dense(x, w)[0, 0].isnan()


@pytest.mark.parametrize("rows,n_in,n_out", [(1, 40, 60), (5, 40, 60), (40, 2100, 300), (70, 40, 60),
                                             (130, 1500, 200), (2000, 40, 1000), (5000, 40, 520)])
def test_fp32_products_that_overflow_do_so_to_their_own_side(rows, n_in, n_out):
    g = gen(7)
    x, w = (1.0 + torch.rand(n, n_in, generator=g, device="cuda") for n in (rows, n_out))
    ref = binding.lstm_dense(x, w)
    x[rows // 2] *= 1e30   # times 1e12 of two columns: far beyond, and to either side
    w[7] *= 1e12
    w[n_out - 1] *= -1e25
    got = binding.lstm_dense(x, w)
    assert (got[rows // 2, 7], got[rows // 2, n_out - 1]) == (float("inf"), -float("inf"))
    keep = [c for c in range(n_out) if c not in (7, n_out - 1)]
    assert got[:, keep].isfinite().all()
    others = [r for r in range(rows) if r != rows // 2]
    assert torch.equal(got[others][:, keep], ref[others][:, keep]) and got[others].isfinite().all()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows", [2, 5, 40, 200, 5000])
def test_values_that_are_not_finite_of_every_type_and_through_each_activation(dtype, rows):
    g, t = gen(1), DTYPES[dtype]
    x, w = normal(g, rows, 100, dtype=t), normal(g, 150, 100, dtype=t)
    y = binding.lstm_dense(x, w)
    x[1, 40], w[70, 99], w[90, 0] = float("inf"), float("nan"), float("-inf")
    got = binding.lstm_dense(x, w)
    assert not got[1].isfinite().any() and not got[:, [70, 90]].isfinite().any()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[1] = False
    keep[:, [70, 90]] = False
    assert torch.equal(got[keep], y[keep])
    # of the residual and the bias too, and nothing is hidden by an activation
    r, b = torch.zeros(rows, 150, dtype=t, device="cuda"), torch.zeros(150, device="cuda")
    r[0, 5], b[6] = float("nan"), float("nan")
    for activation in (None, "relu", "gelu", "gelu_tanh", "silu"):
        got = binding.lstm_dense(x, w, b, activation=activation, residual=r)
        assert got[0, 5].isnan() and got[:, 6].isnan().all() and got[:, 70].isnan().all()


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_rows_beyond_32_bits_of_elements(dtype):
    rows, t = 70001, DTYPES[dtype]
    stride = (1 << 31) // rows + 1024
    stride -= stride % 8
    x, w = normal(gen(1), rows, 40, dtype=t), normal(gen(2), 48, 40, dtype=t)
    r = normal(gen(3), rows, 48, dtype=t)
    ref = binding.lstm_dense(x, w, residual=r)
    far = torch.empty(rows * stride, dtype=t, device="cuda")
    y = far.as_strided((rows, 48), (stride, 1)).copy_(r)
    assert torch.equal(binding.lstm_dense(x, w, residual=y, y=y), ref)
    assert torch.equal(binding.lstm_dense(far.as_strided((rows, 40), (stride, 1)).copy_(x), w, residual=r), ref)


@pytest.mark.parametrize("rows", [4, 70])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_sum_may_take_longer_than_a_wait(rows, dtype):
    # a tile of this K takes milliseconds, the limit is one
    lib = binding.load()
    n_in = 1 << 22 if dtype == "bf16" else 1 << 20
    x = torch.ones(rows, n_in, dtype=DTYPES[dtype], device="cuda")
    w = torch.full((1, n_in), 2.0 ** -20, dtype=DTYPES[dtype], device="cuda")
    assert binding.lstm_fault_status() == 0
    try:
        assert lib.lstm_test_dense_timeout(0, 1000, 0) == 0
        y = binding.lstm_dense(x, w)
        torch.cuda.synchronize()
    finally:
        assert lib.lstm_test_dense_timeout(0, 0, 0) == 0
    assert binding.lstm_fault_status() == 0
    # (powers of two: every partial sum is exact)
    assert (y == n_in * 2.0 ** -20).all()
