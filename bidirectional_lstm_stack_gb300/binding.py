"""ctypes binding of liblstmstack.so (declared in include/lstm_stack.h,
include/lstm_ops.h and include/lstm_layers.h).

Argument marshalling only: the functions compute nothing and forward to the C
entry point of the same name.  Those of lstm_stack.h check nothing the library
does not check again.  Those of lstm_ops.h and lstm_layers.h go through the compiled module
``_native``, which allocates outputs and alone checks shapes, types, devices and
gradients (the C entry points take sizes and strides on trust).  Device buffers
are torch CUDA tensors (their ``data_ptr``), streams are torch streams (their
``cuda_stream`` handle; default: the current stream of the tensor's device).  If
the library or the module is missing, calls raise ``LibraryMissing``: there is no
fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

from .synthetic import FEATURES, HIDDEN, LAYERS

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblstmstack.so")
NATIVE_PATH = os.path.join(os.path.dirname(LIB_PATH), "_native.so")
GATE_COLUMNS = 8 * HIDDEN
OUTPUT = 2 * HIDDEN

LSTM_OK = 0
LSTM_E_INVALID = 1
LSTM_E_LENGTH = 2
LSTM_E_OVERFLOW = 3
LSTM_E_DEVICE = 4
LSTM_E_CUDA = 5
LSTM_E_ALLOC = 6
LSTM_E_FAULT = 7
LSTM_MATH_3XTF32 = 0
LSTM_MATH_TF32 = 1
LSTM_GATES_IFGO = 0
LSTM_GATES_IOFC = 1
LSTM_BOTH_DIRECTIONS = 2
LSTM_F32 = 0
LSTM_BF16 = 1
LSTM_F16 = 2
LSTM_E4M3 = 3
LSTM_ACT_NONE = 0
LSTM_ACT_RELU = 1
LSTM_ACT_GELU = 2
LSTM_ACT_GELU_TANH = 3
LSTM_ACT_SILU = 4

_c_float_p = ctypes.POINTER(ctypes.c_float)
_vp = ctypes.c_void_p


class LibraryMissing(RuntimeError):
    """liblstmstack.so has not been built (run __graft_entry__.build())."""


class LSTMError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"liblstmstack error {code}: {message}")
        self.code = code


class _Weights(ctypes.Structure):
    _fields_ = [("w", _vp * LAYERS), ("r", _vp * LAYERS), ("b", _vp * LAYERS)]


_lock = threading.Lock()
_lib = None


def load():
    """Loads liblstmstack.so (once) and declares its signatures."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise LibraryMissing(f"{LIB_PATH} not found; build it with __graft_entry__.build()")
        lib = ctypes.CDLL(LIB_PATH)
        i, sz = ctypes.c_int, ctypes.c_size_t
        ll, f = ctypes.c_longlong, ctypes.c_float
        sig = {
            "lstm_stack_create": (i, [ctypes.POINTER(_Weights), i, i, i, ctypes.POINTER(_vp)]),
            "lstm_stack_create_ordered": (i, [ctypes.POINTER(_Weights), i, i, i, i,
                                              ctypes.POINTER(_vp)]),
            "lstm_stack_forward": (i, [_vp, _vp, sz, _vp, sz, i, i, _vp]),
            "lstm_stack_forward_host": (i, [_vp, _vp, sz, _vp, sz, i, i, _vp]),
            "lstm_stack_forward_host_async": (i, [_vp, _vp, sz, _vp, sz, i, i, _vp]),
            "lstm_stack_host_sync": (i, [_vp]),
            "lstm_stack_enable_phase_timing": (i, [_vp, i]),
            "lstm_stack_set_graphs": (i, [_vp, i]),
            "lstm_stack_set_math": (i, [_vp, i]),
            "lstm_stack_phase_times": (i, [_vp, _c_float_p]),
            "lstm_stack_destroy": (None, [_vp]),
            "lstm_stack_last_error": (ctypes.c_char_p, []),
            "lstm_pack_layer": (i, [_vp, _vp, _vp, i, i, _vp, _vp, _vp, _vp]),
            "lstm_pack_layer_ordered": (i, [_vp, _vp, _vp, i, i, i, _vp, _vp, _vp, _vp]),
            "lstm_projection": (i, [_vp, i, i, _vp, _vp, i, _vp, _vp]),
            "lstm_projection_math": (i, [_vp, i, i, _vp, _vp, i, _vp, i, _vp]),
            "lstm_recurrence": (i, [_vp, _vp, _vp, _vp, i, i, i, _vp]),
            "lstm_recurrence_variant": (i, [_vp, _vp, _vp, _vp, i, i, i, i, i, i, i, _vp]),
            "lstm_recurrence_max_clusters": (i, [i, i, i, i, i, ctypes.POINTER(i)]),
            "lstm_fault_status": (i, [ctypes.POINTER(ctypes.c_uint)]),
            "lstm_layer_forward_static": (i, [_vp, i, i, i, _vp, _vp, i, _vp, _vp, _vp, _vp]),
            "lstm_heads_create": (i, [_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_float, i, i,
                                      ctypes.POINTER(_vp)]),
            "lstm_heads_forward": (i, [_vp, _vp, sz, _vp, sz, i, _vp]),
            "lstm_heads_destroy": (None, [_vp]),
            "lstm_test_fail_allocations": (i, [i, i]),
            "lstm_test_fail_launches": (i, [i, i]),
            "lstm_test_recurrence_timeout": (i, [i, ctypes.c_uint, i]),
            "lstm_test_projection_timeout": (i, [i, ctypes.c_uint, i]),
            "lstm_test_heads_timeout": (i, [i, ctypes.c_uint, i]),
            "lstm_test_scan_step_timeout": (i, [i, ctypes.c_uint, i]),
            "lstm_test_attention_timeout": (i, [i, ctypes.c_uint, i]),
            "lstm_test_dense_timeout": (i, [i, ctypes.c_uint, i]),
            "lstm_recurrence_floor": (i, [_vp, _vp, _vp, _vp, i, i, i, _vp]),
            "lstm_tf32_rate": (i, [i, i, ctypes.POINTER(ctypes.c_double)]),
            "lstm_recurrence_fused": (i, [_vp, i, _vp, _vp, i, _vp, _vp, _vp, i, i, i, _vp]),
            "lstm_stack_set_fused_batches": (i, [_vp, i]),
            "lstm_causal_conv": (i, [_vp, ll, i, i, i, i, _vp, _vp, i, i, _vp, _vp, i, _vp, _vp,
                                     _vp, ll, _vp]),
            "lstm_causal_conv_step": (i, [_vp, ll, i, i, i, i, _vp, _vp, i, _vp, i, _vp, _vp, ll,
                                          _vp]),
            "lstm_selective_scan": (i, [_vp, ll, _vp, ll, _vp, _vp, ll, _vp, ll, _vp, _vp, ll, _vp,
                                        i, i, i, i, i, i, i, _vp, _vp, i, _vp, _vp, _vp, ll, _vp, sz,
                                        _vp]),
            "lstm_selective_scan_workspace": (sz, [i, i, i, i, i, i]),
            "lstm_selective_scan_step": (i, [_vp, ll, _vp, ll, _vp, _vp, ll, _vp, ll, _vp, _vp, ll,
                                             _vp, i, i, i, i, i, i, _vp, i, _vp, _vp, ll, _vp]),
            "lstm_residual_rms_norm": (i, [_vp, ll, _vp, ll, i, _vp, f, i, i, _vp, ll, _vp, ll, i,
                                           _vp, i, _vp]),
            "lstm_token_logprobs": (i, [_vp, ll, i, i, i, _vp, _vp, _vp, i, _vp, _vp, _vp]),
            "lstm_linear_attention": (i, 3 * [_vp, ll, ll, i] +
                                      [_vp, ll, f, i, i, i, i, i, i, _vp, _vp, i, _vp, _vp, _vp, ll,
                                       _vp, sz, _vp]),
            "lstm_linear_attention_workspace": (sz, [i, i, i, i, i, i]),
            "lstm_linear_attention_step": (i, 3 * [_vp, ll, ll, i] +
                                           [_vp, ll, f, i, i, i, i, i, _vp, i, _vp, _vp, ll, _vp]),
            "lstm_dense": (i, [_vp, ll, _vp, ll, _vp, i, _vp, ll, i, i, i, i, _vp, ll, _vp, sz,
                               _vp]),
            "lstm_dense_workspace": (sz, [_vp, ll, _vp, ll, i, i, i, i]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def lstm_stack_last_error() -> str:
    return load().lstm_stack_last_error().decode()


def _check(code: int) -> None:
    if code != LSTM_OK:
        raise LSTMError(code, lstm_stack_last_error())


def _ptr(t) -> int:
    """Address of a torch tensor's data (None for None)."""
    return None if t is None else t.data_ptr()


def _stream(stream, device=None):
    if stream is None:
        import torch
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _host(a, dtype=np.float32) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=dtype))


def lstm_pack_layer(w, r, b, in_width: int, kp: int, gate_order: int = LSTM_GATES_IFGO):
    """Host packer; returns (wp_hi, wp_lo, rp, bias) numpy arrays."""
    w, r, b = _host(w), _host(r), _host(b)
    wp_hi = np.empty((GATE_COLUMNS, kp), np.float32)
    wp_lo = np.empty((GATE_COLUMNS, kp), np.float32)
    rp = np.empty((2, 4 * HIDDEN, HIDDEN), np.float32)
    bias = np.empty((2, 4 * HIDDEN), np.float32)
    _check(load().lstm_pack_layer_ordered(w.ctypes.data, r.ctypes.data, b.ctypes.data, in_width,
                                          kp, gate_order, wp_hi.ctypes.data, wp_lo.ctypes.data,
                                          rp.ctypes.data, bias.ctypes.data))
    return wp_hi, wp_lo, rp, bias


def lstm_projection(x, rows: int, in_width: int, wp_hi, wp_lo, kp: int, g, stream=None):
    """G = X . Wp^T on the device (torch CUDA tensors)."""
    _check(load().lstm_projection(_ptr(x), rows, in_width, _ptr(wp_hi), _ptr(wp_lo), kp, _ptr(g),
                                  _stream(stream, x.device)))


def lstm_projection_math(x, rows: int, in_width: int, wp_hi, wp_lo, kp: int, g, math: int,
                         stream=None):
    """G = X . Wp^T with the chosen products (LSTM_MATH_*); wp_lo may be None
    for LSTM_MATH_TF32."""
    _check(load().lstm_projection_math(_ptr(x), rows, in_width, _ptr(wp_hi),
                                       _ptr(wp_lo), kp, _ptr(g), math,
                                       _stream(stream, x.device)))


def lstm_recurrence(g, rp, bias, y, batch: int, steps: int, direction: int, stream=None):
    _check(load().lstm_recurrence(_ptr(g), _ptr(rp), _ptr(bias), _ptr(y), batch, steps,
                                  direction, _stream(stream, g.device)))


def lstm_recurrence_floor(g, rp, bias, y, batch: int, steps: int, direction: int, stream=None):
    _check(load().lstm_recurrence_floor(_ptr(g), _ptr(rp), _ptr(bias), _ptr(y), batch, steps,
                                        direction, _stream(stream, g.device)))


def lstm_recurrence_fused(x, in_width: int, wp_hi, wp_lo, kp: int, rp, bias, y, batch: int,
                          steps: int, direction: int, stream=None):
    _check(load().lstm_recurrence_fused(_ptr(x), in_width, _ptr(wp_hi), _ptr(wp_lo), kp,
                                        _ptr(rp), _ptr(bias), _ptr(y), batch, steps, direction,
                                        _stream(stream, x.device)))


def lstm_stack_set_fused_batches(handle, max_batch: int) -> None:
    _check(load().lstm_stack_set_fused_batches(handle, max_batch))


def lstm_tf32_rate(device: int = 0, iterations: int = 20000) -> float:
    v = ctypes.c_double(0.0)
    _check(load().lstm_tf32_rate(device, iterations, ctypes.byref(v)))
    return float(v.value)


def lstm_recurrence_variant(g, rp, bias, y, batch: int, steps: int, direction: int,
                            cluster_size: int, windows_per_chunk: int, chunks: int = 1,
                            threads_per_block: int = 0, stream=None):
    _check(load().lstm_recurrence_variant(_ptr(g), _ptr(rp), _ptr(bias), _ptr(y), batch, steps,
                                          direction, cluster_size, windows_per_chunk, chunks,
                                          threads_per_block, _stream(stream, g.device)))


def lstm_recurrence_max_clusters(cluster_size: int, windows_per_chunk: int, chunks: int = 1,
                                 threads_per_block: int = 0, device: int = 0) -> int:
    v = ctypes.c_int(0)
    _check(load().lstm_recurrence_max_clusters(cluster_size, windows_per_chunk, chunks,
                                               threads_per_block, device, ctypes.byref(v)))
    return int(v.value)


def lstm_layer_forward_static(x, batch: int, steps: int, in_width: int, wp_hi, wp_lo, kp: int,
                              rp, bias, y, stream=None):
    """One bidirectional layer through the entry point that allocates no
    device memory (its gate buffer is a fixed array inside the library)."""
    _check(load().lstm_layer_forward_static(_ptr(x), batch, steps, in_width, _ptr(wp_hi),
                                            _ptr(wp_lo), kp, _ptr(rp), _ptr(bias), _ptr(y),
                                            _stream(stream, x.device)))


def lstm_fault_status() -> int:
    v = ctypes.c_uint(0)
    _check(load().lstm_fault_status(ctypes.byref(v)))
    return int(v.value)


def lstm_stack_create(layers, max_batch: int, max_steps: int, device: int = 0,
                      gate_order: int = LSTM_GATES_IFGO):
    """Creates a stack from source weights (list of dicts w, r, b; numpy) whose
    gate row blocks are in ``gate_order`` (LSTM_GATES_IFGO or _IOFC).

    Returns the opaque handle (an int).  The host arrays are only read during
    the call.
    """
    arrs = [{k: _host(l[k]) for k in ("w", "r", "b")} for l in layers]
    ws = _Weights()
    for l, a in enumerate(arrs):
        ws.w[l] = a["w"].ctypes.data
        ws.r[l] = a["r"].ctypes.data
        ws.b[l] = a["b"].ctypes.data
    h = _vp()
    _check(load().lstm_stack_create_ordered(ctypes.byref(ws), gate_order, max_batch, max_steps,
                                            device, ctypes.byref(h)))
    return h.value


def lstm_stack_forward(handle, x, y, batch: int, steps: int, stream=None):
    _check(load().lstm_stack_forward(handle, _ptr(x), x.numel(), _ptr(y), y.numel(), batch,
                                     steps, _stream(stream, x.device)))


def lstm_stack_forward_host(handle, x: np.ndarray, y: np.ndarray, batch: int, steps: int,
                            stream=None):
    """x, y: C-contiguous float32 host arrays (pinned memory recommended)."""
    assert x.dtype == np.float32 and y.dtype == np.float32
    assert x.flags.c_contiguous and y.flags.c_contiguous
    _check(load().lstm_stack_forward_host(handle, x.ctypes.data, x.size, y.ctypes.data, y.size,
                                          batch, steps, _stream(stream)))


def lstm_stack_forward_host_async(handle, x: np.ndarray, y: np.ndarray, batch: int, steps: int,
                                  stream=None):
    """Enqueue without waiting; x must stay unchanged and y is valid only after
    lstm_stack_host_sync.  x, y: C-contiguous float32 host arrays, pinned for
    the copies to overlap the forward."""
    assert x.dtype == np.float32 and y.dtype == np.float32
    assert x.flags.c_contiguous and y.flags.c_contiguous
    _check(load().lstm_stack_forward_host_async(handle, x.ctypes.data, x.size, y.ctypes.data,
                                                y.size, batch, steps, _stream(stream)))


def lstm_stack_host_sync(handle):
    _check(load().lstm_stack_host_sync(handle))


def lstm_stack_set_graphs(handle, enable: bool = True):
    _check(load().lstm_stack_set_graphs(handle, int(bool(enable))))


def lstm_stack_set_math(handle, math: int):
    _check(load().lstm_stack_set_math(handle, math))


def lstm_stack_enable_phase_timing(handle, enable: bool = True):
    _check(load().lstm_stack_enable_phase_timing(handle, int(bool(enable))))


def lstm_stack_phase_times(handle) -> np.ndarray:
    ms = (ctypes.c_float * (3 * LAYERS))()
    _check(load().lstm_stack_phase_times(handle, ms))
    return np.array(ms[:], dtype=np.float64).reshape(LAYERS, 3)


def lstm_stack_destroy(handle) -> None:
    if handle:
        load().lstm_stack_destroy(handle)


class LSTMStack:
    """Owns a stack handle; ``forward`` takes and returns torch CUDA tensors."""

    def __init__(self, layers, max_batch: int, max_steps: int, device: int = 0,
                 gate_order: int = LSTM_GATES_IFGO):
        self.device = device
        self.max_batch = max_batch
        self.max_steps = max_steps
        self.handle = lstm_stack_create(layers, max_batch, max_steps, device, gate_order)

    def forward(self, x, y=None, stream=None):
        """x: [B, T, 60] float32 CUDA tensor -> y [B, T, 256] (new unless given)."""
        import torch
        B, T, F = x.shape
        if F != FEATURES:
            raise ValueError(f"input width {F}, expected {FEATURES}")
        if y is None:
            y = torch.empty((B, T, OUTPUT), dtype=torch.float32, device=x.device)
        lstm_stack_forward(self.handle, x, y, B, T, stream)
        return y

    __call__ = forward

    def close(self):
        if self.handle:
            lstm_stack_destroy(self.handle)
            self.handle = None

    def __del__(self):  # pragma: no cover
        try:
            self.close()
        except Exception:
            pass


HEADS_CLASSES = 7


class LSTMHeads:
    """The segmentation model's dense heads (linear0, linear1, classifier) on
    stack output rows; ``forward`` takes and returns torch CUDA tensors."""

    def __init__(self, weights, max_rows: int, negative_slope: float = 0.01, device: int = 0):
        arrs = {k: _host(weights[k]) for k in ("w0", "b0", "w1", "b1", "w2", "b2")}
        h = _vp()
        _check(load().lstm_heads_create(*(arrs[k].ctypes.data for k in
                                          ("w0", "b0", "w1", "b1", "w2", "b2")),
                                        float(negative_slope), max_rows, device, ctypes.byref(h)))
        self.handle = h.value
        self.max_rows = max_rows
        self.device = device

    def forward(self, y, out=None, stream=None):
        """y: [..., 256] float32 CUDA tensor -> log-probabilities [..., 7]."""
        import torch
        if y.shape[-1] != OUTPUT:
            raise ValueError(f"input width {y.shape[-1]}, expected {OUTPUT}")
        rows = y.numel() // OUTPUT
        if out is None:
            out = torch.empty((*y.shape[:-1], HEADS_CLASSES), dtype=torch.float32,
                              device=y.device)
        _check(load().lstm_heads_forward(self.handle, _ptr(y), y.numel(), _ptr(out), out.numel(),
                                         rows, _stream(stream, y.device)))
        return out

    __call__ = forward

    def close(self):
        if self.handle:
            load().lstm_heads_destroy(self.handle)
            self.handle = None

    def __del__(self):  # pragma: no cover
        try:
            self.close()
        except Exception:
            pass


# ---- state-space layer and log probabilities (include/lstm_ops.h) -------------
#
# The C entry points take sizes and strides on trust, so these functions check
# that every tensor has the type, shape and device that the call's sizes say.
# Matrices are [rows, columns] with consecutive columns and any row stride of at
# least the columns.  Outputs must not overlap inputs (residual_out may be residual).
# Outputs that are not given are allocated for the stream the call runs on.
# Forward only: while gradients are recorded, tensors that require one are refused.
# Small calls last longer on the host than on the GPU, so checks, outputs and
# the call itself are compiled (csrc/python_ops.cpp): a decode step of one
# sequence takes 5 us from Python, through ctypes it took 25.

_ops = None


def _load_ops():
    """Imports the compiled calls (once)."""
    global _ops
    load()
    import torch  # noqa: F401  (whose libraries the module is linked to)
    try:
        from . import _native
    except ImportError as e:
        raise LibraryMissing(f"{NATIVE_PATH}: {e}; build it with __graft_entry__.build()") from e
    _native.set_error(LSTMError)
    _ops = _native
    return _ops


def lstm_causal_conv(x, w, bias=None, *, silu: bool = True, sequences=None, offsets=None,
                     state=None, slots=None, resume=None, y=None, stream=None):
    """Causal depthwise convolution of packed prompts x [tokens, channels];
    returns y (new unless given) and moves the state, if given, on.

    w [channels, width] and bias [channels] fp32; offsets int32 [sequences + 1]
    (None: `sequences` prompts of equal length, default one); state
    [slots, width - 1, channels] of x's type, slots and resume int32
    [sequences]."""
    return (_ops or _load_ops()).causal_conv(x, w, bias, silu, sequences, offsets, state, slots,
                                             resume, y, stream)


def lstm_causal_conv_step(x, w, bias, state, *, silu: bool = True, slots=None, y=None,
                          stream=None):
    """The next token of every sequence, x [sequences, channels]; returns y
    (new unless given) and moves the state on.  Arguments as lstm_causal_conv."""
    return (_ops or _load_ops()).causal_conv_step(x, w, bias, state, silu, slots, y, stream)


def lstm_selective_scan(u, dt, a, b, c, *, skip=None, z=None, dt_bias=None, softplus: bool = True,
                        groups: int = 1, sequences=None, offsets=None, state=None, slots=None,
                        resume=None, y=None, stream=None):
    """Selective scan of packed prompts u, dt, z [tokens, channels], b and c
    [tokens, groups * states]; returns y (new unless given) and moves the
    state, if given, on.

    a [channels, states] (negative), skip and dt_bias [channels] fp32; offsets
    int32 [sequences + 1] (None: `sequences` prompts of equal length, default
    one); state [slots, channels, states] fp32, slots and resume int32
    [sequences]."""
    return (_ops or _load_ops()).selective_scan(u, dt, a, b, c, skip, z, dt_bias, softplus, groups,
                                                sequences, offsets, state, slots, resume, y, stream)


def lstm_selective_scan_workspace(tokens: int, channels: int, states: int, groups: int,
                                  sequences: int, equal_lengths: bool) -> int:
    """Bytes of workspace of lstm_selective_scan."""
    return load().lstm_selective_scan_workspace(tokens, channels, states, groups, sequences,
                                                int(equal_lengths))


def lstm_selective_scan_step(u, dt, a, b, c, state, *, skip=None, z=None, dt_bias=None,
                             softplus: bool = True, groups: int = 1, slots=None, y=None,
                             stream=None):
    """The next token of every sequence, u, dt, z [sequences, channels]; returns
    y (new unless given) and moves the state on.  Arguments as
    lstm_selective_scan."""
    return (_ops or _load_ops()).selective_scan_step(u, dt, a, b, c, state, skip, z, dt_bias,
                                                     softplus, groups, slots, y, stream)


def lstm_residual_rms_norm(x, weight, eps: float, *, residual=None, residual_out=None,
                           quantize: bool = False, group: int = 0, y=None, scales=None,
                           stream=None):
    """RMS norm of v = x + residual (x alone without one); returns
    (y, scales, v).

    y has x's type, or with quantize torch.float8_e4m3fn, and then scales
    [rows, ceil(cols / group)] fp32 (group 0: one a row) make y * scales stand
    for the norm; else scales is None.  v is rounded to x's type (residual_out:
    where to, may be residual); None without a residual."""
    return (_ops or _load_ops()).residual_rms_norm(x, weight, eps, residual, residual_out,
                                                   quantize, group, y, scales, stream)


def lstm_token_logprobs(logits, tokens=None, *, top: int = 0, entropy: bool = True, stream=None):
    """Log probabilities of tokens (int64 [rows]) under logits [rows, vocab];
    returns (logp, entropy, top_logp, top_ids): fp32 [rows], fp32 [rows], fp32
    and int64 [rows, top]; None for what is not asked for."""
    return (_ops or _load_ops()).token_logprobs(logits, tokens, top, entropy, stream)


# ---- linear attention and dense products (include/lstm_layers.h) -------------------
#
# Checked, allocated and called as the functions above.

def lstm_linear_attention(q, k, v, log_decay, *, scale: float = 1.0, sequences=None, offsets=None,
                          state=None, slots=None, resume=None, y=None, stream=None):
    """Linear attention with a decay for each head over packed prompts,
    S = e^log_decay S + k v^T, y = scale S^T q; returns y [tokens, heads,
    values] (new unless given) and moves the state, if given, on.

    q [tokens, q_heads, keys], k [tokens, k_heads, keys], v [tokens, v_heads,
    values], each with any strides between tokens and heads, their heads shared
    by groups of the call's; log_decay fp32 [heads], or [tokens, heads] for
    each token its own; offsets int32 [sequences + 1] (None: `sequences`
    prompts of equal length, default one); state [slots, heads, keys, values]
    fp32, slots and resume int32 [sequences]."""
    return (_ops or _load_ops()).linear_attention(q, k, v, log_decay, scale, sequences, offsets,
                                                  state, slots, resume, y, stream)


def lstm_linear_attention_workspace(tokens: int, heads: int, keys: int, values: int,
                                    sequences: int, equal_lengths: bool) -> int:
    """Bytes of workspace of lstm_linear_attention."""
    return load().lstm_linear_attention_workspace(tokens, heads, keys, values, sequences,
                                                  int(equal_lengths))


def lstm_linear_attention_step(q, k, v, log_decay, state, *, scale: float = 1.0, slots=None,
                               y=None, stream=None):
    """The next token of every sequence, q [sequences, q_heads, keys] and so on;
    returns y (new unless given) and moves the state on.  Arguments as
    lstm_linear_attention."""
    return (_ops or _load_ops()).linear_attention_step(q, k, v, log_decay, state, scale, slots, y,
                                                       stream)


_ACTIVATIONS = {None: LSTM_ACT_NONE, "relu": LSTM_ACT_RELU, "gelu": LSTM_ACT_GELU,
                "gelu_tanh": LSTM_ACT_GELU_TANH, "silu": LSTM_ACT_SILU}


def lstm_dense(x, w, bias=None, *, activation=None, residual=None, y=None, stream=None):
    """act(x w^T + bias) + residual of x [rows, in] and w [out, in] of one type;
    returns y [rows, out] (new unless given; may be residual).

    bias [out] fp32; activation None, "relu", "gelu", "gelu_tanh" or "silu";
    residual [rows, out] of x's type."""
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation {activation!r}, expected one of {list(_ACTIVATIONS)}")
    return (_ops or _load_ops()).dense(x, w, bias, _ACTIVATIONS[activation], residual, y, stream)


def lstm_dense_workspace(x, x_stride: int, w, w_stride: int, dtype: int, rows: int, inputs: int,
                         outputs: int) -> int:
    """Bytes of workspace of lstm_dense (x and w tensors)."""
    return load().lstm_dense_workspace(_ptr(x), x_stride, _ptr(w), w_stride, dtype, rows, inputs,
                                       outputs)
