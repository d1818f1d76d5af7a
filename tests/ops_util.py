"""Shared helpers of the state-space operators' tests."""
import numpy as np
import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# a rounding to nearest: half the spacing above 1, relatively, and half the
# smallest subnormal (fp32's and bf16's play no part)
ROUND = {name: (torch.finfo(t).eps / 2, 2.0 ** -25 if t == torch.float16 else 0.0)
         for name, t in DTYPES.items()}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def uniform(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def slice_of(t, pad_left, pad_right):
    """The same values as columns of a wider matrix whose other columns are NaN."""
    wide = torch.full((t.shape[0], t.shape[1] + pad_left + pad_right), float("nan"),
                      dtype=t.dtype, device=t.device)
    view = wide[:, pad_left:pad_left + t.shape[1]]
    view.copy_(t)
    return view


def at_element(t, offset):
    """The same values, densely packed, `offset` elements into an allocation that is
    NaN elsewhere."""
    flat = torch.full((t.numel() + 8,), float("nan"), dtype=t.dtype, device=t.device)
    view = flat[offset:offset + t.numel()].view(t.shape)
    view.copy_(t)
    return view


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def assert_close(got, ref, bound, dtype, what=""):
    """got (a tensor of dtype) within the fp32 bound of ref and one rounding."""
    got = f64(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN elsewhere"
    # beyond the type's range a rounding to nearest gives an infinity
    over = np.abs(ref) > torch.finfo(DTYPES[dtype]).max
    ref = np.where(over, np.copysign(np.inf, ref), ref)
    rel, least = ROUND[dtype]
    # the rounding applies to the value that carries the fp32 error
    tol = bound * (1 + rel) + rel * np.abs(ref) + least
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(got - ref) <= tol) | (got == ref) | (np.isnan(got) & np.isnan(ref)))
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - ref) / (tol + 1e-300), 0)), bad.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; worst at {i}: got "
                             f"{got[i]!r}, expected {ref[i]!r}, tolerance {tol[i]:.3e}")
