"""Shared by the GPU tests of the step and q/k entry points: element types with the rounding of one store, and
tensors with poison around them."""
import numpy as np
import torch

# type, and the largest relative error of one rounding to it
TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "fp16": (torch.float16, 2.0 ** -11), "fp32": (torch.float32, 2.0 ** -24)}
U = 2.0 ** -24            # of one FP32 operation
TINY = 2.0 ** -24         # fp16's smallest step: values below its normal range round to multiples of it


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def within(name, got, want, tol):
    """|got - want| <= tol, elementwise; got is finite."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert np.isfinite(got).all(), f"{name}: non-finite values"
    over = np.abs(got - want) - tol
    assert (over <= 0).all(), f"{name}: {np.abs(got - want).max():.3e} off, {over.max():.3e} over, at {np.unravel_index(over.argmax(), over.shape)}"


def strided(x, token, head=None):
    """A copy of x [T, heads, D] or [T, C] on the GPU with `token` elements from token to token (and `head` from head
    to head), poison between the rows."""
    T = x.shape[0]
    flat = torch.full((max(T, 1) * token + 64,), float("nan"), dtype=x.dtype, device="cuda")
    size, stride = tuple(x.shape), (token, head, 1) if x.dim() == 3 else (token, 1)
    v = flat.as_strided(size, stride)
    v.copy_(x)
    return v
