"""The norm of the residual stream on the GPU, its 8-bit output and its gradients, against FP64."""
import numpy as np
import pytest
import torch

import linear_attention_gdn_gb300 as gdn
from tests.step_testutil import TINY, TYPES, U, f64, within

pytestmark = pytest.mark.gpu
EPS = 1e-6


def rows(T, C, dt, g, pad=0, shift=0, size=1.0):
    """[T, C] values, `pad` poisoned ones between the rows, `shift` values past an aligned address."""
    flat = torch.full((T * (C + pad) + shift + 16,), float("nan"), dtype=dt, device="cuda")
    v = flat.as_strided((T, C), (C + pad, 1), shift)
    v.copy_(size * torch.randn(T, C, generator=g))
    return v


def like(x):
    flat = torch.full((x.shape[0] * x.stride(0) + x.storage_offset() + 16,), float("nan"), dtype=x.dtype, device="cuda")
    return flat.as_strided(x.shape, x.stride(), x.storage_offset())


def gaps(x):
    """What lies between the rows."""
    return x.as_strided((max(x.shape[0] - 1, 0), x.stride(0) - x.shape[1]), (x.stride(0), 1), x.storage_offset() + x.shape[1])


def inverse(h, C):
    return 1 / np.sqrt((h * h).sum(-1, keepdims=True) / C + EPS)


# of a row's 1 / sqrt(mean + eps): C squares, each rounded, and summed in any order; then three operations
def root(C):
    return (C / 2 + 6) * U


def forward(T, C, dtype, residual=True, plain=True, group=None, pad=0, shift=0, seed=0, size=1.0, same=None):
    dt, unit = TYPES[dtype]
    g = torch.Generator().manual_seed(seed)
    x = rows(T, C, dt, g, pad, shift, size)
    r = rows(T, C, dt, g, pad, shift, 3 * size) if residual else None
    w = 1 + 0.2 * torch.randn(C, generator=g).cuda()
    X, Rr = f64(x), f64(r) if residual else 0.0
    h = {None: like(x) if residual else None, "x": x, "r": r}[same]
    y = like(x) if plain else None
    y8 = scales = None
    if group is not None:
        y8 = torch.zeros(T * C + 8, dtype=torch.float8_e4m3fn, device="cuda")[:T * C].view(T, C)
        scales = torch.full((T, C // (group or C)), float("nan"), device="cuda")
    prob = gdn.norm_problem(T, C, EPS, dt, group or 0, (C + pad,) * 4)
    gdn.gdn_add_norm_fwd(prob, x, r, w, h, y, y8, scales)
    if residual:
        within("h", h, X + Rr, unit * np.abs(X + Rr) + TINY)
        assert gaps(h).isnan().all()
    held = f64(h) if residual else X      # (the norm is of the rounded sum)
    z = held * inverse(held, C) * f64(w)
    rel = root(C) + 2 * U
    if plain:
        within("y", y, z, (unit + rel) * np.abs(z) + TINY)
        assert gaps(y).isnan().all()
    if group is not None:
        zz = z.reshape(T, -1, group or C)
        s = np.maximum(np.abs(zz).max(-1), 448 * 2.0 ** -100) / 448
        within("scales", scales, s, (rel + 2 * U) * s)
        got = f64(y8.float()).reshape(zz.shape)
        # z / s: the scale's and a product's roundings, then e4m3: 2^-4 of the value, or half its smallest step
        v = zz / s[..., None]
        within("y8", got, v, (2.0 ** -4 + 2 * rel + 8 * U) * np.abs(v) + 2.0 ** -10)
    return x, r, w, h, y, y8, scales


SHAPES = [(1, 1), (1, 8), (3, 40), (5, 100), (2, 256), (7, 512), (4, 1000), (3, 1024), (2, 1032), (200, 2048), (3, 4096), (2, 8200), (1, 16384), (2, 16400)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,C", SHAPES)
def test_forward(T, C, dtype):
    forward(T, C, dtype, group=0, seed=C)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,C,group", [(3, 32, 32), (5, 128, 64), (9, 384, 128), (2, 1024, 32), (300, 1152, 128), (2, 4096, 64), (1, 16384, 128), (1, 16512, 128)])
def test_groups(T, C, group, dtype):
    forward(T, C, dtype, plain=False, group=group, seed=C)
    forward(T, C, dtype, residual=False, group=group, seed=C)


@pytest.mark.parametrize("T,C", [(4, 64), (3, 2048), (2, 77)])
@pytest.mark.parametrize("kw", [dict(pad=8), dict(pad=3), dict(shift=8), dict(shift=1), dict(residual=False), dict(same="x"), dict(same="r"),
                                dict(size=1e-3), dict(size=300.0)])
def test_forward_layouts(T, C, kw):
    for dtype in TYPES:
        forward(T, C, dtype, group=0 if C % 64 else 32, **kw)


def test_general_rows_are_the_fast_ones():
    """A row on an odd address, by the other kernel: the same up to the sums' order."""
    a = forward(3, 512, "bf16", group=128, seed=5)
    b = forward(3, 512, "bf16", group=128, seed=5, shift=1)
    assert torch.equal(a[3], b[3])
    assert (a[6] - b[6]).abs().max() <= 2 * root(512) * a[6].abs().max()


@pytest.mark.parametrize("C", [64, 77, 2048])
def test_rows_of_zeros_and_without_limits(C):
    x = torch.zeros(4, C, dtype=torch.bfloat16, device="cuda")
    x[1, 0] = float("inf")
    x[2, C - 1] = float("nan")
    x[3] = 1
    y, y8 = torch.empty_like(x), torch.empty(4, C, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(4, 1, device="cuda")
    gdn.gdn_add_norm_fwd(gdn.norm_problem(4, C, EPS), x, None, torch.ones(C, device="cuda"), None, y, y8, s)
    assert (y[0] == 0).all() and (y8[0].float() == 0).all() and s[0, 0] == 2.0 ** -100
    assert y[1, 0].isnan() and (y[1, 1:] == 0).all() and y[2].isnan().all()
    assert torch.equal(y[3], x[3]) and (y8[3].float() == 448).all()


def backward(T, C, dtype, along=True, want_dw=True, pad=0, shift=0, same=None, seed=0):
    dt, unit = TYPES[dtype]
    g = torch.Generator().manual_seed(seed)
    h, dy = rows(T, C, dt, g, pad, shift, 2.0), rows(T, C, dt, g, pad, shift)
    res = rows(T, C, dt, g, pad, shift) if along else None
    w = 1 + 0.2 * torch.randn(C, generator=g).cuda()
    H, G, A, W = f64(h), f64(dy), f64(res) if along else 0.0, f64(w)
    dx = {None: like(h), "dy": dy, "dres": res}[same]
    dw = torch.full((C,), float("nan"), device="cuda") if want_dw else None
    prob = gdn.norm_problem(T, C, EPS, dt, 0, (C + pad,) * 4)
    ws = torch.full((max(gdn.gdn_add_norm_workspace_bytes(prob), 16),), 255, dtype=torch.uint8, device="cuda")
    gdn.gdn_add_norm_bwd(prob, h, w, dy, res, dx, dw, ws if want_dw else None)
    rho = inverse(H, C)
    xhat, gw = H * rho, G * W
    mean = (gw * xhat).sum(-1, keepdims=True) / C
    want = rho * (gw - xhat * mean) + A
    rel = root(C) + 8 * U
    loose = rho * (np.abs(gw) + np.abs(xhat) * np.abs(gw * xhat).sum(-1, keepdims=True) / C)
    within("dx", dx, want, unit * np.abs(want) + 3 * rel * loose + 2 * U * np.abs(A) + TINY)
    if pad:
        assert gaps(dx).isnan().all()
    if want_dw:
        within("dw", dw, (G * xhat).sum(0), (rel + (T + 4) * U) * np.abs(G * xhat).sum(0) + 1e-30)
    return h, w, dy, dx, dw


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,C", SHAPES + [(700, 64), (1300, 1100), (2000, 8)])
def test_backward(T, C, dtype):
    backward(T, C, dtype, seed=C)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,C,kw", [(2600, 1096, {}), (1900, 2048, dict(same="dy")), (1300, 4104, dict(same="dres")), (700, 8192, dict(along=False)),
                                    (650, 12296, dict(pad=8)), (500, 16384, {})])
def test_backward_of_more_rows_than_ctas(T, C, kw, dtype):
    backward(T, C, dtype, seed=T, **kw)


@pytest.mark.parametrize("T,C", [(4, 64), (3, 2048), (2, 77)])
@pytest.mark.parametrize("kw", [dict(pad=8), dict(pad=3), dict(shift=8), dict(shift=1), dict(along=False), dict(want_dw=False), dict(same="dy"),
                                dict(same="dres")])
def test_backward_layouts(T, C, kw):
    for dtype in TYPES:
        backward(T, C, dtype, **kw)


def test_backward_is_differences():
    """Central differences of the GPU's own forward in FP32: a step of 2^-7 in one direction.  What the difference leaves out
    is of third order: below 2^-14 of the derivative's size for rows of norm 1 values; the forward's roundings, root(C) of
    each output, are divided by the step."""
    T, C = 3, 96
    h, w, dy, dx, _ = backward(T, C, "fp32", along=False, seed=8)
    step = torch.randn(T, C, generator=torch.Generator().manual_seed(1)).cuda()
    y = [torch.empty(T, C, device="cuda") for _ in range(2)]
    e = 2.0 ** -7
    for s, out in zip((e, -e), y):
        gdn.gdn_add_norm_fwd(gdn.norm_problem(T, C, EPS, torch.float32), (h + s * step).contiguous(), None, w, None, out)
    left = ((f64(y[0]) - f64(y[1])) / (2 * e) * f64(dy)).sum()
    right = (f64(dx) * f64(step)).sum()
    size = np.abs(f64(dx) * f64(step)).sum()
    assert abs(left - right) <= 2.0 ** -14 * size * 8 + 2 * root(C) / (2 * e) * np.abs(f64(y[0]) * f64(dy)).sum()


def test_no_rows():
    dw = torch.full((64,), float("nan"), device="cuda")
    gdn.gdn_add_norm_bwd(gdn.norm_problem(0, 64), None, None, None, None, None, dw, None)
    assert (dw == 0).all()
    gdn.gdn_add_norm_fwd(gdn.norm_problem(0, 64), None, None, None, None, torch.empty(0, device="cuda").data_ptr() or 16, None, None)


def test_same_bits_again():
    a, b = backward(700, 512, "bf16", seed=3), backward(700, 512, "bf16", seed=3)
    assert torch.equal(a[3], b[3]) and torch.equal(a[4], b[4])


def test_rows_past_32_bit_offsets():
    """The last row of a stride that puts it past 2^32 bytes."""
    T, C, stride = 3, 64, 2 ** 30 + 8
    flat = torch.empty(2 * stride + C, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((T, C), (stride, 1))
    g = torch.Generator().manual_seed(0)
    v = torch.randn(T, C, generator=g).bfloat16().cuda()
    x.copy_(v)
    y = torch.empty_like(v)
    gdn.gdn_add_norm_fwd(gdn.norm_problem(T, C, EPS, strides=(stride, 0, 0, 0)), x, None, torch.ones(C, device="cuda"), None, y)
    z = f64(v) * inverse(f64(v), C)
    within("y", y, z, (2.0 ** -8 + root(C) + 2 * U) * np.abs(z))
