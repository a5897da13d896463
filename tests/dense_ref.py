"""Plain float64 evaluation of the training products and of bounds on what the
kernels may differ from it by, element by element.

The bounds follow the kernels' roundings, to first order:
  - a sum of n exact products in fp32, in any order and grouping, is off by at
    most n 2^-24 times the sum of the products' magnitudes per rounding; twice
    that is allowed for, the matrix instructions' inner sums being no IEEE sums;
  - exp, division and the few products of f and f' cost under 2^-18 relative
    (the exponent's argument, up to ~100, is rounded to fp32: 100 * 2^-24);
  - one rounding to a type is at most eps / 2 relative (bf16: 2^-8)."""

import numpy as np
import torch

BF16, F32 = torch.bfloat16, torch.float32
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
FUN = 2.0 ** -18
# smallest normal magnitude of either type: below it a rounding is absolute
TINY = 2.0 ** -126


def act(fn, z):
    """f(z), f'(z), and a bound on |f''|."""
    if fn == "none":
        return z, torch.ones_like(z), 0.0
    if fn == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z)), (z > 0).double(), 0.0
    if fn == "silu":
        s = 1 / (1 + torch.exp(-z))
        return z * s, s * (1 + z * (1 - s)), 0.5
    c = np.sqrt(2 / np.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return (0.5 * z * (1 + t),
            0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z), 1.2)


def dot(a, b, ea=None, eb=None):
    """a b and the bound of its fp32 sum given bounds on a and b."""
    n = a.shape[-1]
    err = 2 * n * 2.0 ** -24 * (a.abs() @ b.abs())
    if ea is not None:
        err = err + ea @ b.abs()
    if eb is not None:
        err = err + a.abs() @ eb
    return a @ b, err


def rounded(v, err, dtype):
    return err + U[dtype] * (v.abs() + err) + TINY


def f_bounds(fn, z, ez):
    """f, f' at z with their bounds when z is off by up to ez."""
    f, df, d2 = act(fn, z)
    fun = FUN if fn in ("silu", "gelu_tanh") else 0.0
    ef = 1.2 * ez + fun * f.abs()
    edf = d2 * 1.2 * ez + 2 * fun + torch.zeros_like(z)
    if fn == "relu":
        edf = torch.where(z.abs() <= ez, torch.ones_like(z), torch.zeros_like(z))
    return f, df, ef, edf


def glu_forward(x, wg, wu, fn, out):
    g, eg = dot(x, wg.T)
    u, eu = dot(x, wu.T)
    f, _, ef, _ = f_bounds(fn, g, eg)
    h = f * u
    eh = ef * u.abs() + f.abs() * eu + ef * eu + 2.0 ** -23 * h.abs()
    return h, rounded(h, eh, out)


def glu_backward(x, wg, wu, dh, fn, grad):
    """(dx, dwg, dwu, h), each with its bound."""
    g, eg = dot(x, wg.T)
    u, eu = dot(x, wu.T)
    f, df, ef, edf = f_bounds(fn, g, eg)
    h = f * u
    eh = rounded(h, ef * u.abs() + f.abs() * eu + ef * eu + 2.0 ** -23 * h.abs(), BF16)
    dg, du = dh * u * df, dh * f
    edg = dh.abs() * (eu * df.abs() + u.abs() * edf + eu * edf) + 2.0 ** -22 * dg.abs()
    edu = dh.abs() * ef + 2.0 ** -23 * du.abs()
    edg, edu = rounded(dg, edg, BF16), rounded(du, edu, BF16)
    # one sum over both halves
    dx, edx = dot(torch.cat([dg, du], 1), torch.cat([wg, wu], 0), torch.cat([edg, edu], 1))
    dwg, edwg = dot(dg.T, x, edg.T)
    dwu, edwu = dot(du.T, x, edu.T)
    return [(dx, rounded(dx, edx, grad)), (dwg, rounded(dwg, edwg, grad)),
            (dwu, rounded(dwu, edwu, grad)), (h, eh)]


def linear_forward(x, w, bias, residual, fn, out):
    z, ez = dot(x, w.T)
    if bias is not None:
        z = z + bias
        ez = ez + 2.0 ** -24 * z.abs()
    f, _, ef, _ = f_bounds(fn, z, ez)
    y = f if residual is None else f + residual
    return y, rounded(y, ef + 2.0 ** -24 * y.abs(), out)


def linear_backward(x, w, bias, dy, fn, grad):
    """(dx, dw, dbias), each with its bound."""
    dz, edz = dy, torch.zeros_like(dy)
    raw = edz
    if fn != "none":
        z, ez = dot(x, w.T)
        if bias is not None:
            z = z + bias
            ez = ez + 2.0 ** -24 * z.abs()
        _, df, _, edf = f_bounds(fn, z, ez)
        dz = dy * df
        raw = dy.abs() * edf + 2.0 ** -23 * dz.abs()
        edz = rounded(dz, raw, BF16)
    dx, edx = dot(dz, w, edz)
    dw, edw = dot(dz.T, x, edz.T)
    # the bias gradient is summed before dz is rounded
    db = dz.sum(0)
    edb = raw.sum(0) + 2 * max(1, dz.shape[0]) * 2.0 ** -24 * dz.abs().sum(0)
    return [(dx, rounded(dx, edx, grad)), (dw, rounded(dw, edw, grad)), (db, edb + TINY)]


def check(name, got, want, bound):
    got = got.double().cpu()
    assert got.shape == want.shape, f"{name}: {got.shape} {want.shape}"
    assert torch.isfinite(got).all(), f"{name}: non-finite output"
    over = (got - want).abs() - bound
    if over.numel() and over.max() > 0:
        i = int(over.argmax())
        raise AssertionError(f"{name}: element {i} is {got.flatten()[i]:.6e}, wanted "
                             f"{want.flatten()[i]:.6e} within {bound.flatten()[i]:.3e}")


def segments(offsets, R, E):
    """(expert, first row, end) from host offsets (None: all rows of expert 0)."""
    if offsets is None:
        return [(0, 0, R)]
    return [(e, offsets[e], offsets[e + 1]) for e in range(E)]
