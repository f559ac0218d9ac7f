"""Plain fp64 definitions of the norm and linear layers and their gradients, 8-bit rows and
checkpoints, with a bound on what stores in fewer bits and fp32 arithmetic may change.

The bounds count half a step of the stored type (bf16 2^-8, e4m3 2^-4 of the value, half a
subnormal step below), 2^-23 of the sum of magnitudes for every 16 products that the matrix
unit adds (it cuts what lies behind an accumulator's 24 bits) and for each of at most 16 further
additions, 2^-24 for every fp32 operation elsewhere, and 2^-20 of the value for the device's
exponential and division.  Where a value is rounded before it is used, the rounding is made here
too, and values so near a rounding's border that fp32 may see them on its other side count
a whole step.
"""

import numpy as np

from .activations import silu
from .bf16 import round_to_bf16

BF16 = 2.0 ** -8
STEP = 2.0 ** -23
FAST = 2.0 ** -20
BLOCK = 32
LEAST = 2.0 ** -126


def round_to_e4m3(x):
    """Nearest e4m3 value, ties to even, of |x| <= 448: four significant bits, subnormal steps of 2^-9."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(x)
    q = np.maximum(e - 4, -9)
    return np.ldexp(np.rint(np.ldexp(x, -q)), q)


# ------------------------------------------------------------------ norm


def norm(X, R, w, eps, rms=True):
    """(S before its rounding, y)."""
    S = X if R is None else X + R
    return S, w * S / np.sqrt((S * S).mean(axis=1, keepdims=True) + eps) if rms else S


def norm_bound(S, y, rms=True):
    """Error of y in fp32: the sum of squares in at most 64 additions one after the other, which counts half
    in its root, and a few operations."""
    return 40 * 2.0 ** -24 * np.abs(y) if rms else 2.0 ** -24 * np.abs(y)


def row_scales(y):
    """Scales of y's rows: infinite and NaN values do not count."""
    most = np.where(np.isfinite(y), np.abs(y), 0.0).max(axis=1)
    return np.maximum(most / 448.0, LEAST)


def norm_grad(S, w, dY, dS, eps):
    """{name: (gradient, bound)}."""
    M, D = S.shape
    r = 1.0 / np.sqrt((S * S).mean(axis=1, keepdims=True) + eps)
    g, xh = w * dY, S * r
    dots = (g * xh).mean(axis=1, keepdims=True)
    dX = r * (g - xh * dots)
    err = 80 * 2.0 ** -24 * r * (np.abs(g) + np.abs(xh) * np.abs(g * xh).mean(axis=1, keepdims=True))
    if dS is not None:
        dX = dX + dS
        err = err + 2.0 ** -24 * np.abs(dX)
    dw = (dY * xh).sum(axis=0)
    e_dw = (M + 112) * 2.0 ** -24 * np.abs(dY * xh).sum(axis=0)
    return {"dX": (dX, err + BF16 * (np.abs(dX) + err)), "dw": (dw, e_dw + BF16 * (np.abs(dw) + e_dw))}


# ------------------------------------------------------------------ linear


_C = np.sqrt(2.0 / np.pi)


def act(z, kind):
    if kind == "swiglu":
        n = z.shape[1] // 2
        return silu(z[:, :n]) * z[:, n:]
    if kind == "gelu":
        return 0.5 * z * (1 + np.tanh(_C * (z + 0.044715 * z ** 3)))
    return np.maximum(z, 0.0) if kind == "relu" else z


def act_bound(z, dz, kind):
    """Error of act(z) for an error dz of z, and the fast exponential's."""
    if kind == "swiglu":
        n = z.shape[1] // 2
        g, u, dg, du = z[:, :n], z[:, n:], dz[:, :n], dz[:, n:]
        return 1.1 * np.abs(u) * dg + np.abs(silu(g)) * du + 1.1 * dg * du + FAST * np.abs(silu(g) * u)
    if kind == "gelu":
        arg = 2 * _C * np.abs(z + 0.044715 * z ** 3)
        t = np.tanh(arg / 2)
        return 1.13 * dz + (FAST + 4 * STEP * arg * (1 - t ** 2)) * np.abs(z)
    return dz


def slope(z, dY, kind):
    """(dZ, its error in fp32)."""
    if kind == "none":
        return dY, np.zeros_like(dY)
    if kind == "relu":
        return np.where(np.isnan(z), np.nan, dY * (z > 0)), np.zeros_like(dY)
    if kind == "gelu":
        t = np.tanh(_C * (z + 0.044715 * z ** 3))
        inner = _C * (1 + 3 * 0.044715 * z ** 2)
        arg = 2 * _C * np.abs(z + 0.044715 * z ** 3)
        fast = FAST + 4 * STEP * arg * (1 - t ** 2)
        return dY * (0.5 * (1 + t) + 0.5 * z * (1 - t ** 2) * inner), np.abs(dY) * fast * (1 + np.abs(z) * 2 * inner)
    n = z.shape[1] // 2
    g, u = z[:, :n], z[:, n:]
    s = np.exp(-np.logaddexp(0.0, -g))
    dz = np.concatenate([dY * u * (s + g * s * (1 - s)), dY * g * s], axis=1)
    err = FAST * np.concatenate([np.abs(dY * u) * s * (1 + np.abs(g) * (2 - s)), np.abs(dY * g) * s], axis=1)
    return dz, err


def pre(X, Xs, Wt, Ws, bias):
    """(z, bound) of 16-bit operands, or of 8-bit rows and their scales."""
    z, mag = X @ Wt.T, np.abs(X) @ np.abs(Wt).T
    if Xs is not None:
        scale = Xs[:, None] * Ws[None, :]
        z, mag = z * scale, mag * np.abs(scale)
    err = (X.shape[1] / 16 + 16) * STEP * mag
    if bias is not None:
        z = z + bias
        err = err + STEP * np.abs(z)
    return z, err


def linear(X, Xs, Wt, Ws, bias, R, kind):
    """(Y, bound, z, bound of z)."""
    z, dz = pre(X, Xs, Wt, Ws, bias)
    Y, err = act(z, kind), act_bound(z, dz, kind)
    if R is not None:
        Y = Y + R
        err = err + STEP * np.abs(Y)
    return Y, err + BF16 * (np.abs(Y) + err), z, dz


def exponents(z, parts):
    """Ze [M, parts, blocks] of z [M, parts * N]."""
    M, N = z.shape[0], z.shape[1] // parts
    blocks = -(-N // BLOCK)
    pad = np.zeros((M, parts, blocks * BLOCK))
    pad[:, :, :N] = np.where(np.isfinite(z), np.abs(z), 0.0).reshape(M, parts, N)
    most = pad.reshape(M, parts, blocks, BLOCK).max(axis=3)
    e = np.full(most.shape, -126)
    # the smallest power of two by which the block fits, found by trying
    for p in range(-126, 121):
        e = np.where((most > 448.0 * 2.0 ** p) & (e <= p), p + 1, e)
    return e + 127


def units(e, parts, N):
    """2^(Ze - 127) for every column, [M, parts * N]."""
    M = e.shape[0]
    return np.repeat(2.0 ** (e.astype(np.float64) - 127), BLOCK, axis=2)[:, :, :N].reshape(M, parts * N)


def checkpoint(z, parts):
    """(values in e4m3, Ze) of z [M, parts * N]."""
    e = exponents(z, parts)
    return round_to_e4m3(z / units(e, parts, z.shape[1] // parts)), e


def linear_grad(X, Xs, Wt, z, dY, kind):
    """{name: (gradient, bound)}; z: what the checkpoint stands for (None for kind "none").  X in bf16,
    or the values of 8-bit rows with scales Xs = f * +-2^e, f in [1, 2): dZ is rounded times f then,
    for dWt, and with an activation for dX, too."""
    dz, err = slope(z, dY, kind)
    err = err + 2.0 ** -24 * np.abs(dz)

    def rounded(f, exact):
        v, e = dz * f, err * f + (0 if np.isscalar(f) else 2.0 ** -24 * np.abs(dz * f))
        if exact:
            return v, np.zeros_like(v)
        d = round_to_bf16(v)
        return d, np.maximum(np.abs(round_to_bf16(v - e) - d), np.abs(round_to_bf16(v + e) - d))
    f, x = 1.0, X
    if Xs is not None:
        fraction, exponent = np.frexp(Xs)
        f, x = 2 * np.abs(fraction[:, None]), X * np.copysign(np.ldexp(1.0, exponent - 1), Xs)[:, None]
    dw, sw = rounded(f, kind == "none" and Xs is None)
    dx, sx = (dw / f, sw / f) if kind != "none" else rounded(1.0, True)
    out = {}
    M, H = dz.shape
    for name, value, mag, loose, depth in (
            ("dX", dx @ Wt, np.abs(dx) @ np.abs(Wt), sx @ np.abs(Wt), H),
            ("dWt", dw.T @ x, np.abs(dw).T @ np.abs(x), sw.T @ np.abs(x), M)):
        e = (depth / 16 + 16) * STEP * mag + loose
        out[name] = (value, e + BF16 * (np.abs(value) + e))
    b = dz.sum(axis=0)
    e = err.sum(axis=0) + (M + 64) * 2.0 ** -24 * np.abs(dz).sum(axis=0)
    out["dbias"] = (b, e + BF16 * (np.abs(b) + e))
    return out
