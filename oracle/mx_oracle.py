"""Plain numpy (fp64) definitions of the microscaled formats and of the layer that uses them.

OCP Microscaling Formats v1.0, blocks of 32 consecutive elements of a row, one E8M0 scale byte e per
block (2^(e - 127); 255: NaN):
  MXFP4   e = max(0, floor(log2 max|x|) - 2 + 127), element E2M1(x 2^(127 - e)), ties to even, to 6
  MXINT8  e = max(0, floor(log2 max|x|) + 127),     element rint(x 2^(133 - e)), to +-127
A block with a NaN or an infinity gets e = 255 and elements 0.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# borders between neighbouring magnitudes, and whether a value on the border goes to the upper one
# (the neighbour whose code is even)
_BORDERS = (E2M1[1:] + E2M1[:-1]) / 2
_TIE_UP = np.arange(7) % 2 == 1


def _block_exponents(b, top):
    """E8M0 bytes of blocks [..., 32]."""
    with np.errstate(invalid="ignore"):
        m = np.max(np.abs(b), axis=-1)
    bad = ~np.isfinite(b).all(axis=-1)
    m = np.where(bad, 1.0, m)
    _, ex = np.frexp(m)                      # m = f 2^ex, f in [0.5, 1): floor(log2 m) = ex - 1
    e = np.where(m > 0, ex - 1 - top + 127, 0)
    return np.where(bad, 255, np.clip(e, 0, 254)).astype(np.int64), bad


def mxfp4_quantize(X):
    """(codes uint8 [rows, cols/2], scale bytes uint8 [rows, cols/32]) of X [rows, cols]."""
    X = np.asarray(X, np.float64)
    rows, cols = X.shape
    b = X.reshape(rows, cols // 32, 32)
    e, bad = _block_exponents(b, 2)
    y = np.where(bad[..., None], 0.0, b) * np.exp2(127.0 - np.where(bad, 127, e))[..., None]
    a = np.abs(y)[..., None]
    mag = np.where(_TIE_UP, a >= _BORDERS, a > _BORDERS).sum(-1)
    code = (mag + 8 * np.signbit(y)).astype(np.uint8).reshape(rows, cols)
    return code[:, 0::2] | (code[:, 1::2] << 4), e.astype(np.uint8)


def mxfp4_values(codes, e):
    rows, cols = codes.shape[0], codes.shape[1] * 2
    c = np.empty((rows, cols), np.int64)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    v = E2M1[c & 7] * np.where(c & 8, -1.0, 1.0)
    return v * _scale(e, 127)


def _scale(e, bias):
    s = np.exp2(e.astype(np.float64) - bias)
    return np.repeat(np.where(e == 255, np.nan, s), 32, axis=1)


def tile_scales(e):
    """Scale bytes [rows, blocks] in the stored order: tiles of 128 rows x 4 blocks, 0 outside."""
    rows, nb = e.shape
    out = np.zeros(((rows + 127) // 128) * ((nb + 3) // 4) * 512, np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    out[((r // 128) * ((nb + 3) // 4) + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4] = e
    return out


def act8_quantize(X):
    """(q int8 [T, d_in], scale bytes uint8 [T, d_in/32])."""
    X = np.asarray(X, np.float64)
    T, d = X.shape
    b = X.reshape(T, d // 32, 32)
    e, bad = _block_exponents(b, 0)
    y = np.where(bad[..., None], 0.0, b) * np.exp2(133.0 - np.where(bad, 133, e))[..., None]
    return np.clip(np.rint(y), -127, 127).astype(np.int8).reshape(T, d), e.astype(np.uint8)


def act8_values(q, e):
    return q.astype(np.float64) * _scale(e, 133)


def layer_forward(W, X, A, B, s):
    """(H, U) for the dequantized weight W and the unquantized X."""
    U = X @ A.T
    return mxfp4_values(*mxfp4_quantize(X)) @ W.T + s * (U @ B.T), U


def layer_backward(W, X, dH, A, B, s, U=None):
    """(dX, dA, dB); X holds the values the backward sees, U the saved one or None."""
    U = X @ A.T if U is None else U
    G = dH @ B
    return dH @ W + s * (G @ A), s * (G.T @ X), s * (dH.T @ U)
