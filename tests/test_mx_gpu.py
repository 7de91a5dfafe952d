"""Microscaled operators on the GPU against the 64-bit oracle.

Stored formats are compared byte for byte.  Products are compared element by element with bounds that
count the roundings the kernels make (u = half a step, relative):
  H, dX   one bf16 rounding of the result, one of each adapter factor s U / s G (u = 2^-8), and
          fp32 accumulation
  dA, dB  the bf16 pair that carries s G (or a recomputed U): 2^-16, and fp32 accumulation
fp32 accumulation of n exact products: at most n roundings of 2^-23 (truncation) of the running sum,
whose magnitude the sum of the products' magnitudes bounds.
"""
import numpy as np
import pytest

from oracle import mx_oracle as M
from qlora_parameter_efficient_b200 import synthetic as S

import oracle as O

pytestmark = pytest.mark.gpu

U16 = 2.0 ** -8      # bf16
PAIR = 2.0 ** -16    # bf16 pair
U32 = 2.0 ** -23     # one fp32 accumulation


@pytest.fixture(scope="module")
def q():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from qlora_parameter_efficient_b200 import build
    build.build_library()
    import qlora_parameter_efficient_b200 as lib
    lib.load()
    return lib


def bf(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(torch.bfloat16)


def f64(t):
    import torch
    return t.detach().to(torch.float64).cpu().numpy()


def within(got, ref, tol, what):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float(np.max((np.abs(got - ref) / tol)[bad])))


def activation(rng, T, d):
    """Tokens with outlier channels, rounded to bf16."""
    x = rng.standard_normal((T, d))
    x[:, :: 61] *= 20
    return S.round_to_bf16(x.astype(np.float32)).astype(np.float64)


def make(seed, T, d_out, d_in, r):
    rng = np.random.default_rng(seed)
    W = rng.standard_normal((d_out, d_in)) * 0.141
    A = S.round_to_bf16((rng.standard_normal((r, d_in)) / np.sqrt(r)).astype(np.float32)).astype(np.float64)
    B = S.round_to_bf16((rng.standard_normal((d_out, r)) * 0.1).astype(np.float32)).astype(np.float64)
    X = activation(rng, T, d_in)
    dH = S.round_to_bf16(rng.standard_normal((T, d_out)).astype(np.float32)).astype(np.float64)
    return W.astype(np.float32), A, B, X, dH


def mx_weight(q, W):
    import torch
    codes, e = M.mxfp4_quantize(W)
    w = q.MXFP4Weight(torch.from_numpy(codes).cuda(), torch.from_numpy(M.tile_scales(e)).cuda(), *W.shape)
    return w, M.mxfp4_values(codes, e)


# ------------------------------------------------------------------ formats


def special_matrix(rows, cols, bf16):
    """Blocks of every kind: normal, zero, negative zero, ties, saturating, tiny, huge, subnormal."""
    rng = np.random.default_rng(rows * 1000 + cols)
    x = rng.standard_normal((rows, cols)).astype(np.float32)
    x *= np.exp2(rng.integers(-20, 20, (rows, cols // 32)).repeat(32, 1)).astype(np.float32)
    b = x.reshape(-1, 32)
    kinds = [np.zeros(32), -np.zeros(32),
             np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0] * 4) * np.array([1, -1] * 16),
             np.array([4.0, 7.9, 6.9, 7.0, 5.0, 6.0, -7.99, 0.1] * 4),
             np.array([1.0, 1.9999, 1.9921875, 0.0078125, 0.00390625, -1.99, 1.5, 0.5] * 4),
             np.full(32, 2.0 ** -120), np.linspace(-1, 1, 32) * 2.0 ** 127, np.linspace(-1, 1, 32) * 2.0 ** -126,
             np.arange(32) * 2.0 ** -133]
    for i, k in enumerate(kinds):
        if i < b.shape[0]:
            b[-1 - i] = k
    return S.round_to_bf16(x) if bf16 else x


SHAPES = [(1, 64), (3, 128), (31, 192), (128, 64), (129, 448), (200, 1088), (257, 320)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_mxfp4_bytes_and_values(q, rows, cols, dtype):
    import torch
    x = special_matrix(rows, cols, dtype == "bf16")
    t = torch.from_numpy(x).cuda()
    w = q.mxfp4_quantize(t.bfloat16() if dtype == "bf16" else t)
    codes, e = M.mxfp4_quantize(x)
    assert np.array_equal(w.codes.cpu().numpy(), codes)
    assert np.array_equal(w.scales.cpu().numpy(), M.tile_scales(e))
    ref = M.mxfp4_values(codes, e)
    assert np.array_equal(f64(q.mxfp4_dequantize(w, torch.float32)), ref)
    assert np.array_equal(f64(q.mxfp4_dequantize(w, torch.bfloat16)), ref)     # every value is a bf16 value


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_act8_bytes_and_values(q, rows, cols, dtype):
    import torch
    x = special_matrix(rows, cols, dtype == "bf16")
    t = torch.from_numpy(x).cuda()
    a = q.act8_quantize(t.bfloat16() if dtype == "bf16" else t)
    qi, e = M.act8_quantize(x)
    assert np.array_equal(a.q.cpu().numpy(), qi)
    assert np.array_equal(a.scales.cpu().numpy(), e)
    ref = M.act8_values(qi, e)
    assert np.array_equal(f64(q.act8_dequantize(a, torch.float32)), ref)
    assert np.array_equal(f64(q.act8_dequantize(a, torch.bfloat16)), ref)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_non_finite_blocks_decode_to_nan(q, bad):
    import torch
    x = np.ones((5, 128), np.float32)
    x[2, 40] = bad
    t = torch.from_numpy(x).cuda()
    for got, ref in ((q.mxfp4_dequantize(q.mxfp4_quantize(t), torch.float32), M.mxfp4_values(*M.mxfp4_quantize(x))),
                     (q.act8_dequantize(q.act8_quantize(t), torch.bfloat16), M.act8_values(*M.act8_quantize(x)))):
        assert np.array_equal(f64(got), ref, equal_nan=True)
        assert np.isnan(ref[2, 32:64]).all() and np.isfinite(ref).sum() == ref.size - 32


def test_every_code_and_scale_decodes(q):
    """All 16 codes under all 255 finite scales and the NaN scale."""
    import torch
    codes = np.tile(np.arange(16, dtype=np.uint8)[None] | (np.arange(16, dtype=np.uint8)[None] << 4), (256, 2))
    e = np.stack([np.arange(256), np.arange(256)], 1).astype(np.uint8)
    w = q.MXFP4Weight(torch.from_numpy(codes).cuda(), torch.from_numpy(M.tile_scales(e)).cuda(), 256, 64)
    with np.errstate(over="ignore"):
        ref = M.mxfp4_values(codes, e).astype(np.float32)
    assert np.array_equal(q.mxfp4_dequantize(w, torch.float32).cpu().numpy(), ref, equal_nan=True)


# ------------------------------------------------------------------ forward


def check_forward(q, T, d_out, d_in, r, seed=0):
    W, A, B, X, _ = make(seed, T, d_out, d_in, r)
    w, Wv = mx_weight(q, W)
    alpha = 2.0 * r
    H, U = q.qlora_linear_fwd_mxfp4(w, bf(X), bf(A), bf(B), alpha)
    assert q.get_device_error() == 0
    Hr, Ur = M.layer_forward(Wv, X, A, B, 2.0)
    X4 = M.mxfp4_values(*M.mxfp4_quantize(X))
    acc_u = d_in * U32 * (np.abs(X) @ np.abs(A).T)
    within(f64(U), Ur, U16 * np.abs(Ur) + acc_u + 1e-30, "U")
    tol = (U16 * np.abs(Hr) + (U16 * 2 * np.abs(Ur) + 2 * acc_u) @ np.abs(B).T
           + (d_in + r) * U32 * (np.abs(X4) @ np.abs(Wv).T + 2 * np.abs(Ur) @ np.abs(B).T))
    within(f64(H), Hr, tol + 1e-30, "H")


FWD = [(1, 64, 64, 1), (1, 256, 256, 16), (1, 1000, 4096, 16), (2, 130, 192, 5), (7, 77, 320, 8), (16, 513, 1088, 64),
       (17, 128, 256, 33), (40, 300, 576, 100), (64, 129, 2048, 128), (65, 64, 64, 8), (127, 200, 448, 12),
       (128, 256, 512, 16), (200, 1001, 1024, 7), (300, 384, 704, 64), (513, 520, 960, 128),
       # 256 x 256 tiles: fewer than the pairs of SMs (split along K), more (a split last wave), whole
       (600, 513, 1088, 64), (1000, 300, 320, 5), (1025, 1000, 2048, 16), (2600, 2100, 1088, 8), (700, 77, 64, 16)]


@pytest.mark.parametrize("T,d_out,d_in,r", FWD)
def test_forward(q, T, d_out, d_in, r):
    check_forward(q, T, d_out, d_in, r, seed=T + d_out)


# ------------------------------------------------------------------ backward


def check_backward(q, T, d_out, d_in, r, base, ckpt, keep_u, seed=0):
    import torch
    W, A, B, X, dH = make(seed, T, d_out, d_in, r)
    if base == "mx":
        w, Wv = mx_weight(q, W)
    else:
        w = q.nf4_quantize(torch.from_numpy(W).cuda())
        Wv = O.nf4_dequantize(*O.nf4_quantize(W)[:3], d_out, d_in, out="bf16").astype(np.float64)
    s, alpha = 2.0, 2.0 * r
    U = S.round_to_bf16((X @ A.T).astype(np.float32)).astype(np.float64) if keep_u else None
    if ckpt:
        qi, e = M.act8_quantize(X)
        act = q.Act8(torch.from_numpy(qi).cuda(), torch.from_numpy(e).cuda())
        X = M.act8_values(qi, e)
    else:
        act = bf(X)
    fn = q.qlora_linear_bwd_mxfp4 if base == "mx" else q.qlora_linear_bwd_act8
    dX, dA, dB = fn(w, act, bf(dH), bf(A), bf(B), alpha, U_saved=bf(U) if keep_u else None)
    assert q.get_device_error() == 0
    dXr, dAr, dBr = M.layer_backward(Wv, X, dH, A, B, s, U)
    G = np.abs(dH @ B)
    acc_g = d_out * U32 * (np.abs(dH) @ np.abs(B))
    Ua = np.abs(X @ A.T)
    acc_u = d_in * U32 * (np.abs(X) @ np.abs(A).T)
    within(f64(dX), dXr, U16 * np.abs(dXr) + s * (U16 * G + acc_g) @ np.abs(A)
           + (d_out + r) * U32 * (np.abs(dH) @ np.abs(Wv) + s * G @ np.abs(A)) + 1e-30, "dX")
    within(f64(dA), dAr, s * ((PAIR + T * U32) * G + acc_g).T @ np.abs(X) + 1e-30, "dA")
    tol_u = (T * U32) * np.abs(U) if keep_u else (PAIR + T * U32) * Ua + acc_u
    within(f64(dB), dBr, s * np.abs(dH).T @ tol_u + U32 * np.abs(dBr) + 1e-30, "dB")


BWD = [(1, 64, 64, 1), (3, 77, 128, 5), (64, 200, 192, 8), (65, 256, 320, 16), (130, 513, 448, 33),
       (257, 128, 1088, 64), (300, 1001, 512, 100), (513, 300, 704, 128), (1100, 2000, 576, 16),
       (2600, 1100, 2112, 8)]


@pytest.mark.parametrize("keep_u", [True, False])
@pytest.mark.parametrize("base,ckpt", [("mx", True), ("mx", False), ("nf4", True)])
@pytest.mark.parametrize("T,d_out,d_in,r", BWD)
def test_backward(q, T, d_out, d_in, r, base, ckpt, keep_u):
    check_backward(q, T, d_out, d_in, r, base, ckpt, keep_u, seed=T + d_in)
