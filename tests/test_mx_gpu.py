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


# ------------------------------------------------------------------ products that are exact


def test_exact_products(q):
    """Values for which every step is exact: the block-scaled product must be the integer sum itself."""
    import torch
    rng = np.random.default_rng(3)
    for T, d_out, d_in in ((1, 130, 320), (40, 256, 512), (150, 129, 704), (700, 512, 1024)):
        mags = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, -6.0, -1.0])
        W, X = (rng.choice(mags, s) for s in ((d_out, d_in), (T, d_in)))
        W[:, ::32] = 6.0                   # every block's scale is 2^0
        X[:, 1::32] = 4.0
        for b in range(d_in // 32):        # and then a power of two of its own
            W[:, 32 * b:32 * b + 32] *= 2.0 ** (b % 3 - 1)
            X[:, 32 * b:32 * b + 32] *= 2.0 ** (b % 2)
        X *= (np.abs(rng.standard_normal((T, 1))) < 0.7)          # some tokens are all zero
        w = q.mxfp4_quantize(torch.from_numpy(W.astype(np.float32)).cuda())
        A, B = np.zeros((8, d_in)), np.zeros((d_out, 8))
        H, _ = q.qlora_linear_fwd_mxfp4(w, bf(X), bf(A), bf(B), 8.0)
        ref = torch.from_numpy((X @ W.T).astype(np.float32)).to(torch.bfloat16).double().numpy()
        assert np.array_equal(f64(H), ref), (T, d_out, d_in)


def test_zero_rank_term_and_zero_activation(q):
    import torch
    W, A, B, X, dH = make(1, 5, 64, 128, 8)
    w, _ = mx_weight(q, W)
    H, U = q.qlora_linear_fwd_mxfp4(w, bf(X * 0), bf(A), bf(B), 16.0)
    assert not H.any() and not U.any()
    a = q.act8_quantize(bf(X * 0))
    assert not a.q.any() and not a.scales.any()
    dX, dA, dB = q.qlora_linear_bwd_mxfp4(w, a, bf(dH * 0), bf(A), bf(B), 16.0)
    assert not dX.any() and not dA.any() and not dB.any()
    torch.cuda.synchronize()


# ------------------------------------------------------------------ NaN and infinity stay where they belong


@pytest.mark.parametrize("T", [3, 16, 50, 130, 700])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_non_finite_token_and_weight_row(q, T, bad):
    import torch
    W, A, B, X, dH = make(2, T, 200, 320, 8)
    t, n = T // 2, 77
    Wb, Xb = W.copy(), X.copy()
    w0, _ = mx_weight(q, W)
    H0, _ = q.qlora_linear_fwd_mxfp4(w0, bf(X), bf(A), bf(B), 16.0)
    Xb[t, 200] = bad
    H1, _ = q.qlora_linear_fwd_mxfp4(w0, bf(Xb), bf(A), bf(B), 16.0)
    H0, H1 = f64(H0), f64(H1)
    assert np.isnan(H1[t]).all()
    keep = np.arange(T) != t
    assert np.array_equal(H1[keep], H0[keep])
    Wb[n, 5] = bad
    wb = q.mxfp4_quantize(torch.from_numpy(Wb).cuda())
    H2 = f64(q.qlora_linear_fwd_mxfp4(wb, bf(X), bf(A), bf(B), 16.0)[0])
    assert np.isnan(H2[:, n]).all()
    cols = np.arange(200) != n
    assert np.array_equal(H2[:, cols], H0[:, cols])
    # backward: a token's bad block reaches dA in its columns only, and no dX
    a0, a1 = q.act8_quantize(bf(X)), q.act8_quantize(bf(Xb))
    U = bf(X @ A.T)
    g0 = [f64(g) for g in q.qlora_linear_bwd_mxfp4(w0, a0, bf(dH), bf(A), bf(B), 16.0, U_saved=U)]
    g1 = [f64(g) for g in q.qlora_linear_bwd_mxfp4(w0, a1, bf(dH), bf(A), bf(B), 16.0, U_saved=U)]
    assert np.array_equal(g0[0], g1[0]) and np.array_equal(g0[2], g1[2])
    block = slice(192, 224)
    assert np.isnan(g1[1][:, block]).all()
    assert np.array_equal(np.delete(g1[1], np.r_[block], 1), np.delete(g0[1], np.r_[block], 1))


def test_infinite_gradient(q):
    """An infinity in dH gives infinities or NaN where the formula does, not everywhere."""
    W, A, B, X, dH = make(4, 70, 96, 128, 8)
    w, Wv = mx_weight(q, W)
    dH[10, 3] = np.inf
    with np.errstate(invalid="ignore"):
        ref = M.layer_backward(Wv, X, dH, A, B, 2.0)
        got = [f64(g) for g in q.qlora_linear_bwd_mxfp4(w, bf(X), bf(dH), bf(A), bf(B), 16.0)]
    for r, g in zip(ref, got):
        assert not np.isfinite(g[~np.isfinite(r)]).any()
    ok = np.arange(70) != 10
    assert np.isfinite(got[0][ok]).all()
    rows = np.arange(96) != 3
    assert np.isfinite(got[2][rows]).all()


# ------------------------------------------------------------------ how a program uses them


def layer(q, T, d_out, d_in, r, seed=0, base="mx"):
    import torch
    W, A, B, X, dH = make(seed, T, d_out, d_in, r)
    w = q.mxfp4_quantize(torch.from_numpy(W).cuda()) if base == "mx" else q.nf4_quantize(torch.from_numpy(W).cuda())
    return w, bf(X), bf(dH), bf(A), bf(B)


@pytest.mark.parametrize("T", [1, 9, 33, 129, 300, 600])
def test_results_do_not_depend_on_the_workspace_or_the_run(q, T):
    """A workspace full of NaN bytes, one full of zeros and a repeated call give the same bits."""
    import torch
    w, X, dH, A, B = layer(q, T, 333, 704, 5)
    outs = []
    for fill in (0xFF, 0, 0x7F):
        need = max(q.workspace_bytes(op, q.BF16, T, 333, 704, 5) for op in (q.OP_FWD_MXFP4, q.OP_BWD_MXFP4))
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        H, U = q.qlora_linear_fwd_mxfp4(w, X, A, B, 10.0, ws=ws)
        ws.fill_(fill)
        a = q.act8_quantize(X)
        g = q.qlora_linear_bwd_mxfp4(w, a, dH, A, B, 10.0, ws=ws)
        ws.fill_(fill)
        g2 = q.qlora_linear_bwd_mxfp4(w, X, dH, A, B, 10.0, U_saved=U, ws=ws)
        outs.append([H, U, *g, *g2])
    assert q.get_device_error() == 0
    for o in outs[1:]:
        for x, y in zip(outs[0], o):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("T,d_out,d_in,r", [(1, 100, 128, 3), (16, 129, 192, 8), (60, 77, 320, 8), (129, 200, 448, 16),
                                            (257, 1001, 640, 33), (600, 300, 704, 100)])
def test_nothing_is_written_past_the_outputs(q, T, d_out, d_in, r):
    import torch
    w, X, dH, A, B = layer(q, T, d_out, d_in, r)

    def guarded(rows, cols, dtype):
        pad = 4096
        buf = torch.full((rows * cols + 2 * pad,), 7, dtype=dtype, device="cuda")
        return buf, buf[pad:pad + rows * cols].view(rows, cols)

    bH, H = guarded(T, d_out, torch.bfloat16)
    bU, U = guarded(T, r, torch.bfloat16)
    bX, dX = guarded(T, d_in, torch.bfloat16)
    bA, dA = guarded(r, d_in, torch.float32)
    bB, dB = guarded(d_out, r, torch.float32)
    bq, aq = guarded(T, d_in, torch.int8)
    bs, asc = guarded(T, d_in // 32, torch.uint8)
    bc, codes = guarded(T, d_in // 2, torch.uint8)
    nsc = 512 * -(-T // 128) * -(-d_in // 128)
    be, sc = guarded(1, nsc, torch.uint8)
    need = max(q.workspace_bytes(op, q.BF16, T, d_out, d_in, r) for op in (q.OP_FWD_MXFP4, q.OP_BWD_MXFP4))
    bw = torch.full((need + 8192,), 7, dtype=torch.uint8, device="cuda")
    ws = bw[4096:4096 + need]
    q.qlora_linear_fwd_mxfp4(w, X, A, B, 2.0 * r, H=H, U_save=U, ws=ws)
    a = q.act8_quantize(X, q=aq, scales=asc)
    q.mxfp4_quantize(X, codes=codes, scales=sc.view(-1))
    q.qlora_linear_bwd_mxfp4(w, a, dH, A, B, 2.0 * r, dX=dX, dA=dA, dB=dB, ws=ws)
    assert q.get_device_error() == 0
    for buf in (bH, bU, bX, bA, bB, bq, bs, bc, be):
        assert (buf[:4096] == 7).all() and (buf[-4096:] == 7).all()
    assert (bw[:4096] == 7).all() and (bw[-4096:] == 7).all()


@pytest.mark.parametrize("base", ["mx", "nf4"])
@pytest.mark.parametrize("T", [20, 129, 400])
def test_phases_and_accumulation(q, T, base):
    import torch
    w, X, dH, A, B = layer(q, T, 264, 640, 16, base=base)
    fn = q.qlora_linear_bwd_mxfp4 if base == "mx" else q.qlora_linear_bwd_act8
    a = q.act8_quantize(X)
    dX, dA, dB = fn(w, a, dH, A, B, 32.0)
    op = q.OP_BWD_MXFP4 if base == "mx" else q.OP_BWD_ACT8
    ws = torch.empty(q.workspace_bytes(op, q.BF16, T, 264, 640, 16), dtype=torch.uint8, device="cuda")
    none, dA2, dB2 = fn(w, a, dH, A, B, 32.0, ws=ws, phase="grads")
    assert none is None
    dX2, n1, n2 = fn(w, a, dH, A, B, 32.0, ws=ws, phase="dx")
    assert n1 is None and n2 is None
    assert torch.equal(dX, dX2) and torch.equal(dA, dA2) and torch.equal(dB, dB2)
    skipped, dA3, dB3 = fn(w, a, dH, A, B, 32.0, want_dx=False)
    assert skipped is None and torch.equal(dA3, dA) and torch.equal(dB3, dB)
    accA, accB = torch.randn_like(dA), torch.randn_like(dB)
    wantA, wantB = accA + dA, accB + dB
    fn(w, a, dH, A, B, 32.0, dA=accA, dB=accB, accumulate=True)
    assert torch.equal(accA, wantA) and torch.equal(accB, wantB)


def test_capture_replay_and_streams(q):
    """A captured step follows its inputs; two streams with a workspace each, and a stream argument."""
    import torch
    T, d_out, d_in, r = 150, 320, 512, 8
    w, X, dH, A, B = layer(q, T, d_out, d_in, r)
    w1, X1, dH1, _, _ = layer(q, T, d_out, d_in, r, seed=9)

    def step(ws, X, dH):
        H, U = q.qlora_linear_fwd_mxfp4(w, X, A, B, 16.0, ws=ws)
        a = q.act8_quantize(X)
        return (H, U, *q.qlora_linear_bwd_mxfp4(w, a, dH, A, B, 16.0, U_saved=U, ws=ws))

    need = max(q.workspace_bytes(op, q.BF16, T, d_out, d_in, r) for op in (q.OP_FWD_MXFP4, q.OP_BWD_MXFP4))
    mk = lambda: torch.empty(need, dtype=torch.uint8, device="cuda")  # noqa: E731
    ref, ref1 = step(mk(), X, dH), step(mk(), X1, dH1)
    # one token too (the decode-size route), in the same graph
    x1 = X[:1].contiguous()
    one = q.qlora_linear_fwd_mxfp4(w, x1, A, B, 16.0)[0]
    sX, sdH, sx1 = X.clone(), dH.clone(), x1.clone()
    ws = mk()
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        out = step(ws, sX, sdH)
        out1 = q.qlora_linear_fwd_mxfp4(w, sx1, A, B, 16.0, ws=ws)[0]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, ref)) and torch.equal(out1, one)
    sX.copy_(X1), sdH.copy_(dH1)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, ref1))
    # eager calls on two streams at once, and with stream=
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for st, (x, d) in zip(streams, ((X, dH), (X1, dH1))):
            with torch.cuda.stream(st):
                got.append(step(mk(), x, d))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, (ref, ref1)[i % 2]))
    H, U = q.qlora_linear_fwd_mxfp4(w, X, A, B, 16.0, stream=streams[0])
    a = q.act8_quantize(X, stream=streams[0])
    g = q.qlora_linear_bwd_mxfp4(w, a, dH, A, B, 16.0, U_saved=U, stream=streams[0])
    wq = q.mxfp4_quantize(X, stream=streams[1])
    v = q.mxfp4_dequantize(wq, torch.float32, stream=streams[1])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((H, U, *g), ref))
    assert np.array_equal(f64(v), M.mxfp4_values(*M.mxfp4_quantize(f64(X))))
    assert q.get_device_error() == 0


def test_training_step(q):
    """A step as it is used: base quantized, forward keeping U and an 8-bit checkpoint, backward from them over
    two micro-batches, AdamW -- against the same step in 64 bits; gradients also against differences."""
    import torch
    d_out, d_in, r, T = 264, 640, 16, 150
    rng = np.random.default_rng(12)
    W, A, B, _, _ = make(12, T, d_out, d_in, r)
    w = q.mxfp4_quantize(torch.from_numpy(W).cuda())
    Wv = M.mxfp4_values(*M.mxfp4_quantize(W))
    tA, tB = bf(A), bf(B)
    dA = torch.zeros((r, d_in), device="cuda")
    dB = torch.zeros((d_out, r), device="cuda")
    rA, rB = np.zeros((r, d_in)), np.zeros((d_out, r))
    for mb in range(2):
        X = activation(rng, T, d_in)
        dH = S.round_to_bf16(rng.standard_normal((T, d_out)).astype(np.float32)).astype(np.float64)
        H, U = q.qlora_linear_fwd_mxfp4(w, bf(X), tA, tB, 32.0)
        ck = q.act8_quantize(bf(X))
        dX, _, _ = q.qlora_linear_bwd_mxfp4(w, ck, bf(dH), tA, tB, 32.0, U_saved=U, dA=dA, dB=dB, accumulate=True)
        Xc = M.act8_values(*M.act8_quantize(X))
        gX, gA, gB = M.layer_backward(Wv, Xc, dH, A, B, 2.0, U=f64(U))
        rA += gA
        rB += gB
        # differences: H is linear in A and in B, and in X with the quantizer passed through
        D = rng.standard_normal(A.shape)
        E = rng.standard_normal(B.shape)
        F = rng.standard_normal(X.shape)

        def value(A_, B_, X_):
            return float(np.sum(dH * (X_ @ Wv.T + 2.0 * (X_ @ A_.T) @ B_.T)))
        gXf, gAf, gBf = M.layer_backward(Wv, X, dH, A, B, 2.0)
        h = 2.0 ** -10
        for num, ana in (((value(A + h * D, B, X) - value(A - h * D, B, X)) / (2 * h), np.sum(gAf * D)),
                         ((value(A, B + h * E, X) - value(A, B - h * E, X)) / (2 * h), np.sum(gBf * E)),
                         ((value(A, B, X + h * F) - value(A, B, X - h * F)) / (2 * h), np.sum(gXf * F))):
            assert abs(num - ana) <= 1e-8 * (abs(num) + np.sum(np.abs(dH)))
        # the bf16 activation's gradients (U recomputed) against those the differences confirmed
        got = q.qlora_linear_bwd_mxfp4(w, bf(X), bf(dH), tA, tB, 32.0)
        for g, ref, tol in zip(got, (gXf, gAf, gBf), (2 * U16, 2.0 ** -14, 2.0 ** -14)):
            assert np.linalg.norm(f64(g) - ref) <= tol * np.linalg.norm(ref)
    for got, ref in ((dA, rA), (dB, rB)):
        # the triples carry 24 bits; what is left is fp32 accumulation over 150 tokens and 264 channels
        assert np.linalg.norm(f64(got) - ref) <= 2.0 ** -16 * np.linalg.norm(ref)
    master = tA.float().clone()
    m, v = torch.zeros_like(master), torch.zeros_like(master)
    q.adamw_step(tA, dA, m, v, 1, 1e-3, master=master, grad_scale=0.5)
    step = -1e-3 * np.sign(rA) * (np.abs(rA) > 1e-3)
    moved = f64(master) - A
    big = np.abs(rA) > 1e-2
    assert np.allclose(moved[big], step[big], rtol=2e-3, atol=1e-9)
    assert q.get_device_error() == 0


def test_matches_the_nf4_layer_in_kind(q):
    """Beside the NF4 layer on the same weight: the 8-bit checkpoint's backward differs from the bf16 one by the
    checkpoint's rounding only."""
    import torch
    W, A, B, X, dH = make(20, 300, 520, 1024, 16)
    w = q.nf4_quantize(torch.from_numpy(W).cuda())
    H, U = q.qlora_linear_fwd(w, bf(X), bf(A), bf(B), 32.0)
    dX, dA, dB = q.qlora_linear_bwd(w, bf(X), bf(dH), bf(A), bf(B), 32.0, U_saved=U)
    dX8, dA8, dB8 = q.qlora_linear_bwd_act8(w, q.act8_quantize(bf(X)), bf(dH), bf(A), bf(B), 32.0, U_saved=U)
    for a, b in ((dX8, dX), (dB8, dB)):         # no activation in them
        assert np.linalg.norm(f64(a) - f64(b)) <= 2 * U16 * np.linalg.norm(f64(b))
    Xc = M.act8_values(*M.act8_quantize(X))
    # a step is 2^-6 2^floor(log2 max) <= 2^-6 max of the block; rounding is off by half of one, or, where the
    # value would round to 128 and 127 is taken, by less than a whole one
    top = np.abs(X).reshape(300, -1, 32).max(-1).repeat(32, 1)
    assert (np.abs(Xc - X) <= 2.0 ** -6 * top).all()
    # dA8 - dA = (s G)^T (Xc - X), beside the NF4 layer's rounding of s G to bf16: element by element
    G = np.abs(dH @ B)
    bound = 2.0 * (G.T @ np.abs(Xc - X) + (U16 + 520 * U32) * G.T @ np.abs(X)) + 300 * U32 * np.abs(dA.cpu().numpy())
    acc = 2.0 * 520 * U32 * (np.abs(dH) @ np.abs(B)).T @ (np.abs(X) + np.abs(Xc))
    within(f64(dA8), f64(dA), bound + acc + 300 * U32 * 2.0 * G.T @ np.abs(X), "dA from the checkpoint")


# ------------------------------------------------------------------ the largest sizes


def test_offsets_past_32_bits(q):
    """More than 2^32 elements: the last rows against the oracle."""
    import torch
    T, d_in = 70000, 65536
    x = torch.zeros((T, d_in), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(1)
    rows = [0, 32767, 32768, 65535, 65536, T - 1]
    for i in rows:
        x[i] = torch.from_numpy(S.round_to_bf16(rng.standard_normal(d_in).astype(np.float32))).to(torch.bfloat16)
    a = q.act8_quantize(x)
    w = q.mxfp4_quantize(x)
    v8, v4 = q.act8_dequantize(a, torch.bfloat16), None
    for i in rows:
        xi = f64(x[i:i + 1])
        assert np.array_equal(f64(v8[i:i + 1]), M.act8_values(*M.act8_quantize(xi)))
    del v8, a
    v4 = q.mxfp4_dequantize(w, torch.bfloat16)
    for i in rows:
        xi = f64(x[i:i + 1])
        assert np.array_equal(f64(v4[i:i + 1]), M.mxfp4_values(*M.mxfp4_quantize(xi)))
    del x, v4, w
    # a forward and a backward whose outputs pass 2^31 elements (H [T, 32768])
    d_out, d_in, r = 32768, 128, 8
    W, A, B, X6, dH6 = make(5, len(rows), d_out, d_in, r)
    w, Wv = mx_weight(q, W)
    X = torch.zeros((T, d_in), dtype=torch.bfloat16, device="cuda")
    X[rows] = bf(X6)
    H, U = q.qlora_linear_fwd_mxfp4(w, X, bf(A), bf(B), 16.0)
    Hr, Ur = M.layer_forward(Wv, X6, A, B, 2.0)
    assert np.linalg.norm(f64(H[rows]) - Hr) <= 2 * U16 * np.linalg.norm(Hr)
    assert not H[1:32767].any()
    dH = H.zero_()
    dH[rows] = bf(dH6)
    dX, dA, dB = q.qlora_linear_bwd_mxfp4(w, X, dH, bf(A), bf(B), 16.0, U_saved=U)
    rX, rA, rB = M.layer_backward(Wv, X6, dH6, A, B, 2.0, U=f64(U[rows]))
    for got, ref, tol in ((dX[rows], rX, 2 * U16), (dA, rA, 2.0 ** -14), (dB, rB, 2.0 ** -14)):
        assert np.linalg.norm(f64(got) - ref) <= tol * np.linalg.norm(ref)
    assert q.get_device_error() == 0
