"""What the microscaled layers carry in more than one bf16 number: the adapter's factor of H and dX.

The base weight is 0, so that the adapter term is the whole result, and ranks and cancellation make the rounding of
its factor the largest error there could be.  u = half a step, relative (bf16 2^-8):
  factor s U, s G   two bf16 terms: the first leaves at most u of the value, the second u of that: 2^-16
  result            one rounding: u
  fp32 sums         2^-23 per term of the sum of the terms' magnitudes (both terms of the factor: 1 + 2^-7 of it)
A factor rounded to one bf16 number (2^-8 of it) fails these bounds.
"""
import numpy as np
import pytest

from oracle import mx_oracle as M

from test_mx_gpu import U16, U32, bf, f64, make, mx_weight, q, within  # noqa: F401 (q: fixture)

pytestmark = pytest.mark.gpu

FACTOR = 2.0 ** -16
BOTH = 1 + 2.0 ** -7
# 16, 32, 48 and 64: where the columns of the two terms change K step; above 64 half a term per step
RANKS = [1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 40, 48, 49, 63, 64, 65, 80, 96, 113, 127, 128]


@pytest.mark.parametrize("T", [1, 5, 16, 17, 64, 65, 130, 385, 700])
@pytest.mark.parametrize("r", RANKS)
def test_adapter_term_of_the_forward(q, T, r):  # noqa: F811
    d_out, d_in = 203, 64
    W, A, B, X, _ = make(100 * r + T, T, d_out, d_in, r)
    w, Wv = mx_weight(q, W * 0)
    assert not Wv.any()
    H, _ = q.qlora_linear_fwd_mxfp4(w, bf(X), bf(A), bf(B), 2.0 * r)
    Hr, Ur = M.layer_forward(Wv, X, A, B, 2.0)
    acc_u = d_in * U32 * (np.abs(X) @ np.abs(A).T)
    tol = U16 * np.abs(Hr) + 2 * (FACTOR * np.abs(Ur) + acc_u + 2 * r * U32 * BOTH * np.abs(Ur)) @ np.abs(B).T
    within(f64(H), Hr, (1 + U16) * tol + 1e-30, "H")


@pytest.mark.parametrize("base", ["mx", "nf4"])
@pytest.mark.parametrize("T", [1, 16, 63, 64, 65, 300])
@pytest.mark.parametrize("r", RANKS)
def test_adapter_term_of_dx(q, T, r, base):  # noqa: F811
    import torch
    d_out, d_in = 72, 192
    W, A, B, X, dH = make(100 * r + T, T, d_out, d_in, r)
    if base == "mx":
        fn, w = q.qlora_linear_bwd_mxfp4, mx_weight(q, W * 0)[0]
    else:
        fn, w = q.qlora_linear_bwd_act8, q.nf4_quantize(torch.zeros(d_out, d_in, device="cuda"))
        assert not q.nf4_dequantize(w, torch.float32).any()
    dX, _, _ = fn(w, q.act8_quantize(bf(X)), bf(dH), bf(A), bf(B), 2.0 * r)
    dXr = M.layer_backward(W * 0.0, X, dH, A, B, 2.0)[0]
    G = np.abs(dH @ B)
    acc_g = d_out * U32 * (np.abs(dH) @ np.abs(B))
    tol = U16 * np.abs(dXr) + 2 * (FACTOR * G + acc_g + 2 * r * U32 * BOTH * G) @ np.abs(A)
    within(f64(dX), dXr, (1 + U16) * tol + 1e-30, "dX")


def test_columns_past_the_rank_are_not_read(q):  # noqa: F811
    """A workspace full of NaN: what pads the factor's terms to whole MMAs is written, the rest not used."""
    import torch
    for T in (3, 40, 150, 500):
        for r in (1, 9, 20, 37, 70, 100):
            W, A, B, X, dH = make(r, T, 100, 128, r)
            w, _ = mx_weight(q, W)
            n = max(q.workspace_bytes(op, q.BF16, T, 100, 128, r) for op in (q.OP_FWD_MXFP4, q.OP_BWD_MXFP4))
            outs = []
            for fill in (0xFF, 0):
                ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
                H, _ = q.qlora_linear_fwd_mxfp4(w, bf(X), bf(A), bf(B), 16.0, ws=ws)
                ws.fill_(fill)
                outs.append((H, *q.qlora_linear_bwd_mxfp4(w, bf(X), bf(dH), bf(A), bf(B), 16.0, ws=ws)))
            for a, b in zip(*outs):
                assert torch.isfinite(a).all() and torch.equal(a, b), (T, r)
    assert q.get_device_error() == 0


# ------------------------------------------------------------------ gradients: three bf16 terms


def bf16(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.float64)).to(torch.bfloat16).double().numpy()


def terms(x, n):
    """The first n bf16 terms of fp32 values, summed."""
    got = np.zeros_like(x)
    for _ in range(n):
        got = got + bf16(x - got)
    return got


@pytest.mark.parametrize("ckpt", [True, False])
@pytest.mark.parametrize("T,d_out", [(1, 3), (1, 8), (2, 3), (2, 5)])
@pytest.mark.parametrize("r", [1, 8, 16, 20, 48, 64, 65, 128])
def test_gradients_carry_24_bits(q, r, T, d_out, ckpt):  # noqa: F811
    """Sums so short that what carries s G and a recomputed U is the largest error: bounds that its third term is
    needed for (without it, in the oracle, they do not hold)."""
    d_in, used = 128, [3, 40, 77, 126]                 # (products with 0 add no error)
    W, A, B, X, dH = make(1000 * r + T, T, d_out, d_in, r)
    keep = np.zeros(d_in)
    keep[used] = 1
    X = X * keep
    w, _ = mx_weight(q, W)
    alpha = np.float32(r / 3)
    s = float(alpha / np.float32(r))                   # as the library forms it: 24 bits, unlike the products' 16
    act = bf(X)
    if ckpt:
        act = q.act8_quantize(act)
        X = M.act8_values(*M.act8_quantize(X))
    _, dA, dB = q.qlora_linear_bwd_mxfp4(w, act, bf(dH), bf(A), bf(B), float(alpha))
    _, dAr, dBr = M.layer_backward(W * 0.0, X, dH, A, B, s)
    sG, U = s * (dH @ B), X @ A.T
    # s G: d_out products summed, scaled; three terms leave 2^-24; T products, two sums of terms
    e_sG = s * d_out * U32 * (np.abs(dH) @ np.abs(B)) + (2.0 ** -24 + 2.0 ** -24) * np.abs(sG)
    e_U = len(used) * U32 * (np.abs(X) @ np.abs(A).T) + 2.0 ** -24 * np.abs(U)
    sums = (T + 3) * U32 * BOTH
    tol_A = e_sG.T @ np.abs(X) + sums * np.abs(sG).T @ np.abs(X)
    tol_B = s * (np.abs(dH).T @ e_U + (sums + 2.0 ** -23) * np.abs(dH).T @ np.abs(U))
    within(f64(dA), dAr, (1 + U16) * tol_A + 1e-30, "dA")
    within(f64(dB), dBr, (1 + U16) * tol_B + 1e-30, "dB")
    # two terms: beyond the bounds somewhere
    two_A = terms(sG, 2).T @ X
    two_B = s * dH.T @ terms(U, 2)
    if r >= 8:
        assert (np.abs(two_A - dAr) > tol_A).any() and (np.abs(two_B - dBr) > tol_B).any()
