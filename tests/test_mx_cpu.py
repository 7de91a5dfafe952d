"""Microscaled formats and entry points, as far as no GPU is needed: the oracle's formats against
exhaustive definitions, sizes, and what the C ABI and the binding refuse before any launch."""
import ctypes

import numpy as np
import pytest

import qlora_parameter_efficient_b200 as q
from oracle import mx_oracle as M


@pytest.fixture(scope="module")
def L():
    from qlora_parameter_efficient_b200 import build
    build.build_library()
    return q.load()


# ------------------------------------------------------------------ the oracle's formats


def test_mxfp4_is_the_nearest_value_with_ties_to_even():
    """Against a search over all 16 codes for a fine grid of values, the borders among them."""
    x = np.concatenate([np.linspace(0, 7.99, 4001), M._BORDERS, np.nextafter(M._BORDERS, 9), np.nextafter(M._BORDERS, 0)])
    x = np.concatenate([x, -x])
    x = x[:len(x) // 31 * 31]
    blocks = np.concatenate([np.full((len(x) // 31, 1), 4.0), x.reshape(-1, 31)], 1)     # max in [4, 8): scale 2^0
    codes, e = M.mxfp4_quantize(blocks.reshape(1, -1))
    assert (e == 127).all()
    got = M.mxfp4_values(codes, e).reshape(blocks.shape)
    for v, g in zip(blocks.ravel(), got.ravel()):
        d = np.abs(M.E2M1 - abs(v))
        best = np.flatnonzero(d == d.min())
        want = M.E2M1[best[0] if len(best) == 1 or best[0] % 2 == 0 else best[1]]
        assert abs(g) == want and (want == 0 or np.sign(g) == np.sign(v)), (v, g)


@pytest.mark.parametrize("top,quant,bias", [(2, M.mxfp4_quantize, 127), (0, M.act8_quantize, 127)])
def test_scales(top, quant, bias):
    for k in range(-149, 128):
        for f in (1.0, 1.5, 1.99999988):
            m = np.float64(np.float32(f * 2.0 ** k)) if k > -149 or f == 1.0 else 2.0 ** -149
            x = np.zeros((1, 32))
            x[0, 7] = -m
            _, e = quant(x)
            assert e[0, 0] == max(0, int(np.floor(np.log2(m))) - top + bias), (k, f)
    for bad in (np.nan, np.inf, -np.inf):
        x = np.ones((1, 64))
        x[0, 3] = bad
        c, e = quant(x)
        assert e.tolist() == [[255, bias - top]] and not c[0, :16].any()


def test_act8_error_bound_and_exactness_in_bf16():
    import torch
    rng = np.random.default_rng(0)
    x = rng.standard_normal((64, 256)) * np.exp2(rng.integers(-60, 60, (64, 8)).repeat(32, 1))
    qi, e = M.act8_quantize(x)
    v = M.act8_values(qi, e)
    top = np.abs(x).reshape(64, 8, 32).max(-1).repeat(32, 1)
    assert (np.abs(v - x) <= 2.0 ** -7 * top + (np.abs(qi) == 127) * 2.0 ** -6 * top).all()
    for ex in (0, 1, 6, 7, 127, 240):
        vals = np.arange(-127, 128) * 2.0 ** (ex - 133)
        t = torch.from_numpy(vals).to(torch.bfloat16).double().numpy()
        assert np.array_equal(t, vals)


def test_scale_tiles_are_a_permutation():
    for rows, nb in ((1, 2), (128, 4), (130, 6), (300, 10)):
        e = (np.arange(rows * nb) % 250 + 1).astype(np.uint8).reshape(rows, nb)
        t = M.tile_scales(e)
        assert t.size == 512 * -(-rows // 128) * -(-nb // 4)
        assert sorted(t[t > 0].tolist()) == sorted(e.ravel().tolist())
    e = np.arange(1, 129, dtype=np.uint8).reshape(128, 1).repeat(4, 1)
    t = M.tile_scales(e).reshape(32, 4, 4)
    assert (t[5, 2] == e[2 * 32 + 5, 0]).all()


# ------------------------------------------------------------------ sizes and refusals of the C ABI


def test_sizes(L):
    for rows, cols in [(4096, 4096), (1, 64), (129, 192), (11008, 4096)]:
        assert q.mxfp4_sizes(rows, cols) == (rows * cols // 2, 512 * -(-rows // 128) * -(-cols // 128))
    for rows, cols in [(0, 64), (1, 32), (1, 100), (-1, 64), (1 << 31, 64)]:
        with pytest.raises(q.QloraError):
            q.mxfp4_sizes(rows, cols)
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert L.qlora_act8_sizes(7, 128, ctypes.byref(a), ctypes.byref(b)) == 0 and (a.value, b.value) == (896, 28)
    assert L.qlora_act8_sizes(7, 96, ctypes.byref(a), ctypes.byref(b)) == 2
    assert L.qlora_act8_sizes(0, 128, ctypes.byref(a), ctypes.byref(b)) == 2
    assert L.qlora_act8_sizes(7, 128, None, ctypes.byref(b)) == 1


def test_workspace_sizes(L):
    for op in (q.OP_FWD_MXFP4, q.OP_BWD_MXFP4, q.OP_BWD_ACT8):
        for T in (1, 16, 17, 64, 65, 129, 600, 4096):
            n = q.workspace_bytes(op, q.BF16, T, 4096, 4096, 16)
            assert n > 0 and n % 256 == 0
            assert q.workspace_bytes(op, q.F32, T, 4096, 4096, 16) == 0
        for T, d_out, d_in, r in [(0, 64, 64, 8), (1, 0, 64, 8), (1, 64, 96, 8), (1, 64, 64, 0), (1, 64, 64, 129)]:
            assert q.workspace_bytes(op, q.BF16, T, d_out, d_in, r) == 0
    assert q.workspace_bytes(19, q.BF16, 1, 64, 64, 8) == 0
    # no bf16 copy of the activation in the backward's workspace: for long batches it grows by less
    grow = (q.workspace_bytes(q.OP_BWD_ACT8, q.BF16, 65536, 256, 4096, 8)
            - q.workspace_bytes(q.OP_BWD_ACT8, q.BF16, 32768, 256, 4096, 8))
    assert grow < 32768 * 4096


def test_refusals_before_any_launch(L):
    big = 1 << 30
    mx = q._MXFP4(16, 16, 128, 128)
    nf4 = q._NF4(16, 16, 16, 128, 128)
    a8 = q._ACT8(16, 16)
    ok = dict(w=mx, X=16, T=4, A=16, B=16, r=8, H=16, U=None, ws=256, n=big)

    def fwd(**kw):
        k = {**ok, **kw}
        w = ctypes.byref(k["w"]) if k["w"] is not None else None
        return L.qlora_linear_fwd_mxfp4(w, k["X"], k["T"], k["A"], k["B"], k["r"], 16.0, k["H"], k["U"], k["ws"], k["n"],
                                        None)
    for kw in ({"w": None}, {"w": q._MXFP4(0, 16, 128, 128)}, {"w": q._MXFP4(16, 24, 128, 128)}, {"X": None}, {"X": 8},
               {"A": 4}, {"B": 0}, {"H": None}, {"U": 20}, {"ws": 0}, {"ws": 128}, {"n": 10}):
        assert fwd(**kw) == 1, kw
    for kw in ({"w": q._MXFP4(16, 16, 128, 96)}, {"w": q._MXFP4(16, 16, 0, 128)}, {"T": 0}, {"T": -3}, {"r": 0},
               {"r": 129}):
        assert fwd(**kw) == 2, kw

    okb = dict(w=mx, X=16, X8=None, dH=16, T=4, A=16, B=16, r=8, U=None, dX=16, dA=16, dB=16, ws=256, n=big, flags=0)

    def bwd(**kw):
        k = {**okb, **kw}
        p8 = ctypes.byref(k["X8"]) if k["X8"] is not None else None
        return L.qlora_linear_bwd_mxfp4(ctypes.byref(k["w"]), k["X"], p8, k["dH"], k["T"], k["A"], k["B"], k["r"], 16.0,
                                        k["U"], k["dX"], k["dA"], k["dB"], k["ws"], k["n"], k["flags"], None)
    for kw in ({"X": None}, {"X8": a8}, {"X": None, "X8": q._ACT8(0, 16)}, {"X": None, "X8": q._ACT8(16, 17)}, {"dH": 2},
               {"A": None}, {"B": 24}, {"U": 8}, {"dX": 8}, {"dA": None}, {"dB": 12}, {"ws": 64}, {"n": 0}, {"flags": 8},
               {"flags": q.BWD_GRADS_ONLY | q.BWD_DX_FROM_WS}, {"flags": q.BWD_DX_FROM_WS, "dX": None},
               {"flags": q.BWD_GRADS_ONLY, "dA": None}):
        assert bwd(**kw) == 1, kw
    for kw in ({"T": 0}, {"r": 200}, {"w": q._MXFP4(16, 16, 128, 100)}):
        assert bwd(**kw) == 2, kw

    def bwd8(w=nf4, X8=a8, **kw):
        k = {**okb, **kw}
        return L.qlora_linear_bwd_act8(ctypes.byref(w), ctypes.byref(X8) if X8 is not None else None, k["dH"], k["T"],
                                       k["A"], k["B"], k["r"], 16.0, k["U"], k["dX"], k["dA"], k["dB"], k["ws"], k["n"],
                                       k["flags"], None)
    for kw in ({"X8": None}, {"X8": q._ACT8(8, 16)}, {"w": q._NF4(16, 8, 16, 128, 128)}, {"dH": None}, {"n": 100}):
        assert bwd8(**kw) == 1, kw
    assert bwd8(w=q._NF4(16, 16, 16, 128, 100)) == 2 and bwd8(T=0) == 2 and bwd8(r=0) == 2

    # quantizers and decoders
    assert L.mxfp4_quantize(None, q.F32, 4, 64, 16, 16, None) == 1
    assert L.mxfp4_quantize(16, 7, 4, 64, 16, 16, None) == 1
    assert L.mxfp4_quantize(16, q.F32, 4, 48, 16, 16, None) == 2
    assert L.mxfp4_quantize(16, q.F32, 0, 64, 16, 16, None) == 2
    assert L.mxfp4_quantize(16, q.F32, 4, 64, 20, 16, None) == 1
    assert L.mxfp4_dequantize(None, 16, q.F32, None) == 1
    assert L.mxfp4_dequantize(ctypes.byref(mx), 17, q.F32, None) == 1
    assert L.mxfp4_dequantize(ctypes.byref(mx), 16, 5, None) == 1
    assert L.qlora_act8_quantize(16, q.BF16, 4, 72, 16, 16, None) == 2
    assert L.qlora_act8_quantize(16, q.BF16, 4, 64, 16, 3, None) == 1
    assert L.qlora_act8_quantize(16, 9, 4, 64, 16, 16, None) == 1
    assert L.qlora_act8_dequantize(None, 4, 64, 16, q.BF16, None) == 1
    assert L.qlora_act8_dequantize(ctypes.byref(a8), 0, 64, 16, q.BF16, None) == 2


# ------------------------------------------------------------------ refusals of the binding


def test_binding_refuses_cpu_tensors_and_wrong_types():
    import torch
    bf = torch.bfloat16
    x = torch.zeros((4, 64), dtype=bf)
    with pytest.raises(ValueError):
        q.mxfp4_quantize(x)
    with pytest.raises(ValueError):
        q.act8_quantize(x)
    with pytest.raises(ValueError):
        q.MXFP4Weight(torch.zeros((4, 32), dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 4, 64)
    with pytest.raises(ValueError):
        q.Act8(torch.zeros((4, 64), dtype=torch.int8), torch.zeros((4, 2), dtype=torch.uint8))
    with pytest.raises(TypeError):
        q.qlora_linear_bwd_act8(None, x, x, x, x, 1.0)


def test_binding_checks_shapes_types_and_layout():
    """On meta tensors that say they are on a GPU nothing can be launched: the checks come first."""
    import torch
    bf = torch.bfloat16
    dev = torch.device("meta")
    t = torch.empty((4, 64), dtype=bf, device=dev)
    q._need("x", t, bf, (4, 64), dev)
    with pytest.raises(TypeError):
        q._need("x", t, torch.float32, (4, 64), dev)
    with pytest.raises(ValueError):
        q._need("x", t, bf, (4, 65), dev)
    with pytest.raises(ValueError):
        q._need("x", t.T, bf, (64, 4), dev)
    with pytest.raises(ValueError):
        q._need("x", t, bf, (4, 64), torch.device("cpu"))
    w = q._made(q.MXFP4Weight, codes=t.to(torch.uint8), scales=t, d_out=8, d_in=64)
    act = q._made(q.Act8, q=torch.empty((4, 128), dtype=torch.int8, device=dev), scales=t)
    dH, A, B = (torch.empty(s, dtype=bf, device=dev) for s in ((4, 8), (2, 64), (8, 2)))
    with pytest.raises(ValueError):                      # the checkpoint's width is not the weight's
        q.qlora_linear_bwd_mxfp4(w, act, dH, A, B, 1.0)
    with pytest.raises(ValueError):
        q.qlora_linear_bwd_mxfp4(w, t, dH, A, B, 1.0, phase="both")
    with pytest.raises(ValueError):                      # phase dx without the workspace of phase grads
        q.qlora_linear_bwd_mxfp4(w, t, dH, A, B, 1.0, phase="dx")
    with pytest.raises(ValueError):                      # accumulation into nothing
        q.qlora_linear_bwd_mxfp4(w, t, dH, A, B, 1.0, accumulate=True)
    with pytest.raises(ValueError):
        q.qlora_linear_bwd_mxfp4(w, t, dH, A, B.T, 1.0)
    with pytest.raises(ValueError):
        q.qlora_linear_fwd_mxfp4(w, t[:, :32], A, B, 1.0)
    with pytest.raises(TypeError):
        q.qlora_linear_fwd_mxfp4(w, t.float(), A, B, 1.0)
