"""Workloads of the microscaled operators: MXFP4 weights and activations, the layer with an MXFP4
base (forward and backward), 8-bit activation checkpoints, and the NF4 layer's backward from one.

Formats (OCP Microscaling v1.0, blocks of 32 consecutive row elements, one E8M0 scale per block):
  MXFP4   value = E2M1(code) 2^(scale - 127);  scale = floor(log2 max|x|) - 2 + 127
  MXINT8  value = q 2^(scale - 127 - 6);       scale = floor(log2 max|x|) + 127,  |q| <= 127
codes and scales of an MXFP4 matrix lie as the framework keeps them: element 2j in the low nibble of
byte j; the scales in 512-byte tiles of 128 rows x 4 blocks, byte (row % 32) 16 + (row / 32 % 4) 4 +
block % 4 of tile (row / 128, block / 4).  Checkpoint scales are row-major [tokens, blocks].
"""
import math

import torch

own = False

# The NF4 levels of the framework's stored base weight (the nf4_gemm backward cases read one).
_NF4 = [-1.0, -0.777601778507232666015625, -0.615571379661560058593750, -0.481248497962951660156250,
        -0.362556546926498413085938, -0.253368556499481201171875, -0.149945825338363647460938,
        -0.0496507771313190460205078125]
_NF4 = _NF4 + [-v for v in reversed(_NF4)]
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def listed():
    return [
        # a weight matrix going into storage, as a whole projection and as an odd small one
        {"name": "mxfp4 weight 4096x11008 f32", "op": "mxfp4", "rows": 4096, "cols": 11008, "f32": True},
        {"name": "mxfp4 activation 203x448 bf16", "op": "mxfp4", "rows": 203, "cols": 448, "f32": False},
        # one new token through a q_proj-sized layer
        {"name": "forward T1 4096x4096 r16", "op": "fwd", "T": 1, "d_out": 4096, "d_in": 4096, "r": 16},
        # a small decode batch through the MLP up projection
        {"name": "forward T13 11008x4096 r64", "op": "fwd", "T": 13, "d_out": 11008, "d_in": 4096, "r": 64},
        # a short prompt, ragged in tokens and rank
        {"name": "forward T200 8192x8192 r5", "op": "fwd", "T": 200, "d_out": 8192, "d_in": 8192, "r": 5},
        # a training micro-batch (4 x 1024 tokens)
        {"name": "forward T4096 4096x4096 r16", "op": "fwd", "T": 4096, "d_out": 4096, "d_in": 4096, "r": 16},
        # its backward, from the 8-bit checkpoint and the U the forward kept
        {"name": "backward T4096 4096x4096 r16 ckpt", "op": "bwd_mx", "T": 4096, "d_out": 4096, "d_in": 4096,
         "r": 16, "ckpt": True, "u": True},
        # a ragged layer, from the bf16 activation, U recomputed
        {"name": "backward T333 1001x2048 r33 bf16", "op": "bwd_mx", "T": 333, "d_out": 1001, "d_in": 2048,
         "r": 33, "ckpt": False, "u": False},
        # the checkpoint itself, written and read back: a micro-batch, and a few fp32 tokens
        {"name": "checkpoint 4096x4096 bf16", "op": "act8", "T": 4096, "d_in": 4096, "f32": False},
        {"name": "checkpoint 37x1344 f32", "op": "act8", "T": 37, "d_in": 1344, "f32": True},
        # the NF4 layer's backward from the checkpoint: the MLP projection, and a short ragged batch
        {"name": "nf4 backward T8192 11008x4096 r64 ckpt", "op": "bwd_nf4", "T": 8192, "d_out": 11008, "d_in": 4096,
         "r": 64, "ckpt": True, "u": True},
        {"name": "nf4 backward T129 4096x4096 r8 ckpt", "op": "bwd_nf4", "T": 129, "d_out": 4096, "d_in": 4096,
         "r": 8, "ckpt": True, "u": False},
    ]


def draw(rng):
    def log(a, b):
        return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))

    op = rng.choice(["mxfp4", "fwd", "fwd", "bwd_mx", "act8", "bwd_nf4"])
    while True:
        T, d_out, d_in, r = log(1, 8192), log(32, 11008), 64 * log(1, 172), rng.randint(1, 128)
        if T * d_out * d_in <= 8192 * 11008 * 4096:
            break
    if op == "mxfp4":
        return {"op": op, "rows": d_out, "cols": d_in, "f32": rng.random() < 0.5}
    if op == "act8":
        return {"op": op, "T": T, "d_in": d_in, "f32": rng.random() < 0.5}
    case = {"op": op, "T": T, "d_out": d_out, "d_in": d_in, "r": r}
    if op != "fwd":
        case["ckpt"] = op == "bwd_nf4" or rng.random() < 0.5
        case["u"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ plain forms (32 bits)


def _blocks32(x):
    return x.float().reshape(x.shape[0], -1, 32)


def _scale_exp(blocks, emax):
    """E8M0 bytes of the blocks: floor(log2 max|x|) - emax + 127, not under 0."""
    _, e = torch.frexp(blocks.abs().amax(-1))           # max = m 2^e with m in [0.5, 1)
    e = e - 1 - emax + 127
    return torch.where(blocks.abs().amax(-1) > 0, e, torch.zeros_like(e)).clamp(0, 254)


def _mxfp4(x):
    """E2M1 magnitudes with sign [rows, nb, 32] and E8M0 bytes [rows, nb] of a matrix."""
    b = _blocks32(x)
    e = _scale_exp(b, 2)
    y = torch.ldexp(b, (127 - e).unsqueeze(-1))
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    v = ((a / step).round() * step).clamp(max=6.0)      # round() takes ties to even
    return torch.copysign(v, y), e


def _mxint8(x):
    b = _blocks32(x)
    e = _scale_exp(b, 0)
    return torch.ldexp(b, (127 + 6 - e).unsqueeze(-1)).round().clamp(-127, 127), e


def _tile_scales(e):
    rows, nb = e.shape
    rt, kt = -(-rows // 128), -(-nb // 4)
    full = torch.zeros((rt * 128, kt * 4), dtype=torch.uint8, device=e.device)
    full[:rows, :nb] = e.to(torch.uint8)
    return full.view(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile_scales(s, rows, nb):
    rt, kt = -(-rows // 128), -(-nb // 4)
    return s.view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:rows, :nb]


def _pack(v):
    """E2M1 values [rows, nb, 32] to packed codes [rows, cols / 2]."""
    mags = torch.tensor(_E2M1, device=v.device)
    code = torch.searchsorted(mags, v.abs().contiguous()) + 8 * torch.signbit(v)
    code = code.to(torch.uint8).reshape(v.shape[0], -1)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _unpack(codes):
    return torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1).long()


def _decode_mxfp4(codes, scales, dtype=torch.float32):
    rows, cols = codes.shape[0], codes.shape[1] * 2
    table = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=dtype, device=codes.device)
    e = _untile_scales(scales, rows, cols // 32).to(torch.int32) - 127
    return torch.ldexp(table[_unpack(codes)].view(rows, -1, 32), e.unsqueeze(-1)).reshape(rows, cols)


def _nf4_weight(w):
    """NF4 codes, uint8 block constants and fp32 group constants of a weight (blocks of 64, groups of 256)."""
    rows, cols = w.shape
    b = w.reshape(-1, 64)
    c1 = b.abs().amax(-1)
    pad = torch.zeros(-(-c1.numel() // 256) * 256, device=w.device)
    pad[: c1.numel()] = c1
    c2 = pad.view(-1, 256).amax(-1)
    q8 = (c1 / c2.repeat_interleave(256)[: c1.numel()] * 127).round().to(torch.uint8)
    levels = torch.tensor(_NF4, device=w.device)
    codes = torch.bucketize(b / c1.unsqueeze(-1), (levels[1:] + levels[:-1]) / 2).to(torch.uint8).view(rows, cols)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), q8, c2


def _decode_nf4(codes, q8, c2):
    """The bf16 weight the layer multiplies with: bf16(level fl32(fl32(q8 c2) / 127))."""
    rows = codes.shape[0]
    scale = q8.float() * c2.repeat_interleave(256)[: q8.numel()] / 127
    levels = torch.tensor(_NF4, device=codes.device)
    return (levels[_unpack(codes)].view(-1, 64) * scale.unsqueeze(-1)).bfloat16().float().view(rows, -1)


# ------------------------------------------------------------------ inputs


def _activation(T, d_in, g):
    """Tokens with a few outlier channels, as a transformer's hidden states have."""
    x = torch.randn((T, d_in), generator=g, device="cuda")
    x[:, torch.randperm(d_in, generator=g, device="cuda")[: max(1, d_in // 200)]] *= 20
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, bf = case["op"], torch.bfloat16
    if op in ("mxfp4", "act8"):
        if op == "mxfp4":
            x = torch.randn((case["rows"], case["cols"]), generator=g, device="cuda") * 0.02 ** 0.5
        else:
            x = _activation(case["T"], case["d_in"], g)
        return {"case": case, "x": x if case["f32"] else x.to(bf)}
    T, d_out, d_in, r = case["T"], case["d_out"], case["d_in"], case["r"]
    w = torch.randn((d_out, d_in), generator=g, device="cuda") * 0.02 ** 0.5
    s = {"case": case, "alpha": 2.0 * r}
    if op == "bwd_nf4":
        s["codes"], s["q8"], s["c2"] = _nf4_weight(w)
    else:
        v, e = _mxfp4(w)
        s["codes"], s["scales"] = _pack(v), _tile_scales(e)
    x = _activation(T, d_in, g).to(bf)
    s["A"] = (torch.randn((r, d_in), generator=g, device="cuda") / r ** 0.5).to(bf)
    s["B"] = (torch.randn((d_out, r), generator=g, device="cuda") * 0.1).to(bf)
    if op == "fwd":
        s["X"] = x
        return s
    s["dH"] = torch.randn((T, d_out), generator=g, device="cuda").to(bf)
    s["U"] = (x.float() @ s["A"].float().T).to(bf) if case["u"] else None
    if case["ckpt"]:
        q, e = _mxint8(x)
        s["q8x"], s["ex"] = q.to(torch.int8).view(T, d_in), e.to(torch.uint8)
    else:
        s["X"] = x
    return s


# ------------------------------------------------------------------ one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    if op == "mxfp4":
        v, e = _mxfp4(state["x"])
        return torch.ldexp(v, (e - 127).unsqueeze(-1)).reshape(state["x"].shape).bfloat16()
    if op == "act8":
        v, e = _mxint8(state["x"])
        return torch.ldexp(v, (e - 127 - 6).unsqueeze(-1)).reshape(state["x"].shape).bfloat16()
    A, B = state["A"].float(), state["B"].float()
    sc = state["alpha"] / A.shape[0]
    if op == "bwd_nf4":
        W = _decode_nf4(state["codes"], state["q8"], state["c2"])
    else:
        W = _decode_mxfp4(state["codes"], state["scales"])
    if op == "fwd":
        v, e = _mxfp4(state["X"])
        X4 = torch.ldexp(v, (e - 127).unsqueeze(-1)).reshape(state["X"].shape)
        U = state["X"].float() @ A.T
        return {"H": (X4 @ W.T + sc * (U @ B.T)).bfloat16(), "U": U.bfloat16()}
    if state["case"]["ckpt"]:
        X = torch.ldexp(state["q8x"].float().view(state["q8x"].shape[0], -1, 32),
                        (state["ex"].int() - 127 - 6).unsqueeze(-1)).reshape(state["q8x"].shape)
    else:
        X = state["X"].float()
    dH = state["dH"].float()
    U = state["U"].float() if state["U"] is not None else X @ A.T
    G = dH @ B
    return {"dX": (dH @ W + sc * (G @ A)).bfloat16(), "dA": sc * (G.T @ X), "dB": sc * (dH.T @ U)}


def _run_own(state, op):
    import qlora_parameter_efficient_b200 as q

    if op == "mxfp4":
        return q.mxfp4_dequantize(q.mxfp4_quantize(state["x"]), torch.bfloat16)
    if op == "act8":
        return q.act8_dequantize(q.act8_quantize(state["x"]), torch.bfloat16)
    case = state["case"]
    T, d_out, d_in, r = case["T"], case["d_out"], case["d_in"], case["r"]
    if "w" not in state:            # the handles and the workspace that a program keeps
        if op == "bwd_nf4":
            state["w"] = q.NF4Weight(state["codes"], state["q8"], state["c2"], d_out, d_in)
        else:
            state["w"] = q.MXFP4Weight(state["codes"], state["scales"], d_out, d_in)
        code = {"fwd": q.OP_FWD_MXFP4, "bwd_mx": q.OP_BWD_MXFP4, "bwd_nf4": q.OP_BWD_ACT8}[op]
        state["ws"] = torch.empty(q.workspace_bytes(code, q.BF16, T, d_out, d_in, r), dtype=torch.uint8, device="cuda")
        if op != "fwd":
            state["act"] = q.Act8(state["q8x"], state["ex"]) if case["ckpt"] else state["X"]
    if op == "fwd":
        H, U = q.qlora_linear_fwd_mxfp4(state["w"], state["X"], state["A"], state["B"], state["alpha"], ws=state["ws"])
        return {"H": H, "U": U}
    bwd = q.qlora_linear_bwd_act8 if op == "bwd_nf4" else q.qlora_linear_bwd_mxfp4
    dX, dA, dB = bwd(state["w"], state["act"], state["dH"], state["A"], state["B"], state["alpha"],
                     U_saved=state["U"], ws=state["ws"])
    return {"dX": dX, "dA": dA, "dB": dB}


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    op = case["op"]
    if op in ("mxfp4", "act8"):
        rows, cols = (case["rows"], case["cols"]) if op == "mxfp4" else (case["T"], case["d_in"])
        stored = 0.5 + 1 / 32 if op == "mxfp4" else 1 + 1 / 32
        n = rows * cols
        return {"bytes": n * ((4 if case["f32"] else 2) + 2 * stored + 2), "flops": 4 * n}
    T, d_out, d_in, r = case["T"], case["d_out"], case["d_in"], case["r"]
    w = d_out * d_in * (0.5 + 1 / 64 if op == "bwd_nf4" else 0.5 + 1 / 32)
    adapters = 2 * r * (d_in + d_out)
    if op == "fwd":
        return {"bytes": w + adapters + 2 * T * (d_in + d_out + r),
                "flops": 2 * T * d_out * d_in + 2 * T * r * (d_in + d_out)}
    x = T * d_in * (1 + 1 / 32 if case["ckpt"] else 2)
    u = 2 * T * r if case["u"] else 0
    return {"bytes": w + adapters + x + u + 2 * T * d_out + 2 * T * d_in + 4 * r * (d_in + d_out),
            "flops": 2 * T * d_out * d_in + 2 * T * r * (2 * d_out + 2 * d_in + (0 if case["u"] else d_in))}


# ------------------------------------------------------------------ the definition in 64 bits


def _ex_pow2(x):
    """2^floor(log2 max|x|) of each block of 32, in 64 bits; 2^-127 where that is less, or the block is 0."""
    m = x.abs().amax(-1, keepdim=True)
    p = torch.exp2(torch.floor(torch.log2(m)))
    p = torch.where(p > m, p / 2, torch.where(2 * p <= m, 2 * p, p))      # log2 near a power of two
    return torch.where(m > 0, p, torch.zeros_like(p))


def _ex_mxfp4(x):
    x = x.double()
    b = x.reshape(x.shape[0], -1, 32)
    unit = (_ex_pow2(b) / 4).clamp(min=2.0 ** -127)
    a = b.abs() / unit
    # E2M1 by its borders: at a tie the value with the even code is taken
    up = ((a > 0.25).double() + (a >= 0.75).double() + (a > 1.25).double() + (a >= 1.75).double()) * 0.5
    up = up + (a > 2.5).double() + (a >= 3.5).double() + 2 * (a > 5.0).double()
    return (torch.sign(b) * up * unit).reshape(x.shape)


def _ex_mxint8(x):
    x = x.double()
    b = x.reshape(x.shape[0], -1, 32)
    unit = _ex_pow2(b).clamp(min=2.0 ** -127) / 64
    low = torch.floor(b / unit)
    part = b / unit - low
    odd = torch.remainder(low, 2)
    q = low + ((part > 0.5) | ((part == 0.5) & (odd == 1))).double()
    return (q.clamp(-127, 127) * unit).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "mxfp4":
        return _ex_mxfp4(s["x"])
    if op == "act8":
        return _ex_mxint8(s["x"])
    A, B = s["A"].double(), s["B"].double()
    sc = s["alpha"] / case["r"]
    rows, cols = case["d_out"], case["d_in"]
    nib = torch.empty((rows, cols), dtype=torch.uint8, device="cuda")
    nib[:, 0::2], nib[:, 1::2] = s["codes"] % 16, s["codes"] // 16
    if op == "bwd_nf4":
        # the stored weight is defined by fp32 products and a bf16 rounding: those steps stay
        block = (s["q8"].float() * s["c2"].repeat_interleave(256)[: s["q8"].numel()]) / 127
        W = (torch.tensor(_NF4, device="cuda")[nib.long()] * block.view(rows, -1).repeat_interleave(64, 1))
        W = W.bfloat16().double()
    else:
        row = torch.arange(rows, device="cuda").view(-1, 1)
        kb = torch.arange(cols // 32, device="cuda").view(1, -1)
        tiles = -(-cols // 128)
        at = ((row // 128) * tiles + kb // 4) * 512 + (row % 32) * 16 + (row // 32 % 4) * 4 + kb % 4
        unit = torch.exp2(s["scales"][at].double() - 127).repeat_interleave(32, 1)
        mag = nib % 8
        exp, man = (mag // 2).double(), (mag % 2).double()
        val = torch.where(mag < 2, man / 2, torch.exp2(exp - 1) * (1 + man / 2))
        W = torch.where(nib >= 8, -val, val) * unit
    if op == "fwd":
        U = s["X"].double() @ A.T
        return {"H": _ex_mxfp4(s["X"]) @ W.T + sc * (U @ B.T), "U": U}
    if case["ckpt"]:
        X = s["q8x"].double() * torch.exp2(s["ex"].double() - 133).repeat_interleave(32, 1)
    else:
        X = s["X"].double()
    dH = s["dH"].double()
    U = s["U"].double() if s["U"] is not None else X @ A.T
    G = dH @ B
    return {"dX": dH @ W + sc * (G @ A), "dA": sc * (G.T @ X), "dB": sc * (dH.T @ U)}
