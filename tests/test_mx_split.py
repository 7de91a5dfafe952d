"""dX of the microscaled backward where the tiles of its last wave are split along K: every form of the schedule
(tiles 256 and 128 wide, 2 to 4 ways, alone and behind whole waves), and that each case here has the one it is for."""
import os
import subprocess

import numpy as np
import pytest

import qlora_parameter_efficient_b200 as q

HERE = os.path.dirname(os.path.abspath(__file__))
U16, U32 = 2.0 ** -8, 2.0 ** -23
FACTOR = 2.0 ** -16                   # s G in two bf16 terms

# T, d_out, d_in, r, base: tile width, whole waves in front, ways
CASES = [((300, 4100, 2048, 8, "mx"), (128, 0, 2)), ((300, 4100, 576, 33, "nf4"), (128, 0, 3)),
         ((300, 8200, 576, 16, "mx"), (128, 0, 4)), ((6400, 28672, 320, 8, "mx"), (128, 1, 4)),
         ((300, 8200, 3328, 8, "mx"), (256, 0, 2)), ((300, 8200, 2560, 70, "nf4"), (256, 0, 3)),
         ((3328, 11008, 192, 16, "mx"), (256, 0, 4)), ((2600, 4100, 2112, 8, "nf4"), (256, 1, 2)),
         ((2048, 4100, 3008, 40, "mx"), (256, 1, 3)), ((1100, 4100, 4096, 16, "mx"), (256, 1, 4)),
         ((4096, 4096, 4096, 16, "mx"), (256, 3, 2)), ((4096, 4096, 4096, 16, "nf4"), (256, 3, 2)),
         # none split: fewer tiles than pairs, whole waves and a rest
         ((1100, 2000, 576, 16, "mx"), (128, 0, 1)), ((2600, 1100, 2112, 8, "mx"), (256, 1, 1))]


@pytest.fixture(scope="module")
def schedule(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("sched") / "pair_schedule")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-o", exe, os.path.join(HERE, "pair_schedule.cpp")],
                   check=True)

    def ask(shapes):
        r = subprocess.run([exe], input="\n".join(" ".join(map(str, s)) for s in shapes), capture_output=True, text=True,
                           check=True)
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    return ask


def test_the_cases_are_split_as_they_say(schedule):
    got = schedule([(T, d_in, -(-d_out // 64), 0) for (T, d_out, d_in, _, _), _ in CASES])
    for (bn, _, whole, tail, split, _), ((T, d_out, d_in, _, _), want) in zip(got, CASES):
        assert (bn, whole, split) == want, (T, d_out, d_in)
        tiles = -(-T // 256) * -(-d_in // bn)
        assert tail == (tiles - 74 * whole if split > 1 else 0)


def test_schedules_fit_the_card_and_their_workspace(schedule):
    """Over all sizes: no more parts than pairs, every tile once, partials and tickets for every split tile; and no
    MXFP4 product is ever split."""
    shapes = [(T, d_in, k, mx) for T in (65, 256, 300, 512, 1100, 2600, 4096, 8192) for d_in in range(64, 11009, 192)
              for k in (1, 3, 4, 16, 64, 448) for mx in (0, 1)]
    for (T, d_in, k, mx), (bn, pairs, whole, tail, split, size) in zip(shapes, schedule(shapes)):
        tiles = -(-T // 256) * -(-d_in // bn)
        assert 1 <= pairs <= 74 and 1 <= split <= (1 if mx else 4) and split <= k and (bn == 256 or (bn == 128 and not mx))
        if split > 1:
            assert tail == tiles % 74 and 0 < tail * split <= pairs and (whole == 0 or pairs == 74)
            assert size >= tail * split * 256 * bn * 4 + tail * 8 * 4
        else:
            assert tail == 0 and size == 0 and pairs == min(tiles, 74)


@pytest.mark.gpu
@pytest.mark.parametrize("case,want", CASES)
def test_split_dx(case, want):
    import torch
    T, d_out, d_in, r, base = case
    g = torch.Generator(device="cuda").manual_seed(T + d_out + d_in)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")                     # noqa: E731
    W, X = rand(d_out, d_in) * 0.141, rand(T, d_in).bfloat16()
    dH, A, B = rand(T, d_out).bfloat16(), (rand(r, d_in) / r ** 0.5).bfloat16(), (rand(d_out, r) * 0.1).bfloat16()
    if base == "mx":
        fn, op, w = q.qlora_linear_bwd_mxfp4, q.OP_BWD_MXFP4, q.mxfp4_quantize(W)
        Wv = q.mxfp4_dequantize(w, torch.float32)
    else:
        fn, op, w = q.qlora_linear_bwd_act8, q.OP_BWD_ACT8, q.nf4_quantize(W)
        Wv = q.nf4_dequantize(w, torch.bfloat16)
    act = q.act8_quantize(X)
    got = []
    for fill in (0xFF, 0x7F, 0):                       # partials and tickets are the call's own business
        ws = torch.full((q.workspace_bytes(op, q.BF16, T, d_out, d_in, r),), fill, dtype=torch.uint8, device="cuda")
        got.append(fn(w, act, dH, A, B, 2.0 * r, ws=ws))
    assert q.get_device_error() == 0
    for o in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, got[0]))
    # whole rows against 64 bits: both ends of every tile of 128 rows, and some between
    rows = sorted({t for t in range(T) if t % 128 in (0, 1, 63, 127)} | {T - 1} | set(range(5, T, 101)))[:400]
    f64 = lambda t: t.double().cpu().numpy()                                          # noqa: E731
    dh, wv, a, b = f64(dH[rows]), f64(Wv), f64(A), f64(B)
    G = dh @ b
    ref = dh @ wv + 2 * G @ a
    acc_g = d_out * U32 * (np.abs(dh) @ np.abs(b))
    tol = (U16 * np.abs(ref) + 2 * (FACTOR * np.abs(G) + acc_g) @ np.abs(a)
           + (d_out + 2 * r) * U32 * (np.abs(dh) @ np.abs(wv) + 2 * np.abs(G) @ np.abs(a)))
    err = np.abs(f64(got[0][0][rows]) - ref)
    assert (err <= (1 + U16) * tol + 1e-30).all(), float((err / tol).max())
    # and close: the result's rounding (2^-8 / 3^(1/2) of a value at most, in the mean square) and a little
    assert np.linalg.norm(err) <= 2.0 ** -8 / 3 ** 0.5 * 1.01 * np.linalg.norm(ref)
