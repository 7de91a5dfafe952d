"""The compiled way into the microscaled calls: it is built and answers None to all that is not a
plain call, and what it answers is bit for bit what the same call through ctypes gives, with the
same refusals."""
import numpy as np
import pytest

import qlora_parameter_efficient_b200 as q
from qlora_parameter_efficient_b200 import _mx_bind_path


@pytest.fixture(scope="module")
def bind():
    from qlora_parameter_efficient_b200 import build
    build.build_library()
    build.build_binding()
    q._load_binding(q.load())       # (looked for before it was built, it stays away otherwise)
    assert q._bind is not None and q._bind.__file__ == _mx_bind_path()
    return q._bind


def cpu(*shape, dtype="bfloat16"):
    import torch
    return torch.zeros(*shape, dtype=getattr(torch, dtype))


def test_no_plain_call_without_a_device(bind):
    import torch
    before = torch.cuda.is_initialized()
    x = cpu(4, 64)
    assert bind.quantize(False, x) is None and bind.quantize(True, x) is None
    assert bind.quantize(False, None) is None and bind.quantize(True, np.zeros((4, 64), np.float32)) is None
    codes, tiles = cpu(4, 32, dtype="uint8"), cpu(512, dtype="uint8")
    assert bind.dequantize(False, codes, tiles, 4, 64, True) is None
    assert bind.dequantize(True, x, tiles, "4", 64, True) is None
    assert bind.forward(codes, tiles, 4, 64, x, cpu(2, 64), cpu(4, 2), 1.0, None, None, True, None) is None
    assert bind.backward(codes, tiles, None, 4, 64, x, None, cpu(4, 4), cpu(2, 64), cpu(4, 2), 1.0, None, None, None,
                         None, True, False, None) is None
    assert torch.cuda.is_initialized() == before


@pytest.mark.parametrize("call,n", [("init", 8), ("quantize", 2), ("dequantize", 6), ("forward", 12), ("backward", 18)])
def test_number_of_arguments(bind, call, n):
    for k in (0, n - 1, n + 1):
        with pytest.raises(TypeError):
            getattr(bind, call)(*range(1, k + 1))


def test_addresses_are_checked(bind):
    with pytest.raises(ValueError):
        bind.init(*[0] * 8)
    q._load_binding(q.load())


# ------------------------------------------------------------------ on the GPU


def both(monkeypatch, f):
    """f() as it is and with the binding away: the results, or the errors, of each."""
    out = []
    for away in (False, True):
        with monkeypatch.context() as m:
            if away:
                m.setattr(q, "_bind", None)
            try:
                out.append(f())
            except Exception as e:               # noqa: BLE001 - compared by type and text
                out.append((type(e), str(e)))
    return out


def same(a, b):
    import torch
    assert type(a) is type(b)
    if isinstance(a, torch.Tensor):
        assert a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride() and a.device == b.device
        assert not a.requires_grad and not b.requires_grad
        assert torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))
    elif isinstance(a, (tuple, list)):
        assert len(a) == len(b)
        for x, y in zip(a, b):
            same(x, y)
    elif isinstance(a, (q.MXFP4Weight, q.Act8)):
        for k in a.__dataclass_fields__:
            same(getattr(a, k), getattr(b, k))
    else:
        assert a == b


class Problem:
    def __init__(self, T, d_out, d_in, r, seed=0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g, device="cuda")    # noqa: E731
        self.W = n(d_out, d_in) * 0.1
        self.X, self.dH = n(T, d_in).bfloat16(), n(T, d_out).bfloat16()
        self.A, self.B = n(r, d_in).bfloat16(), n(d_out, r).bfloat16()
        self.w, self.nf4 = q.mxfp4_quantize(self.W), q.nf4_quantize(self.W)
        self.c = q.act8_quantize(self.X)
        self.U = n(T, r).bfloat16()
        self.T, self.d_out, self.d_in, self.r = T, d_out, d_in, r


@pytest.mark.gpu
@pytest.mark.parametrize("T,d_out,d_in,r", [(1, 96, 128, 4), (17, 200, 192, 8), (130, 129, 320, 64), (520, 256, 256, 128)])
def test_same_results(bind, monkeypatch, T, d_out, d_in, r):
    import torch
    p = Problem(T, d_out, d_in, r)
    ran = []
    for call in (lambda: q.mxfp4_quantize(p.W), lambda: q.mxfp4_quantize(p.X), lambda: q.act8_quantize(p.X),
                 lambda: q.act8_quantize(p.W), lambda: q.mxfp4_dequantize(p.w, torch.bfloat16),
                 lambda: q.mxfp4_dequantize(p.w, torch.float32), lambda: q.act8_dequantize(p.c, torch.bfloat16),
                 lambda: q.act8_dequantize(p.c, torch.float32),
                 lambda: q.qlora_linear_fwd_mxfp4(p.w, p.X, p.A, p.B, 16.0),
                 lambda: q.qlora_linear_fwd_mxfp4(p.w, p.X, p.A, p.B, 16, save_u=False),
                 lambda: q.qlora_linear_fwd_mxfp4(p.w, p.X, p.A, p.B, 16, save_u=1),
                 lambda: q.qlora_linear_fwd_mxfp4(p.w, p.X, p.A, p.B, 16, U_save=torch.zeros_like(p.U), save_u=False)):
        ran.append(both(monkeypatch, call))
    for base in (q.qlora_linear_bwd_mxfp4, q.qlora_linear_bwd_act8):
        w = p.w if base is q.qlora_linear_bwd_mxfp4 else p.nf4
        for X in (p.c,) if w is p.nf4 else (p.c, p.X):
            for kw in (dict(), dict(U_saved=p.U), dict(want_dx=False), dict(want_dx=0, dX=torch.zeros_like(p.X))):
                ran.append(both(monkeypatch, lambda: base(w, X, p.dH, p.A, p.B, 16.0, **kw)))

            def add():
                dA, dB = torch.ones(r, d_in, device="cuda"), torch.ones(d_out, r, device="cuda")
                got = base(w, X, p.dH, p.A, p.B, 16.0, dA=dA, dB=dB, accumulate=1)
                assert got[1] is dA and got[2] is dB
                return got
            ran.append(both(monkeypatch, add))
    for a, b in ran:
        assert not (isinstance(a, tuple) and isinstance(a[0], type)), a
        same(a, b)


@pytest.mark.gpu
def test_the_plain_call_does_not_pass_through_ctypes(bind, monkeypatch):
    """Every plain call is the binding's (the longer way would show itself here)."""
    p = Problem(20, 96, 128, 4)
    import torch

    def gone(*a, **k):
        raise AssertionError("went through ctypes")
    monkeypatch.setattr(q, "_run_on", gone)
    c = q.act8_quantize(p.X)
    q.act8_dequantize(c, torch.float32)
    q.mxfp4_dequantize(q.mxfp4_quantize(p.W), torch.bfloat16)
    q.qlora_linear_fwd_mxfp4(p.w, p.X, p.A, p.B, 16.0)
    q.qlora_linear_bwd_mxfp4(p.w, c, p.dH, p.A, p.B, 16.0)
    q.qlora_linear_bwd_act8(p.nf4, c, p.dH, p.A, p.B, 16.0)


@pytest.mark.gpu
def test_same_refusals(bind, monkeypatch):
    import torch
    p = Problem(20, 96, 128, 4)
    f, b, n = q.qlora_linear_fwd_mxfp4, q.qlora_linear_bwd_mxfp4, q.qlora_linear_bwd_act8
    small = torch.empty(8, dtype=torch.uint8, device="cuda")
    odd = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")[1:]
    for call in (lambda: q.mxfp4_quantize(p.W[:, 1:]), lambda: q.mxfp4_quantize(p.W.double()),
                 lambda: q.mxfp4_quantize(p.W[:0]), lambda: q.mxfp4_quantize(p.W[0]), lambda: q.act8_quantize(p.X.half()),
                 lambda: q.mxfp4_quantize(p.W[:, :32].contiguous()), lambda: q.act8_quantize(p.X.cpu()),
                 lambda: q.act8_quantize(p.X.t()), lambda: q.mxfp4_dequantize(p.w, torch.float16),
                 lambda: f(p.w, p.X.float(), p.A, p.B, 1.0), lambda: f(p.w, p.X[:0], p.A, p.B, 1.0),
                 lambda: f(p.w, p.X, p.A[:, :64], p.B, 1.0), lambda: f(p.w, p.X, p.A, p.B.t(), 1.0),
                 lambda: f(p.w, p.X, p.A, p.B, 1.0, ws=small), lambda: f(p.w, p.X, p.A, p.B, 1.0, ws=odd),
                 lambda: f(p.w, p.X, p.A, p.B, "a"), lambda: f(p.w, p.X, p.A, p.B, 1.0, H=p.U),
                 lambda: f(p.w, p.X, p.A, p.B, 1.0, U_save=p.X),
                 lambda: f(p.w, p.X, torch.zeros(129, 128, device="cuda").bfloat16(),
                           torch.zeros(96, 129, device="cuda").bfloat16(), 1.0),
                 lambda: b(p.w, p.X, p.dH[:3], p.A, p.B, 1.0), lambda: b(p.w, p.c, p.dH, p.A, p.B, 1.0, dA=p.A),
                 lambda: b(p.w, p.c, p.dH, p.A, p.B, 1.0, accumulate=True), lambda: b(p.w, p.X, p.dH, p.A, p.B, 1.0, ws=small),
                 lambda: b(p.w, p.X, p.dH, p.A, p.B, 1.0, phase="no"), lambda: n(p.nf4, p.X, p.dH, p.A, p.B, 1.0),
                 lambda: n(p.nf4, p.c, p.dH.cpu(), p.A, p.B, 1.0), lambda: n(p.nf4, p.c, p.dH, p.A, p.B, 1.0, ws=odd)):
        a, c = both(monkeypatch, call)
        assert isinstance(a, tuple) and isinstance(a[0], type), a
        assert a == c


@pytest.mark.gpu
def test_another_stream_and_capture(bind):
    import torch
    p = Problem(64, 96, 128, 4)
    ref = q.qlora_linear_fwd_mxfp4(p.w, p.X, p.A, p.B, 16.0)[0].clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)             # the call has to wait behind this, on the same stream
        x = p.X * 1
        got = q.qlora_linear_fwd_mxfp4(p.w, x, p.A, p.B, 16.0)[0]
    s.synchronize()
    same(got, ref)
    graph = torch.cuda.CUDAGraph()
    x.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = q.qlora_linear_fwd_mxfp4(p.w, x, p.A, p.B, 16.0)[0]
    x.copy_(p.X)
    graph.replay()
    torch.cuda.synchronize()
    same(got, ref)


@pytest.mark.gpu
def test_threads(bind):
    """Calls from four threads at once, each on its own stream."""
    import threading

    import torch
    ps = [Problem(40, 96, 128, 4, seed=i) for i in range(4)]
    ref = [q.qlora_linear_bwd_mxfp4(p.w, p.c, p.dH, p.A, p.B, 16.0) for p in ps]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                got = q.qlora_linear_bwd_mxfp4(ps[i].w, ps[i].c, ps[i].dH, ps[i].A, ps[i].B, 16.0)
            s.synchronize()
        for a, b in zip(got, ref[i]):
            if not torch.equal(a, b):
                bad.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
