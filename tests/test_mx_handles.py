"""Handles of stored matrices: malformed ones are refused before anything is launched."""
import numpy as np
import pytest

import qlora_parameter_efficient_b200 as q


def nf4_parts(dev, d_out=128, d_in=192):
    import torch
    blocks = d_out * d_in // 64                                   # 384 blocks, two groups
    return dict(codes=torch.zeros((d_out, d_in // 2), dtype=torch.uint8, device=dev),
                absmax_q=torch.zeros(blocks, dtype=torch.uint8, device=dev),
                c2=torch.zeros(-(-blocks // 256), dtype=torch.float32, device=dev), d_out=d_out, d_in=d_in)


def bad_nf4(dev):
    """(error, fields) of NF4 handles with a buffer too short, of another type, strided or of another shape."""
    import torch
    ok = nf4_parts(dev)
    for err, kw in ((ValueError, dict(absmax_q=ok["absmax_q"][:-1])), (ValueError, dict(absmax_q=ok["absmax_q"][:0])),
                    (ValueError, dict(absmax_q=ok["absmax_q"].repeat(2)[::2])), (TypeError, dict(absmax_q=ok["absmax_q"].to(torch.int8))),
                    (TypeError, dict(absmax_q=ok["absmax_q"].float())), (ValueError, dict(c2=ok["c2"][:1])),
                    (TypeError, dict(c2=ok["c2"].double())), (TypeError, dict(c2=ok["c2"].half())),
                    (ValueError, dict(c2=ok["c2"].repeat(2)[::2])), (TypeError, dict(codes=ok["codes"].to(torch.int8))),
                    (ValueError, dict(codes=ok["codes"][:-1])), (ValueError, dict(d_out=129)), (ValueError, dict(d_in=256))):
        yield err, {**ok, **kw}


def call(dev, fields):
    import torch
    T, d_out, d_in, r = 4, fields["d_out"], fields["d_in"], 8
    bf = torch.bfloat16
    x8 = q._made(q.Act8, q=torch.zeros((T, d_in), dtype=torch.int8, device=dev),
                 scales=torch.zeros((T, d_in // 32), dtype=torch.uint8, device=dev))
    dH, A, B = (torch.zeros(s, dtype=bf, device=dev) for s in ((T, d_out), (r, d_in), (d_out, r)))
    return q.qlora_linear_bwd_act8(q.NF4Weight(**fields), x8, dH, A, B, 16.0)


def test_malformed_nf4_handles(monkeypatch):
    """On meta tensors that pass for a GPU's nothing can be launched: the checks come first."""
    monkeypatch.setattr(q, "_need_cuda", lambda name, t: t.device)
    for err, fields in bad_nf4("meta"):
        with pytest.raises(err):
            call("meta", fields)


@pytest.mark.gpu
@pytest.mark.parametrize("binding", [True, False])
def test_malformed_nf4_handles_on_the_gpu(monkeypatch, binding):
    import torch
    if not binding:
        monkeypatch.setattr(q, "_bind", None)
        monkeypatch.setattr(q, "_bind_looked_for", True)
    n0 = q.launch_count()
    for err, fields in bad_nf4("cuda"):
        with pytest.raises(err):
            call("cuda", fields)
    with pytest.raises(ValueError):
        call("cuda", {**nf4_parts("cuda"), "c2": nf4_parts("cpu")["c2"]})
    assert q.launch_count() == n0
    # buffers of another shape, or longer ones, hold the same weight
    ok = nf4_parts("cuda")
    ref = call("cuda", ok)
    for kw in (dict(absmax_q=ok["absmax_q"].view(128, 3)), dict(absmax_q=ok["absmax_q"].repeat(2)), dict(c2=ok["c2"].repeat(3))):
        for a, b in zip(call("cuda", {**ok, **kw}), ref):
            assert torch.equal(a, b)
    assert np.isfinite(ref[0].float().cpu().numpy()).all() and q.get_device_error() == 0


def test_a_handle_keeps_no_addresses(monkeypatch):
    """What a call passes on are the buffers as they are then, checked; a used handle can be copied."""
    import copy

    import torch
    monkeypatch.setattr(q, "_need_cuda", lambda name, t: t.device)
    u8 = torch.uint8
    w = q.MXFP4Weight(torch.zeros((8, 32), dtype=u8), torch.zeros(512, dtype=u8), 8, 64)
    a = q.Act8(torch.zeros((4, 64), dtype=torch.int8), torch.zeros((4, 2), dtype=u8))
    assert w._c()._obj.codes == w.codes.data_ptr() and a._c().q == a.q.data_ptr()
    for t in (w.codes, w.scales, a.q, a.scales):
        t.data = torch.ones_like(t)                   # other memory (the old one is freed)
    c, c8 = w._c()._obj, a._c()
    assert (c.codes, c.scales) == (w.codes.data_ptr(), w.scales.data_ptr())
    assert (c8.q, c8.scales) == (a.q.data_ptr(), a.scales.data_ptr())
    for h, name in ((w, "codes"), (a, "q")):
        d = copy.deepcopy(h)
        assert getattr(d, name).data_ptr() != getattr(h, name).data_ptr()
        d._c()
    w.scales.data = torch.zeros(512, dtype=u8)[:256]
    with pytest.raises(ValueError):
        w._c()
    a.scales.data = torch.zeros((3, 2), dtype=u8)
    with pytest.raises(ValueError):
        a._c()


@pytest.mark.gpu
def test_a_weight_that_was_given_other_memory():
    """The same handle before and after its buffers moved, by either way into the library."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    W, X = torch.randn(96, 128, generator=g, device="cuda"), torch.randn(20, 128, generator=g, device="cuda").bfloat16()
    A, B = torch.randn(4, 128, generator=g, device="cuda").bfloat16(), torch.randn(96, 4, generator=g, device="cuda").bfloat16()
    w, s = q.mxfp4_quantize(W), torch.cuda.current_stream()
    H = q.qlora_linear_fwd_mxfp4(w, X, A, B, 8.0, stream=s)[0]
    for t in (w.codes, w.scales):
        old = t.data
        t.data = old.clone()
        old.fill_(0x55)
    for kw in (dict(), dict(stream=s)):
        assert torch.equal(q.qlora_linear_fwd_mxfp4(w, X, A, B, 8.0, **kw)[0], H)
        assert torch.equal(q.mxfp4_dequantize(w, torch.float32, **kw), q.mxfp4_dequantize(q.mxfp4_quantize(W), torch.float32))
