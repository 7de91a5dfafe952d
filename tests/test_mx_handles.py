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
