"""The norm, the gated activation, the few-token layer and the clip refuse operands on another device than the
first one, or than the current one, before any kernel gets their addresses (stand-ins for tensors)."""
import pytest
import torch

import mxfp8_quantization_amax_gb300 as fq
from test_device_checks import BF, F32, I32, U8, Stand

COPIES = dict(q=((16, 32), U8), scale_inv=((16, 1), F32), q_t=((32, 16), U8), scale_inv_t=((32, 1), F32))


def copies(t):
    return {k: t[k] for k in COPIES}


CALLS = {
    "rmsnorm": (dict(x=((16, 32), BF), w=((32,), F32), res=((16, 32), F32), h=((16, 32), F32), rstd=((16,), F32), y=((16, 32), BF), **COPIES),
                lambda t: fq.fp8q_rmsnorm(t["x"], t["w"], t["res"], direction=fq.BOTH, want_y=True,
                                          out={"h": t["h"], "rstd": t["rstd"], "y": t["y"], **copies(t)})),
    "rmsnorm_backward": (dict(d_y=((16, 32), BF), h=((16, 32), F32), w=((32,), BF), rstd=((16,), F32), d_h=((16, 32), F32),
                              d_x=((16, 32), F32), d_w=((32,), F32)),
                         lambda t: fq.fp8q_rmsnorm_backward(t["d_y"], t["h"], t["w"], t["rstd"], t["d_h"], out={"d_x": t["d_x"], "d_weight": t["d_w"]})),
    "swiglu": (dict(h=((16, 64), BF), a=((16, 32), BF), **COPIES),
               lambda t: fq.fp8q_swiglu(t["h"], direction=fq.BOTH, want_a=True, out={"a": t["a"], **copies(t)})),
    "swiglu_backward": (dict(h=((16, 32), BF), d_a=((16, 16), BF), d_h=((16, 32), BF), **COPIES),
                        lambda t: fq.fp8q_swiglu_backward(t["h"], t["d_a"], want_d_h=True, out={"d_h": t["d_h"], **copies(t)})),
    "decode": (dict(x=((4, 32), BF), ids=((4, 2), I32), w=((4, 2), F32), w1=((3, 32, 32), U8), s1=((3, 1, 1), F32), w2=((3, 32, 16), U8),
                    s2=((3, 1, 1), F32), out=((4, 32), BF)),
               lambda t: fq.fp8q_moe_decode(t["x"], t["ids"], t["w"], t["w1"], t["s1"], t["w2"], t["s2"], out=t["out"])),
    "clip": (dict(a=((7,), F32), b=((3, 4), BF), oa=((7,), F32), ob=((3, 4), BF)),
             lambda t: fq.fp8q_clip_grads([t["a"], t["b"]], 1.0, out=[t["oa"], t["ob"]])),
    "grad_norm": (dict(a=((7,), F32), b=((3, 4), BF), out=((1,), F32)), lambda t: fq.fp8q_grad_norm([t["a"], t["b"]], out=t["out"])),
}


@pytest.mark.parametrize("call", CALLS)
def test_operands_of_other_devices_are_refused(call, monkeypatch):
    fq.build()
    shapes, run = CALLS[call]
    monkeypatch.setattr(fq, "_current_device", lambda: 0)
    real = torch.empty
    monkeypatch.setattr(fq, "_empty", lambda *a, **k: real(*a, **{**k, "device": "cpu"}))  # workspaces of a machine without a GPU
    for moved in shapes:
        t = {name: Stand(*spec, index=int(name == moved)) for name, spec in shapes.items()}
        with pytest.raises(ValueError, match="cuda:"):
            run(t)
    monkeypatch.setattr(fq.torch, "empty", lambda *a, **k: real(*a, **{**k, "device": "cpu"}))
    with pytest.raises(AssertionError, match="address"):  # all on the current one: the checks pass
        run({name: Stand(*spec) for name, spec in shapes.items()})
    monkeypatch.setattr(fq, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="not the current device"):
        run({name: Stand(*spec) for name, spec in shapes.items()})
