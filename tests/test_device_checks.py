"""Operands on another device than the first one, or than the current one, are refused before any kernel gets
their addresses.  Stand-ins for tensors, since no second device is needed to say so."""
import pytest
import torch

import mxfp8_quantization_amax_gb300 as fq


class Stand:
    """What the checks ask of a contiguous CUDA tensor."""

    is_cuda = True

    def __init__(self, shape, dtype, index=0):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", index)

    def get_device(self):
        return self.device.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        raise AssertionError("an address was taken")


U8, F32, I32, I64, BF = torch.uint8, torch.float32, torch.int32, torch.int64, torch.bfloat16


def plan(t):
    return {"row_of": t["row_of"], "src": t["src"]}


CALLS = {
    "blockwise": (dict(a=((4, 128), U8), sa=((4, 1), F32), b=((8, 128), U8), sb=((1, 1), F32), out=((4, 8), BF)),
                  lambda t: fq.fp8q_matmul_blockwise(t["a"], t["sa"], t["b"], t["sb"], out=t["out"])),
    "grouped": (dict(a=((4, 128), U8), sa=((4, 1), F32), b=((2, 8, 128), U8), sb=((2, 1, 1), F32), out=((4, 8), BF)),
                lambda t: fq.fp8q_matmul_grouped(t["a"], t["sa"], t["b"], t["sb"], Stand((3,), I64), out=t["out"])),
    "wgrad": (dict(a=((4, 128), U8), sa=((4, 1), F32), b=((8, 128), U8), sb=((8, 1), F32), out=((2, 4, 8), F32)),
              lambda t: fq.fp8q_matmul_grouped_wgrad(t["a"], t["sa"], t["b"], t["sb"], Stand((3,), I64), out=t["out"])),
    "route": (dict(x=((4, 8), F32), bias=((8,), F32), w=((4, 2), F32), ids=((4, 2), I32)),
              lambda t: fq.fp8q_moe_route(t["x"], 2, bias=t["bias"], out={"weights": t["w"], "ids": t["ids"]})),
    "route_backward": (dict(x=((4, 8), F32), ids=((4, 2), I32), d=((4, 2), F32), out=((4, 8), F32)),
                       lambda t: fq.fp8q_moe_route_backward(t["x"], t["ids"], t["d"], out=t["out"])),
    "plan": (dict(ids=((4, 2), I32), offsets=((9,), I64), row_of=((4, 2), I32), src=((8,), I32)),
             lambda t: fq.fp8q_moe_plan(t["ids"], 8, out={k: t[k] for k in ("offsets", "row_of", "src")})),
    "dispatch": (dict(x=((4, 16), BF), row_of=((4, 2), I32), src=((8,), I32), q=((8, 16), U8), s=((8, 1), F32)),
                 lambda t: fq.fp8q_moe_dispatch(t["x"], plan(t), out={"q": t["q"], "scale_inv": t["s"]})),
    "combine": (dict(y=((8, 16), F32), row_of=((4, 2), I32), w=((4, 2), F32), out=((4, 16), F32)),
                lambda t: fq.fp8q_moe_combine(t["y"], {"row_of": t["row_of"]}, t["w"], out=t["out"])),
    "combine_backward": (dict(y=((8, 16), F32), d=((4, 16), F32), row_of=((4, 2), I32), src=((8,), I32), w=((4, 2), F32),
                              d_y=((8, 16), F32), d_w=((4, 2), F32)),
                         lambda t: fq.fp8q_moe_combine_backward(t["d"], t["y"], plan(t), t["w"], out={"d_y": t["d_y"], "d_weights": t["d_w"]})),
}


@pytest.mark.parametrize("call", CALLS)
def test_operands_of_other_devices_are_refused(call, monkeypatch):
    fq.build()
    shapes, run = CALLS[call]
    monkeypatch.setattr(fq, "_current_device", lambda: 0)
    monkeypatch.setattr(fq, "_group_offsets", lambda offsets, device: (offsets, 2))  # offsets are brought to the device
    for moved in shapes:
        t = {name: Stand(*spec, index=int(name == moved)) for name, spec in shapes.items()}
        with pytest.raises(ValueError, match="cuda:"):
            run(t)
    with pytest.raises(AssertionError, match="address"):  # all on the current one: the checks pass
        run({name: Stand(*spec) for name, spec in shapes.items()})
    monkeypatch.setattr(fq, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="not the current device"):
        run({name: Stand(*spec) for name, spec in shapes.items()})
