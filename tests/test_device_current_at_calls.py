"""Every library call runs with its tensors' device current.  Streams are passed
as raw handles and a default stream's handle is 0 on every device, so a call made
while another device is current would run there.  CPU only: fake tensors on a
second device and stubs that record the current one."""
import os

import pytest
import torch
from torch._subclasses import FakeTensorMode

from combine_top_route_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="library not built")

DEV = torch.device("cuda", 1)
BF, I32, U8, F32 = torch.bfloat16, torch.int32, torch.uint8, torch.float32
T, d, E, k, I = 4, 128, 4, 2, 128
R = T * k


def z(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device=DEV)


def routing():
    return B.Routing.empty(T, E, k, DEV, logits=z(T, E))


def tensors():
    r = routing()
    return (r.topk_ids, r.topk_w, r.counts, r.offsets, r.row_of, r.src_of)


def step(**kw):
    layer = B.MoeLayer(T, d, E, k, I, device=DEV, **kw)
    layer.forward(z(T, d), z(E, 2 * I, d), z(E, d, I), logits=z(T, E))
    layer.backward(z(T, d), z(T, d), z(E, 2 * I, d), z(E, d, I))


def op_backward(name, size, *more):
    from combine_top_route_amd import autograd as A
    saved = z(size(B.make_shape(T, d, E, k, I, BF, BF)), dtype=U8)
    getattr(A, name)._init_fn(z(T, d), z(T, d), z(T, E), z(E, 2 * I, d), z(E, d, I), saved, *tensors(), k, *more)


def op(name, *more):
    from combine_top_route_amd import autograd as A
    getattr(A, name)._init_fn(z(T, d), z(T, E), z(E, 2 * I, d), z(E, d, I), k, *more)


CALLS = {
    "layer": (step, ["moe_forward", "moe_backward"]),
    "layer save8": (lambda: step(save8=True), ["moe_forward8", "moe_backward8"]),
    "moe_fwd": (lambda: op("moe_fwd", "native", True), ["moe_forward"]),
    "moe_bwd": (lambda: op_backward("moe_bwd", B.saved_size, "native"), ["moe_backward"]),
    "moe_fwd8": (lambda: op("moe_fwd8"), ["moe_forward8"]),
    "moe_bwd8": (lambda: op_backward("moe_bwd8", B.saved8_size), ["moe_backward8"]),
    "decoder": (lambda: B.MoeDecoder(T, d, E, k, I, device=DEV).forward(
        z(T, d), z(E, 2 * I, d), z(E, d, I), logits=z(T, E)), ["moe_decode"]),
    "router_logits": (lambda: B.router_logits(z(T, d), z(E, d)), ["moe_router_forward"]),
    "router_backward": (lambda: B.router_backward(z(T, E), z(T, d), z(E, d)), ["moe_router_backward"]),
    "swiglu_save8": (lambda: B.swiglu_save8(z(R, 2 * I), routing(), T, k), ["moe_swiglu_save8"]),
    "swiglu_backward8": (lambda: B.swiglu_backward8(z(R, I), z(R, 2 * I, dtype=U8), z(R, 2 * (I // 32), dtype=U8),
                                                    routing(), T, k), ["moe_swiglu_backward8"]),
    "route": (lambda: B.route(z(T, E), k), ["moe_route"]),
    "route_ids": (lambda: B.route_ids(z(T, k, dtype=I32), z(T, k, dtype=F32), E), ["moe_route"]),
    "route_noalloc": (lambda: B.route_noalloc(routing(), T, E, k), ["moe_route_noalloc"]),
    "permute": (lambda: B.permute(z(T, d), routing(), k), ["moe_permute"]),
    "combine": (lambda: B.combine(z(R, d), routing(), T, k), ["moe_combine"]),
    "quantize_fp8": (lambda: B.quantize_fp8(z(E, d, I), B.QUANT_WEIGHT), ["moe_quantize_fp8"]),
    "quantize_mxfp8": (lambda: B.quantize_mxfp8(z(R, d)), ["moe_quantize_mxfp8"]),
    "quantize_tokens_fp8": (lambda: B.quantize_tokens_fp8(z(T, d), routing(), T, k, True),
                            ["moe_quantize_tokens_fp8"]),
    "quantize_tokens_mxfp8": (lambda: B.quantize_tokens_mxfp8(z(R, d), routing(), T, k, False),
                              ["moe_quantize_tokens_mxfp8"]),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_the_tensors_device_is_current(name, monkeypatch):
    current, calls, real = [0], [], B.lib()

    class Guard:
        def __init__(self, device):
            self.index = torch.device(device).index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *a):
            current[0] = self.before

    class Stub:
        def __getattr__(self, entry):
            if entry.endswith(("_size", "_bytes", "_error", "_string")):
                return getattr(real, entry)
            return lambda *a: calls.append((entry, current[0])) or 0

    monkeypatch.setattr(B, "lib", lambda: Stub())
    monkeypatch.setattr(B, "_ptr", lambda t: None if t is None else 1 << 20)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    run, entries = CALLS[name]
    with FakeTensorMode():
        run()
    assert calls == [(e, DEV.index) for e in entries] and current == [0]
