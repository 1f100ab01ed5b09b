"""Every public function of the binding refuses tensors in host memory before
the library's entry point is called: a host address in a kernel is a memory
fault.  The entry points are stubs here that record a call; the host-side size
queries are the library's own."""
import inspect
import os

import pytest
import torch

from combine_top_route_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="library not built")

BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8
T, d, E, k, I = 4, 128, 4, 2, 128
R = T * k


class HostOnly:
    """The loaded library's host-side queries; any other entry point records
    that it was reached."""

    def __init__(self, real):
        self.real, self.reached = real, []

    def __getattr__(self, name):
        if name.endswith(("_size", "_bytes", "_error", "_string")):
            return getattr(self.real, name)
        return lambda *a: self.reached.append(name) or 0


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def routing():
    return B.Routing.empty(T, E, k, torch.device("cpu"), logits=z(T, E))


def layer(**kw):
    return B.MoeLayer(T, d, E, k, I, device="cpu", **kw)


def forward(l):
    return l.forward(z(T, d), z(E, 2 * I, d), z(E, d, I), logits=z(T, E))


def backward(l):
    l.routing.logits = z(T, E)
    return l.backward(z(T, d), z(T, d), z(E, 2 * I, d), z(E, d, I))


CALLS = {
    "MoeLayer.forward": lambda: forward(layer()),
    "MoeLayer.forward ids": lambda: layer().forward(z(T, d), z(E, 2 * I, d), z(E, d, I), topk_ids=z(T, k, dtype=I32),
                                                    topk_w=z(T, k, dtype=torch.float32)),
    "MoeLayer.forward save8": lambda: forward(layer(save8=True)),
    "MoeLayer.backward": lambda: backward(layer()),
    "MoeLayer.backward recompute": lambda: backward(layer(save=False)),
    "MoeLayer.backward save8": lambda: backward(layer(save8=True)),
    "MoeDecoder.forward": lambda: B.MoeDecoder(T, d, E, k, I, device="cpu").forward(
        z(T, d), z(E, 2 * I, d), z(E, d, I), logits=z(T, E)),
    "router_logits": lambda: B.router_logits(z(T, d), z(E, d)),
    "router_backward": lambda: B.router_backward(z(T, E), z(T, d), z(E, d)),
    "swiglu_save8": lambda: B.swiglu_save8(z(R, 2 * I), routing(), T, k),
    "swiglu_backward8": lambda: B.swiglu_backward8(z(R, I), z(R, 2 * I, dtype=U8), z(R, 2 * (I // 32), dtype=U8),
                                                   routing(), T, k),
    "route": lambda: B.route(z(T, E), k),
    "route_ids": lambda: B.route_ids(z(T, k, dtype=I32), z(T, k, dtype=torch.float32), E),
    "route_noalloc": lambda: B.route_noalloc(routing(), T, E, k),
    "permute": lambda: B.permute(z(T, d), routing(), k),
    "combine": lambda: B.combine(z(R, d), routing(), T, k),
    "quantize_fp8": lambda: B.quantize_fp8(z(E, d, I), B.QUANT_WEIGHT),
    "quantize_mxfp8": lambda: B.quantize_mxfp8(z(R, d)),
    "quantize_tokens_fp8": lambda: B.quantize_tokens_fp8(z(T, d), routing(), T, k, True),
    "quantize_tokens_mxfp8": lambda: B.quantize_tokens_mxfp8(z(R, d), routing(), T, k, False),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_host_memory_is_refused_before_the_library(name, monkeypatch):
    host = HostOnly(B.lib())
    monkeypatch.setattr(B, "lib", lambda: host)
    # as on a machine with a GPU, where a stream handle would be found
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    with pytest.raises(ValueError, match="cpu"):
        CALLS[name]()
    assert host.reached == []


def test_every_function_that_takes_tensors_is_listed():
    """A function of the binding that enqueues work names the stream."""
    names = {n for n, f in vars(B).items() if inspect.isfunction(f) and "_stream(" in inspect.getsource(f)
             and n != "_stream"}
    names |= {f"{c.__name__}.{n}" for c in (B.MoeLayer, B.MoeDecoder) for n, f in vars(c).items()
              if inspect.isfunction(f) and "_stream(" in inspect.getsource(f)}
    assert names <= set(CALLS), names - set(CALLS)
