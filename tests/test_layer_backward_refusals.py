"""MoeLayer.backward refuses x and weights that are not the layer's, in the plain
and the 8-bit form: the kernels take their extents from the layer's shape.  CPU
only, with a stub in place of the entry points."""
import os

import pytest
import torch

from combine_top_route_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="library not built")

T, d, E, k, I = 4, 64, 4, 2, 32
BF = torch.bfloat16


class HostOnly:
    def __init__(self, real):
        self.real, self.reached = real, []

    def __getattr__(self, name):
        if name.endswith(("_size", "_bytes", "_error", "_string")):
            return getattr(self.real, name)
        return lambda *a: self.reached.append(name) or 0


def z(*shape, dtype=BF, device="cpu"):
    return torch.zeros(shape, dtype=dtype, device=device)


BAD = {
    "dout has shape": dict(dout=z(T, d + 8)),
    "x has shape": dict(x=z(T - 1, d)),
    "x has dtype": dict(x=z(T, d, dtype=torch.float32)),
    "x is on meta": dict(x=z(T, d, device="meta")),
    "x must be contiguous": dict(x=z(T, 2 * d)[:, ::2]),
    "x is required": dict(x=None),
    "w_gate_up has shape": dict(w_gate_up=z(E, I, d)),
    "w_gate_up has dtype": dict(w_gate_up=z(E, 2 * I, d, dtype=torch.float32)),
    "w_down has shape": dict(w_down=z(E, d, 2 * I)),
    "w_down must be contiguous": dict(w_down=z(E, I, d).transpose(1, 2)),
}


@pytest.mark.parametrize("save8", [False, True])
@pytest.mark.parametrize("match", sorted(BAD))
def test_refused(match, save8, monkeypatch):
    host = HostOnly(B.lib())
    monkeypatch.setattr(B, "lib", lambda: host)
    monkeypatch.setattr(B, "_on", lambda device: B._HERE)
    monkeypatch.setattr(B, "_stream", lambda device: 0)
    layer = B.MoeLayer(T, d, E, k, I, device="cpu", save8=save8)
    layer.routing.logits = z(T, E)
    good = dict(dout=z(T, d), x=z(T, d), w_gate_up=z(E, 2 * I, d), w_down=z(E, d, I))
    layer.backward(**good)
    assert host.reached == ["moe_backward8" if save8 else "moe_backward"]
    with pytest.raises(ValueError, match=match):
        layer.backward(**{**good, **BAD[match]})
    assert len(host.reached) == 1
