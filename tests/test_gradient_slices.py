"""The backward operators bring gradients that start off a 16-byte boundary to
one before the library is called (CPU: the calls are stubs)."""
import os

import pytest
import torch

from combine_top_route_amd import autograd as A
from combine_top_route_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="library not built")

T, d, E, k, I = 5, 64, 3, 2, 32
BF = torch.bfloat16


def sliced(*shape, dtype=BF):
    n = torch.Size(shape).numel()
    t = torch.arange(n + 3, dtype=torch.float32).to(dtype)[3:].view(shape)
    assert t.data_ptr() % 16
    return t


def test_router(monkeypatch):
    got = {}
    monkeypatch.setattr(A, "_check_devices", lambda **t: got.update(t))
    monkeypatch.setattr(B, "router_backward", lambda dl, x, w, dx_in: got.update(dl=dl, add=dx_in))
    dl, add = sliced(T, E, dtype=torch.float32), sliced(T, d)
    A.router_bwd._init_fn(dl, torch.zeros(T, d, dtype=BF), torch.zeros(E, d, dtype=BF), add)
    assert got["dl"].data_ptr() % 16 == 0 and torch.equal(got["dl"], dl)
    assert got["add"].data_ptr() % 16 == 0 and torch.equal(got["add"], add)


@pytest.mark.parametrize("name", ["moe_bwd", "moe_bwd8"])
def test_layer(name, monkeypatch):
    seen = []

    def devices(x, dout, **rest):
        seen.append(dout)
        raise ValueError("far enough")

    monkeypatch.setattr(A, "_check_devices", devices)
    dout = sliced(T, d)
    shape = B.make_shape(T, d, E, k, I, BF, torch.float32)
    r = B.Routing.empty(T, E, k, "cpu")
    saved = torch.empty(B.saved8_size(shape) if name == "moe_bwd8" else B.saved_size(shape), dtype=torch.uint8)
    with pytest.raises(ValueError, match="far enough"):
        getattr(A, name)._init_fn(dout, torch.zeros(T, d, dtype=BF), torch.zeros(T, E),
                                  torch.zeros(E, 2 * I, d, dtype=BF), torch.zeros(E, d, I, dtype=BF), saved, r.topk_ids,
                                  r.topk_w, r.counts, r.offsets, r.row_of, r.src_of, k,
                                  *(["native"] if name == "moe_bwd" else []))
    assert seen[0].data_ptr() % 16 == 0 and torch.equal(seen[0], dout)
