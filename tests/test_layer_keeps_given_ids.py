"""A MoeLayer called with ids and then with logits writes the second call's ids and
weights into its own tensors, not into those it was given.  CPU only, with a stub
that writes where the library would."""
import os

import pytest
import torch

from combine_top_route_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="library not built")

T, d, E, k, I = 4, 64, 4, 2, 32
BF = torch.bfloat16


@pytest.mark.parametrize("save8", [False, True])
def test_given_ids_are_not_written(save8, monkeypatch):
    layer = B.MoeLayer(T, d, E, k, I, device="cpu", save8=save8)
    real = B.lib()

    class Stub:
        def __getattr__(self, name):
            if name.endswith(("_size", "_bytes", "_error", "_string")):
                return getattr(real, name)
            def forward(*a):
                if layer.routing.logits is not None:
                    layer.routing.topk_ids.fill_(7)
                    layer.routing.topk_w.fill_(7.0)
                return 0
            return forward

    monkeypatch.setattr(B, "lib", lambda: Stub())
    monkeypatch.setattr(B, "_on", lambda device: B._HERE)
    monkeypatch.setattr(B, "_stream", lambda device: 0)
    args = torch.zeros(T, d, dtype=BF), torch.zeros(E, 2 * I, d, dtype=BF), torch.zeros(E, d, I, dtype=BF)
    ids, w = torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k)
    layer.forward(*args, topk_ids=ids, topk_w=w)
    assert layer.routing.topk_ids is ids and layer.routing.topk_w is w and layer.routing.logits is None
    layer.forward(*args, logits=torch.zeros(T, E, dtype=BF))
    assert not ids.any() and not w.any()
    assert bool((layer.routing.topk_ids == 7).all()) and bool((layer.routing.topk_w == 7).all())
    layer.forward(*args, topk_ids=ids, topk_w=w)
    assert layer.routing.topk_ids is ids and layer.routing.topk_w is w and not ids.any()
