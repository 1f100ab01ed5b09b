"""Functions that take a Routing refuse one whose tensors lie elsewhere than the
rows, in host memory or on another GPU, before the library is called.  CPU only:
fake tensors, stubs in place of the entry points."""
import os

import pytest
import torch
from torch._subclasses import FakeTensorMode

from combine_top_route_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="library not built")

T, d, E, k = 4, 128, 4, 2
HERE, OTHER, HOST = torch.device("cuda", 0), torch.device("cuda", 1), torch.device("cpu")


def z(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device=HERE)


CALLS = {
    "permute": lambda r: B.permute(z(T, d), r, k),
    "combine": lambda r: B.combine(z(T * k, d), r, T, k),
    "quantize_tokens_fp8": lambda r: B.quantize_tokens_fp8(z(T, d), r, T, k, True),
    "quantize_tokens_mxfp8": lambda r: B.quantize_tokens_mxfp8(z(T, d), r, T, k, True),
    "route_noalloc": lambda r: B.route_noalloc(r, T, E, k),
}


# the tensors of the Routing that a call reads or writes
USED = {
    "permute": ("src_of", "row_of"), "combine": ("row_of", "topk_w"), "quantize_tokens_fp8": ("offsets", "src_of"),
    "quantize_tokens_mxfp8": ("offsets", "src_of"),
    "route_noalloc": ("logits", "topk_ids", "topk_w", "offsets", "row_of", "src_of"),
}


@pytest.mark.parametrize("where", [HOST, OTHER], ids=str)
@pytest.mark.parametrize("name", sorted(CALLS))
def test_refused(name, where, monkeypatch):
    reached, real = [], B.lib()

    class Stub:
        def __getattr__(self, entry):
            if entry.endswith(("_size", "_bytes", "_error", "_string")):
                return getattr(real, entry)
            return lambda *a: reached.append(entry) or 0

    monkeypatch.setattr(B, "lib", lambda: Stub())
    monkeypatch.setattr(B, "_ptr", lambda t: None if t is None else 1 << 20)
    monkeypatch.setattr(B, "_on", lambda device: B._HERE)
    monkeypatch.setattr(B, "_stream", lambda device: 0)
    with FakeTensorMode():
        make = lambda: B.Routing.empty(T, E, k, HERE, logits=z(T, E))
        CALLS[name](make())
        assert len(reached) == 1
        for field in USED[name]:
            r = make()
            t = getattr(r, field)
            setattr(r, field, torch.empty(t.shape, dtype=t.dtype, device=where))
            with pytest.raises(ValueError, match=f"routing.{field} is on {where}"):
                CALLS[name](r)
    assert len(reached) == 1
