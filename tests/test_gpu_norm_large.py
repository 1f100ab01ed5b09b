"""The norms' backward where its rows pass the last-level cache (256 MiB of operands:
rows loaded past the caches, the next one on its way), for every spread of a row over
lanes; in place and in a replayed graph there; and a few long rows.  Bounds are
those of test_gpu_norm.py."""
import ctypes

import pytest
import torch

from combine_top_route_amd import binding as B
from test_gpu_norm import EPS, args, check, inputs

pytestmark = pytest.mark.gpu

# (T, d) with 6 T d values above 256 MiB, by the lanes of a row and 16-byte pieces a lane
BF16 = {"8": (1 << 20, 24), "8 full": ((1 << 19) + 7, 64), "16": (300001, 80), "32": (200003, 136), "64": (110001, 264),
        "128": (60007, 520), "256 idle": (30011, 1032), "256": (16387, 2048), "320": (9001, 2560), "384": (8999, 2880),
        "512": (6001, 4096), "512x2": (4501, 5000), "512x4": (1501, 16376)}
F32 = {"8": (1 << 19, 24), "16": (300001, 40), "32": (130003, 96), "64": (60007, 200), "128": (40009, 296),
       "256": (15001, 1000), "320": (9001, 1280), "384": (8999, 1440), "512": (9001, 2048), "512x2": (3001, 4096),
       "512x4": (2801, 5000), "512x8": (701, 16376)}


def past_cache(T, d, size):
    return 6 * T * d * size > 256 << 20


@pytest.mark.parametrize("name", list(BF16))
def test_bf16(name):
    T, d = BF16[name]
    assert past_cache(T, d, 2)
    check(T, d, "bf16", "all")


@pytest.mark.parametrize("name", list(F32))
def test_f32(name):
    T, d = F32[name]
    assert past_cache(T, d, 4)
    check(T, d, "f32", "all")


@pytest.mark.parametrize("form", ["pre", "token", "plain", "last", "gate"])
def test_forms(form):
    check(33001, 2048, "bf16", form)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [2048, 4096, 4104, 8192, 16384])
@pytest.mark.parametrize("T", [2, 3, 4, 5])
def test_few_rows(T, d, dtype):
    check(T, d, dtype, "all")


@pytest.mark.parametrize("T,d", [(16387, 2048), (9001, 2560)])
def test_in_place(T, d):
    """dx over dz gives the same, and rows behind the last stay as they were."""
    t, scale = inputs(T, d, "bf16", "all")
    z, _ = B.norm_residual(t["x"], t["y"], **args(t, scale))
    want = B.norm_residual_backward(t["dz"], t["dh"], z, t["y"], **args(t, scale))
    pad = lambda v: torch.cat([v, torch.full((3, d), 7.0, dtype=v.dtype, device="cuda")])
    dz, dy = pad(t["dz"]), pad(torch.zeros_like(z))
    sh = B.MoeNormShape(T, d, 1, B.GATE_CHANNEL, scale, EPS)
    p, stream = B._ptr, torch.cuda.current_stream().cuda_stream
    ws = torch.empty(B.norm_workspace_size(sh), dtype=torch.uint8, device="cuda")
    dw = [torch.empty_like(t["gate"]) for _ in range(3)]
    assert B.lib().moe_norm_backward(ctypes.byref(sh), p(dz), p(t["dh"]), p(z), p(t["y"]), p(t["w_post"]), p(t["gate"]),
                                     p(t["w_next"]), p(dz), p(dy), *map(p, dw), p(ws), ws.numel(), stream) == 0
    for got, ref in ((dz, want["dx"]), (dy, want["dy"])):
        assert torch.equal(got[:T], ref) and bool((got[T:] == 7).all())
    for got, n in zip(dw, ("dw_post", "dgate", "dw_next")):
        assert torch.equal(got, want[n]), n


@pytest.mark.parametrize("T,d,dtype", [(16387, 2048, "bf16"), (3001, 4096, "f32"), (3, 16384, "bf16")])
def test_replayed(T, d, dtype):
    t, scale = inputs(T, d, dtype, "all")
    step = lambda: list(B.norm_residual_backward(t["dz"], t["dh"], t["x"], t["y"], **args(t, scale)).values())
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        t["x"].mul_(1.25)
        t["dz"].add_(0.5)
        want = step()
        for o in out:
            o.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
