"""The router's projection and its gradients against float64 matrix products.

Tolerances.  Sums run in float32: n terms are off by at most n 2^-24 times the
sum of their magnitudes, plus the product's 2^-24; a float32 dlogits beside
bf16 tensors is carried to 2^-17 (two bf16 values); the result is rounded once.
"""
import pytest
import torch

from combine_top_route_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}

# one token and one expert; every tile of the forward; E and d tails; E odd
# (rows of dlogits that are not 16-byte aligned); more experts than one block;
# runs of tokens with a short last step
SIZES = [(1, 8, 1), (5, 64, 3), (33, 2048, 128), (17, 40, 16), (200, 136, 17), (333, 72, 40), (130, 264, 64),
         (1000, 200, 128), (64, 1000, 129), (300, 24, 1024), (5000, 40, 8), (12300, 16, 100), (6200, 72, 33),
         (3100, 136, 200)]


def inputs(T, d, E, dtype, ldtype, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    return (rn(T, d).to(DT[dtype]), (rn(E, d) * d ** -0.5).to(DT[dtype]), rn(T, E).to(DT[ldtype]),
            rn(T, d).to(DT[dtype]))


def near(got, ref, mag, n, extra=0.0):
    tol = ((n + 2) * 2.0 ** -24 + extra) * mag + STEP[got.dtype] * ref.abs() * (1 + 2.0 ** -6) + 1e-37
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), f"worst error over bound {float((err / tol).max()):.3g}"


@pytest.mark.parametrize("ldtype", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E", SIZES)
def test_forward(T, d, E, dtype, ldtype):
    x, w, _, _ = inputs(T, d, E, dtype, ldtype)
    got = B.router_logits(x, w, logits_dtype=DT[ldtype])
    assert got.shape == (T, E) and got.dtype == DT[ldtype]
    x, w = x.double(), w.double()
    near(got, x @ w.t(), x.abs() @ w.abs().t(), d)


@pytest.mark.parametrize("ldtype", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E", SIZES)
def test_backward(T, d, E, dtype, ldtype):
    x, w, dl, dx_in = inputs(T, d, E, dtype, ldtype)
    split = 2.0 ** -17 if dtype == "bf16" and ldtype == "f32" else 0.0
    x64, w64, l64 = x.double(), w.double(), dl.double()
    for add in (dx_in, None):
        dx, dw = B.router_backward(dl, x, w, dx_in=add)
        a = add.double() if add is not None else torch.zeros_like(x64)
        near(dx, a + l64 @ w64, a.abs() + l64.abs() @ w64.abs(), E + 1, split)
        near(dw, l64.t() @ x64, l64.abs().t() @ x64.abs(), T, split)


def test_add_in_place_and_repeatable():
    T, d, E = 700, 136, 40
    x, w, dl, dx_in = inputs(T, d, E, "bf16", "f32")
    dx, dw = B.router_backward(dl, x, w, dx_in=dx_in)
    again = B.router_backward(dl, x, w, dx_in=dx_in)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    import ctypes
    sh = B.make_shape(T, d, E, 1, 8, torch.bfloat16, torch.float32)
    ws = torch.full((B.router_workspace_size(sh),), 255, dtype=torch.uint8, device=DEV)
    dw2 = torch.empty_like(w)
    B._check("moe_router_backward", B.lib().moe_router_backward(
        ctypes.byref(sh), B._ptr(dl), B._ptr(x), B._ptr(w), B._ptr(dx_in), B._ptr(dx_in), B._ptr(dw2), B._ptr(ws),
        ws.numel(), B._stream(DEV)))
    assert torch.equal(dx_in, dx) and torch.equal(dw2, dw)


def test_nan_and_infinity_stay_where_they_are():
    T, d, E = 70, 72, 20
    x, w, dl, _ = inputs(T, d, E, "bf16", "f32")
    x[3, 5] = float("nan")
    w[7, 1] = float("inf")
    dl[11, 2] = float("inf")
    dl[12, 4] = 3.4e38              # rounds to infinity in bf16
    lg = B.router_logits(x, w)
    bad = torch.zeros(T, E, dtype=torch.bool, device=DEV)
    bad[3] = True
    bad[:, 7] = True
    assert torch.equal(~lg.isfinite(), bad)
    w = w.nan_to_num(0.0, 0.0, 0.0)
    dx, dw = B.router_backward(dl, x, w)
    assert torch.equal(dx.isfinite().all(1), ~torch.isin(torch.arange(T, device=DEV), torch.tensor([11, 12], device=DEV)))
    assert not bool(dx[11].isnan().any())
    ok = torch.ones(E, d, dtype=torch.bool, device=DEV)
    ok[2] = False
    ok[4] = False
    ok[:, 5] = False
    assert bool(dw[ok].isfinite().all()) and bool(dw[:, 5].isnan().all())


def test_captured_and_replayed():
    T, d, E = 500, 128, 24
    x, w, dl, dx_in = inputs(T, d, E, "bf16", "f32")
    B.router_logits(x, w)
    B.router_backward(dl, x, w, dx_in=dx_in)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lg = B.router_logits(x, w)
        dx, dw = B.router_backward(dl, x, w, dx_in=dx_in)
    for i in range(4):
        for t, n in zip((x, w, dl, dx_in), inputs(T, d, E, "bf16", "f32", seed=5 + i)):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(lg, B.router_logits(x, w))
        want = B.router_backward(dl, x, w, dx_in=dx_in)
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
