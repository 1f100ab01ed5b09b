"""The router at the sizes of training: runs of many steps of tokens, rows of dx
beyond 32 MiB (whose work-groups start first), the forward's largest tile over
several units of K.  Bounds of test_gpu_router."""
import pytest
import torch

from test_gpu_router import DT, inputs, near

pytestmark = pytest.mark.gpu

# one run of four steps, full and with a short last one; eight runs of twelve
# steps, the last short; sixteen of eighteen and more than 32 MiB of rows in
# bfloat16; the same in float32; many blocks of experts over many tokens; one
# run a tile of d and E, hundreds of steps
BACKWARD = [(128, 40, 16), (97, 72, 5), (3001, 2048, 130), (9000, 2048, 128), (4200, 2056, 64), (2000, 520, 1000),
            (20000, 16384, 3), (1100, 16384, 300)]


@pytest.mark.parametrize("ldtype", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E", BACKWARD)
def test_backward(T, d, E, dtype, ldtype):
    from combine_top_route_amd import binding as B
    x, w, dl, dx_in = inputs(T, d, E, dtype, ldtype, seed=40)
    split = 2.0 ** -17 if dtype == "bf16" and ldtype == "f32" else 0.0
    x64, w64, l64 = x.double(), w.double(), dl.double()
    dw_ref, dw_mag = l64.t() @ x64, l64.abs().t() @ x64.abs()
    dx_ref, dx_mag = l64 @ w64, l64.abs() @ w64.abs()
    del x64
    for add in (dx_in, None):
        dx, dw = B.router_backward(dl, x, w, dx_in=add)
        a = add.double() if add is not None else torch.zeros((), dtype=torch.float64, device=x.device)
        near(dx, a + dx_ref, a.abs() + dx_mag, E + 1, split)
        near(dw, dw_ref, dw_mag, T, split)
        again = B.router_backward(dl, x, w, dx_in=add)
        assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("ldtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,E,dtype", [(12300, 1032, 100, "bf16"), (16384, 2048, 128, "bf16"), (12400, 1096, 70, "f32"),
                                         (6200, 16384, 40, "bf16")])
def test_forward(T, d, E, dtype, ldtype):
    from combine_top_route_amd import binding as B
    x, w, _, _ = inputs(T, d, E, dtype, ldtype, seed=41)
    got = B.router_logits(x, w, logits_dtype=DT[ldtype])
    x, w = x.double(), w.double()
    near(got, x @ w.t(), x.abs() @ w.abs().t(), d)
