"""The router's backward with infinities in x and w: a float32 dlogits beside
bfloat16 enters as two values, and the second must not meet an infinity."""
import math

import pytest
import torch

from combine_top_route_amd import binding as B
from test_gpu_router import DT, inputs, near

pytestmark = pytest.mark.gpu


# one run and several; one and more blocks of experts
@pytest.mark.parametrize("ldtype", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E", [(70, 72, 20), (300, 136, 40), (700, 264, 150)])
def test_infinities(T, d, E, dtype, ldtype):
    x, w, dl, dx_in = inputs(T, d, E, dtype, ldtype, seed=50)
    dl[:, 3] = torch.where(torch.arange(T, device=x.device) % 2 == 0, 0.5, -1.25).to(dl.dtype)   # exact in bfloat16
    x[7, 5], x[40, 9] = math.inf, -math.inf
    w[2, 11], w[3, 60] = math.inf, -math.inf
    x[13, 20] = math.nan
    x64, w64, l64 = x.double(), w.double(), dl.double()
    dx_ref = dx_in.double() + l64 @ w64
    dw_ref = l64.t() @ x64
    dx, dw = B.router_backward(dl, x, w, dx_in=dx_in)
    split = 2.0 ** -17 if dtype == "bf16" and ldtype == "f32" else 0.0
    for got, ref, mag, n in ((dx, dx_ref, dx_in.double().abs() + l64.abs() @ w64.abs(), E + 1),
                             (dw, dw_ref, l64.abs().t() @ x64.abs(), T)):
        assert torch.equal(got.isnan(), ref.isnan())
        inf = ref.isinf()
        assert bool(inf.any())
        assert torch.equal(torch.where(inf, got.double(), 0.0), torch.where(inf, ref, 0.0))
        ok = ref.isfinite()
        near(torch.where(ok, got, 0.0), torch.where(ok, ref, 0.0), torch.where(ok, mag, 0.0), n, split)
    assert bool(dx[:, [11, 60]].isinf().all()) and bool(dw[:, [5, 9]].isinf().all())
