"""The gate/up GEMM's encoding epilogue (moe_forward8 in bfloat16) where an
expert has more rows than a tile, and on pre-activations that are hard to
encode: against the row pass on the H that the plain layer keeps."""
import math

import pytest
import torch

import test_gpu_save8 as S8
from combine_top_route_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = S8.DEV


# tiles of 256 rows with a short last one, of 128 and of 64 rows; I with a last
# tile of 8 columns (264), of a short block (136, 40), of whole blocks (128)
@pytest.mark.parametrize("T,d,E,k,I,limit", [
    (700, 64, 2, 1, 264, 0.0), (300, 72, 1, 1, 136, 0.0), (600, 136, 3, 2, 40, 0.6), (1100, 64, 4, 1, 128, 0.0),
    (258, 40, 1, 1, 392, 0.0)])
def test_layer_of_long_segments(T, d, E, k, I, limit):
    S8.test_layer(T, d, E, k, I, "bf16", limit)


def same(a, b):
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))


@pytest.mark.parametrize("special", ["finite", "not finite"])
@pytest.mark.parametrize("T,I", [(30, 40), (100, 264), (300, 136), (600, 128)])
def test_hard_blocks(T, I, special):
    """x holds unit vectors, so that a row of H is a column of W_gate_up: zero
    rows, magnitudes down to 2^-43, blocks whose largest value is 1.75 2^e or just
    past it, ties; or infinities and NaN."""
    d, E, k = 64, 2, 1
    x = torch.nn.functional.one_hot(torch.arange(T, device=DEV) % d, d).bfloat16()
    wgu = torch.stack([S8.test_matrix(d, I, torch.bfloat16, seed=60 + e).t().contiguous() for e in range(E)])
    if special != "finite":
        wgu[0, 3, 1], wgu[0, I + 33, 2], wgu[1, 34, 4] = math.inf, -math.inf, math.nan
        x[5] = math.inf
        x[6, 10] = math.nan
    wd = torch.randn((E, d, I), generator=S8.gen(61), device=DEV).bfloat16()
    lg = torch.randn((T, E), generator=S8.gen(62), device=DEV)
    plain = B.MoeLayer(T, d, E, k, I, logits_dtype=torch.float32, device=DEV)
    layer = B.MoeLayer(T, d, E, k, I, logits_dtype=torch.float32, device=DEV, save8=True)
    layer.saved.fill_(171)
    same(layer.forward(x, wgu, wd, logits=lg), plain.forward(x, wgu, wd, logits=lg))
    H = plain.saved_views()[0].contiguous()
    if special == "finite":
        r = plain.routing
        tok = r.src_of.long()
        assert torch.equal(H, wgu[r.topk_ids.view(-1)[tok].long()].transpose(1, 2)[torch.arange(T, device=DEV), tok % d])
    _, codes, scales = B.swiglu_save8(H, None, T, k)
    got = layer.saved_views()
    assert torch.equal(got[0], codes) and torch.equal(got[1], scales)
    assert bool((scales == 255).any()) == (special != "finite")
    if special == "finite":
        v, s = S8.encode64(H)
        assert torch.equal(got[1], s) and torch.equal(got[0].view(torch.float8_e4m3fn).double(), v)
