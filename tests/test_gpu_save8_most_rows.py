"""The checkpoint's row passes at 2^26 rows of a wave each: 2^32 threads, more than
one dimension of a launch takes.  Rows repeat with a period, so the results of
every period equal the first one's, which a call of its own gives."""
import pytest
import torch

from combine_top_route_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
T, k, I, P = 1 << 24, 4, 264, 4096
R = T * k


def rows(width, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    base = torch.randn((P, width), generator=g, device=DEV).bfloat16()
    full = torch.empty((R, width), dtype=torch.bfloat16, device=DEV)
    full.view(R // P, P, width).copy_(base)
    return base, full


def repeats(full, base):
    full = full.view(R // P, *base.shape)
    return all(bool((part == base).all()) for part in full.split(512))


def test_rows_beyond_one_launch_dimension():
    need = 190 << 30
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip("needs 190 GiB of free GPU memory")
    src = torch.arange(R, dtype=torch.int32, device=DEV)
    w = (torch.arange(R, device=DEV) % P + 1).float().view(T, k) / P
    r = B.Routing(None, w, None, None, None, src)
    r0 = B.Routing(None, w.view(-1)[:P].view(P, 1).contiguous(), None, None, None, src[:P].contiguous())
    h0, H = rows(2 * I, 80)
    _, c0, s0 = B.swiglu_save8(h0, None, P, 1)
    _, codes, scales = B.swiglu_save8(H, None, T, k)
    assert repeats(codes, c0) and repeats(scales, s0)
    del H
    torch.cuda.empty_cache()
    g0, G = rows(I, 81)
    dh0, aw0, dw0 = B.swiglu_backward8(g0, c0, s0, r0, P, 1)
    dh, aw, dw = B.swiglu_backward8(G, codes, scales, r, T, k)
    assert repeats(dh, dh0) and repeats(aw, aw0) and repeats(dw, dw0)
    del G, codes, scales, dh, aw, dw
    torch.cuda.empty_cache()
