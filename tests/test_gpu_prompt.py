"""The prompt layer from MXFP4 weights against 64 bits, and moe_combine's masked
form.

Bound of the layer.  The weights are bfloat16 numbers and the sums float32, so a
sum over n terms errs by at most (n + 16) 2^-24 of its terms' magnitudes; the
activation passes on its two sums' errors (slope below 1.1 in the gate, |silu| in
the up value) and adds 1e-6 of itself (hardware exp and reciprocal); activations
and each slot's product are rounded to bf16, by 2^-8 at most.  The weights are a
float32 softmax: l - max errs by 2^-24 of at most |l| + |max|, exp by 2^-22, the
sum of k and its quotient by (k + 2) 2^-24.  The weighted sum adds (k + 2) 2^-24 of
its terms and the output's rounding 2^-8."""
import math

import pytest
import torch

from combine_top_route_amd import autograd as A
from combine_top_route_amd import binding as B
from test_gpu_grouped import DEV, values_of, weight

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, 2.0 ** -8


def reference(x, lg, gu, dn, k, limit):
    """(out, bound) of the layer in 64 bits, expert by expert."""
    T, d = x.shape
    I, lim = dn[0].shape[2] * 2, limit if limit > 0 else math.inf
    v, ids = torch.sort(lg.double(), dim=1, descending=True, stable=True)
    v, ids = v[:, :k], ids[:, :k]
    on = v > -math.inf
    top = torch.where(on[:, :1], v[:, :1], 0.0)
    ex = torch.where(on, torch.exp(v - top), 0.0)
    w = ex / ex.sum(1, keepdim=True).clamp(min=1e-300)
    far = torch.where(on, v.abs() + top.abs(), 0.0)
    wrel = 2 * (far * U + 2.0 ** -22) + (k + 2) * U      # a weight's own and its sum's
    out = torch.zeros((T, d), dtype=torch.float64, device=DEV)
    tol, mag = torch.zeros_like(out), torch.zeros_like(out)
    for e in range(lg.shape[1]):
        t, j = torch.nonzero((ids == e) & on, as_tuple=True)
        if not t.numel():
            continue
        W, D, xe = values_of(gu[0][e], gu[1][e]), values_of(dn[0][e], dn[1][e]), x[t].double()
        h, dh = xe @ W.t(), (d + 16) * U * (xe.abs() @ W.abs().t())
        g, u = h[:, :I].clamp(max=lim), h[:, I:].clamp(-lim, lim)
        s = g * torch.sigmoid(g)
        a = s * u
        da = 1.1 * dh[:, :I] * (u.abs() + dh[:, I:]) + s.abs() * dh[:, I:] + 1e-6 * a.abs()
        da = da + HALF * (a.abs() + da)
        y = a @ D.t()
        dy = da @ D.abs().t() + (I + 16) * U * ((a.abs() + da) @ D.abs().t())
        dy = dy + HALF * (y.abs() + dy)
        we = w[t, j, None]
        out.index_add_(0, t, we * y)
        mag.index_add_(0, t, we * (y.abs() + dy))
        tol.index_add_(0, t, we * (dy + wrel[t, j, None] * (y.abs() + dy)))
    tol = tol + (k + 2) * U * mag
    return out, tol + HALF * (out.abs() + tol) + 2.0 ** -130


def layer(T, d, E, k, I, lt=torch.float32, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + T)
    x = torch.randn((T, d), generator=g, device=DEV).bfloat16()
    return x, torch.randn((T, E), generator=g, device=DEV).to(lt), weight(E, 2 * I, d, 7), weight(E, d, I, 8)


# one token to thousands, on either side of what moe_decode takes; one expert and
# all of them; rows of the combine's two wide forms; more slots than a wave has lanes
@pytest.mark.parametrize("limit", [0.0, 0.75])
@pytest.mark.parametrize("T,d,E,k,I", [(1, 128, 1, 1, 128), (1, 2048, 16, 8, 256), (33, 2048, 40, 8, 384),
                                       (256, 256, 8, 3, 128), (257, 256, 8, 3, 128), (700, 4096, 12, 4, 256),
                                       (3001, 640, 32, 6, 128), (20, 384, 80, 70, 128), (513, 1152, 64, 9, 256)])
def test_prompt(T, d, E, k, I, limit):
    x, lg, gu, dn = layer(T, d, E, k, I, torch.bfloat16 if d == 640 else torch.float32)
    if E > 1:
        lg[:, E // 3] = -math.inf                       # a masked expert
        lg[T // 2, 1:] = -math.inf                      # one left
        lg[T // 2, 0] = 3.0
    if T > 2:
        lg[T - 1] = -math.inf                           # none left
        lg[T - 2] *= 20                                 # weights far from each other
    got = A.moe_prompt(x, lg, gu[0], dn[0], k, gu[1], dn[1], limit)
    want, tol = reference(x, lg, gu, dn, k, limit)
    over = ((got.double() - want).abs() / tol).max().item()
    assert over <= 1, f"worst error over bound {over:.3g}"
    assert T <= 2 or not bool(got[T - 1].any())


@pytest.mark.parametrize("lt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [1, 3, 4, 8, 9, 21])
@pytest.mark.parametrize("d", [8, 136, 2048, 4096])
def test_combine(d, k, dt, lt):
    """Masked slots add nothing, whatever their rows and weights hold; without the
    flag, and without masks, nothing changes."""
    T, E = 37, 24
    g = torch.Generator(device=DEV).manual_seed(d + k)
    lg = torch.randn((T, E), generator=g, device=DEV).to(lt)
    clean = B.route(lg, k)
    rows = torch.randn((T * k, d), generator=g, device=DEV).to(dt)
    assert torch.equal(B.combine(rows, clean, T, k, skip_masked=True), B.combine(rows, clean, T, k))
    lg[:, 5:9] = -math.inf
    lg[3, 2:] = -math.inf
    lg[11] = -math.inf
    lg[12, 4] = math.nan
    r = B.route(lg, k)
    off = lg.gather(1, r.topk_ids.long()) == -math.inf
    assert bool(off[11].all()) and bool(off.any()) and not bool(off[0, 0])
    at = r.row_of.view(T, k).long()
    junk = torch.tensor([math.nan, math.inf, -math.inf], device=DEV)
    rows[at[off]] = junk[torch.arange(int(off.sum()), device=DEV) % 3, None].to(dt)
    w = torch.where(off, math.nan, torch.rand((T, k), generator=g, device=DEV))
    r.topk_w = w.contiguous()
    got = B.combine(rows, r, T, k, skip_masked=True)
    terms = torch.where(off[..., None], 0.0, w[..., None].double() * rows[at].double())
    want, mag = terms.sum(1), terms.abs().sum(1)
    half = torch.finfo(dt).eps / 2
    assert bool(((got.double() - want).abs() <= (k + 2) * U * mag * (1 + half) + half * want.abs()).all())
    assert not bool(got[11].any())


def test_captured():
    """The layer in a graph, replayed with other values."""
    T, d, E, k, I = 300, 256, 16, 4, 128
    x, lg, gu, dn = layer(T, d, E, k, I)
    lg[:, 3] = -math.inf
    lg[7] = -math.inf
    run = lambda: A.moe_prompt(x, lg, gu[0], dn[0], k, gu[1], dn[1])
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(4):
        x.copy_(torch.randn((T, d), device=DEV))
        lg[:, 4 + i] = -math.inf
        x[7] = math.nan
        want = run()
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and bool(out.isfinite().all()), i


@pytest.mark.parametrize("d", [8, 136, 2048, 4096])
@pytest.mark.parametrize("k", [64, 65, 70, 130])
def test_combine_more_slots_than_lanes(d, k):
    T, E = 9, 140
    g = torch.Generator(device=DEV).manual_seed(d + k)
    lg = torch.randn((T, E), generator=g, device=DEV)
    lg[:, ::3] = -math.inf
    lg[4] = -math.inf
    r = B.route(lg, k)
    off = lg.gather(1, r.topk_ids.long()) == -math.inf
    rows = torch.randn((T * k, d), generator=g, device=DEV).bfloat16()
    at = r.row_of.view(T, k).long()
    rows[at[off]] = math.nan
    r.topk_w = torch.where(off, math.inf, torch.rand((T, k), generator=g, device=DEV)).contiguous()
    got = B.combine(rows, r, T, k, skip_masked=True)
    terms = torch.where(off[..., None], 0.0, r.topk_w[..., None].double() * rows[at].double())
    want, mag = terms.sum(1), terms.abs().sum(1)
    assert bool(off.any()) and bool(((got.double() - want).abs() <= (k + 2) * U * mag * 1.01 + HALF * want.abs()).all())
    assert not bool(got[4].any())
