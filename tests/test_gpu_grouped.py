"""Products of expert-sorted rows with MXFP4 matrices, and the prompt layer made
of them, against 64 bits.

Bounds.  The operands are exact in bfloat16 (a code times its scale is a bfloat16
number), sums are float32: an output errs by at most (K + 16) 2^-24 of the sum of
its terms' magnitudes, and by half a step of its rounding, 2^-8.  With SwiGLU the
two sums' errors pass through it (its slope below 1.1 in the gate, |silu| in the
up value), and the hardware exp and reciprocal add 1e-6 of the value."""
import math

import pytest
import torch

from combine_top_route_amd import autograd as A
from combine_top_route_amd import binding as B
from test_gpu_mxfp4 import DEV, values_of

pytestmark = pytest.mark.gpu


def weight(E, N, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return B.quantize_mxfp4((torch.randn((E, N, K), generator=g, device=DEV) * K ** -0.5).bfloat16())


def routing(counts, k, seed=0):
    """A routing with these rows per expert: T tokens of k slots, the slots in
    any order (an expert may come twice in a token; the products do not mind)."""
    R = sum(counts)
    assert R % k == 0
    g = torch.Generator().manual_seed(seed)
    ids = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))[torch.randperm(R, generator=g)]
    r = B.route_ids(ids.view(-1, k).to(torch.int32).to(DEV), torch.rand((R // k, k), generator=g).to(DEV), len(counts))
    assert r.counts.tolist() == list(counts)
    return r


def reference(x, w, r, k, gather, swiglu, limit):
    """(y, bound) in 64 bits."""
    R, lim = r.src_of.numel(), limit if limit > 0 else math.inf
    N, K = w[0].shape[1], x.shape[1]
    y = torch.zeros((R, N // 2 if swiglu else N), dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(y)
    off = r.offsets.tolist()
    for e in range(len(off) - 1):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        a = (x[r.src_of[lo:hi].long() // k] if gather else x[lo:hi]).double()
        W = values_of(w[0][e], w[1][e])
        h, dh = a @ W.t(), (K + 16) * 2.0 ** -24 * (a.abs() @ W.abs().t())
        if swiglu:
            g, u = h[:, :N // 2], h[:, N // 2:]
            gc, uc = g.clamp(max=lim), u.clamp(-lim, lim)
            s = gc * torch.sigmoid(gc)
            y[lo:hi] = s * uc
            tol[lo:hi] = 1.1 * dh[:, :N // 2] * (uc.abs() + dh[:, N // 2:]) + s.abs() * dh[:, N // 2:] + \
                1e-6 * (s * uc).abs()
        else:
            y[lo:hi], tol[lo:hi] = h, dh
    return y, tol + 2.0 ** -8 * (y.abs() + tol) + 2.0 ** -130


def near(got, y, tol):
    over = (got.double() - y).abs() / tol
    assert got.shape == y.shape and bool((over <= 1).all()), f"worst error over bound {over.max().item():.3g}"


# rows per expert: none, one, around every tile height, several tiles, one expert
COUNTS = {"one": ([1], 1), "few": ([0, 3, 0, 1, 2, 0], 2), "tiles": ([64, 0, 65, 128, 129, 256, 257, 63, 1, 37], 4),
          "many": ([700, 3, 0, 1025], 4), "spread": ([2] * 130 + [0] * 7 + [5] * 20, 6),
          "lone": ([0, 0, 0, 90, 0], 3), "hundreds": ([1, 0, 2] * 200 + [3] * 40, 8), "mid": ([17, 33, 49, 16, 32, 8, 45], 5)}


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N,K", [(256, 128), (528, 384), (16, 256), (1040, 640), (784, 1024)])
@pytest.mark.parametrize("name", list(COUNTS))
def test_products(name, N, K, gather, swiglu):
    counts, k = COUNTS[name]
    E, R = len(counts), sum(counts)
    r = routing(counts, k)
    w = weight(E, N, K, seed=N)
    x = torch.randn((R // k if gather else R, K), generator=torch.Generator(device=DEV).manual_seed(K), device=DEV)
    x = x.bfloat16()
    limit = 0.75 if K == 640 else 0.0
    got = B.grouped_product(x, w, r, R // k, k, gather=gather, swiglu=swiglu, swiglu_limit=limit)
    near(got, *reference(x, w, r, k, gather, swiglu, limit))


# enough work-groups for the larger tiles: 64 rows by 256 columns, then 128 by 256
# (segments around each tile height, none, several tiles, K of one to five times
# 128), and 64 by 128; more experts than 128
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("K", [128, 256, 384, 640])
@pytest.mark.parametrize("E,mean,N", [(64, 30, 1040), (130, 33, 528), (66, 90, 1040), (140, 75, 528), (300, 7, 144)])
def test_many(E, mean, N, K, swiglu):
    g = torch.Generator().manual_seed(E + K)
    counts = torch.poisson(torch.full((E,), float(mean)), generator=g).long().tolist()
    edges = [0, 1, 15, 16, 17, 31, 32, 33, 48, 49, 63, 64, 65, 95, 96, 97, 127, 128, 129, 257]
    counts[:len(edges)] = edges
    k = 2
    counts[-1] += sum(counts) % k
    r = routing(counts, k, seed=E)
    R = sum(counts)
    w = weight(E, N, K, seed=N)
    x = torch.randn((R // k, K), generator=torch.Generator(device=DEV).manual_seed(K), device=DEV).bfloat16()
    near(B.grouped_product(x, w, r, R // k, k, swiglu=swiglu), *reference(x, w, r, k, True, swiglu, 0.0))


# K over the waves: every number of stages a wave from none to four, one or two
# blocks of 16 rows
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("K", [1024, 1152, 1280, 1408, 2048])
def test_split(K, swiglu):
    counts, k, N = [3, 0, 16, 17, 32, 33, 1, 2], 8, 208
    r, w = routing(counts, k), weight(8, N, K, seed=K)
    R = sum(counts)
    x = torch.randn((R // k, K), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).bfloat16()
    near(B.grouped_product(x, w, r, R // k, k, swiglu=swiglu), *reference(x, w, r, k, True, swiglu, 0.0))


@pytest.mark.parametrize("N", [8, 24, 248, 264])
def test_narrow(N):
    r = routing([5, 70, 0, 300, 1], 4)
    w, x = weight(5, N, 256, 1), torch.randn((94, 256), device=DEV).bfloat16()
    near(B.grouped_product(x, w, r, 94, 4), *reference(x, w, r, 4, True, False, 0.0))


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,k", [([20] * 30, 4), ([300, 0, 500], 2), ([1, 2, 3, 2], 2), ([70] * 140, 4),
                                      ([30] * 140, 4)])
def test_rows_behind_and_odd_offsets(counts, k, swiglu):
    """Rows of no expert are left as they were; offsets outside or out of order
    reach no memory but y's rows."""
    R, N, K = sum(counts), 272, 256
    r = routing(counts, k)
    w, x = weight(len(counts), N, K, 2), torch.randn((R // k, K), device=DEV).bfloat16()
    full = B.grouped_product(x, w, r, R // k, k, swiglu=swiglu)
    short = B.Routing(r.topk_ids, r.topk_w, r.counts, r.offsets.clamp(max=R - 7), r.row_of, r.src_of)
    out = torch.full_like(full, 5.0)
    assert B.grouped_product(x, w, short, R // k, k, swiglu=swiglu, out=out) is out
    assert torch.equal(out[:R - 7], full[:R - 7]) and bool((out[R - 7:] == 5).all())
    pad = torch.full((R + 2, full.shape[1]), 5.0, dtype=torch.bfloat16, device=DEV)
    for off in (r.offsets + 1000000, r.offsets - 1000000, r.offsets.flip(0).contiguous(), r.offsets * 3 - R):
        odd = B.Routing(r.topk_ids, r.topk_w, r.counts, off, r.row_of, r.src_of * 1000 - 7)
        B.grouped_product(x, w, odd, R // k, k, swiglu=swiglu, out=pad[:R])
    torch.cuda.synchronize()
    assert bool((pad[R:] == 5).all())


@pytest.mark.parametrize("counts,k", [([3, 0, 5, 4], 2), ([200, 90, 0, 34], 4), ([12] * 40, 8), ([68] * 140, 8),
                                      ([28] * 140, 8)])
def test_nan_and_infinity_stay_where_they_are(counts, k):
    E, R, N, K = len(counts), sum(counts), 272, 384
    r = routing(counts, k)
    w = tuple(t.clone() for t in weight(E, N, K, 3))
    x = torch.randn((R // k, K), generator=torch.Generator(device=DEV).manual_seed(5), device=DEV).bfloat16()
    clean = B.grouped_product(x, w, r, R // k, k)
    x[1, 100], x[R // k - 1, 7] = math.nan, math.inf
    hit = torch.isin(r.src_of.long() // k, torch.tensor([1, R // k - 1], device=DEV))
    got = B.grouped_product(x, w, r, R // k, k)
    assert torch.equal(got[~hit], clean[~hit])
    assert not bool(got[hit].isfinite().any())
    x[1, 100], x[R // k - 1, 7] = 0.0, 0.0
    clean = B.grouped_product(x, w, r, R // k, k)
    w[1][0, 13, 5] = 255                                   # a block of one column of expert 0
    got = B.grouped_product(x, w, r, R // k, k)
    lo = counts[0]
    assert bool(got[:lo, 13].isnan().all())
    got[:lo, 13] = clean[:lo, 13]
    assert torch.equal(got, clean)


def test_graph_and_stream():
    counts, k = [30, 0, 70, 200, 4], 4
    R = sum(counts)
    r, w = routing(counts, k), weight(5, 528, 256, 4)
    x = torch.randn((R // k, 256), device=DEV).bfloat16()
    want = B.grouped_product(x, w, r, R // k, k, swiglu=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = B.grouped_product(x, w, r, R // k, k, swiglu=True)
    side.synchronize()
    assert torch.equal(want, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = B.grouped_product(x, w, r, R // k, k, swiglu=True)
    for i in range(4):
        x.mul_(1.25)
        eager = B.grouped_product(x, w, r, R // k, k, swiglu=True)
        out.fill_(2.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i


@pytest.mark.parametrize("T,d,E,k,I", [(1, 256, 8, 2, 128), (300, 256, 16, 4, 256), (1000, 384, 6, 2, 128)])
def test_prompt(T, d, E, k, I):
    """The layer from its parts, and beside the few-token form: both round to
    bf16, moe_prompt also the activations and each slot's product."""
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn((T, d), generator=g, device=DEV).bfloat16()
    lg = torch.randn((T, E), generator=g, device=DEV)
    lg[:, 3] = -math.inf
    if T > 1:
        lg[1] = -math.inf
        lg[2, 1:] = -math.inf
    gu, dn = weight(E, 2 * I, d, 7), weight(E, d, I, 8)
    got = A.moe_prompt(x, lg, gu[0], dn[0], k, gu[1], dn[1], 1.5)
    n = min(T, 256)
    dec = B.MoeDecoder(n, d, E, k, I, weights="mxfp4", device=DEV, swiglu_limit=1.5, logits_dtype=torch.float32)
    want = dec.forward(x[:n], gu, dn, logits=lg[:n].contiguous())
    # magnitudes: sum over slots and columns of |w a W|
    W, D = values_of(*gu), values_of(*dn)
    mag = torch.zeros((n, d), dtype=torch.float64, device=DEV)
    for j in range(k):
        for e in range(E):
            t = (dec.topk_ids[:, j] == e).nonzero()[:, 0]
            h = x[t].double() @ W[e].t()
            a = torch.nn.functional.silu(h[:, :I].clamp(max=1.5)) * h[:, I:].clamp(-1.5, 1.5)
            y = a @ D[e].t()
            mag[t] += dec.topk_w[t, j, None].double() * (2.0 ** -8 * (a.abs() @ D[e].abs().t()) + 2.0 ** -8 * y.abs())
    tol = 1.1 * mag + 2.0 ** -7 * want.double().abs() + 1e-6
    assert bool(((got[:n].double() - want.double()).abs() <= tol).all())
    if T > 1:
        assert not bool(got[1].any())
    f = torch.compile(lambda *a: A.moe_prompt(*a[:4], k, *a[4:], 1.5), fullgraph=True, backend="aot_eager")
    assert torch.equal(f(x, lg, gu[0], dn[0], gu[1], dn[1]), got)


def test_prompt_masks_what_is_not_finite():
    """A masked slot adds nothing, whatever its token and its expert hold."""
    T, d, E, k, I = 40, 256, 8, 3, 128
    x = torch.randn((T, d), device=DEV).bfloat16()
    lg = torch.randn((T, E), device=DEV)
    gu, dn = weight(E, 2 * I, d, 7), weight(E, d, I, 8)
    dn[1][5] = 255  # expert 5 makes NaN
    lg[:, 5] = -math.inf
    lg[4, :4] = lg[4, 6:] = -math.inf  # one expert left
    lg[7] = -math.inf
    lg[9] = -math.inf
    x[7] = math.nan
    x[9] = math.inf
    got = A.moe_prompt(x, lg, gu[0], dn[0], k, gu[1], dn[1])
    dec = B.MoeDecoder(T, d, E, k, I, weights="mxfp4", device=DEV, logits_dtype=torch.float32)
    want = dec.forward(x, gu, dn, logits=lg)
    assert bool(got.isfinite().all()) and bool(want.isfinite().all())
    assert not bool(got[[7, 9]].any()) and not bool(want[[7, 9]].any())
    one = A.moe_prompt(x[4:5], lg[4:5], gu[0], dn[0], k, gu[1], dn[1])  # the expert alone, weight 1
    near = (got[4:5].double() - one.double()).abs()
    assert bool((near <= 2.0 ** -7 * one.double().abs() + 2.0 ** -7 * one.double().abs().max()).all())
