"""The 8-bit activation checkpoint: its row passes against a plain float64
evaluation and the library's own MXFP8 encoder, and the layer's forward and
backward through it.

Tolerances.  Codes and scale bytes are exact.  The row passes compute in
float32 with the hardware exp and reciprocal (z = g or a few of its sums, each
operation within 2^-23; the exponential's argument reaches |g| log2 e, off by
|g| 2^-23): values within (16 + 2 |g|) 2^-23 of the magnitudes that enter them,
plus the result's rounding.  The layer's backward rounds G, Aw and dH to the
storage type (2^-8 for bf16) before the products that read them and every
result once, so a gradient is off by at most the sums of the products'
magnitudes times 2 (G through dH) or 1 such steps, plus one for itself; the
small terms are covered by counting three steps for two and two for one.
"""
import math

import pytest
import torch

from combine_top_route_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def routing(T, k, E, seed=0):
    g = gen(seed)
    ids = torch.rand((T, E), generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32).contiguous()
    w = torch.rand((T, k), generator=g, device=DEV) + 0.1
    return B.route_ids(ids, w, E)


def row_weight(r):
    return r.topk_w.double().view(-1)[r.src_of.long()][:, None]


def encode64(H):
    """(values of the codes, scale bytes) of H [R, 2I], in float64."""
    R, two_i = H.shape
    I = two_i // 2
    nb = -(-I // 32)
    h = torch.nn.functional.pad(H.double().view(R, 2, I), (0, 32 * nb - I)).view(R, 2, nb, 32)
    amax = h.abs().amax(3)
    m, e = torch.frexp(amax)
    X = torch.where(amax > 0, (e - 9 + (m > 0.875)).clamp(min=-127), 0)
    y = h * torch.exp2(-X.double())[..., None]
    ex = torch.frexp(y)[1].clamp(min=-5) - 1                 # floor(log2), from 2^-6 on
    step = torch.exp2(ex.double() - 3)
    v = torch.round(y / step) * step
    return v.view(R, 2, 32 * nb)[:, :, :I].reshape(R, two_i), (X + 127).to(torch.uint8).view(R, 2 * nb)


def decode64(codes, scales):
    R, two_i = codes.shape
    I = two_i // 2
    v = codes.view(torch.float8_e4m3fn).double().view(R, 2, I)
    s = torch.exp2(scales.double().view(R, 2, -1) - 127.0).repeat_interleave(32, 2)[:, :, :I]
    v = v * s
    return v[:, 0], v[:, 1]


def act64(g, u, limit):
    lim = limit if limit > 0 else math.inf
    gc, uc = g.clamp(max=lim), u.clamp(-lim, lim)
    s = torch.sigmoid(gc)
    return gc, uc, s


def test_matrix(R, I, dtype, seed=0):
    """Rows of very different magnitudes, an all-zero row, exact ties, blocks
    whose largest magnitude is 1.75 2^e or just past it."""
    g = gen(seed)
    H = torch.randn((R, 2 * I), generator=g, device=DEV)
    H *= torch.exp(torch.rand((R, 1), generator=g, device=DEV) * 40 - 30)
    if R > 1:
        H[R // 2:] = torch.randn((R - R // 2, 2 * I), generator=g, device=DEV)
        H[-1] = 0.0
    H[0, :8] = torch.tensor([448.0, 224.0, 17.0, -17.0, 19.0, 0.5, -0.001, 0.0], device=DEV)
    H[0, I:I + 4] = torch.tensor([1.7578125, 1.75, 1.0, -0.25], device=DEV)
    return H.to(dtype)


test_matrix.__test__ = False

SIZES = [(1, 1, 1, 8), (5, 1, 2, 24), (7, 3, 9, 40), (33, 2, 4, 64), (64, 8, 16, 136), (3, 2, 5, 520), (2, 1, 2, 2056)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,I", SIZES)
def test_save8_rows(T, k, E, I, dtype):
    R = T * k
    r = routing(T, k, E)
    H = test_matrix(R, I, DT[dtype])
    for limit in (0.0, 0.5):
        aw, codes, scales = B.swiglu_save8(H, r, T, k, swiglu_limit=limit)
        v, s = encode64(H)
        assert torch.equal(scales, s)
        assert torch.equal(codes.view(torch.float8_e4m3fn).double(), v)
        g, u = H.double()[:, :I], H.double()[:, I:]
        gc, uc, sg = act64(g, u, limit)
        ref = row_weight(r) * gc * sg * uc
        # float32's sigmoid is 0 where the true one lies below 2^-126: exp(-g)
        # overflows from g = -88.73 on (2^-128 there), and the reciprocal of a
        # number above 2^126 is flushed; that is at most 2^-126 of |w g u|
        flush = 2.0 ** -126 * (row_weight(r) * gc * uc).abs()
        tol = ((16 + 2 * gc.abs()) * 2.0 ** -23 + STEP[DT[dtype]]) * ref.abs() + flush + 1e-37
        err = (aw.double() - ref).abs()
        worst = int((err / tol).argmax())
        assert bool((err <= tol).all()), [float(t.reshape(-1)[worst]) for t in (aw, ref, tol, gc, uc)]
        only = B.swiglu_save8(H, None, T, k, swiglu_limit=limit)
        assert only[0] is None and torch.equal(only[1], codes) and torch.equal(only[2], scales)


# widths on both sides of those where a wave takes one, two, four or eight rows,
# with a last group of rows that is not full
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("I", [16, 64, 72, 128, 136, 256, 264])
def test_rows_of_a_wave(I, dtype):
    test_save8_rows(37, 1, 3, I, dtype)
    test_backward8_rows(37, 1, 3, I, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_past_the_cache(dtype):
    """More than 256 MiB written (non-temporal stores): the same results, bit
    for bit, as the same rows in pieces below that."""
    k, I, dt = 1, 1000, DT[dtype]
    T = 150000 if dtype == "bf16" else 70000
    r = routing(T, k, 2)
    H = torch.randn((T, 2 * I), generator=gen(12), device=DEV).to(dt)
    G = torch.randn((T, I), generator=gen(13), device=DEV).to(dt)
    aw, codes, scales = B.swiglu_save8(H, r, T, k)
    back = B.swiglu_backward8(G, codes, scales, r, T, k)
    w = r.topk_w.view(-1)[r.src_of.long()]
    for lo in range(0, T, T // 10):
        s = slice(lo, lo + T // 10)
        n = T // 10
        part = B.Routing(r.topk_ids[s], w[s].view(n, 1).contiguous(), r.counts, r.offsets, r.row_of[:n],
                         torch.arange(n, dtype=torch.int32, device=DEV))
        p = B.swiglu_save8(H[s], part, n, k)
        assert all(torch.equal(a[s], b) for a, b in zip((aw, codes, scales), p))
        assert all(torch.equal(a[s], b) for a, b in zip(back, B.swiglu_backward8(G[s], *p[1:], part, n, k)))


def test_save8_codes_are_the_mxfp8_row_encoding():
    T, k, I = 40, 2, 128
    H = test_matrix(T * k, I, torch.bfloat16, seed=3)
    _, codes, scales = B.swiglu_save8(H, None, T, k)
    q, s = B.quantize_mxfp8(H)
    assert torch.equal(codes, q) and torch.equal(scales, s)


def test_non_finite_blocks_decode_to_nan():
    T, k, I = 4, 1, 72
    r = routing(T, k, 2)
    H = torch.randn((T, 2 * I), generator=gen(1), device=DEV).bfloat16()
    H[0, 33] = float("inf")          # gate block 1
    H[1, I + 70] = float("nan")      # up block 2 (short)
    H[2, 3] = -float("inf")          # gate block 0
    aw, codes, scales = B.swiglu_save8(H, r, T, k)
    want = torch.zeros(T, 6, dtype=torch.bool, device=DEV)
    want[0, 1] = want[1, 5] = want[2, 0] = True
    assert torch.equal(scales == 255, want)
    G = torch.ones((T, I), device=DEV).bfloat16()
    dh, aw8, dw = B.swiglu_backward8(G, codes, scales, r, T, k)
    bad = torch.zeros(T, I, dtype=torch.bool, device=DEV)
    bad[0, 32:64] = True
    bad[1, 64:] = True
    bad[2, :32] = True
    assert torch.equal(aw8.isnan(), bad)
    assert torch.equal(dh.isnan()[:, :I], bad) and bool(dh.isnan()[2, I:I + 32].all())
    assert torch.equal(dw.isnan(), bad.any(1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,E,I", SIZES)
def test_backward8_rows(T, k, E, I, dtype):
    R, dt = T * k, DT[dtype]
    r = routing(T, k, E)
    H = torch.randn((R, 2 * I), generator=gen(5), device=DEV).to(dt)
    _, codes, scales = B.swiglu_save8(H, None, T, k)
    G = torch.randn((R, I), generator=gen(6), device=DEV).to(dt)
    w = row_weight(r)
    for limit in (0.0, 0.5):
        dh, aw, dw = B.swiglu_backward8(G, codes, scales, r, T, k, swiglu_limit=limit)
        lim = limit if limit > 0 else math.inf
        g, u = decode64(codes, scales)
        gc, uc, s = act64(g, u, limit)
        G64 = G.double()
        a = gc * s * uc
        dg = torch.where(g <= lim, w * G64 * uc * s * (1 + gc * (1 - s)), 0.0)
        du = torch.where(u.abs() <= lim, w * G64 * gc * s, 0.0)
        f = (16 + 2 * gc.abs()) * 2.0 ** -23
        assert bool(((aw.double() - w * a).abs() <= (f + STEP[dt]) * (w * a).abs() + 1e-37).all())
        # dg: 1 + g (1 - s) may cancel, so count its terms' magnitudes
        mag = w.abs() * G64.abs() * uc.abs() * s * (1 + gc.abs() * (1 - s) + gc.abs())
        assert bool(((dh[:, :I].double() - dg).abs() <= f * mag + STEP[dt] * dg.abs() + 1e-37).all())
        assert bool(((dh[:, I:].double() - du).abs() <= (f + STEP[dt]) * du.abs() + 1e-37).all())
        terms = (G64 * a).abs()
        assert bool(((dw.double() - (G64 * a).sum(1)).abs() <= (f * terms).sum(1) + (I + 64) * 2.0 ** -24 * terms.sum(1)
                     + 1e-37).all())


def layer_inputs(T, d, E, k, I, dtype, seed=0):
    g = gen(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    return ((rn(T, d)).to(dtype), rn(T, E), (rn(E, 2 * I, d) * d ** -0.5).to(dtype),
            (rn(E, d, I) * I ** -0.5).to(dtype), rn(T, d).to(dtype))


def layer_backward64(x, wgu, wd, dout, r, g, u, k, limit, step):
    """Gradients from the decoded g, u (rows in expert order), and their error
    bounds, in float64."""
    x, wgu, wd, dout = (t.double() for t in (x, wgu, wd, dout))
    E, two_i, d = wgu.shape
    I = two_i // 2
    lim = limit if limit > 0 else math.inf
    gc, uc, s = act64(g, u, limit)
    a = gc * s * uc
    w = row_weight(r)
    tok = (r.src_of.long() // k)
    off = r.offsets.tolist()
    R = a.shape[0]
    T = x.shape[0]
    ref = dict(dx=torch.zeros_like(x), dwgu=torch.zeros_like(wgu), dwd=torch.zeros_like(wd),
               dw=torch.zeros(R, dtype=torch.float64, device=DEV))
    tol = {n: torch.zeros_like(v) for n, v in ref.items()}
    slack = (d + 2 * I + R + 64) * 2.0 ** -23
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        t = tok[rows]
        G, Gm = dout[t] @ wd[e], dout[t].abs() @ wd[e].abs()
        dA = w[rows] * G
        sl = s[rows] * (1 + gc[rows] * (1 - s[rows]))
        dh = torch.cat([torch.where(g[rows] <= lim, dA * uc[rows] * sl, 0.0),
                        torch.where(u[rows].abs() <= lim, dA * (gc * s)[rows], 0.0)], 1)
        ga = torch.cat([(w[rows] * uc[rows] * sl).abs(), (w[rows] * (gc * s)[rows]).abs()], 1)
        ddh = 3 * step * dh.abs() + slack * ga * torch.cat([Gm, Gm], 1)   # dh's own error
        aw = w[rows] * a[rows]
        ref["dw"][rows] = (G * a[rows]).sum(1)
        tol["dw"][rows] = (2 * step * (G * a[rows]).abs() + slack * Gm * a[rows].abs()).sum(1)
        ref["dwd"][e] = dout[t].t() @ aw
        tol["dwd"][e] = (2 * step + slack) * (dout[t].abs().t() @ aw.abs())
        ref["dwgu"][e] = dh.t() @ x[t]
        tol["dwgu"][e] = (ddh + slack * dh.abs()).t() @ x[t].abs()
        # each row's product is rounded to the storage type before the reduction
        ref["dx"].index_add_(0, t, dh @ wgu[e])
        tol["dx"].index_add_(0, t, (ddh + slack * dh.abs()) @ wgu[e].abs() + step * (dh @ wgu[e]).abs())
    for n in ("dx", "dwgu", "dwd"):
        tol[n] += step * ref[n].abs() + 1e-30
    tol["dw"] += 1e-30
    return ref, tol


@pytest.mark.parametrize("T,d,E,k,I,dtype,limit", [
    (1, 8, 1, 1, 8, "bf16", 0.0), (37, 72, 5, 2, 40, "bf16", 0.0), (130, 256, 4, 3, 128, "bf16", 0.6),
    (300, 136, 3, 1, 264, "bf16", 0.0), (1, 16, 2, 1, 8, "f32", 0.0), (61, 64, 6, 2, 72, "f32", 0.6)])
def test_layer(T, d, E, k, I, dtype, limit):
    dt = DT[dtype]
    x, lg, wgu, wd, dout = layer_inputs(T, d, E, k, I, dt)
    plain = B.MoeLayer(T, d, E, k, I, dtype=dt, logits_dtype=torch.float32, device=DEV, swiglu_limit=limit)
    want = plain.forward(x, wgu, wd, logits=lg)
    layer = B.MoeLayer(T, d, E, k, I, dtype=dt, logits_dtype=torch.float32, device=DEV, swiglu_limit=limit,
                       save8=True)
    layer.saved.fill_(171)
    got = layer.forward(x, wgu, wd, logits=lg)
    assert torch.equal(got, want)
    assert layer.saved.numel() * 2.5 < plain.saved.numel() + 2048
    codes, scales = layer.saved_views()
    _, c, s = B.swiglu_save8(plain.saved_views()[0].contiguous(), None, T, k)   # the H the plain layer keeps
    assert torch.equal(codes, c) and torch.equal(scales, s)
    layer.ws_bwd.fill_(255)
    grads = layer.backward(dout, x, wgu, wd)
    g, u = decode64(codes, scales)
    r = layer.routing
    ref, tol = layer_backward64(x, wgu, wd, dout, r, g, u, k, limit, STEP[dt])
    for n, m in (("dx", "dx"), ("dW_gate_up", "dwgu"), ("dW_down", "dwd")):
        err = (grads[n].double() - ref[m]).abs()
        assert bool((err <= tol[m]).all()), (n, float((err / tol[m]).max()))
    dw = ref["dw"][r.row_of.long()].view(T, k)
    dw_tol = tol["dw"][r.row_of.long()].view(T, k)
    assert bool(((grads["d_topk_w"].double() - dw).abs() <= dw_tol).all())
    w = r.topk_w.double()
    inner = (w * dw).sum(1, keepdim=True)
    dl = torch.zeros((T, E), dtype=torch.float64, device=DEV).scatter_(1, r.topk_ids.long(), w * (dw - inner))
    lt = torch.zeros((T, E), dtype=torch.float64, device=DEV).scatter_(
        1, r.topk_ids.long(), w * (dw_tol + (w * dw_tol).sum(1, keepdim=True)) * 1.01
        + 2.0 ** -20 * w * (dw.abs() + (w * dw).abs().sum(1, keepdim=True)))
    assert bool(((grads["dlogits"].double() - dl).abs() <= lt + 1e-30).all())


def test_ids_form():
    T, d, E, k, I = 50, 64, 4, 2, 32
    x, _, wgu, wd, dout = layer_inputs(T, d, E, k, I, torch.bfloat16)
    r = routing(T, k, E)
    a = B.MoeLayer(T, d, E, k, I, device=DEV)
    b = B.MoeLayer(T, d, E, k, I, device=DEV, save8=True)
    assert torch.equal(a.forward(x, wgu, wd, topk_ids=r.topk_ids, topk_w=r.topk_w),
                       b.forward(x, wgu, wd, topk_ids=r.topk_ids, topk_w=r.topk_w))
    g = b.backward(dout, x, wgu, wd)
    assert "dlogits" not in g and all(bool(v.isfinite().all()) for v in g.values())


def test_autograd_equals_the_layer_object():
    from combine_top_route_amd.autograd import moe_layer
    T, d, E, k, I = 70, 128, 4, 2, 64
    x, lg, wgu, wd, dout = layer_inputs(T, d, E, k, I, torch.bfloat16)
    layer = B.MoeLayer(T, d, E, k, I, logits_dtype=torch.float32, device=DEV, save8=True)
    out = layer.forward(x, wgu, wd, logits=lg)
    g = layer.backward(dout, x, wgu, wd)
    leaves = [t.clone().requires_grad_() for t in (x, lg, wgu, wd)]
    y = moe_layer(*leaves, k, save8=True)
    y.backward(dout)
    assert torch.equal(y, out)
    for t, n in zip(leaves, ("dx", "dlogits", "dW_gate_up", "dW_down")):
        assert torch.equal(t.grad, g[n]), n


def test_finite_differences_through_the_exact_part():
    """On H that 8 bits hold exactly, the row pass's dH is the derivative of
    sum(G w silu(g) u): central differences in float64."""
    T, k, I = 6, 1, 32
    r = routing(T, k, 2)
    vals = torch.tensor([-2.0, -1.0, -0.5, 0.25, 1.0, 1.5, 2.0, 3.0], device=DEV)
    H = vals[torch.randint(0, 8, (T, 2 * I), generator=gen(9), device=DEV)]
    _, codes, scales = B.swiglu_save8(H, None, T, k)
    g, u = decode64(codes, scales)
    assert torch.equal(torch.cat([g, u], 1), H.double())
    G = torch.randn((T, I), generator=gen(10), device=DEV)
    dh, aw, dw = B.swiglu_backward8(G, codes, scales, r, T, k)
    w = row_weight(r)
    f = lambda g, u: G.double() * w * g * torch.sigmoid(g) * u
    h = 1e-5
    ng = (f(g + h, u) - f(g - h, u)) / (2 * h)
    nu = (f(g, u + h) - f(g, u - h)) / (2 * h)
    # differences: h^2/6 times the third derivative (below 1 per factor) and 1e-16/h of rounding
    assert bool(((dh.double() - torch.cat([ng, nu], 1)).abs() <= 1e-5 * (1 + torch.cat([ng, nu], 1).abs())).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed(dtype):
    T, d, E, k, I = 90, 64, 4, 2, 40
    dt = DT[dtype]
    x, lg, wgu, wd, dout = layer_inputs(T, d, E, k, I, dt)
    layer = B.MoeLayer(T, d, E, k, I, dtype=dt, logits_dtype=torch.float32, device=DEV, save8=True)
    eager = B.MoeLayer(T, d, E, k, I, dtype=dt, logits_dtype=torch.float32, device=DEV, save8=True)
    layer.forward(x, wgu, wd, logits=lg)
    layer.backward(dout, x, wgu, wd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.forward(x, wgu, wd, logits=lg)
        g = layer.backward(dout, x, wgu, wd)
    for i in range(4):
        for t, n in zip((x, lg, wgu, wd, dout), layer_inputs(T, d, E, k, I, dt, seed=20 + i)):
            t.copy_(n)
        graph.replay()
        want = eager.forward(x, wgu, wd, logits=lg)
        wg = eager.backward(dout, x, wgu, wd)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        for n in wg:
            assert torch.equal(g[n], wg[n]), n
