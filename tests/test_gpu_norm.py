"""The norms around a block, with its gate and residual scale, and their
gradients, against the formulas in 64 bits.

Bounds.  The kernels compute in float32: every value is a few products and sums
of terms whose magnitudes add up to `mag`, and a sum over a row or over tokens
runs over at most SEQ terms in one accumulator before tree-like joins, so its
rounding is below (SEQ + a few) 2^-24 of the terms' magnitudes.  SEQ: 32 columns
a lane and 16 waves in a row; 32 (work-groups a slice) + 32 (slices) + 32 (rows of
lanes) + rows a work-group over tokens.  Results are then rounded once, by at
most half a step of their type."""
import math

import pytest
import torch

from combine_top_route_amd import autograd as A
from combine_top_route_amd import binding as B

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6
U = 2.0 ** -24

# block, post, gate, after, scale
FORMS = {"pre": (False, False, None, True, 1.0), "all": (True, True, "channel", True, 0.7),
         "token": (True, True, "token", True, -1.3), "plain": (True, False, None, True, 1.0),
         "last": (True, True, None, False, 0.0), "gate": (True, False, "token", False, 1.0),
         "scale": (True, False, "channel", True, 2.0)}
# one row to several a work-group; a row in 8 lanes to 16 waves; one piece a lane
# to four; several rows a work-group takes in turn
SIZES = [(1, 8), (1, 2048), (3, 64), (5, 200), (37, 520), (130, 1000), (33, 2056), (9, 4096), (2, 8200), (3, 16384),
         (700, 136), (2049, 72), (2100, 1024), (2051, 2048), (2100, 4104), (2048, 8200), (2050, 16384),
         (600, 2304), (1100, 2880), (700, 1032), (513, 528)]


def inputs(T, d, dtype, form, seed=0):
    block, post, gate, after, scale = FORMS[form]
    g = torch.Generator(device="cuda").manual_seed(seed + T * 7 + d)
    dt = DT[dtype]
    r = lambda shape, std=1.0, mean=0.0: (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dt)
    t = {"x": r((T, d), 2.0), "y": r((T, d), 0.5) if block else None, "w_post": r(d, 0.2, 1.0) if post else None,
         "w_next": r(d, 0.2, 1.0) if after else None, "gate": None, "dz": r((T, d)), "dh": r((T, d)) if after else None}
    if gate:
        t["gate"] = r(d if gate == "channel" else (T, 1), 0.5, 0.5)
    return t, scale


def d64(t):
    return None if t is None else t.double()


def rms(v):
    return v.square().mean(1, keepdim=True).sqrt()


def rstd(v):
    return 1.0 / (v.square().mean(1, keepdim=True) + EPS).sqrt()


def near(got, ref, mag, seq):
    assert got.shape == ref.shape
    half = torch.finfo(got.dtype).eps / 2
    err = (got.double() - ref).abs()
    tol = (seq + 16) * U * mag + half * ref.abs() * (1 + 2.0 ** -6) + 2.0 ** -126
    worst = ((err - tol) / tol).max().item()
    assert worst <= 0, f"off by {worst + 1:.3g} of the bound"


def forward_ref(t, scale):
    x, y, wp, g, wn = (d64(t[n]) for n in ("x", "y", "w_post", "gate", "w_next"))
    z, mag = x, x.abs()
    if y is not None:
        b = y if wp is None else y * rstd(y) * wp
        b = b if g is None else b * g
        z, mag = scale * x + b, abs(scale) * x.abs() + b.abs()
    if wn is None:
        return z, mag, None, None
    h = z * rstd(z) * wn
    # z's error reaches h by itself and through the row's root mean square
    hmag = mag * rstd(z) * wn.abs() + h.abs() * (1 + rms(mag) * rstd(z))
    return z, mag, h, hmag


def backward_ref(t, z, scale, use_dz=True, use_dh=True):
    """The formulas of the gradients and the magnitudes of their terms."""
    y, wp, g, wn, dz, dh = (d64(t[n]) for n in ("y", "w_post", "gate", "w_next", "dz", "dh"))
    z, out = z.double(), {}
    G = dz if use_dz else torch.zeros_like(z)
    m = G.abs()
    if wn is not None and use_dh:
        rz = rstd(z)
        zh, s = z * rz, dh * wn
        G = G + rz * (s - zh * (s * zh).mean(1, keepdim=True))
        m = m + rz * (s.abs() + zh.abs() * (s * zh).abs().mean(1, keepdim=True))
        out["dw_next"] = (dh * zh).sum(0), (dh * zh).abs().sum(0)
    out["dx"] = scale * G, abs(scale) * m
    if y is None:
        return out
    u = y if wp is None else y * rstd(y)
    w = 1.0 if wp is None else wp
    gt = 1.0 if g is None else g
    s, sm = G * gt * w, m * abs(gt) * abs(w)
    if wp is None:
        out["dy"] = s, sm
    else:
        ry = rstd(y)
        out["dy"] = (ry * (s - u * (s * u).mean(1, keepdim=True)),
                     ry * (sm + u.abs() * (sm * u.abs()).mean(1, keepdim=True)))
        out["dw_post"] = (G * gt * u).sum(0), (m * abs(gt) * u.abs()).sum(0)
    if g is not None:
        k = 0 if g.dim() == 1 else 1
        f = lambda v: v.sum(k) if k == 0 else v.sum(k, keepdim=True)
        out["dgate"] = f(G * u * w), f(m * u.abs() * abs(w))
    return out


def args(t, scale):
    return dict(w_post=t["w_post"], gate=t["gate"], res_scale=scale, w_next=t["w_next"], eps=EPS)


def check(T, d, dtype, form):
    t, scale = inputs(T, d, dtype, form)
    z, h = B.norm_residual(t["x"], t["y"], **args(t, scale))
    zr, zm, hr, hm = forward_ref(t, scale)
    if t["y"] is None:
        assert z is t["x"]
    else:
        near(z, zr, zm, 48)
    if h is None:
        assert t["w_next"] is None
    else:
        near(h, hr, hm, 48)
    grads = B.norm_residual_backward(t["dz"], t["dh"], z, t["y"], **args(t, scale))
    ref = backward_ref(t, z, scale)
    assert {n for n, v in grads.items() if v is not None} == set(ref)
    for n, (r, m) in ref.items():
        assert grads[n].dtype == z.dtype
        # a gradient's terms carry the row sums' rounding on top of their own
        near(grads[n], r, m, 48 if n in ("dx", "dy") else 48 + 128 + T / 256)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SIZES)
def test_all(T, d, dtype):
    check(T, d, dtype, "all")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", [f for f in FORMS if f != "all"])
@pytest.mark.parametrize("T,d", [(1, 72), (33, 1000), (2500, 2048)])
def test_forms(T, d, form, dtype):
    check(T, d, dtype, form)


@pytest.mark.parametrize("form", ["all", "token"])
@pytest.mark.parametrize("use_dz,use_dh", [(True, False), (False, True)])
def test_one_gradient_only(form, use_dz, use_dh):
    t, scale = inputs(70, 264, "f32", form)
    z, _ = B.norm_residual(t["x"], t["y"], **args(t, scale))
    a = args(t, scale)
    if not use_dh:
        a["w_next"] = None
    got = B.norm_residual_backward(t["dz"] if use_dz else None, t["dh"] if use_dh else None, z, t["y"], **a)
    ref = backward_ref(t, z, scale, use_dz, use_dh)
    for n, (r, m) in ref.items():
        near(got[n], r, m, 200)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_odd_values(dtype):
    """Zero rows, rows with an infinity or a NaN, tiny and huge rows: the others
    keep their values bit for bit."""
    t, scale = inputs(40, 328, dtype, "all")
    z0, h0 = B.norm_residual(t["x"], t["y"], **args(t, scale))
    x, y = t["x"].clone(), t["y"].clone()
    x[3], y[3] = 0, 0
    x[5, 7] = math.inf
    y[8, 300] = math.nan
    y[11, 0] = -math.inf
    x[13], y[13] = x[13] * 1e-30, y[13] * 1e-30
    x[17], y[17] = x[17] * 1e15, y[17] * 1e15
    z, h = B.norm_residual(x, y, **args(t, scale))
    odd = [3, 5, 8, 11, 13, 17]
    rest = [i for i in range(40) if i not in odd]
    assert torch.equal(z[rest], z0[rest]) and torch.equal(h[rest], h0[rest])
    assert bool((z[3] == 0).all()) and bool((h[3] == 0).all())
    assert math.isinf(z[5, 7]) and bool(z[5].isfinite().sum() == 327) and math.isnan(h[5, 7])
    assert bool(z[8].isnan().all()) and bool(h[8].isnan().all())
    assert math.isnan(z[11, 0])
    t2 = dict(t, x=x, y=y)
    zr, zm, hr, hm = forward_ref(t2, scale)
    for r in (13, 17):
        near(z[r:r + 1], zr[r:r + 1], zm[r:r + 1], 48)
        near(h[r:r + 1], hr[r:r + 1], hm[r:r + 1], 48)
    grads = B.norm_residual_backward(t["dz"], t["dh"], z, y, **args(t, scale))
    g0 = B.norm_residual_backward(t["dz"], t["dh"], z0, t["y"], **args(t, scale))
    assert torch.equal(grads["dx"][rest], g0["dx"][rest]) and torch.equal(grads["dy"][rest], g0["dy"][rest])
    assert bool(grads["dx"][3].isfinite().all()) and bool(grads["dy"][3].isfinite().all())


def test_rows_behind_and_in_place():
    """Only T rows are written; z over x and dx over dz give the same."""
    import ctypes
    t, scale = inputs(37, 520, "bf16", "all")
    z0, h0 = B.norm_residual(t["x"], t["y"], **args(t, scale))
    g0 = B.norm_residual_backward(t["dz"], t["dh"], z0, t["y"], **args(t, scale))
    pad = lambda v: torch.cat([v, torch.full((3, 520), 7.0, dtype=v.dtype, device="cuda")])
    x, h, dz, dy = pad(t["x"]), pad(torch.zeros_like(h0)), pad(t["dz"]), pad(torch.zeros_like(h0))
    sh = B.MoeNormShape(37, 520, 1, B.GATE_CHANNEL, scale, EPS)
    p, stream = B._ptr, torch.cuda.current_stream().cuda_stream
    assert B.lib().moe_norm_forward(ctypes.byref(sh), p(x), p(t["y"]), p(t["w_post"]), p(t["gate"]), p(t["w_next"]),
                                    p(x), p(h), stream) == 0
    ws = torch.empty(B.norm_workspace_size(sh), dtype=torch.uint8, device="cuda")
    dw = [torch.empty_like(t["gate"]) for _ in range(3)]
    assert B.lib().moe_norm_backward(ctypes.byref(sh), p(dz), p(t["dh"]), p(x), p(t["y"]), p(t["w_post"]),
                                     p(t["gate"]), p(t["w_next"]), p(dz), p(dy), *map(p, dw), p(ws), ws.numel(),
                                     stream) == 0
    for got, ref in ((x, z0), (h, h0), (dz, g0["dx"]), (dy, g0["dy"])):
        assert torch.equal(got[:37], ref) and bool((got[37:] == 7).all())
    for got, n in zip(dw, ("dw_post", "dgate", "dw_next")):
        assert torch.equal(got, g0[n])


def test_same_every_time_and_on_a_stream():
    t, scale = inputs(3000, 1032, "bf16", "all")
    z, h = B.norm_residual(t["x"], t["y"], **args(t, scale))
    g = B.norm_residual_backward(t["dz"], t["dh"], z, t["y"], **args(t, scale))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        z2, h2 = B.norm_residual(t["x"], t["y"], **args(t, scale))
        g2 = B.norm_residual_backward(t["dz"], t["dh"], z2, t["y"], **args(t, scale))
    side.synchronize()
    assert torch.equal(z, z2) and torch.equal(h, h2)
    for n in g:
        assert torch.equal(g[n], g2[n])


def test_graph():
    t, scale = inputs(2100, 1024, "bf16", "all")
    step = lambda: (lambda z, h: (z, h, *B.norm_residual_backward(t["dz"], t["dh"], z, t["y"], **args(t, scale))
                                  .values()))(*B.norm_residual(t["x"], t["y"], **args(t, scale)))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        t["x"].mul_(1.25)
        t["dz"].add_(0.5)
        want = step()
        for o in out:
            o.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


# ------------------------------------------------------------------ autograd
def leaves(t):
    return {n: v.detach().clone().requires_grad_() for n, v in t.items() if v is not None and not n.startswith("d")}


@pytest.mark.parametrize("form", list(FORMS))
def test_autograd(form):
    t, scale = inputs(33, 264, "f32", form)
    p = leaves(t)
    q = {n: v.detach().double().requires_grad_() for n, v in p.items()}
    z, h = A.norm_residual(p["x"], p.get("y"), p.get("w_post"), p.get("gate"), scale, p.get("w_next"), EPS)
    loss = (z * t["dz"]).sum() + (0 if h is None else (h * t["dh"]).sum())
    loss.backward()
    zq = q["x"]
    if "y" in q:
        b = q["y"] if "w_post" not in q else q["y"] * rstd(q["y"]) * q["w_post"]
        zq = scale * q["x"] + (b * q["gate"] if "gate" in q else b)
    want = (zq * t["dz"].double()).sum()
    if h is not None:
        want = want + (zq * rstd(zq) * q["w_next"] * t["dh"].double()).sum()
    want.backward()
    for n in p:
        ref = q[n].grad
        assert p[n].grad is not None, n
        # the kernel's z is rounded to float32, which moves the gradient by about as much
        err = (p[n].grad.double() - ref).abs().max().item()
        assert err <= 2.0 ** -16 * ref.abs().max().item() + 1e-12, (n, err)


def test_autograd_unused_outputs():
    t, scale = inputs(20, 136, "f32", "all")
    for use in ("z", "h"):
        p = leaves(t)
        z, h = A.norm_residual(p["x"], p["y"], p["w_post"], p["gate"], scale, p["w_next"], EPS)
        ((z * t["dz"]) if use == "z" else (h * t["dh"])).sum().backward()
        a = args(t, scale)
        if use == "z":
            a["w_next"] = None
            assert p["w_next"].grad is None
        want = B.norm_residual_backward(t["dz"] if use == "z" else None, t["dh"] if use == "h" else None, z.detach(),
                                        t["y"], **a)
        for n, g in (("x", "dx"), ("y", "dy"), ("w_post", "dw_post"), ("gate", "dgate")):
            assert torch.equal(p[n].grad, want[g]), (use, n)
    # a gradient that is a broadcast scalar, and a slice that starts anywhere
    p = leaves(t)
    z, h = A.norm_residual(p["x"], p["y"], p["w_post"], p["gate"], scale, p["w_next"], EPS)
    torch.cat([z.flatten()[1:], h.flatten()]).sum().backward()
    one = torch.ones_like(z)
    first = one.clone()
    first[0, 0] = 0
    want = B.norm_residual_backward(first, one, z.detach(), t["y"], **args(t, scale))
    assert torch.equal(p["x"].grad, want["dx"]) and torch.equal(p["gate"].grad, want["dgate"])


def test_differences():
    """Gradients against central differences of the forward, in float32 along one
    direction: the third-order rest is h^2 of it, the roundings 2^-24 / h."""
    t, scale = inputs(6, 64, "f32", "token")
    z, h = B.norm_residual(t["x"], t["y"], **args(t, scale))
    grads = B.norm_residual_backward(t["dz"], t["dh"], z, t["y"], **args(t, scale))
    loss = lambda v: sum((a.double() * b.double()).sum().item() for a, b in
                         zip(B.norm_residual(v["x"], v["y"], **args(v, scale)), (t["dz"], t["dh"])))
    step = 2.0 ** -6
    for n, g in (("x", "dx"), ("y", "dy"), ("w_post", "dw_post"), ("gate", "dgate"), ("w_next", "dw_next")):
        way = torch.randn(t[n].shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
        up, down = dict(t), dict(t)
        up[n], down[n] = t[n] + step * way, t[n] - step * way
        got = (grads[g].double() * way.double()).sum().item()
        diff = (loss(up) - loss(down)) / (2 * step)
        size = grads[g].double().norm().item() * way.double().norm().item()
        assert abs(got - diff) <= 4 * step ** 2 * size, (n, got, diff)


@pytest.mark.parametrize("save8", [False, True])
def test_block(save8):
    """A block as it is used: norm, router, experts, gate, norm, residual, next
    norm, against the same pieces one by one."""
    T, d, E, k, I = 96, 256, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(torch.bfloat16).requires_grad_()
    p = dict(x=r(T, d), w_router=r(E, d, std=0.06), w_gate_up=r(E, 2 * I, d, std=0.06), w_down=r(E, d, I, std=0.09),
             w_pre=r(d), w_post=r(d), gate=r(d), w_next=r(d))
    z, h = A.moe_residual_block(**p, k=k, res_scale=0.5, save8=save8)
    dz, dh = torch.randn_like(z), torch.randn_like(h)
    torch.autograd.backward((z, h), (dz, dh))
    q = {n: v.detach() for n, v in p.items()}
    _, h0 = B.norm_residual(q["x"], w_next=q["w_pre"])
    leaf = {n: q[n].clone().requires_grad_() for n in ("w_router", "w_gate_up", "w_down")}
    h0 = h0.requires_grad_()
    y = A.moe_block(h0, leaf["w_router"], leaf["w_gate_up"], leaf["w_down"], k, save8=save8)
    rest = dict(w_post=q["w_post"], gate=q["gate"], res_scale=0.5, w_next=q["w_next"])
    z1, h1 = B.norm_residual(q["x"], y.detach(), **rest)
    assert torch.equal(z, z1) and torch.equal(h, h1)
    g1 = B.norm_residual_backward(dz, dh, z1, y.detach(), **rest)
    y.backward(g1["dy"])
    g0 = B.norm_residual_backward(g1["dx"], h0.grad, q["x"], w_next=q["w_pre"])
    for n, want in (("x", g0["dx"]), ("w_pre", g0["dw_next"]), ("w_post", g1["dw_post"]), ("gate", g1["dgate"]),
                    ("w_next", g1["dw_next"]), *((n, leaf[n].grad) for n in leaf)):
        assert torch.equal(p[n].grad, want), n
    with torch.no_grad():  # the next block takes h as it is
        a = A.moe_residual_block(z, *(q[n] for n in ("w_router", "w_gate_up", "w_down")), k, h=h)
        b = z + A.moe_block(h, *(q[n] for n in ("w_router", "w_gate_up", "w_down")), k)
    assert a[1] is None
    near(a[0], (z.double() + (A.moe_block(h, *(q[n] for n in ("w_router", "w_gate_up", "w_down")), k)).double()),
         z.double().abs() + 8, 4)
    assert b.shape == a[0].shape


def test_captured_step_beside_a_live_eager_graph():
    """A whole block's forward and backward in a graph, on leaves of its own, while
    an eager graph of the same weights lives; every replay against eager."""
    T, d, E, k, I = 96, 256, 8, 2, 128
    names = ("x", "w_router", "w_gate_up", "w_down", "w_pre", "w_post", "gate", "w_next")
    shapes = ((T, d), (E, d), (E, 2 * I, d), (E, d, I), (d,), (d,), (T, 1), (d,))

    def fresh(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda s: (torch.randn(s, generator=g, device="cuda") * (0.1 if len(s) == 3 else 1)).to(torch.bfloat16)
        return [r(s) for s in shapes], [r((T, d)), r((T, d))]

    def step(p):
        z, h = A.moe_residual_block(**dict(zip(names, p)), k=k, res_scale=0.5)
        return [z, h, *torch.autograd.grad((z, h), p, douts)]

    data, douts = fresh(1)
    own = lambda: [t.detach().requires_grad_() for t in data]
    live = A.moe_residual_block(**dict(zip(names, own())), k=k)  # kept until the end
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(own())
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    leaf = own()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(leaf)
    for i in range(3):
        for t, f in zip([*data, *douts], sum(fresh(20 + i), [])):
            t.copy_(f)
        graph.replay()
        want = step(own())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
    assert live[0].shape == (T, d)


def test_compiled():
    T, d = 64, 128
    x, y, w = (torch.randn(s, device="cuda", requires_grad=True) for s in ((T, d), (T, d), (d,)))

    def f(x, y, w):
        z, h = A.norm_residual(x, y, w_post=w, res_scale=0.5, w_next=w)
        return (z * h).sum()

    f(x, y, w).backward()
    want = [t.grad.clone() for t in (x, y, w)]
    for t in (x, y, w):
        t.grad = None
    torch.compile(f, fullgraph=True, backend="aot_eager")(x, y, w).backward()
    for t, g in zip((x, y, w), want):
        assert (t.grad - g).abs().max().item() <= 2.0 ** -20 * g.abs().max().item()


def test_blocks_beyond_one_launch_dimension():
    """Two rows a work-group: more work-groups than one dimension of the grid takes."""
    T, d = (1 << 22) + 3, 2056
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GiB of free GPU memory")
    w = torch.randn(d, device="cuda").bfloat16()
    few = torch.randn((64, d), device="cuda").bfloat16()
    # 64 rows alone are spread over other lanes, whose sums differ in the last bits:
    # the bound is the formula's
    _, _, want, mag = forward_ref(dict(x=few, y=None, w_post=None, gate=None, w_next=w), 1.0)
    x = torch.zeros((T, d), dtype=torch.bfloat16, device="cuda")
    x[:32], x[-32:] = few[:32], few[32:]
    _, h = B.norm_residual(x, w_next=w)
    near(torch.cat((h[:32], h[-32:])), want, mag, 64)
    assert not any(bool(part.any()) for part in h[32:-32].split(1 << 20))
