"""The operators together: router, layer with the 8-bit checkpoint, their
backward, and then the trained weights served by the decoder."""
import pytest
import torch

from combine_top_route_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
T, d, E, k, I = 96, 128, 8, 2, 64


def tensors(dtype, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    return [t.to(dtype) for t in (rn(T, d), rn(E, d) * d ** -0.5, rn(E, 2 * I, d) * d ** -0.5,
                                  rn(E, d, I) * I ** -0.5)], rn(T, d).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("save8", [False, True])
def test_block_is_its_parts(dtype, save8):
    from combine_top_route_amd.autograd import moe_block, moe_layer, router
    leaves, dout = tensors(dtype)
    leaves = [t.requires_grad_() for t in leaves]
    out = moe_block(*leaves, k, save8=save8)
    grads = torch.autograd.grad(out, leaves, dout)
    # by hand: logits, layer, layer backward, router backward added to its dx
    x, wr, wgu, wd = (t.detach() for t in leaves)
    logits = B.router_logits(x, wr)
    layer = B.MoeLayer(T, d, E, k, I, dtype=dtype, logits_dtype=torch.float32, device=DEV, save8=save8)
    want = layer.forward(x, wgu, wd, logits=logits)
    g = layer.backward(dout, x, wgu, wd)
    dx, dwr = B.router_backward(g["dlogits"], x, wr, dx_in=g["dx"])
    assert torch.equal(out, want)
    for a, b in zip(grads, (dx, dwr, g["dW_gate_up"], g["dW_down"])):
        assert torch.equal(a, b)
    # the same through the separate functions: torch adds x's two gradients,
    # one rounding of the router's part (half a step of it) more
    out2 = moe_layer(leaves[0], router(leaves[0], leaves[1]), *leaves[2:], k, save8=save8)
    g2 = torch.autograd.grad(out2, leaves, dout)
    eps = torch.finfo(dtype).eps / 2
    part = B.router_backward(g["dlogits"], x, wr)[0].double().abs()
    assert bool(((g2[0].double() - dx.double()).abs() <= 1.01 * eps * (part + 2 * dx.double().abs()) + 1e-30).all())
    for a, b in zip(g2[1:], grads[1:]):
        assert torch.equal(a, b)


def test_gradients_against_differences():
    """Float32, the plain checkpoint: the directional derivative of the block
    against central differences of its own forward in float64 arithmetic."""
    from combine_top_route_amd.autograd import moe_block
    leaves, dout = tensors(torch.float32, seed=4)
    leaves = [t.requires_grad_() for t in leaves]
    grads = torch.autograd.grad(moe_block(*leaves, k), leaves, dout)

    def forward64(x, wr, wgu, wd):
        lg = x @ wr.T
        v, ids = lg.topk(k, 1)
        w = torch.softmax(v, 1)
        out = torch.zeros_like(x)
        for j in range(k):
            h = torch.bmm(wgu[ids[:, j]], x[:, :, None])[:, :, 0]
            a = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
            out = out + w[:, j:j + 1] * torch.bmm(wd[ids[:, j]], a[:, :, None])[:, :, 0]
        return (out * dout.double()).sum(), ids

    base = [t.detach().double() for t in leaves]
    _, ids0 = forward64(*base)
    for i, (t, g) in enumerate(zip(base, grads)):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(30 + i)
        dirn = torch.randn(t.shape, generator=gen, device=DEV).double()
        h = 1e-7
        vals = []
        for s in (h, -h):
            moved = list(base)
            moved[i] = t + s * dirn
            f, ids = forward64(*moved)
            assert torch.equal(ids, ids0)      # the direction crosses no change of experts
            vals.append(f)
        num = float((vals[0] - vals[1]) / (2 * h))
        ana = float((g.double() * dirn).sum())
        mag = float((g.double() * dirn).abs().sum())
        # rounding of the differences 2^-52 |f| / h, float32 gradients within
        # (d + I + T) 2^-23 of the magnitudes that make them
        assert abs(num - ana) <= (d + I + T) * 2.0 ** -20 * mag + 1e-6 * abs(float(vals[0]) + 1), i


def test_train_steps_then_decode():
    """A few steps with 8-bit checkpoints run and move the weights; the decoder
    on the result agrees with the layer's forward on a few tokens."""
    from combine_top_route_amd.autograd import moe_block
    leaves, target = tensors(torch.bfloat16, seed=7)
    x, ws = leaves[0], [t.requires_grad_() for t in leaves[1:]]
    for _ in range(3):
        out = moe_block(x, *ws, k, save8=True)
        grads = torch.autograd.grad(((out - target).float() ** 2).mean(), ws)
        assert all(bool(g.isfinite().all()) and bool(g.any()) for g in grads)
        with torch.no_grad():
            for w, g in zip(ws, grads):
                w -= 0.1 * g
    wr, wgu, wd = (w.detach() for w in ws)
    few = x[:9].contiguous()
    logits = B.router_logits(few, wr)
    dec = B.MoeDecoder(16, d, E, k, I, logits_dtype=torch.float32, device=DEV)
    got = dec.forward(few, wgu, wd, logits=logits)
    layer = B.MoeLayer(9, d, E, k, I, logits_dtype=torch.float32, device=DEV)
    want = layer.forward(few, wgu, wd, logits=logits)
    assert torch.equal(dec.topk_ids, layer.routing.topk_ids)
    # both round w silu(g) u to bf16 before the down product, then the layer
    # rounds each slot's product and both the sum: five half steps of the
    # sum of magnitudes cover the difference
    mag = torch.zeros_like(few, dtype=torch.float64)
    for t in range(9):
        for j in range(k):
            e = int(dec.topk_ids[t, j])
            h = wgu[e].double() @ few[t].double()
            a = float(dec.topk_w[t, j]) * torch.nn.functional.silu(h[:I]) * h[I:]
            mag[t] += wd[e].double().abs() @ a.abs()
    assert bool(((got.double() - want.double()).abs() <= 5 * 2.0 ** -8 * mag).all())


def test_compiled_block_traces():
    from combine_top_route_amd.autograd import moe_block
    leaves, dout = tensors(torch.bfloat16, seed=9)
    leaves = [t.requires_grad_() for t in leaves]
    want = torch.autograd.grad(moe_block(*leaves, k, save8=True), leaves, dout)
    fn = torch.compile(lambda *a: moe_block(*a, k, save8=True), fullgraph=True, backend="aot_eager")
    got = torch.autograd.grad(fn(*leaves), leaves, dout)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_captured_step_beside_a_live_eager_graph():
    """Forward and backward of the block in a HIP graph, on leaves of its own,
    while an eager autograd graph of the same weights lives; every replay
    against the eager gradients."""
    from combine_top_route_amd.autograd import moe_block
    leaves, dout = tensors(torch.bfloat16, seed=11)
    leaves = [t.requires_grad_() for t in leaves]
    live = moe_block(*leaves, k, save8=True)               # kept until the end
    own = [t.detach().requires_grad_() for t in leaves]    # the same memory
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = [t.detach().requires_grad_() for t in leaves]
        torch.autograd.grad(moe_block(*warm, k, save8=True), warm, dout)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe_block(*own, k, save8=True)
        grads = torch.autograd.grad(out, own, dout)
    for i in range(3):
        fresh, d2 = tensors(torch.bfloat16, seed=20 + i)
        with torch.no_grad():
            for t, f in zip(leaves, fresh):
                t.detach().copy_(f)
            dout.copy_(d2)
        graph.replay()
        eager = [t.detach().requires_grad_() for t in leaves]
        want_out = moe_block(*eager, k, save8=True)
        want = torch.autograd.grad(want_out, eager, dout)
        torch.cuda.synchronize()
        assert torch.equal(out, want_out)
        for a, b in zip(grads, want):
            assert torch.equal(a, b)
    assert live.shape == (T, d)


def test_router_alone():
    """Without a gradient through x's other use nothing is added; compiled and
    eager calls agree; logits that nothing uses leave x's gradient as it is."""
    from combine_top_route_amd.autograd import _Router, router
    leaves, _ = tensors(torch.bfloat16, seed=9)
    x, wr = (t.requires_grad_() for t in leaves[:2])
    g = torch.randn((T, E), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    want = B.router_backward(g, x.detach(), wr.detach())
    for fn in (router, torch.compile(lambda *a: router(*a), fullgraph=True, backend="aot_eager")):
        logits = fn(x, wr)
        assert torch.equal(logits, B.router_logits(x.detach(), wr.detach()))
        for a, b in zip(torch.autograd.grad(logits, (x, wr), g), want):
            assert torch.equal(a, b)
    dx_in = torch.randn((T, d), generator=torch.Generator(device=DEV).manual_seed(4), device=DEV).bfloat16()
    through = _Router.apply(x, wr, torch.float32)[1]
    got = torch.autograd.grad(through, (x, wr), dx_in, allow_unused=True)
    assert torch.equal(got[0], dx_in) and got[1] is None
