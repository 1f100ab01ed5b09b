"""The norms and the residual block by the calls that a training or serving loop
makes of them: compiled whole, with a stream each at once, twice through one graph."""
import pytest
import torch

from combine_top_route_amd import autograd as A
from combine_top_route_amd import binding as B
from test_gpu_mxfp4 import make
from test_gpu_norm import args, inputs

pytestmark = pytest.mark.gpu


def leaves(ts):
    return [t.detach().clone().requires_grad_() for t in ts]


@pytest.mark.parametrize("use", ["z", "h", "both"])
def test_norm_alone_compiled(use):
    """Without a block z is x itself: what comes back along it is added."""
    x0, w0 = torch.randn((64, 264), device="cuda"), torch.randn(264, device="cuda")

    def f(x, w):
        z, h = A.norm_residual(x * 1.5, w_next=w)
        return {"z": (z * z).sum(), "h": (h * h * x).sum(), "both": (z * h).sum()}[use]

    got, want = leaves((x0, w0)), leaves((x0, w0))
    f(*want).backward()
    torch.compile(f, fullgraph=True, backend="aot_eager")(*got).backward()
    for a, b in zip(got, want):
        if b.grad is None:
            assert a.grad is None or not bool(a.grad.any())
        else:
            assert (a.grad - b.grad).abs().max().item() <= 2.0 ** -20 * b.grad.abs().max().item()


def block_leaves(seed=1, T=96, d=256, E=8, I=128):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shapes = dict(x=(T, d), w_router=(E, d), w_gate_up=(E, 2 * I, d), w_down=(E, d, I), w_pre=(d,), w_post=(d,),
                  gate=(T, 1), w_next=(d,))
    return {n: (torch.randn(s, generator=g, device="cuda") * (0.1 if len(s) == 3 else 1)).bfloat16().requires_grad_()
            for n, s in shapes.items()}


@pytest.mark.parametrize("save8", [False, True])
def test_block_compiled(save8):
    f = lambda **p: A.moe_residual_block(**p, k=2, res_scale=0.5, save8=save8)
    p, q = block_leaves(), block_leaves()
    z, h = f(**p)
    dz, dh = torch.randn_like(z), torch.randn_like(h)
    torch.autograd.backward((z, h), (dz, dh))
    zc, hc = torch.compile(f, fullgraph=True, backend="aot_eager")(**q)
    torch.autograd.backward((zc, hc), (dz, dh))
    assert torch.equal(z, zc) and torch.equal(h, hc)
    for n in p:
        assert torch.equal(p[n].grad, q[n].grad), n


def test_two_streams_at_once():
    """Calls in flight together share nothing."""
    t, scale = inputs(3000, 2048, "bf16", "all")
    u, _ = inputs(3000, 2048, "bf16", "all", seed=9)
    step = lambda v: list(B.norm_residual_backward(v["dz"], v["dh"], v["x"], v["y"], **args(v, scale)).values())
    x, gu, dn, lg = make(300, 256, 16, 4, 256)
    prompt = lambda: [A.moe_prompt(x, lg, gu[0], dn[0], 4, gu[1], dn[1])]
    want = [step(t), step(u), prompt()]
    streams = [torch.cuda.Stream() for _ in want]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, f in zip(streams, (lambda: step(t), lambda: step(u), prompt)):
            with torch.cuda.stream(s):
                got.append(f())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(c, d) for c, d in zip(a, b))


def test_second_order_is_refused():
    """A gradient of the gradient has no formula here and says so."""
    t, scale = inputs(20, 136, "f32", "all")
    x, y = leaves((t["x"], t["y"]))
    z, h = A.norm_residual(x, y, t["w_post"], t["gate"], scale, t["w_next"])
    (g,) = torch.autograd.grad((z * h).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="autograd"):
        (g * g).sum().backward()
