"""Two layers as they are served from MXFP4 weights: norm, router, experts, then
gate, norm and residual with the next layer's norm in the same pass; few tokens
through moe_decode, a prompt through moe_prompt, and both in a captured graph."""
import math

import pytest
import torch

from combine_top_route_amd import autograd as A
from combine_top_route_amd import binding as B
from test_gpu_norm import forward_ref, near

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
D, E, K, I, LAYERS = 512, 16, 4, 256, 2


def model(seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s, std=1.0, mean=0.0: (torch.randn(s, generator=g, device=DEV) * std + mean).bfloat16()
    layers = []
    for _ in range(LAYERS):
        gu, dn = B.quantize_mxfp4(r(E, 2 * I, D, std=D ** -0.5)), B.quantize_mxfp4(r(E, D, I, std=I ** -0.5))
        layers.append(dict(w_router=r(E, D, std=D ** -0.5), gu=gu, dn=dn, w_pre=r(D, std=0.2, mean=1.0),
                           w_post=r(D, std=0.2, mean=1.0), gate=r(D, std=0.3, mean=0.5)))
    return layers


def experts(p, h, lg, prompt):
    f = A.moe_prompt if prompt else A.moe_decode
    return f(h, lg, p["gu"][0], p["dn"][0], K, p["gu"][1], p["dn"][1])


def served(layers, x, prompt, ban=None):
    """(residual stream, last norm's output, what passed between the operators)"""
    seen = []
    _, h = A.norm_residual(x, w_next=layers[0]["w_pre"])
    for p, nxt in zip(layers, layers[1:] + layers[:1]):
        lg = B.router_logits(h, p["w_router"])
        if ban is not None:
            lg = lg.masked_fill(ban, -math.inf)
        y = experts(p, h, lg, prompt)
        z, hn = A.norm_residual(x, y, w_post=p["w_post"], gate=p["gate"], res_scale=0.5, w_next=nxt["w_pre"])
        seen.append((x, h, lg, y, z, hn, p, nxt))
        x, h = z, hn
    return x, h, seen


def ban_of(T):
    ban = torch.zeros((T, E), dtype=torch.bool, device=DEV)
    ban[:, 2] = True
    if T > 1:
        ban[T // 2] = True  # a token without experts
    return ban


@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("T", [1, 7, 64, 256, 700])
@torch.no_grad()
def test_layers(T, prompt):
    if T > 256 and not prompt:
        with pytest.raises(Exception, match="T="):
            served(model(), torch.zeros((T, D), dtype=torch.bfloat16, device=DEV), False)
        return
    layers = model()
    x = (torch.randn((T, D), generator=torch.Generator(device=DEV).manual_seed(T), device=DEV) * 2).bfloat16()
    ban = ban_of(T)
    z, h, seen = served(layers, x, prompt, ban)
    for xi, hi, lg, y, zi, hn, p, nxt in seen:
        assert T == 1 or not bool(y[T // 2].any())
        t = dict(x=xi, y=y, w_post=p["w_post"], gate=p["gate"], w_next=nxt["w_pre"])
        zr, zm, hr, hm = forward_ref(t, 0.5)
        near(zi, zr, zm, 64)
        near(hn, hr, hm, 64)
        if prompt:  # in pieces of a decode step each
            few = torch.cat([experts(p, hi[i:i + 256], lg[i:i + 256], False) for i in range(0, T, 256)])
            # moe_prompt rounds the activations and the products of the K slots once more, by
        # 2^-8 each, and both round y
            size = y.double().norm(dim=1) + few.double().norm(dim=1)
            assert bool(((y.double() - few.double()).norm(dim=1) <= 4 * 2.0 ** -8 * size).all())


@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("T", [1, 24, 200])
@torch.no_grad()
def test_captured(T, prompt):
    layers = model(1)
    x = torch.randn((T, D), device=DEV).bfloat16()
    ban = ban_of(T)
    served(layers, x, prompt, ban)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z, h, _ = served(layers, x, prompt, ban)
    for i in range(4):
        x.copy_(torch.randn((T, D), device=DEV))
        want = served(layers, x, prompt, ban)[:2]
        z.fill_(3.0), h.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, want[0]) and torch.equal(h, want[1]), i
