"""Gradients that autograd hands over as slices of a larger one: joining outputs
(torch.cat) gives each part's backward a contiguous slice that may start at any
element, where the kernels want 16-byte aligned rows."""
import pytest
import torch

from combine_top_route_amd.autograd import moe_layer, router

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)


def rn(*shape, seed=0, dtype=torch.float32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("ldtype", [torch.float32, torch.bfloat16])
def test_router_of_two_batches_joined(ldtype):
    """E odd: the second batch's rows of dlogits start off any 16-byte boundary.
    Each batch's gradients equal those of its own backward, bit for bit."""
    d, E, sizes = 72, 7, (3, 18)
    xs = [rn(T, d, seed=T, dtype=torch.bfloat16).requires_grad_() for T in sizes]
    w = rn(E, d, seed=1, dtype=torch.bfloat16)
    dl = rn(sum(sizes), E, seed=2, dtype=ldtype)
    ws = [w.clone().requires_grad_() for _ in sizes]
    torch.cat([router(x, v, ldtype) for x, v in zip(xs, ws)]).backward(dl)
    for x, v, part in zip(xs, ws, dl.split(sizes)):
        x1, v1 = x.detach().clone().requires_grad_(), w.clone().requires_grad_()
        router(x1, v1, ldtype).backward(part.clone())
        assert torch.equal(x.grad, x1.grad) and torch.equal(v.grad, v1.grad)


@pytest.mark.parametrize("save8", [False, True])
def test_layer_output_joined_behind_other_values(save8):
    """dout starts three elements into the joined gradient."""
    T, d, E, k, I = 9, 64, 4, 2, 40
    args = (rn(T, d, dtype=torch.bfloat16), rn(T, E, seed=1), rn(E, 2 * I, d, seed=2, dtype=torch.bfloat16) * d ** -0.5,
            rn(E, d, I, seed=3, dtype=torch.bfloat16) * I ** -0.5)
    dout = rn(3 + T * d, seed=4, dtype=torch.bfloat16)
    a = [t.clone().requires_grad_() for t in args]
    b = [t.clone().requires_grad_() for t in args]
    torch.cat([torch.zeros(3, device=DEV, dtype=torch.bfloat16), moe_layer(*a, k, save8=save8).flatten()]).backward(dout)
    moe_layer(*b, k, save8=save8).backward(dout[3:].clone().view(T, d))
    for s, t in zip(a, b):
        assert torch.equal(s.grad, t.grad)
