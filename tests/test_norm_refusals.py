"""The norms' entry points refuse bad arguments on the host, before any HIP
call, and their torch operators trace on the CPU."""
import ctypes
import math
import os

import pytest
import torch

from combine_top_route_amd import autograd as A
from combine_top_route_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="library not built")

BIG = 1 << 40
P = lambda n, off=0: ctypes.c_void_p((n << 24) + off)


def shape(T=4, d=64, dtype=1, gate=0, scale=1.0, eps=1e-6):
    return B.MoeNormShape(T, d, dtype, gate, scale, eps)


def forward(sh=None, x=P(1), y=P(2), w_post=P(3), gate=None, w_next=P(5), z=P(6), h=P(7)):
    return B.lib().moe_norm_forward(ctypes.byref(sh or shape()), x, y, w_post, gate, w_next, z, h, None)


def backward(sh=None, dz=P(1), dh=P(2), z=P(3), y=P(4), w_post=P(5), gate=None, w_next=P(7), dx=P(8), dy=P(9),
             dw_post=P(10), dgate=None, dw_next=P(12), ws=P(13), n=BIG):
    return B.lib().moe_norm_backward(ctypes.byref(sh or shape()), dz, dh, z, y, w_post, gate, w_next, dx, dy, dw_post,
                                     dgate, dw_next, ws, n, None)


BAD_SHAPES = [dict(T=0), dict(T=(1 << 24) + 1), dict(d=0), dict(d=12), dict(d=16392), dict(dtype=2), dict(gate=3),
              dict(gate=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
              dict(scale=math.nan), dict(scale=math.inf)]


@pytest.mark.parametrize("bad", BAD_SHAPES, ids=str)
def test_shapes(bad):
    g = P(4) if bad.get("gate") else None
    assert forward(shape(**bad), gate=g) == 1
    assert backward(shape(**bad), gate=g, dgate=g) == 1
    n = ctypes.c_size_t()
    assert B.lib().moe_norm_workspace_size(ctypes.byref(shape(**bad)), ctypes.byref(n)) == 1


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(z=None), dict(h=None), dict(w_next=None), dict(y=None), dict(gate=P(4)),
    dict(sh=shape(gate=1)), dict(sh=shape(gate=2)), dict(y=None, z=None, w_post=None, sh=shape(scale=0.5)),
    dict(y=None, z=None, w_post=None, w_next=None, h=None), dict(x=P(1, 8)), dict(y=P(2, 4)), dict(w_post=P(3, 8)),
    dict(w_next=P(5, 8)), dict(z=P(6, 8)), dict(h=P(7, 8)), dict(sh=shape(gate=1), gate=P(4, 8)),
    dict(sh=shape(gate=2), gate=P(4, 1)), dict(h=P(6)), dict(h=P(1)), dict(h=P(2, 496)), dict(z=P(3)),
    dict(z=P(1, 16)), dict(z=P(5, 112)), dict(sh=shape(gate=1), gate=P(4), z=P(4))], ids=str)
def test_forward(bad):
    assert forward(**bad) == 1


@pytest.mark.parametrize("bad", [
    dict(dx=None), dict(dz=None, dh=None), dict(dh=None), dict(w_next=None), dict(dw_next=None), dict(z=None),
    dict(y=None), dict(dy=None), dict(dw_post=None), dict(w_post=None), dict(gate=P(6)), dict(dgate=P(11)),
    dict(sh=shape(gate=1), gate=P(6)), dict(sh=shape(gate=1), dgate=P(11)), dict(ws=None), dict(ws=P(13, 64)),
    dict(dy=None, w_post=None, dw_post=None, sh=shape(scale=0.5)), dict(dz=P(1, 8)), dict(dh=P(2, 8)),
    dict(z=P(3, 8)), dict(y=P(4, 8)), dict(dx=P(8, 8)), dict(dy=P(9, 8)), dict(dw_post=P(10, 1)),
    dict(dw_next=P(12, 1)), dict(sh=shape(gate=2), gate=P(6), dgate=P(11, 1)), dict(dx=P(2)), dict(dx=P(1, 16)),
    dict(dx=P(9)), dict(dy=P(4)), dict(dw_post=P(5)), dict(dw_next=P(7)), dict(dw_next=P(13)),
    dict(sh=shape(gate=2), gate=P(6), dgate=P(6)), dict(sh=shape(gate=2), gate=P(6), dgate=P(10))], ids=str)
def test_backward(bad):
    assert backward(**bad) == 1


def test_workspace():
    assert backward(n=16) == 3
    for T, d in ((1, 8), (100, 2048), (1 << 24, 16384)):  # bounded as T grows
        assert 0 < B.norm_workspace_size(shape(T, d)) < 1 << 27


def test_binding():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w, t = torch.zeros(64, dtype=torch.bfloat16), torch.zeros(4, 1, dtype=torch.bfloat16)
    for kw in (dict(w_next=w.float()), dict(w_next=w[:32]), dict(y=x.float()), dict(y=x[:2]), dict(y=x, gate=t[:3]),
               dict(y=x, gate=w[:8]), dict(y=x, gate=t.float()), dict(y=x, w_post=torch.zeros(128)[::2]),
               dict(w_next=w)):                      # the last: right, but not on a GPU
        with pytest.raises(ValueError):
            B.norm_residual(x, **kw)
        with pytest.raises(ValueError):
            A.norm_residual(x, **kw)
    for bad in (x[0], x.half(), torch.zeros(4, 128, dtype=torch.bfloat16)[:, ::2]):
        with pytest.raises(ValueError):
            B.norm_residual(bad, w_next=w)
        with pytest.raises(ValueError):
            A.norm_residual(bad, w_next=w)
    for kw in (dict(), dict(w_next=w, res_scale=0.5), dict(w_next=w, gate=t), dict(w_post=w, w_next=w)):
        with pytest.raises(ValueError):
            A.norm_residual(x, **kw)
    with pytest.raises(ValueError, match="dh and w_next"):
        B.norm_residual_backward(x, None, x, w_next=w)
    with pytest.raises(ValueError, match="dz has shape"):
        B.norm_residual_backward(x[:2], x, x, w_next=w)
    with pytest.raises(ValueError, match="w_pre, or h"):
        A.moe_residual_block(x, None, None, None, 1)


def test_operators_trace():
    """Shapes of the operators' outputs, without a device."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        x, w, g = torch.empty(4, 64), torch.empty(64), torch.empty(4, 1)
        z, h = A.norm_fwd(x, x, w, g, w, 0.5, 1e-6)
        assert z.shape == h.shape == x.shape
        z, h = A.norm_fwd(x, None, None, None, w, 1.0, 1e-6)
        assert z.numel() == 0 and h.shape == x.shape
        out = A.norm_bwd(x, x, x, x, w, g, w, 0.5, 1e-6)
        assert [tuple(t.shape) for t in out] == [(4, 64), (4, 64), (64,), (4, 1), (64,)]
        out = A.norm_bwd(None, x, x, None, None, None, w, 1.0, 1e-6)
        assert [t.numel() for t in out] == [256, 0, 0, 0, 64]
