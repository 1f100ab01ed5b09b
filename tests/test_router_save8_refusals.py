"""The router's and the 8-bit checkpoint's entry points refuse bad arguments
on the host, before any HIP call, and their torch operators trace on the CPU."""
import ctypes
import os

import pytest
import torch

from combine_top_route_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="library not built")

P = lambda off=0: ctypes.c_void_p((1 << 20) + off)
BIG = 1 << 40


def shape(T=4, d=256, E=8, k=2, I=128, dtype=torch.bfloat16, precision="native", **kw):
    return B.make_shape(T, d, E, k, I, dtype, torch.float32, precision, **kw)


def routing(**null):
    r = B.MoeRouting(*[P()] * 7)
    for n in null:
        setattr(r, n, None)
    return r


def each(call, names, bad_status=1, make_bad=lambda: None):
    for n in names:
        assert call(**{n: make_bad()}) == bad_status, n


def test_router_forward():
    def call(sh=None, x=P(), w=P(), logits=P()):
        return B.lib().moe_router_forward(ctypes.byref(sh or shape()), x, w, logits, None)
    each(call, ("x", "w", "logits"))
    each(call, ("x", "w", "logits"), make_bad=lambda: P(4))
    assert call(sh=shape(T=0)) == 1 and call(sh=shape(d=12)) == 1 and call(sh=shape(E=1025)) == 1


def test_router_backward():
    def call(sh=None, dl=P(), x=P(), w=P(), dx_in=None, dx=P(), dw=P(), ws=P(), n=BIG):
        return B.lib().moe_router_backward(ctypes.byref(sh or shape()), dl, x, w, dx_in, dx, dw, ws, n, None)
    each(call, ("dl", "x", "w", "dx", "dw", "ws"))
    each(call, ("dl", "x", "w", "dx_in", "dx", "dw"), make_bad=lambda: P(8))
    assert call(ws=P(64)) == 1
    assert call(n=16) == 3 and "workspace" in B.lib().moe_last_error().decode()
    # outputs over inputs and over each other: a byte of overlap is enough
    far = dict(dl=P(1 << 20), x=P(2 << 20), w=P(3 << 20), dx=P(4 << 20), dw=P(5 << 20), ws=P(6 << 20))
    rows, wide, lg = 4 * 256 * 2, 8 * 256 * 2, 4 * 8 * 4
    for out, n_out in (("dx", rows), ("dw", wide)):
        for other, base, n in (("dl", 1, lg), ("x", 2, rows), ("w", 3, wide)):
            for off in (0, n - 16, 16 - n_out):
                assert call(**{**far, out: P((base << 20) + off)}) == 1
                assert "overlap" in B.lib().moe_last_error().decode()
        assert call(**{**far, out: P((7 << 20) + 16), "dx_in": P(7 << 20)}) == 1
    assert call(**{**far, "dx": P(5 << 20)}) == 1
    for T in (1, 100, 1 << 24):       # the parts' size stays bounded as T grows
        n = B.router_workspace_size(shape(T=T, k=1))
        assert 0 < n < 1 << 29
    assert B.router_workspace_size(shape(T=1 << 24, E=1024, k=1, d=16384)) > 0
    with pytest.raises(B.MoeError):
        B.router_workspace_size(shape(T=0))


def test_router_binding():
    bf = torch.bfloat16
    x, w = torch.zeros(4, 64, dtype=bf), torch.zeros(8, 64, dtype=bf)
    for a in ((x, torch.zeros(8, 32, dtype=bf)), (x[0], w), (x, w.float()), (x.half(), w.half()),
              (x, torch.zeros(64, 8, dtype=bf).t()), (torch.zeros(4, 128, dtype=bf)[:, ::2], w), (x, w)):
        with pytest.raises(ValueError):            # the last: right, but not on a GPU
            B.router_logits(*a)
    with pytest.raises(ValueError):
        B.router_logits(x, w, logits_dtype=torch.float16)
    with pytest.raises(ValueError, match="dlogits has shape"):
        B.router_backward(torch.zeros(4, 7), x, w)
    with pytest.raises(ValueError, match="dx_in has dtype"):
        B.router_backward(torch.zeros(4, 8), x, w, dx_in=torch.zeros(4, 64))


def test_save8_rows():
    L = B.lib()

    def save(sh=None, H=P(), r=None, aw=P(), codes=P(), scales=P(1)):
        return L.moe_swiglu_save8(ctypes.byref(sh or shape()), H, ctypes.byref(r or routing()), aw, codes, scales, None)
    each(save, ("H", "codes", "scales"))
    each(save, ("H", "aw", "codes"), make_bad=lambda: P(8))
    for n in ("src_of", "topk_w"):
        assert save(r=routing(**{n: 1})) == 1
    assert save(sh=shape(precision="fp8_block")) == 2 and save(sh=shape(I=12)) == 1

    def back(sh=None, G=P(), codes=P(), scales=P(1), r=None, dH=P(), aw=P(), dw=P()):
        return L.moe_swiglu_backward8(ctypes.byref(sh or shape()), G, codes, scales, ctypes.byref(r or routing()), dH,
                                      aw, dw, None)
    each(back, ("G", "codes", "scales", "dH", "dw"))
    each(back, ("G", "codes", "dH", "aw"), make_bad=lambda: P(8))
    for n in ("src_of", "topk_w"):
        assert back(r=routing(**{n: 1})) == 1
    assert back(sh=shape(precision="mxfp8")) == 2


def test_save8_layer():
    L = B.lib()

    def fwd(sh=None, x=P(), r=None, wgu=P(), wd=P(), out=P(), saved=P(), ws=P(), n=BIG):
        return L.moe_forward8(ctypes.byref(sh or shape()), x, ctypes.byref(r or routing()), wgu, wd, out, saved, ws, n,
                              None)
    each(fwd, ("x", "wgu", "wd", "out", "saved", "ws"))
    each(fwd, ("x", "wgu", "wd", "out", "saved", "ws"), make_bad=lambda: P(8))
    assert fwd(r=routing(row_of=1)) == 1 and fwd(n=16) == 3
    for p in ("fp8_block", "mxfp8", "fp8_bwd"):
        assert fwd(sh=shape(precision=p)) == 2

    def bwd(sh=None, dout=P(), x=P(), r=None, wgu=P(), wd=P(), saved=P(), dx=P(), dwgu=P(), dwd=P(), dtw=P(),
            dlg=P(), ws=P(), n=BIG):
        return L.moe_backward8(ctypes.byref(sh or shape()), dout, x, ctypes.byref(r or routing()), wgu, wd, saved, dx,
                               dwgu, dwd, dtw, dlg, ws, n, None)
    each(bwd, ("dout", "x", "wgu", "wd", "saved", "dx", "dwgu", "dwd", "dtw", "ws"))
    each(bwd, ("dout", "x", "wgu", "wd", "saved", "dx", "dwgu", "dwd", "ws"), make_bad=lambda: P(8))
    assert bwd(r=routing(logits=1)) == 1 and b"dlogits" in L.moe_last_error()
    assert bwd(n=16) == 3


def test_save8_sizes():
    for kw in (dict(), dict(I=8), dict(I=40, dtype=torch.float32), dict(T=1000, k=8)):
        sh = shape(**kw)
        R, I = sh.T * sh.k, sh.I
        n = B.saved8_size(sh)
        assert n == -(-R * 2 * I // 256) * 256 + R * 2 * -(-I // 32)
        for op, plain in ((B.OP_FORWARD, B.OP_FORWARD), (B.OP_BACKWARD, B.OP_BACKWARD)):
            assert B.workspace8_size(sh, op) >= B.workspace_size(sh, plain)
        for op in (B.OP_ROUTE, B.OP_BACKWARD_RECOMPUTE, 9):
            with pytest.raises(B.MoeError):
                B.workspace8_size(sh, op)
    with pytest.raises(B.MoeError, match="NATIVE"):
        B.saved8_size(shape(precision="fp8_bwd"))
    with pytest.raises(ValueError, match="save8"):
        B.MoeLayer(4, 64, 4, 2, 32, device="cpu", save=False, save8=True)


def test_save8_binding():
    bf = torch.bfloat16
    r = B.Routing.empty(4, 4, 2, torch.device("cpu"))
    for H in (torch.zeros(8, 64, dtype=bf), torch.zeros(7, 64, dtype=bf), torch.zeros(8, 63, dtype=bf),
              torch.zeros(8, 64).half(), torch.zeros(8, 128, dtype=bf)[:, ::2], torch.zeros(8, dtype=bf)):
        with pytest.raises(ValueError):            # the first: right, but not on a GPU
            B.swiglu_save8(H, r, 4, 2)
    with pytest.raises(B.MoeError):
        B.swiglu_save8(torch.zeros(8, 24, dtype=bf), None, 4, 2)      # I = 12
    G, c, s = torch.zeros(8, 32, dtype=bf), torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="codes has shape"):
        B.swiglu_backward8(G, c[:, :32].contiguous(), s, r, 4, 2)
    with pytest.raises(ValueError, match="scales has dtype"):
        B.swiglu_backward8(G, c, s.float(), r, 4, 2)
    with pytest.raises(ValueError, match="src_of has shape"):
        B.swiglu_backward8(G, c, s, B.Routing.empty(3, 4, 2, torch.device("cpu")), 4, 2)


def test_operators_refuse_and_trace():
    from torch.fx.experimental.proxy_tensor import make_fx

    from combine_top_route_amd.autograd import moe_block, moe_layer, router
    T, d, E, k, I = 16, 64, 4, 2, 32
    bf = torch.bfloat16
    x, wr, wgu, wd = (torch.empty(s, dtype=bf) for s in ((T, d), (E, d), (E, 2 * I, d), (E, d, I)))
    with pytest.raises(ValueError, match="w_router"):
        router(x, wr[:, :32])
    with pytest.raises(ValueError, match="contiguous"):
        router(x, torch.empty(d, E, dtype=bf).t())
    with pytest.raises(ValueError, match="recompute"):
        moe_layer(x, torch.empty(T, E), wgu, wd, k, recompute=True, save8=True)
    with pytest.raises(ValueError, match="native"):
        moe_layer(x, torch.empty(T, E), wgu, wd, k, precision="mxfp8", save8=True)
    with pytest.raises(ValueError, match="GPU"):
        router(x, wr)
    with pytest.raises(ValueError, match="GPU"):
        moe_layer(x, torch.empty(T, E), wgu, wd, k, save8=True)

    def step(x, wr, wgu, wd, dout):
        out = moe_block(x, wr, wgu, wd, k, save8=True)
        return torch.autograd.grad(out, (x, wr, wgu, wd), dout)

    leaves = [t.requires_grad_() for t in (x, wr, wgu, wd)]
    gm = make_fx(step, tracing_mode="fake")(*leaves, torch.empty(T, d, dtype=bf))
    names = [str(n.target) for n in gm.graph.nodes if n.op == "call_function"]
    for op in ("router_fwd", "moe_fwd8", "moe_bwd8", "router_bwd"):
        assert any(op in n for n in names), op
