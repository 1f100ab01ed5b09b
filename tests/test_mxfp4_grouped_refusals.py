"""MXFP4 weights and the grouped products: bad arguments are refused on the host
before any HIP call; the calls that this binding makes for the norms, the encoder
and the products refuse host memory and run with their tensors' device current."""
import ctypes
import inspect
import os

import pytest
import torch
from torch._subclasses import FakeTensorMode

from combine_top_route_amd import autograd as A
from combine_top_route_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="library not built")

P = lambda n, off=0: ctypes.c_void_p((n << 24) + off)
BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


def shape(T=8, d=256, E=4, k=2, dtype=BF, precision="native", **kw):
    return B.make_shape(T, d, E, k, 128, dtype, BF, precision, **kw)


def routing(offsets=P(5), src_of=P(6)):
    r = B.MoeRouting()
    r.offsets, r.src_of = offsets, src_of
    return r


def product(sh=None, weights=3, x=P(1), gather=1, r=None, codes=P(2), scales=P(3), N=256, swiglu=0, y=P(4)):
    return B.lib().moe_grouped_product(ctypes.byref(sh or shape()), weights, x, gather,
                                       ctypes.byref(r or routing()), codes, scales, N, swiglu, y, None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(codes=None), dict(scales=None), dict(y=None), dict(r=routing(offsets=None)),
    dict(r=routing(src_of=None)), dict(x=P(1, 8)), dict(codes=P(2, 4)), dict(scales=P(3, 2)), dict(y=P(4, 8)),
    dict(N=0), dict(N=-8), dict(N=12), dict(N=32776), dict(N=24, swiglu=1), dict(N=8, swiglu=1), dict(weights=-1),
    dict(weights=4), dict(sh=shape(T=0)), dict(sh=shape(k=5)), dict(y=P(1, 16)), dict(y=P(2, 16)), dict(y=P(3)),
    dict(y=P(5)), dict(y=P(6, 16)), dict(y=P(1, 4080))], ids=str)
def test_product_arguments(bad):
    assert product(**bad) == 1


def test_product_unsupported():
    for w in (0, 1, 2):
        assert product(weights=w) == 2
    assert product(sh=shape(d=192)) == 2
    assert product(sh=shape(dtype=torch.float32)) == 2


def test_encoder_arguments():
    def call(src=P(1), n0=2, n1=3, n2=128, q=P(2), s=P(3)):
        return B.lib().moe_quantize_mxfp4(src, n0, n1, n2, q, s, None)
    for bad in (dict(src=None), dict(q=None), dict(s=None), dict(n0=0), dict(n1=0), dict(n2=0), dict(n2=64),
                dict(n2=-128), dict(n0=65536), dict(n1=65535 * 128 + 1), dict(n2=65536 * 128), dict(src=P(1, 8)),
                dict(q=P(2, 4)), dict(s=P(3, 2)), dict(n0=65535, n1=65535 * 128, n2=65535 * 128)):
        assert call(**bad) == 1, bad


def test_decode_arguments():
    r = B.MoeRouting(*[P(9)] * 7)

    def call(sh=None, weights=3, gs=P(3), ds=P(5)):
        return B.lib().moe_decode(ctypes.byref(sh or shape()), weights, P(1), ctypes.byref(r), P(2), gs, P(4), ds, P(6),
                                  P(7), 1 << 40, None)
    assert call(weights=4) == 1 and call(gs=None) == 1 and call(ds=None) == 1 and call(gs=P(3, 2)) == 1
    assert call(sh=shape(dtype=torch.float32)) == 2 and call(sh=shape(d=192)) == 2 and call(sh=shape(T=257)) == 2


# ------------------------------------------------------------------- binding
T, d, E, k, I, N = 4, 128, 4, 2, 128, 64
R = T * k
F = torch.float32


def tensors(device):
    z = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device=device)
    w = lambda n, m: (z(E, n, m // 2, dtype=U8), z(E, n, m // 32, dtype=U8))
    r = B.Routing.empty(T, E, k, torch.device(device), logits=z(T, E))
    return z, w, r


def calls(device):
    z, w, r = tensors(device)
    return {
        "norm_residual": lambda: B.norm_residual(z(T, d), z(T, d), w_post=z(d), gate=z(T, 1), w_next=z(d)),
        "norm_residual alone": lambda: B.norm_residual(z(T, d), w_next=z(d)),
        "norm_residual_backward": lambda: B.norm_residual_backward(z(T, d), z(T, d), z(T, d), z(T, d), w_post=z(d),
                                                                   gate=z(d), w_next=z(d)),
        "quantize_mxfp4": lambda: B.quantize_mxfp4(z(E, N, d)),
        "grouped_product": lambda: B.grouped_product(z(T, d), w(N, d), r, T, k, swiglu=True),
        "grouped_product rows": lambda: B.grouped_product(z(R, d), w(N, d), r, T, k, gather=False),
        "MoeDecoder.forward": lambda: B.MoeDecoder(T, d, E, k, I, device=device, weights="mxfp4").forward(
            z(T, d), w(2 * I, d), w(d, I), logits=z(T, E)),
    }


ENTRY = {"norm_residual": "moe_norm_forward", "norm_residual alone": "moe_norm_forward",
         "norm_residual_backward": "moe_norm_backward", "quantize_mxfp4": "moe_quantize_mxfp4",
         "grouped_product": "moe_grouped_product", "grouped_product rows": "moe_grouped_product",
         "MoeDecoder.forward": "moe_decode"}


class Stub:
    """The library's host-side queries; other entry points record what device
    was current."""

    def __init__(self, real, current, reached):
        self.__dict__.update(real=real, current=current, reached=reached)

    def __getattr__(self, name):
        if name.endswith(("_size", "_bytes", "_error", "_string")):
            return getattr(self.real, name)
        return lambda *a: self.reached.append((name, self.current[0])) or 0


@pytest.fixture
def stub(monkeypatch):
    current, reached = [0], []

    class Guard:
        def __init__(self, device):
            self.index = torch.device(device).index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *a):
            current[0] = self.before

    s = Stub(B.lib(), current, reached)
    monkeypatch.setattr(B, "lib", lambda: s)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
    return reached


@pytest.mark.parametrize("name", sorted(ENTRY))
def test_host_memory_is_refused(name, stub):
    with pytest.raises(ValueError, match="cpu"):
        calls("cpu")[name]()
    assert stub == []


@pytest.mark.parametrize("name", sorted(ENTRY))
def test_the_tensors_device_is_current(name, stub, monkeypatch):
    monkeypatch.setattr(B, "_ptr", lambda t: None if t is None else 1 << 20)
    with FakeTensorMode():
        calls("cuda:1")[name]()
    assert stub == [(ENTRY[name], 1)]


def test_every_entry_is_listed():
    entries = {v.name for v in vars(B).values() if isinstance(v, B._Entry)}
    assert entries <= set(ENTRY.values())
    used = {n for n, f in vars(B).items() if inspect.isfunction(f)
            and any(e + "(dev" in inspect.getsource(f) for e, v in vars(B).items() if isinstance(v, B._Entry))}
    assert used and used <= {n.split()[0] for n in ENTRY}


def test_binding_refusals():
    z, w, r = tensors("cpu")
    x = z(T, d)
    for bad in (dict(x=x[0]), dict(x=x.float()), dict(x=z(R, d)), dict(weight=z(E, N, d)), dict(weight=w(N, 256)),
                dict(weight=(w(N, d)[0], z(E, N, d // 32))), dict(gather=False), dict(out=z(R, N + 8)),
                dict(routing=B.Routing.empty(T, E + 1, k, torch.device("cpu"))),
                dict(routing=B.Routing.empty(T + 1, E, k, torch.device("cpu")))):
        with pytest.raises(ValueError):
            B.grouped_product(**{**dict(x=x, weight=w(N, d), routing=r, T=T, k=k), **bad})
    for bad in (z(E, N, d).float(), z(N, d), z(E, d, N).transpose(1, 2)):
        with pytest.raises(ValueError, match="src must"):
            B.quantize_mxfp4(bad)
    dec = B.MoeDecoder(T, d, E, k, I, device="cpu", weights="mxfp4")
    for gu in (z(E, 2 * I, d), (z(E, 2 * I, d, dtype=U8), z(E, 2 * I, d // 32, dtype=U8)), w(2 * I, 256)):
        with pytest.raises(ValueError):
            dec.forward(x, gu, w(d, I), logits=z(T, E))


def test_operators():
    z, w, r = tensors("cpu")
    gu, dn = w(2 * I, d), w(d, I)
    good = (z(T, d), z(T, E), gu[0], dn[0], k, gu[1], dn[1])
    for at, bad in ((0, z(T, d).float()), (0, z(T, 256)), (1, z(T, E + 1)), (2, z(E, 2 * I, d, dtype=U8)),
                    (3, z(E, d, I, dtype=U8)), (4, 5), (5, gu[1][:, :, :1]), (6, dn[1].float()), (0, z(T, d))):
        with pytest.raises(ValueError):                   # the last: right, but not on a GPU
            A.moe_prompt(*good[:at], bad, *good[at + 1:])
    with FakeTensorMode():
        z, w, r = tensors("cuda:0")
        gu, dn = w(2 * I, d), w(d, I)
        assert A.moe_prompt(z(T, d), z(T, E), gu[0], dn[0], k, gu[1], dn[1]).shape == (T, d)
        assert A.moe_decode(z(T, d), z(T, E), gu[0], dn[0], k, gu[1], dn[1]).shape == (T, d)
