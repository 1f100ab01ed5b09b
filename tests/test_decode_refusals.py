"""moe_decode and MoeDecoder refuse bad arguments on the host, before any HIP
call (no GPU here: device pointers are fakes that are never read)."""
import ctypes
import os

import pytest
import torch

from combine_top_route_amd import binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="library not built")

P = lambda off=0: ctypes.c_void_p((1 << 20) + off)


def shape(T=4, d=256, E=8, k=2, I=128, dtype=torch.bfloat16, precision="native", **kw):
    return B.make_shape(T, d, E, k, I, dtype, torch.float32, precision, **kw)


def call(sh=None, weights=0, x=P(), ids=P(), w=P(), wgu=P(), sgu=None, wd=P(), sd=None, out=P(), ws=P(), n=1 << 40,
         routing=True):
    sh = shape() if sh is None else sh
    r = B.MoeRouting(None, ids, w, None, None, None, None)
    return B.lib().moe_decode(ctypes.byref(sh), weights, x, ctypes.byref(r) if routing else None, wgu, sgu, wd, sd, out,
                              ws, n, None)


def size(sh):
    n = ctypes.c_size_t()
    return B.lib().moe_decode_workspace_size(ctypes.byref(sh), ctypes.byref(n)), n.value


def test_workspace_sizes():
    for kw in (dict(), dict(T=1), dict(T=17), dict(T=256), dict(dtype=torch.float32), dict(d=8, I=8)):
        st, n = size(shape(**kw))
        assert st == 0 and n > 0
    # grows with T, so a workspace for the largest batch serves the smaller
    sizes = [size(shape(T=T))[1] for T in range(1, 257)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    assert size(shape(T=256, E=1024, k=256, I=16384, d=16384))[1] > 1 << 32   # sizes beyond 32 bits
    assert size(shape(T=256, E=1024, k=512, I=16384))[0] == 2 and b"4 GiB" in B.lib().moe_last_error()
    assert size(shape(T=257))[0] == 2 and b"moe_forward" in B.lib().moe_last_error()
    assert size(shape(T=0))[0] == 1
    assert size(shape(precision="fp8_block"))[0] == 2
    assert size(shape(k=9))[0] == 1


def test_null_and_misaligned_pointers():
    for name in ("x", "ids", "w", "wgu", "wd", "out", "ws"):
        assert call(**{name: None}) == 1, name
    assert call(routing=False) == 1
    for name in ("x", "wgu", "wd", "out"):
        assert call(**{name: P(8)}) == 1, name
    assert call(ws=P(128)) == 1
    assert call(n=16) == 3


def test_weight_formats():
    assert call(weights=3) == 1 and call(weights=-1) == 1
    assert call(sgu=P()) == 1 and call(sd=P()) == 1                 # scales for uncoded weights
    for w in (1, 2):
        ok = dict(weights=w, sgu=P(), sd=P())
        assert call(**{**ok, "sgu": None}) == 1 and call(**{**ok, "sd": None}) == 1
        assert call(**{**ok, "sgu": P(2)}) == 1 and call(**{**ok, "sd": P(1)}) == 1
        assert call(sh=shape(dtype=torch.float32), **ok) == 2
        assert call(sh=shape(d=264), **ok) == 2 and call(sh=shape(I=136), **ok) == 2


def decoder(**kw):
    a = dict(max_T=8, d=64, E=4, k=2, I=32, device="cpu")
    a.update(kw)
    return B.MoeDecoder(**a)


def test_decoder_constructor():
    with pytest.raises(B.MoeError, match="moe_forward"):
        decoder(max_T=257)
    with pytest.raises(B.MoeError):
        decoder(max_T=0)
    with pytest.raises(ValueError, match="weights"):
        decoder(weights="int4")
    with pytest.raises(B.MoeError):
        decoder(k=5)


def test_decoder_arguments():
    bf = torch.bfloat16
    good = dict(x=torch.zeros(3, 64, dtype=bf), w_gate_up=torch.zeros(4, 64, 64, dtype=bf),
                w_down=torch.zeros(4, 64, 32, dtype=bf), logits=torch.zeros(3, 4, dtype=bf))
    dec = decoder()

    def bad(match, **kw):
        with pytest.raises(ValueError, match=match):
            dec.forward(**{**good, **kw})

    bad("on cpu")                                       # everything right but the memory
    bad("9 tokens", x=torch.zeros(9, 64, dtype=bf))
    bad("0 tokens", x=torch.zeros(0, 64, dtype=bf))
    bad("x has shape", x=torch.zeros(3, 32, dtype=bf))
    bad("x has dtype", x=torch.zeros(3, 64))
    bad("contiguous", x=torch.zeros(3, 128, dtype=bf)[:, ::2])
    bad("contiguous", w_down=torch.zeros(4, 32, 64, dtype=bf).transpose(1, 2))
    bad("w_gate_up has shape", w_gate_up=torch.zeros(4, 32, 64, dtype=bf))
    bad("logits has shape", logits=torch.zeros(2, 4, dtype=bf))
    bad("logits has dtype", logits=torch.zeros(3, 4))
    bad("topk_ids is required", logits=None)
    bad("not both", topk_ids=torch.zeros(3, 2, dtype=torch.int32))
    bad("topk_ids has dtype", logits=None, topk_ids=torch.zeros(3, 2, dtype=torch.int64),
        topk_w=torch.zeros(3, 2))
    for weights in ("fp8_block", "mxfp8"):
        dec = decoder(weights=weights, d=128, I=128)
        good = dict(x=torch.zeros(3, 128, dtype=bf), logits=torch.zeros(3, 4, dtype=bf))
        codes = torch.zeros(4, 256, 128, dtype=torch.uint8), torch.zeros(4, 128, 128, dtype=torch.uint8)
        sh = ((4, 2, 1), (4, 1, 1)) if weights == "fp8_block" else ((4, 256, 4), (4, 128, 4))
        dt = torch.float32 if weights == "fp8_block" else torch.uint8
        gu, dn = (codes[0], torch.zeros(sh[0], dtype=dt)), (codes[1], torch.zeros(sh[1], dtype=dt))
        bad("pair", w_gate_up=torch.zeros(4, 256, 128, dtype=bf), w_down=dn)
        bad("scales has shape", w_gate_up=gu, w_down=(dn[0], gu[1]))
        bad("codes has shape", w_gate_up=(dn[0], gu[1]), w_down=dn)
        bad("scales has dtype", w_gate_up=(gu[0], gu[1].to(torch.int32)), w_down=dn)


def test_operator_refuses_and_traces():
    from combine_top_route_amd.autograd import moe_decode
    bf, u8 = torch.bfloat16, torch.uint8
    good = dict(x=torch.zeros(3, 128, dtype=bf), logits=torch.zeros(3, 4), w_gate_up=torch.zeros(4, 256, 128, dtype=bf),
                w_down=torch.zeros(4, 128, 128, dtype=bf), k=2)

    def bad(match, **kw):
        with pytest.raises(ValueError, match=match):
            moe_decode(**{**good, **kw})

    bad("GPU")
    bad("w_gate_up", x=torch.zeros(3, 64, dtype=bf))
    bad("w_down", w_down=torch.zeros(4, 128, 64, dtype=bf))
    bad("logits", logits=torch.zeros(2, 4))
    bad("k=5", k=5)
    bad("weights must be", w_down=torch.zeros(4, 128, 128))
    bad("both weights or of neither", s_down=torch.zeros(4, 1, 1))
    bad("weights must be", s_gate_up=torch.zeros(4, 2, 1), s_down=torch.zeros(4, 1, 1))
    bad("s_down must be", s_gate_up=torch.zeros(4, 2, 1), s_down=torch.zeros(4, 2, 1))
    bad("contiguous", x=torch.zeros(3, 256, dtype=bf)[:, ::2])
    meta = {n: t.to("meta") if isinstance(t, torch.Tensor) else t for n, t in good.items()}
    assert moe_decode(**meta).shape == (3, 128)
    codes = dict(meta, w_gate_up=torch.zeros(4, 256, 128, dtype=u8, device="meta"),
                 w_down=torch.zeros(4, 128, 128, dtype=u8, device="meta"),
                 s_gate_up=torch.zeros(4, 256, 4, dtype=u8, device="meta"),
                 s_down=torch.zeros(4, 128, 4, dtype=u8, device="meta"))
    assert moe_decode(**codes).dtype == bf
