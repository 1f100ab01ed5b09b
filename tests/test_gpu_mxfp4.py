"""MXFP4 weights: the encoder bit for bit, and the few-token layer from them.
The layer's bounds are those of test_gpu_decode.py: a code times its scale is
exact in bfloat16, so a coded weight is a bfloat16 weight."""
import math

import pytest
import torch

from combine_top_route_amd import autograd as A
from combine_top_route_amd import binding as B
from test_gpu_decode import DEV, check, plain, topk64

pytestmark = pytest.mark.gpu

VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def values_of(codes, scales):
    """float64 [.., K] of codes [.., K/2] and scale bytes [.., K/32]."""
    codes = codes.long()
    nib = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    v = VALUES.to(codes.device)[nib & 7] * (1 - 2 * (nib >> 3))
    s = torch.where(scales == 255, math.nan, torch.exp2(scales.double() - 127.0))
    return (v.view(*scales.shape, 32) * s[..., None]).flatten(-2)


def encode_ref(w):
    """Codes and scales of w [.., K] by looking at every code."""
    b = w.double().cpu().reshape(*w.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    X = torch.full(amax.shape, 200.0, dtype=torch.float64)
    for x in range(130, -128, -1):
        X = torch.where(amax <= 6.0 * 2.0 ** x, float(x), X)
    X = torch.where(amax > 0, X, 0.0)
    y = b * torch.exp2(-X)[..., None]
    dist = (y.abs()[..., None] - VALUES).abs()
    near = dist == dist.amin(-1, keepdim=True)
    even = near & (torch.arange(8) % 2 == 0)
    code = torch.where(even.any(-1), even.double().argmax(-1), near.double().argmax(-1))
    code = code + 8 * y.signbit()
    bad = ~b.isfinite().all(-1)
    code = torch.where(bad[..., None], 7, code).flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), torch.where(bad, 255, X + 127).to(torch.uint8)


@pytest.mark.parametrize("n0,n1,n2", [(1, 1, 128), (3, 5, 384), (2, 130, 256)])
def test_encoder(n0, n1, n2):
    g = torch.Generator().manual_seed(n1)
    w = torch.randn((n0, n1, n2), generator=g) * torch.exp2(torch.randint(-8, 8, (n0, n1, 1), generator=g).float())
    w = w.bfloat16()
    w[0, 0, :32] = 0.0
    w[0, 0, 32:40] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])  # ties, under a scale of one
    w[0, 0, 40:48] = -w[0, 0, 32:40]
    w[0, 0, 48:64] = 0.0
    w[0, 0, 64:96] = torch.linspace(-6.03125, 6.03125, 32)                       # just past a scale's largest
    w[0, 0, 96:128] = torch.randn(32, generator=g) * 2.0 ** -128                 # subnormal
    if n1 > 1:
        w[0, 1, :32] = 2.0 ** -133
        w[0, 1, 32:64] = torch.finfo(torch.bfloat16).max
        w[0, 2, 3], w[0, 2, 40], w[0, 3, 100] = math.inf, math.nan, -math.inf
        w[0, 4, :32] = torch.arange(32) / 4
    q, s = B.quantize_mxfp4(w.to(DEV))
    qr, sr = encode_ref(w)
    assert torch.equal(s.cpu(), sr)
    same = q.cpu() == qr
    # -0 and what rounds to it keep their sign; every code is as nearest, ties to even
    assert bool(same.all()), (w.flatten()[(~same).flatten().repeat_interleave(2).nonzero()[:4, 0]], (~same).sum())


def make(T, d, E, k, I, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    x = rn(T, d).bfloat16()
    wgu = B.quantize_mxfp4((rn(E, 2 * I, d) * d ** -0.5).bfloat16())
    wd = B.quantize_mxfp4((rn(E, d, I) * I ** -0.5).bfloat16())
    return x, wgu, wd, rn(T, E)


def decoder(x, E, k, I, limit=0.0, logits_dtype=torch.float32, max_T=None):
    return B.MoeDecoder(max_T or x.shape[0], x.shape[1], E, k, I, weights="mxfp4", device=DEV, swiglu_limit=limit,
                        logits_dtype=logits_dtype)


# one token, odd counts, on and around a column block, up to the largest; extents
# of one and of odd numbers of 128 columns; one expert; k = E; weights past the
# last-level cache; wide row tiles; an expert's tokens split over work-groups
CASES = [(1, 128, 1, 1, 128), (1, 256, 16, 4, 128), (2, 256, 8, 8, 384), (3, 384, 5, 5, 640), (8, 640, 30, 4, 256),
         (9, 128, 6, 2, 256), (16, 384, 7, 3, 128), (17, 256, 7, 3, 256), (33, 128, 1, 1, 384), (49, 896, 4, 2, 128),
         (100, 128, 2, 1, 256), (256, 256, 40, 6, 128), (130, 1024, 200, 4, 1024), (12, 4096, 48, 6, 1024),
         (9, 1024, 200, 8, 1024), (20, 256, 256, 6, 128), (256, 1152, 128, 5, 256), (250, 128, 20, 2, 256),
         (97, 640, 2, 1, 128), (4, 128, 64, 64, 128), (8, 128, 128, 8, 128), (3, 128, 200, 150, 128)]


def cut(wgu, wd, ids):
    """The experts in use, in 64 bits, and ids among them."""
    used = [e for e in torch.unique(ids).tolist() if 0 <= e < wgu[0].shape[0]]
    remap = torch.full((wgu[0].shape[0] + 1,), -1, device=DEV)
    remap[used] = torch.arange(len(used), device=DEV)
    outside = (ids < 0) | (ids >= wgu[0].shape[0])
    return values_of(wgu[0][used], wgu[1][used]), values_of(wd[0][used], wd[1][used]), torch.where(
        outside, -1, remap[ids.long().clamp(0, wgu[0].shape[0])])


@pytest.mark.parametrize("T,d,E,k,I", CASES)
def test_logits(T, d, E, k, I):
    x, wgu, wd, logits = make(T, d, E, k, I)
    for lt in (torch.float32, torch.bfloat16):
        dec = decoder(x, E, k, I, logits_dtype=lt)
        got = dec.forward(x, wgu, wd, logits=logits.to(lt))
        ids, w = topk64(logits.to(lt), k)
        assert torch.equal(dec.topk_ids.long(), ids)
        a, b, used = cut(wgu, wd, ids)
        check(got, x, a, b, used, w)


@pytest.mark.parametrize("T,d,E,k,I", CASES)
def test_ids_with_empty_slots_and_repeats(T, d, E, k, I):
    x, wgu, wd, _ = make(T, d, E, k, I, seed=1)
    g = torch.Generator().manual_seed(2)
    ids = torch.randint(-2, E + 2, (T, k), generator=g, dtype=torch.int32)
    w = torch.randn((T, k), generator=g)
    ids[T // 2] = -1                                                         # a row left empty
    w[ids < 0] = float("nan")
    ids, w = ids.to(DEV), w.to(DEV)
    got = decoder(x, E, k, I, limit=0.75).forward(x, wgu, wd, topk_ids=ids, topk_w=w)
    if bool(((ids >= 0) & (ids < E)).any()):
        a, b, used = cut(wgu, wd, ids)
        check(got, x, a, b, used, w, limit=0.75)
    assert not bool(got[T // 2].any())


# gate/up in 128-column tiles from 256 of them on (more experts than slots, and
# fewer), down in tiles of 128 and of 256; an expert with every token, one with
# none, one with 20; d and I of one and of odd numbers of 128
@pytest.mark.parametrize("T,d,E,k,I", [(256, 128, 64, 4, 256), (200, 384, 128, 5, 128), (70, 640, 40, 6, 512),
                                       (9, 256, 200, 3, 384), (100, 1152, 128, 8, 640), (33, 1024, 130, 2, 128),
                                       (256, 2176, 33, 3, 512), (17, 256, 128, 8, 1152), (4, 2176, 40, 8, 640),
                                       (8, 4096, 9, 4, 1280)])
def test_tiles(T, d, E, k, I):
    x, wgu, wd, logits = make(T, d, E, k, I, seed=6)
    logits[:, 5] = 9.0
    logits[:, 7] = -9.0
    logits[:20, 2] = 8.0
    logits[20:, 2] = -9.0
    dec = decoder(x, E, k, I, limit=1.25)
    got = dec.forward(x, wgu, wd, logits=logits)
    ids, w = topk64(logits, k)
    assert torch.equal(dec.topk_ids.long(), ids)
    a, b, used = cut(wgu, wd, ids)
    check(got, x, a, b, used, w, limit=1.25)
    again = decoder(x, E, k, I, limit=1.25)
    assert torch.equal(again.forward(x, wgu, wd, logits=logits), got)


@pytest.mark.parametrize("T", [40, 200])
def test_nan_stays_in_its_tokens(T):
    d, E, k, I = 256, 128, 2, 256
    x, wgu, wd, _ = make(T, d, E, k, I, seed=9)
    ids = (torch.arange(T, device=DEV)[:, None] % 3 + torch.tensor([0, 3], device=DEV)).to(torch.int32).contiguous()
    w = torch.full((T, k), 0.5, device=DEV)
    ids[4] = -1
    clean = decoder(x, E, k, I).forward(x, wgu, wd, topk_ids=ids, topk_w=w).clone()
    x[1, 7], x[4] = math.nan, math.inf
    wgu[1][2, 3, 5] = 255                                  # experts 2 and 5: tokens 2, 5, 8, ...
    got = decoder(x, E, k, I).forward(x, wgu, wd, topk_ids=ids, topk_w=w)
    hit = torch.arange(T, device=DEV) % 3 == 2
    hit[1] = True
    assert bool(got[hit].isnan().all()) and torch.equal(got[~hit], clean[~hit]) and not bool(got[4].any())


@pytest.mark.parametrize("T,d,E,k,I", [(1, 256, 16, 4, 128), (8, 256, 16, 8, 256), (16, 256, 3, 2, 128),
                                       (40, 128, 20, 4, 256), (130, 1024, 128, 9, 256)])
def test_activations_keep_sixteen_bits(T, d, E, k, I):
    x, wgu, wd, logits = make(T, d, E, k, I, seed=8)
    got = decoder(x, E, k, I).forward(x, wgu, wd, logits=logits)
    ids, w = topk64(logits, k)
    ref, tol = plain(x, values_of(*wgu), values_of(*wd), ids, w, eps_act=2.0 ** -17)
    assert bool(((got.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("T", [1, 3, 40])
def test_special_scales(T):
    """Byte 255 is NaN for the block's rows alone; byte 0 is 2^-127."""
    d, E, k, I = 384, 3, 1, 256
    x, wgu, wd, _ = make(T, d, E, k, I, seed=4)
    ids = (torch.arange(T, device=DEV)[:, None] % 3).to(torch.int32)
    w = torch.ones((T, 1), device=DEV)
    wd[1][0, 7, 3] = 255                                  # expert 0, row 7
    wd[1][1, 9, :] = 0
    wd[1][1, 9, 7] = 127                                  # the rest is far below that block
    got = decoder(x, E, k, I).forward(x, wgu, wd, topk_ids=ids, topk_w=w)
    first = ids[:, 0] == 0
    assert bool(got[first, 7].isnan().all())
    wd[1][0, 7, 3] = 127
    a, b = values_of(*wgu), values_of(*wd)
    ref = torch.where(got.isnan(), decoder(x, E, k, I).forward(x, wgu, wd, topk_ids=ids, topk_w=w), got)
    check(ref, x, a, b, ids, w)
    assert int(got.isnan().sum()) == int(first.sum())


def test_codes_as_they_are():
    """Every code byte under several scales, one product each: the value read is
    the code's, exactly."""
    d, I = 256, 128
    codes = torch.zeros((1, d, I // 2), dtype=torch.uint8, device=DEV)
    codes[0, :, 0] = torch.arange(256, device=DEV).to(torch.uint8)
    for scale in (127, 100, 131):
        scales = torch.full((1, d, I // 32), scale, dtype=torch.uint8, device=DEV)
        for col in (0, 1):
            # the gate/up product gives a = silu(8) 1 in column `col`, else 0
            gu = torch.zeros((1, 2 * I, d), device=DEV)
            gu[0, col, 0], gu[0, I + col, 1] = 1.0, 1.0
            x = torch.zeros((1, d), device=DEV, dtype=torch.bfloat16)
            x[0, 0], x[0, 1] = 8.0, 1.0
            wgu = B.quantize_mxfp4(gu.bfloat16())
            got = decoder(x, 1, 1, I).forward(x, wgu, (codes, scales), topk_ids=torch.zeros((1, 1), dtype=torch.int32, device=DEV),
                                              topk_w=torch.ones((1, 1), device=DEV))
            act = 8.0 / (1.0 + math.exp(-8.0))
            want = values_of(codes, scales)[0, :, col] * act
            assert bool(((got[0].double() - want).abs() <= 2.0 ** -8 * 1.02 * want.abs()).all())


def test_operator_graph_and_stream():
    T, d, E, k, I = 5, 256, 16, 4, 256
    x, wgu, wd, logits = make(T, d, E, k, I, seed=5)
    dec = decoder(x, E, k, I)
    want = dec.forward(x, wgu, wd, logits=logits).clone()
    got = A.moe_decode(x, logits, wgu[0], wd[0], k, wgu[1], wd[1])
    assert torch.equal(got, want)
    f = torch.compile(lambda *a: A.moe_decode(*a[:4], k, *a[4:]), fullgraph=True, backend="aot_eager")
    assert torch.equal(f(x, logits, wgu[0], wd[0], wgu[1], wd[1]), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = decoder(x, E, k, I)
        assert torch.equal(other.forward(x, wgu, wd, logits=logits).clone(), want)
    side.synchronize()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dec.forward(x, wgu, wd, logits=logits)
    for i in range(4):
        x.mul_(1.5)
        eager = other.forward(x, wgu, wd, logits=logits).clone()
        out.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i


def test_encoding_beyond_one_launch_dimension():
    """2^35 values: 2^32 threads of eight values, more than one dimension of a launch takes."""
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GiB of free GPU memory")
    few = torch.randn((1, 128, 4096), device=DEV).bfloat16()
    q0, s0 = B.quantize_mxfp4(few)
    src = few.expand(64, 128, 4096).reshape(1, 8192, 4096).repeat(1024, 1, 1)
    assert src.numel() == 1 << 35
    q, s = B.quantize_mxfp4(src)
    for got, want in ((q, q0), (s, s0)):
        got = got.view(-1, *want.shape[1:])
        assert all(bool((part == want).all()) for part in got.split(4096))
