"""moe_decode's dispatch: masked logits through each routing form, the gate/up
kernel that routes for itself at four waves and with non-temporal loads.
Against the plain float64 evaluation and bounds of test_gpu_decode."""
import math

import pytest
import torch

from test_gpu_decode import DEV, check, decoder, make, topk64

pytestmark = pytest.mark.gpu


def check_routing(dec, logits, k):
    """Ids exactly; weights: exp within two steps of 2^-23 and its argument
    within one (at most 2^-23 |argument| <= 2^-23 times 104 before it underflows,
    where the weight is below e^-|argument|: 40 steps of the largest), k sums,
    one division."""
    ids, w = topk64(logits, k)
    assert torch.equal(dec.topk_ids.long(), ids)
    assert bool(((dec.topk_w.double() - w).abs() <= (k + 8) * 2.0 ** -23 * w + 40 * 2.0 ** -23 * w * (1 - w) + 1e-37).all())
    return ids, w


def mask(lg, k, dtype):
    """Rows with nothing left, with fewer than k left, with the type's lowest
    value beside the mask, with ties of both zeros; the last row masked too."""
    inf = math.inf
    T, E = lg.shape
    lg = lg.to(dtype)
    lg[0] = -inf
    if T > 1:
        lg[1, : E - k // 2] = -inf
        lg[T - 1] = -inf
    if T > 3:
        lg[2] = -inf
        lg[2, E // 2:E // 2 + 2] = torch.finfo(dtype).min
    if T > 5:
        lg[3] = 0.0
        lg[3, ::2] = -0.0
        lg[4] = -inf
        lg[4, E - 1] = 3.0
    return lg


# routed inside the gate/up kernel by eight and by four waves; by a kernel of its
# own: more than 8 tokens, more work-groups, more than 64 slots a token, than
# 256 slots, than 128 and than 512 experts
MASKED = [
    (6, 64, 16, 4, 32, "bf16", "native"), (8, 72, 64, 8, 136, "bf16", "native"),
    (9, 64, 16, 8, 32, "bf16", "native"), (40, 128, 16, 8, 128, "bf16", "fp8_block"),
    (7, 72, 64, 8, 328, "f32", "native"), (3, 64, 200, 150, 32, "bf16", "native"),
    (8, 64, 60, 40, 24, "f32", "native"), (6, 128, 130, 5, 128, "bf16", "mxfp8"),
    (2, 24, 600, 300, 16, "bf16", "native"), (12, 16, 130, 129, 8, "f32", "native"),
]


@pytest.mark.parametrize("ldtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d,E,k,I,dtype,weights", MASKED)
def test_masked_logits(T, d, E, k, I, dtype, weights, ldtype):
    x, wgu, wd, lg = make(T, d, E, k, I, dtype, weights, seed=20)
    lg = mask(lg, k, ldtype)
    dec = decoder(x, E, k, I, weights, logits_dtype=ldtype)
    dec.workspace.fill_(255)
    got = dec.forward(x, wgu, wd, logits=lg)
    ids, w = check_routing(dec, lg, k)
    check(got, x, wgu, wd, ids, w)
    assert not bool(got[0].any()) and bool((dec.topk_ids[0] == -1).all()) and not bool(dec.topk_w[0].any())


# 513 to 1024 work-groups of 16 rows: the gate/up kernel routes with four waves;
# weights above 256 MiB with at most 512 and with more work-groups
INLINE = [
    (2, 72, 64, 8, 640, "f32", "native"), (2, 72, 64, 8, 640, "bf16", "native"),
    (2, 128, 64, 8, 640, "bf16", "fp8_block"), (2, 256, 64, 8, 640, "bf16", "mxfp8"),
    (8, 136, 20, 5, 520, "bf16", "native"), (1, 8, 128, 64, 208, "bf16", "native"),
    (2, 4096, 20, 8, 768, "bf16", "native"), (2, 8192, 20, 8, 512, "bf16", "native"),
    (3, 4096, 16, 5, 720, "f32", "native"), (2, 8192, 17, 8, 1024, "bf16", "fp8_block"),
    (2, 8192, 17, 8, 1024, "bf16", "mxfp8"), (8, 1032, 64, 8, 696, "bf16", "native"),
]


@pytest.mark.parametrize("T,d,E,k,I,dtype,weights", INLINE)
def test_routed_inside(T, d, E, k, I, dtype, weights):
    x, wgu, wd, lg = make(T, d, E, k, I, dtype, weights, seed=21)
    lg[T - 1, : E - k + 1] = -math.inf                 # one slot of the last token stays empty
    dec = decoder(x, E, k, I, weights)
    dec.workspace.fill_(255)
    got = dec.forward(x, wgu, wd, logits=lg).clone()
    ids, w = check_routing(dec, lg, k)
    used = torch.unique(ids[ids >= 0]).tolist()
    remap = torch.full((E + 1,), -1, device=DEV)
    remap[used] = torch.arange(len(used), device=DEV)
    cut = lambda m: m[used] if isinstance(m, torch.Tensor) else tuple(t[used] for t in m)
    check(got, x, cut(wgu), cut(wd), remap[ids], w)
    # the same slots given as ids, with one of them named twice
    gid, gw = dec.topk_ids.clone(), dec.topk_w.clone()
    again = dec.forward(x, wgu, wd, topk_ids=gid, topk_w=gw)
    assert torch.equal(again, got)
    if k > 1:
        gid[0, 1] = gid[0, 0]
        check(dec.forward(x, wgu, wd, topk_ids=gid, topk_w=gw), x, cut(wgu), cut(wd), remap[gid.long()], gw)


@pytest.mark.parametrize("T", [1, 7, 12, 40])
def test_one_decoder_for_layers_in_a_row(T):
    """The decoder's own output as the next layer's x."""
    d, E, k, I = 136, 12, 3, 72
    layers = [make(T, d, E, k, I, seed=90 + i) for i in range(4)]
    one = decoder(layers[0][0], E, k, I)
    h = g = layers[0][0]
    for _, wgu, wd, lg in layers:
        h = one.forward(h, wgu, wd, logits=lg)
        g = decoder(g, E, k, I).forward(g.clone(), wgu, wd, logits=lg)
        assert torch.equal(h, g)
    assert bool(g.any())
