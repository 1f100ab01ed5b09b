"""The layer for few tokens (moe_decode) against a plain float64 evaluation.

Tolerances.  The output of a bf16 call is off by: at most one rounding to bf16
of the weighted SwiGLU output (each factor of every product within 2^-8; a
test of its own holds it to 2^-17), that of the result
(2^-8), float32 sums and the hardware exp and reciprocal (both far below).
With s_t = sum over slots and columns of |w a W_down| an output's error is at
most 2^-8 s_t + 2^-8 |out|; float32 calls: the products' sums run over K = d
and I terms in float32, at most (d + I + 64) 2^-24 of the sums of magnitudes,
through SwiGLU (whose slope stays below 1.1 in the gate and |silu| in the up
value).  bound() adds these up from magnitudes computed in float64.
"""
import math

import pytest
import torch

from combine_top_route_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def weights64(w):
    if isinstance(w, torch.Tensor):
        return w.double()
    codes, scales = w
    v = codes.view(torch.float8_e4m3fn).double()
    if scales.dtype == torch.float32:
        return v * scales.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
    return v * torch.exp2(scales.double() - 127.0).repeat_interleave(32, 2)


def topk64(logits, k):
    v, i = torch.sort(logits.double(), dim=1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    none = v == -math.inf
    w = torch.where(none, 0.0, torch.exp(v - v[:, :1]))
    w = torch.where(none, 0.0, w / w.sum(1, keepdim=True))
    return torch.where(none, -1, i), w


def plain(x, wgu, wd, ids, w, limit=0.0, eps_act=2.0 ** -8, eps_out=2.0 ** -8):
    """(out, error bound), float64 [T, d]."""
    x, wgu, wd = x.double(), weights64(wgu), weights64(wd)
    E, two_i, d = wgu.shape
    I = two_i // 2
    lim = limit if limit > 0 else math.inf
    out = torch.zeros_like(x)
    mag = torch.zeros_like(x)
    sums = (d + I + 64) * 2.0 ** -24
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            h = wgu[e] @ x[t]
            dh = sums * (wgu[e].abs() @ x[t].abs())
            g, u = h[:I], h[I:]
            gc, uc = g.clamp(max=lim), u.clamp(-lim, lim)
            a = gc * torch.sigmoid(gc) * uc
            da = 1.1 * dh[:I] * uc.abs() + (gc * torch.sigmoid(gc)).abs() * dh[I:] + 1e-6 * a.abs()
            wj = float(w[t, j])
            out[t] += wj * (wd[e] @ a)
            mag[t] += abs(wj) * (wd[e].abs() @ ((eps_act + sums) * a.abs() + da))
    return out, mag + (eps_out + sums) * out.abs() + 1e-30


def make(T, d, E, k, I, dtype="bf16", weights="native", seed=0, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = DT[dtype]
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    x = (scale * rn(T, d)).to(dt)
    wgu = (rn(E, 2 * I, d) * d ** -0.5).to(dt)
    wd = (rn(E, d, I) * I ** -0.5).to(dt)
    logits = rn(T, E)
    if weights == "fp8_block":
        wgu, wd = B.quantize_fp8(wgu, B.QUANT_WEIGHT), B.quantize_fp8(wd, B.QUANT_WEIGHT)
    elif weights == "mxfp8":
        wgu, wd = B.quantize_mxfp8(wgu, B.QUANT_WEIGHT), B.quantize_mxfp8(wd, B.QUANT_WEIGHT)
    return x, wgu, wd, logits


def decoder(x, E, k, I, weights="native", limit=0.0, max_T=None, logits_dtype=torch.float32):
    T, d = x.shape
    return B.MoeDecoder(max_T or T, d, E, k, I, dtype=x.dtype, logits_dtype=logits_dtype, weights=weights,
                        device=DEV, swiglu_limit=limit)


def check(got, x, wgu, wd, ids, w, limit=0.0):
    eps = (2.0 ** -24 if x.dtype == torch.float32 else 2.0 ** -8)
    ref, tol = plain(x, wgu, wd, ids, w, limit, eps_act=eps, eps_out=eps)
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), f"worst error over bound {float((err / tol).max()):.3g}"


# one token, odd counts, exactly one and just over one column block, up to the
# largest; extents with K tails and partial row tiles; one expert; k = E
CASES = [
    # T, d, E, k, I, dtype, weights
    (1, 256, 16, 4, 128, "bf16", "native"),
    (1, 8, 1, 1, 8, "bf16", "native"),
    (3, 72, 5, 5, 40, "bf16", "native"),
    (16, 200, 7, 3, 104, "bf16", "native"),
    (17, 200, 7, 3, 104, "bf16", "native"),
    (33, 136, 1, 1, 264, "bf16", "native"),
    (64, 264, 3, 2, 72, "bf16", "native"),
    (100, 64, 2, 1, 24, "bf16", "native"),
    (256, 136, 40, 6, 40, "bf16", "native"),
    (5, 1000, 19, 3, 360, "f32", "native"),
    (1, 8, 2, 2, 8, "f32", "native"),
    (16, 40, 9, 9, 24, "f32", "native"),
    (49, 104, 4, 2, 56, "f32", "native"),
    (1, 128, 4, 2, 128, "bf16", "fp8_block"),
    (9, 384, 6, 2, 256, "bf16", "fp8_block"),
    (70, 256, 3, 3, 128, "bf16", "fp8_block"),
    (2, 256, 8, 8, 384, "bf16", "mxfp8"),
    (40, 128, 2, 1, 128, "bf16", "mxfp8"),
    (130, 384, 12, 4, 256, "bf16", "mxfp8"),
    # more slots a token than a wave has lanes; more experts than 128 and 512
    (3, 16, 200, 150, 16, "bf16", "native"),
    (2, 24, 600, 64, 8, "f32", "native"),
    (20, 16, 130, 129, 8, "bf16", "native"),
    # a few tokens with the most slots that are routed inside the first kernel,
    # one more token, and one more slot
    (4, 40, 64, 64, 24, "bf16", "native"),
    (8, 72, 128, 8, 40, "f32", "native"),
    (9, 72, 128, 8, 40, "bf16", "native"),
    (4, 40, 66, 65, 24, "bf16", "native"),
]


@pytest.mark.parametrize("T,d,E,k,I,dtype,weights", CASES)
def test_logits_form(T, d, E, k, I, dtype, weights):
    x, wgu, wd, logits = make(T, d, E, k, I, dtype, weights)
    for lt in (torch.float32, torch.bfloat16):
        lg = logits.to(lt)
        dec = decoder(x, E, k, I, weights, logits_dtype=lt)
        got = dec.forward(x, wgu, wd, logits=lg)
        ids, w = topk64(lg, k)
        assert torch.equal(dec.topk_ids.long(), ids)
        assert float((dec.topk_w.double() - w).abs().max()) <= 1e-6
        check(got, x, wgu, wd, ids, w)


@pytest.mark.parametrize("T,d,E,k,I,dtype,weights", CASES)
def test_ids_form_with_empty_slots_and_repeats(T, d, E, k, I, dtype, weights):
    x, wgu, wd, _ = make(T, d, E, k, I, dtype, weights, seed=1)
    g = torch.Generator().manual_seed(2)
    ids = torch.randint(-2, E + 2, (T, k), generator=g, dtype=torch.int32)   # repeats and ids outside
    w = torch.randn((T, k), generator=g)
    ids[T // 2] = -1                                                         # a row left empty
    w[ids < 0] = float("nan")                                                # an empty slot's weight is not read
    ids, w = ids.to(DEV), w.to(DEV)
    dec = decoder(x, E, k, I, weights, limit=0.75)
    got = dec.forward(x, wgu, wd, topk_ids=ids, topk_w=w)
    check(got, x, wgu, wd, ids, w, limit=0.75)
    assert not bool(got[T // 2].any())
    assert dec.topk_ids is ids and dec.topk_w is w


# weights beyond the last-level cache (256 MiB) take the kernels' non-temporal
# loads: more than 16 tokens, 9 to 16, and 9 to 16 at a larger d
@pytest.mark.parametrize("T,d,E,k,I,dtype,weights", [
    (20, 1024, 48, 3, 1024, "bf16", "native"), (40, 1024, 24, 2, 1032, "f32", "native"),
    (24, 1024, 96, 5, 1024, "bf16", "fp8_block"), (130, 1024, 96, 2, 1024, "bf16", "mxfp8"),
    (12, 1032, 48, 6, 1024, "bf16", "native"), (9, 1024, 30, 8, 1024, "f32", "native"),
    (10, 4096, 16, 8, 1024, "bf16", "native"), (16, 4096, 8, 5, 1024, "f32", "native"),
    (13, 4096, 24, 6, 1024, "bf16", "fp8_block"), (9, 4096, 24, 8, 1024, "bf16", "mxfp8"),
])
def test_weights_past_the_cache(T, d, E, k, I, dtype, weights):
    x, wgu, wd, logits = make(T, d, E, k, I, dtype, weights, seed=3)
    dec = decoder(x, E, k, I, weights)
    got = dec.forward(x, wgu, wd, logits=logits)
    ids, w = topk64(logits, k)
    assert torch.equal(dec.topk_ids.long(), ids)
    used = torch.unique(ids).tolist()                       # the plain form on the experts in use
    remap = torch.full((E,), -1, device=DEV)
    remap[used] = torch.arange(len(used), device=DEV)
    cut = lambda m: m[used] if isinstance(m, torch.Tensor) else tuple(t[used] for t in m)
    check(got, x, cut(wgu), cut(wd), remap[ids], w)


# more experts and rows than 1024 work-groups of 32 rows: gate/up for a few
# rows an expert, then also the down product (8 rows an expert and more), with
# extents that end inside a tile of 32 and an expert with more than 32 rows
@pytest.mark.parametrize("T,d,E,k,I,dtype,weights", [
    (17, 72, 128, 8, 264, "bf16", "native"), (20, 40, 256, 6, 136, "f32", "native"),
    (33, 128, 256, 4, 128, "bf16", "fp8_block"), (20, 256, 256, 6, 128, "bf16", "mxfp8"),
    (130, 1032, 120, 9, 264, "bf16", "native"), (90, 1144, 114, 11, 280, "f32", "native"),
    (101, 1024, 128, 12, 256, "bf16", "fp8_block"), (256, 1152, 128, 5, 256, "bf16", "mxfp8"),
])
def test_wide_row_tiles(T, d, E, k, I, dtype, weights):
    x, wgu, wd, logits = make(T, d, E, k, I, dtype, weights, seed=6)
    logits[: T // 3, 5] = 9.0                                 # one expert with many rows
    logits[:, 7] = -9.0                                       # one that no token selects
    dec = decoder(x, E, k, I, weights)
    got = dec.forward(x, wgu, wd, logits=logits)
    ids, w = topk64(logits, k)
    assert torch.equal(dec.topk_ids.long(), ids)
    check(got, x, wgu, wd, ids, w)


# few experts with many rows each: the tokens of one are split over work-groups
# in blocks of 32, up to and over one work-group per CU, with a last block that
# is short and an expert whose rows fill the first block alone
@pytest.mark.parametrize("T,d,E,k,I,dtype,weights", [
    (200, 136, 30, 4, 40, "f32", "native"), (33, 200, 2, 2, 24, "f32", "native"),
    (256, 24, 3, 2, 136, "bf16", "native"), (255, 520, 9, 3, 88, "bf16", "native"),
    (250, 256, 16, 3, 256, "bf16", "fp8_block"), (65, 384, 1, 1, 128, "bf16", "fp8_block"),
    (250, 128, 20, 2, 256, "bf16", "mxfp8"), (97, 640, 2, 1, 128, "bf16", "mxfp8"),
])
def test_tokens_split(T, d, E, k, I, dtype, weights):
    x, wgu, wd, logits = make(T, d, E, k, I, dtype, weights, seed=7)
    if E > 2:
        logits[:, 2] = -9.0
        logits[:20, 2] = 9.0                                  # an expert with 20 rows
    dec = decoder(x, E, k, I, weights)
    got = dec.forward(x, wgu, wd, logits=logits)
    ids, w = topk64(logits, k)
    assert torch.equal(dec.topk_ids.long(), ids)
    check(got, x, wgu, wd, ids, w)
    assert torch.equal(dec.forward(x, wgu, wd, logits=logits), got)


# bf16 calls keep the activations between the products in two bf16 parts: hi =
# rn(v) leaves |v - hi| <= 2^(e - 8) at |v| >= 2^e, and rounding that rest to 8
# bits errs by half a step of its exponent, at most 2^(e - 17): 2^-17 of v.  So
# an output is off by its own rounding and 2^-17 of the sum of magnitudes.
@pytest.mark.parametrize("T,d,E,k,I,dtype,weights", [
    (1, 256, 16, 4, 128, "bf16", "native"), (4, 264, 12, 8, 200, "bf16", "native"),
    (8, 256, 16, 8, 256, "bf16", "fp8_block"), (12, 136, 40, 3, 72, "bf16", "native"),
    (16, 256, 3, 2, 128, "bf16", "mxfp8"), (40, 128, 20, 4, 256, "bf16", "mxfp8"),
    (200, 264, 5, 2, 136, "bf16", "native"), (130, 1024, 128, 9, 256, "bf16", "fp8_block"),
])
def test_activations_keep_sixteen_bits(T, d, E, k, I, dtype, weights):
    x, wgu, wd, logits = make(T, d, E, k, I, dtype, weights, seed=8)
    dec = decoder(x, E, k, I, weights)
    got = dec.forward(x, wgu, wd, logits=logits)
    ids, w = topk64(logits, k)
    ref, tol = plain(x, wgu, wd, ids, w, eps_act=2.0 ** -17)
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), f"worst error over bound {float((err / tol).max()):.3g}"


def test_masked_logits():
    """-inf logits are empty slots: none left, fewer left than k, ties."""
    T, d, E, k, I = 6, 64, 8, 4, 32
    x, wgu, wd, lg = make(T, d, E, k, I)
    inf = float("inf")
    lg[0] = -inf
    lg[1, 1:] = -inf
    lg[2, :] = -inf
    lg[2, 5:7] = torch.finfo(torch.float32).min    # the type's lowest value is a value
    lg[3] = 0.0
    lg[3, ::2] = -0.0                               # -0 ties with +0: lowest index first
    lg[4, 3] = 200.0
    dec = decoder(x, E, k, I)
    got = dec.forward(x, wgu, wd, logits=lg)
    ids, w = topk64(lg, k)
    assert torch.equal(dec.topk_ids.long(), ids)
    assert dec.topk_ids[0].tolist() == [-1] * 4 and dec.topk_ids[2].tolist() == [5, 6, -1, -1]
    assert dec.topk_ids[3].tolist() == [0, 1, 2, 3]
    check(got, x, wgu, wd, ids, w)
    assert not bool(got[0].any())


@pytest.mark.parametrize("T", [5, 40])
def test_nan_and_infinity_stay_where_they_are(T):
    """A token's NaN reaches its own row alone; an expert's, the tokens that
    chose it; an empty token's row is zero whatever it holds."""
    d, E, k, I = 72, 6, 2, 40
    x, wgu, wd, _ = make(T, d, E, k, I)
    ids = (torch.arange(T, device=DEV)[:, None] % 3 + torch.tensor([0, 3], device=DEV)).to(torch.int32).contiguous()
    w = torch.full((T, k), 0.5, device=DEV)
    ids[4] = -1
    x[1, 7] = float("nan")
    x[4] = float("inf")
    wgu[2, 3, 5] = float("nan")       # experts 2 and 5: tokens 2, 5, 8, ...
    wd[2, 11, 0] = float("inf")
    dec = decoder(x, E, k, I)
    got = dec.forward(x, wgu, wd, topk_ids=ids, topk_w=w)
    hit = torch.arange(T, device=DEV) % 3 == 2
    hit[4] = False
    ok = ~hit
    ok[1] = False
    assert bool(got[1].isnan().all()) and bool(got[hit].isnan().all())
    x1 = torch.where(ok[:, None], x, 0.0)
    ids1 = torch.where(ok[:, None], ids, -1)
    check(torch.where(ok[:, None], got, 0.0), x1, wgu.nan_to_num(0, 0), wd.nan_to_num(0, 0, 0), ids1, w)
    assert not bool(got[4].any())


def test_smaller_batches_leave_the_rows_behind_alone():
    d, E, k, I = 64, 8, 2, 32
    x, wgu, wd, lg = make(40, d, E, k, I)
    dec = decoder(x, E, k, I)
    full = dec.forward(x, wgu, wd, logits=lg).clone()
    ids_full = dec.topk_ids.clone()
    for T in (7, 40, 1, 17):
        part = dec.forward(x[:T], wgu, wd, logits=lg[:T])
        assert part.shape == (T, d) and torch.equal(dec.topk_ids, ids_full[:T])
        ids, w = topk64(lg[:T], k)
        check(part, x[:T], wgu, wd, ids, w)
    dec._out.copy_(full)
    dec.forward(x[:7], wgu, wd, logits=lg[:7])
    assert torch.equal(dec._out[7:], full[7:])


def test_same_as_the_layer_forward():
    """Against moe_forward on the same inputs: both round the activations and
    the result to bf16, so they differ by at most twice the bound."""
    T, d, E, k, I = 24, 256, 8, 2, 128
    x, wgu, wd, lg = make(T, d, E, k, I)
    lg = lg.bfloat16()
    layer = B.MoeLayer(T, d, E, k, I, device=DEV)
    want = layer.forward(x, wgu, wd, logits=lg)
    dec = decoder(x, E, k, I, logits_dtype=torch.bfloat16)
    got = dec.forward(x, wgu, wd, logits=lg)
    assert torch.equal(dec.topk_ids, layer.routing.topk_ids)
    ids, w = topk64(lg, k)
    _, tol = plain(x, wgu, wd, ids, w)
    # the layer also rounds each slot's product before the combine
    assert bool(((got.double() - want.double()).abs() <= 4 * tol).all())


def test_repeatable_and_on_another_stream():
    T, d, E, k, I = 20, 136, 8, 3, 72
    x, wgu, wd, lg = make(T, d, E, k, I)
    dec = decoder(x, E, k, I)
    want = dec.forward(x, wgu, wd, logits=lg).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = dec.forward(x, wgu, wd, logits=lg).clone()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(want, again)


@pytest.mark.parametrize("T", [1, 30])
def test_captured_and_replayed(T):
    d, E, k, I = 128, 8, 2, 64
    x, wgu, wd, lg = make(T, d, E, k, I)
    dec = decoder(x, E, k, I)
    dec.forward(x, wgu, wd, logits=lg)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dec.forward(x, wgu, wd, logits=lg)
    eager = decoder(x, E, k, I)
    for i in range(4):
        x.copy_(make(T, d, E, k, I, seed=10 + i)[0])
        lg.copy_(make(T, d, E, k, I, seed=10 + i)[3])
        dec.workspace.fill_(255)            # nothing is expected in the workspace
        graph.replay()
        want = eager.forward(x, wgu, wd, logits=lg)
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_two_decoders_at_once():
    """Two decoders on two streams at a time, each against its own result alone."""
    cases = [make(24, 136, 8, 3, 72, seed=1), make(3, 264, 6, 2, 104, seed=2)]
    decs = [decoder(cases[0][0], 8, 3, 72), decoder(cases[1][0], 6, 2, 104)]
    want = [d.forward(x, wgu, wd, logits=lg).clone() for d, (x, wgu, wd, lg) in zip(decs, cases)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for d, s, (x, wgu, wd, lg) in zip(decs, streams, cases):
            with torch.cuda.stream(s):
                d.forward(x, wgu, wd, logits=lg)
        torch.cuda.synchronize()
        for d, w in zip(decs, want):
            assert torch.equal(d.out, w)


@pytest.mark.parametrize("T,dtype,weights", [(3, "bf16", "native"), (40, "f32", "native"), (20, "bf16", "fp8_block"),
                                             (2, "bf16", "mxfp8")])
def test_operator(T, dtype, weights):
    from combine_top_route_amd.autograd import moe_decode
    d, E, k, I = 128, 6, 2, 128
    x, wgu, wd, lg = make(T, d, E, k, I, dtype, weights)
    want = decoder(x, E, k, I, weights, limit=0.5).forward(x, wgu, wd, logits=lg)
    args = (wgu, wd, k) if weights == "native" else (wgu[0], wd[0], k, wgu[1], wd[1])
    got = moe_decode(x, lg, *args, swiglu_limit=0.5)
    assert torch.equal(got, want)
    fn = torch.compile(lambda x, lg: moe_decode(x, lg, *args, swiglu_limit=0.5), fullgraph=True, backend="aot_eager")
    assert torch.equal(fn(x, lg), want)
    xr = (x.clone() if weights == "native" else x.float().to(x.dtype)).requires_grad_()
    with pytest.raises(RuntimeError):
        moe_decode(xr, lg, *args).sum().backward()
