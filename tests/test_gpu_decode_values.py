"""moe_decode at extreme values: infinite weights, and the ends of the MXFP8
scale range.  Bounds of test_gpu_decode."""
import math

import pytest
import torch

from test_gpu_decode import DEV, decoder, make, plain

pytestmark = pytest.mark.gpu


# the down product in one kernel, through y in its eight-row and other forms,
# split over I and not, with one and two column blocks
@pytest.mark.parametrize("T,d,E,k,I,dtype", [
    (1, 64, 6, 2, 40, "bf16"), (5, 72, 6, 2, 40, "bf16"), (5, 72, 6, 2, 40, "f32"), (12, 72, 6, 2, 40, "bf16"),
    (40, 72, 6, 2, 40, "bf16"), (40, 72, 6, 2, 40, "f32"), (150, 136, 6, 2, 72, "bf16"),
    (200, 1032, 120, 9, 264, "bf16"), (30, 4096, 8, 2, 24, "bf16")])
def test_infinite_down_weight(T, d, E, k, I, dtype):
    """An infinity in W_down meets every token of its expert as the formula has
    it: w a inf, of a's sign, in its row alone; never NaN."""
    x, wgu, wd, _ = make(T, d, E, k, I, dtype, seed=30)
    g = torch.Generator(device=DEV).manual_seed(31)
    ids = torch.rand((T, E), generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32).contiguous()
    ids[0, 0], ids[0, 1:] = 3, -1
    w = torch.rand((T, k), generator=g, device=DEV) + 0.25
    wd[3, 11, 5] = math.inf
    wd[3, 20, I - 1] = -math.inf
    dec = decoder(x, E, k, I)
    got = dec.forward(x, wgu, wd, topk_ids=ids, topk_w=w).double()
    used = torch.unique(ids[ids >= 0]).tolist()
    remap = torch.full((E + 1,), -1, device=DEV)
    remap[used] = torch.arange(len(used), device=DEV)
    ref, tol = plain(x, wgu[used], wd[used], remap[ids.long()], w)
    assert not bool(ref.isnan().any()) and bool(ref[0, 11].isinf())
    hit = ref.isinf()
    assert torch.equal(hit.any(1), (ids == 3).any(1)) and int(hit.sum()) == 2 * int((ids == 3).sum())
    assert torch.equal(torch.where(hit, got, 0.0), torch.where(hit, ref, 0.0))
    assert bool(((got - ref).abs() <= tol)[~hit].all())


def test_infinite_gate_up_weight():
    T, d, E, k, I = 20, 72, 4, 2, 40
    x, wgu, wd, _ = make(T, d, E, k, I, seed=32)
    ids = (torch.arange(T, device=DEV)[:, None] % 2 + torch.tensor([0, 2], device=DEV)).to(torch.int32).contiguous()
    w = torch.full((T, k), 0.5, device=DEV)
    wgu[1, I + 7, 3] = math.inf                     # an up row: a = silu(g) (+-inf)
    wd[1, 5, 7] = 0.0                               # 0 inf: NaN in the formula
    got = decoder(x, E, k, I).forward(x, wgu, wd, topk_ids=ids, topk_w=w).double()
    ref, tol = plain(x, wgu, wd, ids, w)
    assert bool(ref[1, 5].isnan()) and bool(ref[1].isinf().any()) and bool(ref[0].isfinite().all())
    assert torch.equal(got.isnan(), ref.isnan())
    inf = ref.isinf()
    assert torch.equal(torch.where(inf, got, 0.0), torch.where(inf, ref, 0.0))
    ok = ref.isfinite()
    assert bool(((got - ref).abs() <= tol)[ok].all())


# one kernel for the down product, and rows of y; wide tiles of 32 rows
@pytest.mark.parametrize("T,d,E,k,I", [(1, 640, 4, 2, 512), (6, 640, 4, 3, 512), (20, 640, 4, 2, 512),
                                       (40, 640, 128, 8, 512)])
def test_mxfp8_scale_bytes(T, d, E, k, I):
    """Scale bytes from 0 (2^-127) to 240, each block of gate/up's K meeting x of
    the inverse size, and rows of W_down of very different sizes.  A weight that
    is no bfloat16 number (below 2^-126, in steps of 2^-133) is off by half a
    step."""
    g = torch.Generator(device=DEV).manual_seed(33)
    byte = torch.tensor([0, 1, 2, 7, 8, 60, 126, 127, 128, 200, 240], device=DEV)
    codes = lambda *s: (torch.randn(s, generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    kb = byte[torch.arange(d // 32, device=DEV) % len(byte)]
    x = torch.randn((T, d), generator=g, device=DEV) * d ** -0.5 * torch.exp2(120.0 - kb.repeat_interleave(32))
    x = x.bfloat16()
    assert bool(x.isfinite().all())
    wgu = (codes(E, 2 * I, d).view(torch.uint8), kb.to(torch.uint8).expand(E, 2 * I, d // 32).contiguous())
    rows = byte[:9][torch.arange(d, device=DEV) % 9]                        # up to 128: outputs stay finite
    rows = torch.where(torch.arange(d, device=DEV) % 10 == 9, 200, rows)
    wd = (codes(E, d, I).view(torch.uint8), rows.to(torch.uint8)[None, :, None].expand(E, d, I // 32).contiguous())
    ids = torch.rand((T, E), generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32).contiguous()
    w = torch.rand((T, k), generator=g, device=DEV) + 0.25
    got = decoder(x, E, k, I, "mxfp8").forward(x, wgu, wd, topk_ids=ids, topk_w=w).double()
    used = torch.unique(ids).tolist()
    remap = torch.full((E,), -1, device=DEV)
    remap[used] = torch.arange(len(used), device=DEV)
    cut = lambda m: tuple(t[used] for t in m)
    ref, tol = plain(x, cut(wgu), cut(wd), remap[ids.long()], w)
    # what half a step of W_gate_up leaves in h: 2^-134 |x|_1, through SwiGLU and
    # W_down; relative to the sums of magnitudes it is below 2^-134 / 2^-127
    # times the smallest weight that counts, so: the same relative part of each
    h_part = 2.0 ** -134 * x.double().abs().sum(1, keepdim=True)
    amp = torch.zeros_like(ref)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            h = (wgu[0][e].view(torch.float8_e4m3fn).double() * torch.exp2(kb.double() - 127).repeat_interleave(32)) @ x[t].double()
            gg, u = h[:I], h[I:]
            a = gg * torch.sigmoid(gg) * u
            da = h_part[t] * (1.1 * u.abs() + (gg * torch.sigmoid(gg)).abs() + 1.1 * h_part[t])
            m = wd[0][e].view(torch.float8_e4m3fn).double().abs() * torch.exp2(rows.double() - 127)[:, None]
            amp[t] += float(w[t, j]) * (m @ da + 2.0 ** -134 * (a.abs() + da).sum())
    tol = (tol - 1e-30) + amp + 2.0 ** -134                                  # out itself in steps of 2^-133
    err = (got - ref).abs()
    assert bool(got.isfinite().all())
    assert bool((err <= tol).all()), [float((err / tol)[:, rows == b].max()) for b in rows.unique()]
    assert bool((ref.abs().amax(0)[rows == 0] > 0).any())
