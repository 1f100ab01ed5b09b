"""The 8-bit checkpoint with MOE_FLAG_PERSISTENT: the encoding gate/up GEMM has a
persistent form too, with the same results bit for bit."""
import pytest
import torch

import test_gpu_save8 as S8
from combine_top_route_amd import binding as B

pytestmark = pytest.mark.gpu

DEV = S8.DEV


def run(args, T, d, E, k, I, persistent, limit=0.0):
    x, lg, wgu, wd, dout = args
    layer = B.MoeLayer(T, d, E, k, I, logits_dtype=torch.float32, device=DEV, swiglu_limit=limit, save8=True,
                       persistent=persistent)
    layer.saved.fill_(171)
    layer.forward(x, wgu, wd, logits=lg)
    res = dict(out=layer.out, saved=layer.saved)
    return {n: v.clone() for n, v in {**res, **layer.backward(dout, x, wgu, wd)}.items()}


# many tiles a work-group with K and column tails, one K step, one token, an
# expert with one row beside a hot one, wide I, short rows
@pytest.mark.parametrize("T,d,E,k,I,limit", [
    (3001, 2000, 40, 6, 712, 0.0), (500, 64, 12, 3, 40, 0.6), (1, 128, 8, 2, 128, 0.0), (2000, 512, 64, 2, 256, 0.0),
    (700, 136, 2, 1, 648, 0.0), (333, 8, 6, 2, 8, 0.0)])
def test_same_as_the_default_engine(T, d, E, k, I, limit):
    args = S8.layer_inputs(T, d, E, k, I, torch.bfloat16, seed=70)
    if E == 64:
        args[1][:, 5] = 9.0
        args[1][:, 9] = -9.0
        args[1][17, 9] = 10.0
    a = run(args, T, d, E, k, I, True, limit)
    b = run(args, T, d, E, k, I, False, limit)
    used = B.saved8_size(B.make_shape(T, d, E, k, I))
    assert a["saved"].numel() == used
    for n in b:
        assert torch.equal(a[n], b[n]), n
    plain = B.MoeLayer(T, d, E, k, I, logits_dtype=torch.float32, device=DEV, swiglu_limit=limit, persistent=True)
    assert torch.equal(plain.forward(args[0], args[2], args[3], logits=args[1]), a["out"])


def test_the_flag_reaches_every_bf16_gemm():
    from torch.profiler import ProfilerActivity, profile
    T, d, E, k, I = 300, 128, 4, 2, 128
    args = S8.layer_inputs(T, d, E, k, I, torch.bfloat16, seed=71)
    names = {}
    for persistent in (True, False):
        run(args, T, d, E, k, I, persistent)
        torch.cuda.synchronize()
        with profile(activities=[ProfilerActivity.CUDA]) as prof:
            run(args, T, d, E, k, I, persistent)
            torch.cuda.synchronize()
        names[persistent] = [e.name for e in prof.events()]
        count = lambda part: sum(part in n for n in names[persistent])
        want, other = ("persist_kernel", "rows_gemm_kernel") if persistent else ("rows_gemm_kernel", "persist_kernel")
        # gate/up and down forward, their data gradients; with the flag both weight gradients too
        assert count(want) == (6 if persistent else 4) and count(other) == 0, names[persistent]
