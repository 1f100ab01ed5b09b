"""Offsets that go back and forth between nothing and every row, at the size where
the tiles that they count pass 32 bits: the products reach y's rows alone, and
hold what an expert that those offsets name makes of them."""
import pytest
import torch

from combine_top_route_amd import binding as B
from test_gpu_grouped import DEV, weight

pytestmark = pytest.mark.gpu


def test_tiles_beyond_32_bits():
    """512 of 1024 experts claim all 2^27 rows: 2^29 row tiles of 128, by 4 column
    tiles.  All experts hold the same matrix, so whichever makes a row, its result
    is that of one expert alone."""
    T, k, E, N, K = 1 << 17, 1024, 1024, 1024, 128
    R = T * k
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 160 GiB of free GPU memory")
    assert (E // 2) * (R // 128) * (N // 256) >= 1 << 31
    x = torch.randn((T, K), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).bfloat16()
    one = weight(1, N, K, 2)
    all_of = tuple(t.expand(E, -1, -1).contiguous() for t in one)
    i32 = dict(dtype=torch.int32, device=DEV)
    rows = lambda n: B.Routing(*[None] * 5, src_of=torch.arange(n, **i32))
    alone = rows(T)
    alone.offsets = torch.tensor([0, T], **i32)
    want = B.grouped_product(x, one, alone, T, 1, swiglu=True)
    odd = rows(R)
    odd.offsets = (torch.arange(E + 1, **i32) % 2) * R
    buf = torch.full((R + 64, N // 2), 5.0, dtype=torch.bfloat16, device=DEV)
    got = B.grouped_product(x, all_of, odd, T, k, swiglu=True, out=buf[:R])
    for part, ref in zip(got.view(T, k, N // 2).split(1 << 11), want.split(1 << 11)):
        assert bool((part == ref[:, None]).all())
    assert bool((buf[R:] == 5).all())
