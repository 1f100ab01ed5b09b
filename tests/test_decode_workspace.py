"""The few-token layer's workspace: a format that keeps no down products in memory
takes a buffer without room for them, MXFP4 needs the room.  No GPU here: a call
whose workspace is large enough goes on to the next check, which a misaligned
output fails."""
import pytest
import torch

from combine_top_route_amd import binding as B
from test_decode_refusals import P, call, pytestmark, shape, size  # noqa: F401

up = lambda n: -(-n // 256) * 256
LAST_CHECK = b"out must be 16-byte aligned"


def parts(T, d, k, I):
    """Bytes without and of the down products."""
    R = T * k
    return 2 * up(4 * R) + up(4 * R * I), up(4 * R * d)


def reached(**kw):
    """Whether the call passes the workspace's check (else its status is 3)."""
    st = call(out=P(8), **kw)
    assert st == 3 or (st == 1 and LAST_CHECK in B.lib().moe_last_error()), st
    return st == 1


@pytest.mark.parametrize("T,k", [(1, 8), (4, 8), (8, 4)])
@pytest.mark.parametrize("weights", [0, 1, 2])
def test_few_tokens_take_the_small_workspace(T, k, weights):
    small, y = parts(T, 256, k, 128)
    kw = dict(sh=shape(T=T, k=k), weights=weights)
    if weights:
        kw.update(sgu=P(), sd=P())
    assert reached(n=small, **kw) and not reached(n=small - 256, **kw)
    kw = dict(sh=shape(T=T, k=k), weights=3, sgu=P(), sd=P())
    assert reached(n=small + y, **kw) and not reached(n=small + y - 256, **kw)
    assert size(shape(T=T, k=k)) == (0, small + y)


def test_sizes_of_shapes_that_no_coded_weight_has():
    for kw in (dict(dtype=torch.float32), dict(d=264), dict(I=136)):
        s = shape(T=4, k=8, **kw)
        assert size(s) == (0, parts(4, s.d, 8, s.I)[0])


def test_more_tokens_need_all_of_it():
    small, y = parts(9, 256, 4, 128)
    assert size(shape(T=9, k=4)) == (0, small + y)
    for weights in (0, 3):
        sc = dict(sgu=P(), sd=P()) if weights else {}
        kw = dict(sh=shape(T=9, k=4), weights=weights, **sc)
        assert reached(n=small + y, **kw) and not reached(n=small, **kw)
