"""The few-token layer from MXFP4 weights beyond the last-level cache (256 MiB of codes
and more) through the kernels that are not streaming tiles: gate/up with too few
work-groups for those (long rows, few experts), routing for itself and not, and a
down product with I below 512 and few rows an expert."""
import pytest
import torch

from test_gpu_decode import check, topk64
from test_gpu_mxfp4 import cut, decoder, make

pytestmark = pytest.mark.gpu


def served(T, d, E, k, I, seed=0):
    x, wgu, wd, logits = make(T, d, E, k, I, seed)
    dec = decoder(x, E, k, I)
    got = dec.forward(x, wgu, wd, logits=logits).clone()
    ids, w = topk64(logits, k)
    assert torch.equal(dec.topk_ids.long(), ids)
    check(got, x, *cut(wgu, wd, ids), w)
    again = decoder(x, E, k, I)
    again.workspace.fill_(255)
    assert torch.equal(again.forward(x, wgu, wd, logits=logits), got)


@pytest.mark.parametrize("T,d,E,k,I", [(2, 16384, 16, 8, 896), (12, 16384, 16, 8, 896), (40, 16384, 8, 4, 1920),
                                       (5, 14336, 9, 9, 1664)])
def test_gateup_of_long_rows(T, d, E, k, I):
    items = min(T * k, E)
    assert items * (I // 128) < 128 and items * 3 * I * d / 2 > 256 << 20
    served(T, d, E, k, I)


@pytest.mark.parametrize("T,d,E,k,I", [(40, 8192, 128, 8, 256), (20, 16384, 64, 3, 384), (4, 16384, 32, 8, 384)])
def test_down_of_short_rows(T, d, E, k, I):
    items = min(T * k, E)
    assert I < 512 and T * k < 16 * items and items * 3 * I * d / 2 > 256 << 20
    served(T, d, E, k, I)
