"""moe_combine's masked form on the host: what it refuses, and that moe_prompt is
made of the library's calls alone, with the rows that moe_combine's contract
names (no GPU here)."""
import ctypes

import pytest
import torch
from torch._subclasses import FakeTensorMode
from torch.utils._python_dispatch import TorchDispatchMode

from combine_top_route_amd import autograd as A
from combine_top_route_amd import binding as B
from test_mxfp4_grouped_refusals import E, I, P, T, d, k, pytestmark, stub, tensors  # noqa: F401

R = T * k


def call(flags, rows=P(1), out=P(2), logits=P(3), ids=P(4), row_of=P(5), w=P(6)):
    sh = B.make_shape(T, d, E, k, 8)
    sh.flags = flags
    r = B.MoeRouting(logits, ids, w, None, None, row_of, None)
    return B.lib().moe_combine(ctypes.byref(sh), rows, ctypes.byref(r), out, None)


def test_masked_needs_logits_and_ids():
    for bad in (dict(logits=None), dict(ids=None), dict(row_of=None), dict(w=None), dict(rows=None), dict(out=None),
                dict(rows=P(1, 8)), dict(out=P(2, 8))):
        assert call(2, **bad) == 1, bad
    assert call(4) == 1 and call(6) == 1 and call(-1) == 1      # flags that there are none of
    assert B.lib().moe_combine(None, P(1), None, P(2), None) == 1
    # without the flag neither is looked at: the next check fails
    assert call(0, logits=None, ids=None, out=P(2, 8)) == 1 and b"out must be" in B.lib().moe_last_error()


def test_other_calls_refuse_the_flag():
    sh = B.make_shape(T, d, E, k, I)
    sh.flags = B.FLAG_SKIP_MASKED
    n = ctypes.c_size_t()
    r = B.MoeRouting(*[P(9)] * 7)
    assert B.lib().moe_workspace_size(ctypes.byref(sh), B.OP_FORWARD, ctypes.byref(n)) == 1
    assert B.lib().moe_permute(ctypes.byref(sh), P(1), ctypes.byref(r), P(2), None) == 1
    assert B.lib().moe_route(ctypes.byref(sh), ctypes.byref(r), P(1), 1 << 40, None) == 1


def test_binding_refuses_rows_that_are_not_there():
    z, _, r = tensors("cpu")
    for bad in (z(R - 1, d), z(R, d).t(), z(R, 2 * d)[:, ::2], z(R * d), z(R, d).half()):
        with pytest.raises(ValueError, match="rows must be"):
            B.combine(bad, r, T, k)
    for name, t in (("logits", None), ("logits", z(T, E + 1)), ("logits", z(T, E).half()), ("topk_ids", z(T, k))):
        odd = tensors("cpu")[2]
        setattr(odd, name, t)
        with pytest.raises(ValueError, match="logits|topk_ids"):
            B.combine(z(R, d), odd, T, k, skip_masked=True)


def test_prompt_is_made_of_the_librarys_calls(stub, monkeypatch):  # noqa: F811
    """No torch operation computes anything in between, and the combine gets T k rows."""
    monkeypatch.setattr(B, "_ptr", lambda t: None if t is None else 1 << 20)
    rows, ops = [], []
    combine = B.combine
    monkeypatch.setattr(B, "combine", lambda y, *a, **kw: rows.append(tuple(y.shape)) or combine(y, *a, **kw))

    class Log(TorchDispatchMode):
        def __torch_dispatch__(self, f, types, args=(), kwargs=None):
            ops.append(f.overloadpacket.__name__)
            return f(*args, **(kwargs or {}))

    with FakeTensorMode():
        z, w, _ = tensors("cuda:1")
        gu, dn = w(2 * I, d), w(d, I)
        x, lg = z(T, d), z(T, E)
        with Log():
            A.moe_prompt._init_fn(x, lg, gu[0], dn[0], k, gu[1], dn[1])
    assert [n for n, _ in stub] == ["moe_route", "moe_grouped_product", "moe_grouped_product", "moe_combine"]
    assert all(dev == 1 for _, dev in stub)
    assert rows == [(R, d)]
    assert set(ops) <= {"empty", "new_empty", "empty_strided"}, ops
