"""The fused MoE layer as PyTorch operators with autograd.

The pages' integration registers the layer's backward as a custom operator
so that the compiler accepts the tensors the forward saves, and runs the
layer under activation checkpointing ("Mario/overlap moe kernel
integration", overview and commits on the custom autograd ops;
"Prime Intellect added the missing backward pass to DeepSeek's fused MoE
kernel ...").  Here:

* ``ctr_moe::moe_fwd`` and ``ctr_moe::moe_bwd`` are ``torch.library`` custom
  operators over ``moe_forward`` / ``moe_backward`` of the C ABI, with fake
  (shape-only) implementations, so ``torch.compile(fullgraph=True)`` traces
  through them without graph breaks;
* ``moe_fwd`` carries an autograd formula that calls ``moe_bwd``;
* ``recompute=True`` keeps nothing from the forward: the backward reruns the
  gate/up GEMM from x (``moe_backward`` with ``saved == NULL``).

Beside the layer: ``moe_fwd8`` / ``moe_bwd8`` (``save8=True``: the activations
kept in 8 bits), ``router_fwd`` / ``router_bwd`` (the projection that makes the
logits; ``router`` and, with the layer, ``moe_block``), and ``moe_decode`` (the
layer for at most 256 tokens, without a gradient), ``moe_prompt`` (the layer for
more, from MXFP4 weights), ``norm_fwd`` / ``norm_bwd``
(the norms before and after the block with its gate and residual scale;
``norm_residual`` and, around the block, ``moe_residual_block``).

Every call allocates its outputs and workspace from torch's caching
allocator on the inputs' device and enqueues on torch's current stream.
Routing comes from router logits; the gradient reaches them through the
renormalised top-k softmax.
"""
from __future__ import annotations

import ctypes

import torch
from torch import Tensor

from . import binding as B

_NS = "ctr_moe"


_FLOATS = (torch.float32, torch.bfloat16)


def _require(ok: bool, msg: str):
    if not ok:
        raise ValueError(msg)


def _check_layer_args(x: Tensor, logits: Tensor, w_gate_up: Tensor, w_down: Tensor, k: int,
                      precision: str):
    """Shapes, dtypes and contiguity of the layer's inputs, checked before
    anything is launched: x [T,d], logits [T,E], w_gate_up [E,2I,d],
    w_down [E,d,I], 1 <= k <= E."""
    _require(x.dim() == 2, f"x must be [T, d], got {tuple(x.shape)}")
    T, d = x.shape
    _require(w_gate_up.dim() == 3 and w_gate_up.shape[2] == d and w_gate_up.shape[1] % 2 == 0,
             f"w_gate_up must be [E, 2I, d={d}], got {tuple(w_gate_up.shape)}")
    E, two_i, _ = w_gate_up.shape
    _require(tuple(w_down.shape) == (E, d, two_i // 2),
             f"w_down must be [E={E}, d={d}, I={two_i // 2}], got {tuple(w_down.shape)}")
    _require(tuple(logits.shape) == (T, E), f"logits must be [T={T}, E={E}], got {tuple(logits.shape)}")
    _require(1 <= k <= E, f"k={k} outside [1, E={E}]")
    _require(precision in B._PREC, f"precision {precision!r} unknown")
    _require(x.dtype in _FLOATS and w_gate_up.dtype == x.dtype and w_down.dtype == x.dtype,
             f"x and both weights need one dtype of {_FLOATS}, got {x.dtype}, {w_gate_up.dtype}, "
             f"{w_down.dtype}")
    _require(logits.dtype in _FLOATS, f"logits dtype {logits.dtype} not in {_FLOATS}")
    for name, t in (("x", x), ("logits", logits), ("w_gate_up", w_gate_up), ("w_down", w_down)):
        _require(t.is_contiguous(), f"{name} must be contiguous")


def _check_devices(**tensors):
    """Every tensor on the first one's GPU (checked last, after the shapes)."""
    dev = next(iter(tensors.values())).device
    for name, t in tensors.items():
        _require(t.device.type == "cuda" and t.device == dev, f"{name} is on {t.device}; every tensor "
                 f"must be on one GPU ({dev})")


def _check_backward_args(dout: Tensor, x: Tensor, saved: Tensor, routing, k: int, precision: str):
    """dout [T,d] in x's dtype, `saved` empty or of the forward's size, and the
    routing tensors the forward returned, on x's device."""
    T, d = x.shape
    _require(tuple(dout.shape) == (T, d) and dout.dtype == x.dtype,
             f"dout must be [T={T}, d={d}] {x.dtype}, got {tuple(dout.shape)} {dout.dtype}")
    ids, w, counts, offsets, row_of, src_of = routing
    E = counts.numel()
    for name, t, shape, dt in (("topk_ids", ids, (T, k), torch.int32), ("topk_w", w, (T, k), torch.float32),
                               ("counts", counts, (E,), torch.int32), ("offsets", offsets, (E + 1,), torch.int32),
                               ("row_of", row_of, (T * k,), torch.int32), ("src_of", src_of, (T * k,), torch.int32),
                               ("saved", saved, (saved.numel(),), torch.uint8)):
        _require(tuple(t.shape) == shape and t.dtype == dt, f"{name} must be {shape} {dt}, got "
                 f"{tuple(t.shape)} {t.dtype}")
        _require(t.is_contiguous(), f"{name} must be contiguous")


def _dense(grad: Tensor) -> Tensor:
    """A gradient as the library takes it: contiguous and 16-byte aligned.  What
    autograd hands over may be a slice of a larger gradient at any element."""
    grad = grad.contiguous()
    return grad if grad.data_ptr() % 16 == 0 else grad.clone()


def _shape(x: Tensor, logits: Tensor, w_gate_up: Tensor, k: int, precision: str, swiglu_limit: float = 0.0):
    T, d = x.shape
    E, two_i, _ = w_gate_up.shape
    return B.make_shape(T, d, E, k, two_i // 2, x.dtype, logits.dtype, precision, swiglu_limit)


def _workspace(shape, op, device) -> Tensor:
    return torch.empty(B.workspace_size(shape, op), dtype=torch.uint8, device=device)


def _routing_empty(T, E, k, device):
    i32 = dict(dtype=torch.int32, device=device)
    return (torch.empty((T, k), **i32), torch.empty((T, k), dtype=torch.float32, device=device),
            torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T * k, **i32),
            torch.empty(T * k, **i32))


@torch.library.custom_op(f"{_NS}::moe_fwd", mutates_args=())
def moe_fwd(x: Tensor, logits: Tensor, w_gate_up: Tensor, w_down: Tensor, k: int, precision: str,
            save: bool, swiglu_limit: float = 0.0
            ) -> tuple[Tensor, Tensor, Tensor, Tensor, Tensor, Tensor, Tensor, Tensor]:
    """Layer forward.  Returns (out [T,d], saved (uint8; empty unless save),
    topk_ids, topk_w, counts, offsets, row_of, src_of).  swiglu_limit > 0:
    the clamped SwiGLU."""
    _check_layer_args(x, logits, w_gate_up, w_down, k, precision)
    _check_devices(x=x, logits=logits, w_gate_up=w_gate_up, w_down=w_down)
    shape = _shape(x, logits, w_gate_up, k, precision, swiglu_limit)
    T, d = x.shape
    E = w_gate_up.shape[0]
    dev = x.device
    with B._on(dev):
        out = torch.empty((T, d), dtype=x.dtype, device=dev)
        saved = torch.empty(B.saved_size(shape) if save else 0, dtype=torch.uint8, device=dev)
        rt = _routing_empty(T, E, k, dev)
        r = B.Routing(*rt, logits=logits)
        cr = r.c()
        ws = _workspace(shape, B.OP_FORWARD, dev)
        B._check("moe_forward", B.lib().moe_forward(
            ctypes.byref(shape), B._ptr(x), ctypes.byref(cr), B._ptr(w_gate_up), B._ptr(w_down), B._ptr(out),
            B._ptr(saved) if save else None, B._ptr(ws), ws.numel(), B._stream(dev)))
    return (out, saved) + rt


@moe_fwd.register_fake
def _(x, logits, w_gate_up, w_down, k, precision, save, swiglu_limit=0.0):
    T, d = x.shape
    E = w_gate_up.shape[0]
    shape = _shape(x, logits, w_gate_up, k, precision, swiglu_limit)
    n = B.saved_size(shape) if save else 0
    i32 = dict(dtype=torch.int32)
    return (x.new_empty((T, d)), x.new_empty((n,), dtype=torch.uint8), x.new_empty((T, k), **i32),
            x.new_empty((T, k), dtype=torch.float32), x.new_empty((E,), **i32),
            x.new_empty((E + 1,), **i32), x.new_empty((T * k,), **i32), x.new_empty((T * k,), **i32))


@torch.library.custom_op(f"{_NS}::moe_bwd", mutates_args=())
def moe_bwd(dout: Tensor, x: Tensor, logits: Tensor, w_gate_up: Tensor, w_down: Tensor, saved: Tensor,
            topk_ids: Tensor, topk_w: Tensor, counts: Tensor, offsets: Tensor, row_of: Tensor,
            src_of: Tensor, k: int, precision: str, swiglu_limit: float = 0.0
            ) -> tuple[Tensor, Tensor, Tensor, Tensor]:
    """Layer backward: (dx, dlogits, dw_gate_up, dw_down).  An empty `saved`
    selects recomputation."""
    _check_layer_args(x, logits, w_gate_up, w_down, k, precision)
    dout = _dense(dout)
    _check_backward_args(dout, x, saved, (topk_ids, topk_w, counts, offsets, row_of, src_of), k, precision)
    shape = _shape(x, logits, w_gate_up, k, precision, swiglu_limit)
    _require(saved.numel() in (0, B.saved_size(shape)),
             f"saved holds {saved.numel()} bytes, expected 0 or {B.saved_size(shape)}")
    _check_devices(x=x, dout=dout, logits=logits, w_gate_up=w_gate_up, w_down=w_down, saved=saved,
                   topk_ids=topk_ids, topk_w=topk_w, counts=counts, offsets=offsets, row_of=row_of,
                   src_of=src_of)
    T, d = x.shape
    E, two_i, _ = w_gate_up.shape
    dev = x.device
    recompute = saved.numel() == 0
    with B._on(dev):
        dx = torch.empty_like(x)
        dlogits = torch.empty_like(logits)
        dwgu = torch.empty_like(w_gate_up)
        dwd = torch.empty_like(w_down)
        d_topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
        r = B.Routing(topk_ids, topk_w, counts, offsets, row_of, src_of, logits=logits)
        cr = r.c()
        ws = _workspace(shape, B.OP_BACKWARD_RECOMPUTE if recompute else B.OP_BACKWARD, dev)
        B._check("moe_backward", B.lib().moe_backward(
            ctypes.byref(shape), B._ptr(dout), B._ptr(x), ctypes.byref(cr), B._ptr(w_gate_up), B._ptr(w_down),
            None if recompute else B._ptr(saved), B._ptr(dx), B._ptr(dwgu), B._ptr(dwd), B._ptr(d_topk_w),
            B._ptr(dlogits), B._ptr(ws), ws.numel(), B._stream(dev)))
    return dx, dlogits, dwgu, dwd


@moe_bwd.register_fake
def _(dout, x, logits, w_gate_up, w_down, saved, topk_ids, topk_w, counts, offsets, row_of, src_of,
      k, precision, swiglu_limit=0.0):
    return (torch.empty_like(x), torch.empty_like(logits), torch.empty_like(w_gate_up),
            torch.empty_like(w_down))


def _setup_context(ctx, inputs, output):
    x, logits, w_gate_up, w_down, k, precision, save, swiglu_limit = inputs
    ctx.save_for_backward(x, logits, w_gate_up, w_down, *output[1:])
    ctx.k, ctx.precision, ctx.swiglu_limit = k, precision, swiglu_limit


def _backward(ctx, dout, *unused):
    x, logits, w_gate_up, w_down, saved, ids, w, counts, offsets, row_of, src_of = ctx.saved_tensors
    dx, dlogits, dwgu, dwd = moe_bwd(dout, x, logits, w_gate_up, w_down, saved, ids, w, counts, offsets,
                                     row_of, src_of, ctx.k, ctx.precision, ctx.swiglu_limit)
    return dx, dlogits, dwgu, dwd, None, None, None, None


moe_fwd.register_autograd(_backward, setup_context=_setup_context)


# The same pair with the 8-bit activation checkpoint (moe_forward8 and
# moe_backward8): `saved` holds H as e4m3 codes and scale bytes.
@torch.library.custom_op(f"{_NS}::moe_fwd8", mutates_args=())
def moe_fwd8(x: Tensor, logits: Tensor, w_gate_up: Tensor, w_down: Tensor, k: int, swiglu_limit: float = 0.0
             ) -> tuple[Tensor, Tensor, Tensor, Tensor, Tensor, Tensor, Tensor, Tensor]:
    """Layer forward.  Returns (out [T,d], saved8 (uint8), topk_ids, topk_w,
    counts, offsets, row_of, src_of)."""
    _check_layer_args(x, logits, w_gate_up, w_down, k, "native")
    _check_devices(x=x, logits=logits, w_gate_up=w_gate_up, w_down=w_down)
    shape = _shape(x, logits, w_gate_up, k, "native", swiglu_limit)
    T, d = x.shape
    E = w_gate_up.shape[0]
    dev = x.device
    with B._on(dev):
        out = torch.empty((T, d), dtype=x.dtype, device=dev)
        saved = torch.empty(B.saved8_size(shape), dtype=torch.uint8, device=dev)
        rt = _routing_empty(T, E, k, dev)
        cr = B.Routing(*rt, logits=logits).c()
        ws = torch.empty(B.workspace8_size(shape, B.OP_FORWARD), dtype=torch.uint8, device=dev)
        B._check("moe_forward8", B.lib().moe_forward8(
            ctypes.byref(shape), B._ptr(x), ctypes.byref(cr), B._ptr(w_gate_up), B._ptr(w_down), B._ptr(out),
            B._ptr(saved), B._ptr(ws), ws.numel(), B._stream(dev)))
    return (out, saved) + rt


@moe_fwd8.register_fake
def _(x, logits, w_gate_up, w_down, k, swiglu_limit=0.0):
    T, d = x.shape
    E = w_gate_up.shape[0]
    n = B.saved8_size(_shape(x, logits, w_gate_up, k, "native", swiglu_limit))
    i32 = dict(dtype=torch.int32)
    return (x.new_empty((T, d)), x.new_empty((n,), dtype=torch.uint8), x.new_empty((T, k), **i32),
            x.new_empty((T, k), dtype=torch.float32), x.new_empty((E,), **i32),
            x.new_empty((E + 1,), **i32), x.new_empty((T * k,), **i32), x.new_empty((T * k,), **i32))


@torch.library.custom_op(f"{_NS}::moe_bwd8", mutates_args=())
def moe_bwd8(dout: Tensor, x: Tensor, logits: Tensor, w_gate_up: Tensor, w_down: Tensor, saved: Tensor,
             topk_ids: Tensor, topk_w: Tensor, counts: Tensor, offsets: Tensor, row_of: Tensor,
             src_of: Tensor, k: int, swiglu_limit: float = 0.0) -> tuple[Tensor, Tensor, Tensor, Tensor]:
    """Layer backward from the 8-bit checkpoint: (dx, dlogits, dw_gate_up,
    dw_down)."""
    _check_layer_args(x, logits, w_gate_up, w_down, k, "native")
    dout = _dense(dout)
    _check_backward_args(dout, x, saved, (topk_ids, topk_w, counts, offsets, row_of, src_of), k, "native")
    shape = _shape(x, logits, w_gate_up, k, "native", swiglu_limit)
    _require(saved.numel() == B.saved8_size(shape),
             f"saved holds {saved.numel()} bytes, expected {B.saved8_size(shape)}")
    _check_devices(x=x, dout=dout, logits=logits, w_gate_up=w_gate_up, w_down=w_down, saved=saved,
                   topk_ids=topk_ids, topk_w=topk_w, counts=counts, offsets=offsets, row_of=row_of,
                   src_of=src_of)
    T, d = x.shape
    dev = x.device
    with B._on(dev):
        dx = torch.empty_like(x)
        dlogits = torch.empty_like(logits)
        dwgu = torch.empty_like(w_gate_up)
        dwd = torch.empty_like(w_down)
        d_topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
        cr = B.Routing(topk_ids, topk_w, counts, offsets, row_of, src_of, logits=logits).c()
        ws = torch.empty(B.workspace8_size(shape, B.OP_BACKWARD), dtype=torch.uint8, device=dev)
        B._check("moe_backward8", B.lib().moe_backward8(
            ctypes.byref(shape), B._ptr(dout), B._ptr(x), ctypes.byref(cr), B._ptr(w_gate_up), B._ptr(w_down),
            B._ptr(saved), B._ptr(dx), B._ptr(dwgu), B._ptr(dwd), B._ptr(d_topk_w), B._ptr(dlogits), B._ptr(ws),
            ws.numel(), B._stream(dev)))
    return dx, dlogits, dwgu, dwd


@moe_bwd8.register_fake
def _(dout, x, logits, w_gate_up, w_down, saved, topk_ids, topk_w, counts, offsets, row_of, src_of, k,
      swiglu_limit=0.0):
    return (torch.empty_like(x), torch.empty_like(logits), torch.empty_like(w_gate_up),
            torch.empty_like(w_down))


def _setup_context8(ctx, inputs, output):
    x, logits, w_gate_up, w_down, k, swiglu_limit = inputs
    ctx.save_for_backward(x, logits, w_gate_up, w_down, *output[1:])
    ctx.k, ctx.swiglu_limit = k, swiglu_limit


def _backward8(ctx, dout, *unused):
    x, logits, w_gate_up, w_down, saved, ids, w, counts, offsets, row_of, src_of = ctx.saved_tensors
    return moe_bwd8(dout, x, logits, w_gate_up, w_down, saved, ids, w, counts, offsets, row_of, src_of, ctx.k,
                    ctx.swiglu_limit) + (None, None)


moe_fwd8.register_autograd(_backward8, setup_context=_setup_context8)


# ---------------------------------------------------------------- few tokens
def _check_decode_args(x, logits, w_gate_up, w_down, k, s_gate_up, s_down) -> str:
    """Shapes and dtypes of moe_decode; returns the weights' format."""
    # two e2m1 codes to a byte
    per = 2 if s_gate_up is not None and x.dim() == 2 and w_gate_up.shape[-1] * 2 == x.shape[1] else 1
    _require(x.dim() == 2 and w_gate_up.dim() == 3 and w_gate_up.shape[2] * per == x.shape[1]
             and w_gate_up.shape[1] % 2 == 0,
             f"x must be [T, d] and w_gate_up [E, 2I, d], got {tuple(x.shape)} and {tuple(w_gate_up.shape)}")
    T, d = x.shape
    E, two_i, _ = w_gate_up.shape
    I = two_i // 2
    _require(tuple(w_down.shape) == (E, d, I // per),
             f"w_down must be [E={E}, d={d}, I={I}], got {tuple(w_down.shape)}" + " of two codes a byte" * (per - 1))
    _require(tuple(logits.shape) == (T, E) and logits.dtype in _FLOATS,
             f"logits must be [T={T}, E={E}] of one of {_FLOATS}, got {tuple(logits.shape)} {logits.dtype}")
    _require(1 <= k <= E, f"k={k} outside [1, E={E}]")
    _require(x.dtype in _FLOATS, f"x dtype {x.dtype} not in {_FLOATS}")
    _require((s_gate_up is None) == (s_down is None), "give the scales of both weights or of neither")
    tensors = [("x", x), ("logits", logits), ("w_gate_up", w_gate_up), ("w_down", w_down)]
    if s_gate_up is None:
        fmt, dt = "native", x.dtype
    else:
        fmt, dt = ("mxfp4" if per == 2 else "fp8_block" if s_gate_up.dtype == torch.float32 else "mxfp8"), torch.uint8
        _require(d % 128 == 0 and I % 128 == 0, f"coded weights need d and I multiples of 128, got {d} and {I}")
        shapes = (((E, two_i // 128, d // 128), (E, d // 128, I // 128)) if fmt == "fp8_block"
                  else ((E, two_i, d // 32), (E, d, I // 32)))
        sdt = torch.float32 if fmt == "fp8_block" else torch.uint8
        for name, t, sh in (("s_gate_up", s_gate_up, shapes[0]), ("s_down", s_down, shapes[1])):
            _require(tuple(t.shape) == sh and t.dtype == sdt, f"{name} must be {sh} {sdt}, got {tuple(t.shape)} {t.dtype}")
            tensors.append((name, t))
    _require(w_gate_up.dtype == dt and w_down.dtype == dt,
             f"the weights must be {dt}, got {w_gate_up.dtype}, {w_down.dtype}")
    for name, t in tensors:
        _require(t.is_contiguous(), f"{name} must be contiguous")
    return fmt


@torch.library.custom_op(f"{_NS}::moe_decode", mutates_args=())
def moe_decode(x: Tensor, logits: Tensor, w_gate_up: Tensor, w_down: Tensor, k: int,
               s_gate_up: Tensor | None = None, s_down: Tensor | None = None, swiglu_limit: float = 0.0) -> Tensor:
    """The layer for at most 256 tokens (binding.MoeDecoder as one operator that
    allocates its output and workspace): out [T,d].  With s_gate_up and s_down
    the weights are e4m3 codes, their scales float32 per 128x128 block or E8M0
    bytes per 32 columns, or pairs of e2m1 codes ([E, 2I, d/2] and [E, d, I/2])
    with E8M0 bytes.  No gradient."""
    fmt = _check_decode_args(x, logits, w_gate_up, w_down, k, s_gate_up, s_down)
    tensors = dict(x=x, logits=logits, w_gate_up=w_gate_up, w_down=w_down)
    if fmt != "native":
        tensors.update(s_gate_up=s_gate_up, s_down=s_down)
    _check_devices(**tensors)
    E, two_i, _ = w_gate_up.shape
    with B._on(x.device):
        dec = B.MoeDecoder(x.shape[0], x.shape[1], E, k, two_i // 2, x.dtype, logits.dtype, fmt, x.device, swiglu_limit)
        pair = (lambda w, s: w) if fmt == "native" else (lambda w, s: (w, s))
        return dec.forward(x, pair(w_gate_up, s_gate_up), pair(w_down, s_down), logits=logits)


@moe_decode.register_fake
def _(x, logits, w_gate_up, w_down, k, s_gate_up=None, s_down=None, swiglu_limit=0.0):
    return torch.empty_like(x)


@torch.library.custom_op(f"{_NS}::moe_prompt", mutates_args=())
def moe_prompt(x: Tensor, logits: Tensor, w_gate_up: Tensor, w_down: Tensor, k: int, s_gate_up: Tensor,
               s_down: Tensor, swiglu_limit: float = 0.0) -> Tensor:
    """The layer for any number of tokens from the MXFP4 weights that moe_decode
    takes: routing, the two grouped products and the combine; out [T,d].  bf16
    x; the activations and each slot's product are rounded to bf16 in between, as
    in moe_forward.  A masked expert (a logit of -inf) adds nothing, so a token of
    masked experts alone gets zeros.  No gradient."""
    fmt = _check_decode_args(x, logits, w_gate_up, w_down, k, s_gate_up, s_down)
    _require(fmt == "mxfp4" and x.dtype == torch.bfloat16, "moe_prompt takes bf16 x and MXFP4 weights")
    _check_devices(x=x, logits=logits, w_gate_up=w_gate_up, w_down=w_down, s_gate_up=s_gate_up, s_down=s_down)
    T = x.shape[0]
    with B._on(x.device):
        r = B.route(logits, k)
        a = B.grouped_product(x, (w_gate_up, s_gate_up), r, T, k, swiglu=True, swiglu_limit=swiglu_limit)
        y = B.grouped_product(a, (w_down, s_down), r, T, k, gather=False)
        return B.combine(y, r, T, k, skip_masked=True)


@moe_prompt.register_fake
def _(x, logits, w_gate_up, w_down, k, s_gate_up, s_down, swiglu_limit=0.0):
    return torch.empty_like(x)


def moe_layer(x: Tensor, logits: Tensor, w_gate_up: Tensor, w_down: Tensor, k: int,
              precision: str = "native", recompute: bool = False, swiglu_limit: float = 0.0,
              save8: bool = False) -> Tensor:
    """out [T,d] of the layer, differentiable in x, logits and both weights.
    recompute=True: activation checkpointing inside the operator (nothing
    kept between forward and backward but the routing).  swiglu_limit > 0:
    the clamped SwiGLU with that limit.  save8=True (precision "native"): the
    activations are kept in 8 bits between forward and backward.

    In a HIP graph, capture forward and backward on leaves of the graph's own
    (t.detach().requires_grad_()): a leaf that an eager autograd graph still
    holds takes its gradient on the stream it was first used on, and torch
    ends the capture, or the process, when that stream is drawn in."""
    for name, t in (("x", x), ("logits", logits), ("w_gate_up", w_gate_up), ("w_down", w_down)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if save8:
        _require(not recompute, "save8 keeps a checkpoint, recompute keeps none: give one of them")
        _require(precision == "native", f"save8 needs precision 'native', got {precision!r}")
        return moe_fwd8(x, logits, w_gate_up, w_down, k, swiglu_limit)[0]
    return moe_fwd(x, logits, w_gate_up, w_down, k, precision, not recompute, swiglu_limit)[0]


# ------------------------------------------------------------------ router
def _check_router_args(x: Tensor, w_router: Tensor, logits_dtype: torch.dtype):
    """x [T,d] and w_router [E,d], contiguous, of one float type."""
    _require(x.dim() == 2 and w_router.dim() == 2 and w_router.shape[1] == x.shape[1],
             f"x must be [T, d] and w_router [E, d], got {tuple(x.shape)} and {tuple(w_router.shape)}")
    _require(x.dtype in _FLOATS and w_router.dtype == x.dtype,
             f"x and w_router need one dtype of {_FLOATS}, got {x.dtype}, {w_router.dtype}")
    _require(logits_dtype in _FLOATS, f"logits dtype {logits_dtype} not in {_FLOATS}")
    for name, t in (("x", x), ("w_router", w_router)):
        _require(t.is_contiguous(), f"{name} must be contiguous")


@torch.library.custom_op(f"{_NS}::router_fwd", mutates_args=())
def router_fwd(x: Tensor, w_router: Tensor, logits_dtype: torch.dtype) -> Tensor:
    """Router logits x w_router^T [T,E]."""
    _check_router_args(x, w_router, logits_dtype)
    _check_devices(x=x, w_router=w_router)
    return B.router_logits(x, w_router, logits_dtype)


@router_fwd.register_fake
def _(x, w_router, logits_dtype):
    return x.new_empty((x.shape[0], w_router.shape[0]), dtype=logits_dtype)


@torch.library.custom_op(f"{_NS}::router_bwd", mutates_args=())
def router_bwd(dlogits: Tensor, x: Tensor, w_router: Tensor, dx_in: Tensor | None) -> tuple[Tensor, Tensor]:
    """(dx, dw_router): dx = dx_in + dlogits w_router, dw_router = dlogits^T x."""
    _check_router_args(x, w_router, dlogits.dtype)
    dlogits = _dense(dlogits)
    _require(tuple(dlogits.shape) == (x.shape[0], w_router.shape[0]),
             f"dlogits must be [T={x.shape[0]}, E={w_router.shape[0]}], got {tuple(dlogits.shape)}")
    tensors = dict(x=x, w_router=w_router, dlogits=dlogits)
    if dx_in is not None:
        dx_in = _dense(dx_in)
        _require(dx_in.shape == x.shape and dx_in.dtype == x.dtype,
                 f"dx_in must be {tuple(x.shape)} {x.dtype}, got {tuple(dx_in.shape)} {dx_in.dtype}")
        tensors["dx_in"] = dx_in
    _check_devices(**tensors)
    return B.router_backward(dlogits, x, w_router, dx_in=dx_in)


@router_bwd.register_fake
def _(dlogits, x, w_router, dx_in):
    return torch.empty_like(x), torch.empty_like(w_router)


class _Router(torch.autograd.Function):
    """logits, and x passed through: what comes back to x from the layer
    enters the router's backward, which adds its own part in the same pass."""

    @staticmethod
    def forward(ctx, x, w_router, logits_dtype):
        ctx.save_for_backward(x, w_router)
        ctx.set_materialize_grads(False)  # no zeros to add where only the logits were used
        return router_fwd(x, w_router, logits_dtype), x.view_as(x)

    @staticmethod
    def backward(ctx, dlogits, dx_in):
        x, w_router = ctx.saved_tensors
        if dlogits is None:  # the logits were not used
            return dx_in, None, None
        dx, dw = router_bwd(dlogits, x, w_router, dx_in)
        return dx, dw, None


def router(x: Tensor, w_router: Tensor, logits_dtype: torch.dtype = torch.float32) -> Tensor:
    """Router logits x w_router^T [T,E], differentiable in both."""
    _check_router_args(x, w_router, logits_dtype)
    return _Router.apply(x, w_router, logits_dtype)[0]


def moe_block(x: Tensor, w_router: Tensor, w_gate_up: Tensor, w_down: Tensor, k: int, precision: str = "native",
              recompute: bool = False, swiglu_limit: float = 0.0, save8: bool = False,
              logits_dtype: torch.dtype = torch.float32) -> Tensor:
    """The router and the layer: out [T,d] of moe_layer at the logits
    x w_router^T, differentiable in x and the three weights; x's gradient is
    written once, by the router's backward."""
    _check_router_args(x, w_router, logits_dtype)
    logits, x = _Router.apply(x, w_router, logits_dtype)
    return moe_layer(x, logits, w_gate_up, w_down, k, precision, recompute, swiglu_limit, save8)


# ------------------------------------------------------- norms and residual
def _check_norm_args(rows: Tensor, name: str, same: dict, w_post, gate, w_next):
    """rows [T,d] and whatever is given of `same` (like rows), the weights [d]
    and the gate ([d] or [T,1]): one float type, contiguous."""
    _require(rows.dim() == 2 and rows.dtype in _FLOATS,
             f"{name} must be [T, d] of one of {_FLOATS}, got {tuple(rows.shape)} {rows.dtype}")
    T, d = rows.shape
    want = {name: (rows, [(T, d)]), "w_post": (w_post, [(d,)]), "w_next": (w_next, [(d,)]),
            "gate": (gate, [(d,), (T, 1)])}
    want.update({n: (t, [(T, d)]) for n, t in same.items()})
    for n, (t, shapes) in want.items():
        if t is not None:
            _require(tuple(t.shape) in shapes and t.dtype == rows.dtype,
                     f"{n} must be {shapes} {rows.dtype}, got {tuple(t.shape)} {t.dtype}")
            _require(t.is_contiguous(), f"{n} must be contiguous")
    return {n: t for n, (t, _) in want.items() if t is not None}


@torch.library.custom_op(f"{_NS}::norm_fwd", mutates_args=())
def norm_fwd(x: Tensor, y: Tensor | None, w_post: Tensor | None, gate: Tensor | None, w_next: Tensor | None,
             res_scale: float, eps: float) -> tuple[Tensor, Tensor]:
    """(z, h) of binding.norm_residual; empty where there is no y, or no w_next."""
    _check_devices(**_check_norm_args(x, "x", {"y": y}, w_post, gate, w_next))
    z, h = B.norm_residual(x, y, w_post, gate, res_scale, w_next, eps)
    return x.new_empty(0) if y is None else z, x.new_empty(0) if h is None else h


@norm_fwd.register_fake
def _(x, y, w_post, gate, w_next, res_scale, eps):
    return (x.new_empty(0) if y is None else torch.empty_like(x),
            x.new_empty(0) if w_next is None else torch.empty_like(x))


@torch.library.custom_op(f"{_NS}::norm_bwd", mutates_args=())
def norm_bwd(dz: Tensor | None, dh: Tensor | None, z: Tensor, y: Tensor | None, w_post: Tensor | None,
             gate: Tensor | None, w_next: Tensor | None, res_scale: float, eps: float
             ) -> tuple[Tensor, Tensor, Tensor, Tensor, Tensor]:
    """(dx, dy, dw_post, dgate, dw_next) of binding.norm_residual_backward;
    empty where there is none."""
    dz = None if dz is None else _dense(dz)
    dh = None if dh is None else _dense(dh)
    _check_devices(**_check_norm_args(z, "z", {"dz": dz, "dh": dh, "y": y}, w_post, gate, w_next))
    g = B.norm_residual_backward(dz, dh, z, y, w_post, gate, res_scale, w_next, eps)
    return tuple(z.new_empty(0) if g[n] is None else g[n] for n in ("dx", "dy", "dw_post", "dgate", "dw_next"))


@norm_bwd.register_fake
def _(dz, dh, z, y, w_post, gate, w_next, res_scale, eps):
    return tuple(z.new_empty(0) if t is None else torch.empty_like(t) for t in (z, y, w_post, gate, w_next))


class _NormResidual(torch.autograd.Function):
    """z is saved as it leaves (x itself without a y, passed through so that
    what comes back along the residual stream is added in the same pass)."""

    @staticmethod
    def forward(ctx, x, y, w_post, gate, w_next, res_scale, eps):
        z, h = norm_fwd(x, y, w_post, gate, w_next, res_scale, eps)
        if y is None:
            z = x.view_as(x)
        ctx.save_for_backward(z, y, w_post, gate, w_next)
        ctx.scales = res_scale, eps
        ctx.set_materialize_grads(False)  # no zeros to add where z or h was not used
        return z, None if w_next is None else h

    @staticmethod
    def backward(ctx, dz, dh):
        z, y, w_post, gate, w_next = ctx.saved_tensors
        if dz is None and dh is None:
            return (None,) * 7
        if dh is None and y is None:
            return (dz,) + (None,) * 6
        used = None if dh is None else w_next
        grads = norm_bwd(dz, dh, z, y, w_post, gate, used, *ctx.scales)
        return tuple(g if t is not None else None for g, t in zip(grads, (z, y, w_post, gate, used))) + (None, None)


def norm_residual(x: Tensor, y: Tensor | None = None, w_post: Tensor | None = None, gate: Tensor | None = None,
                  res_scale: float = 1.0, w_next: Tensor | None = None, eps: float = 1e-6
                  ) -> tuple[Tensor, Tensor | None]:
    """(z, h) around a block, differentiable in every tensor: z = res_scale x +
    gate N(y; w_post) and h = N(z; w_next), N(v; w) = v / sqrt(mean(v^2) + eps) w.
    Without y z is x, without w_next h is None; gate: [d], or [T, 1] for one per
    token.  In a HIP graph, capture on leaves of the graph's own (see
    moe_layer)."""
    _check_norm_args(x, "x", {"y": y}, w_post, gate, w_next)
    if y is None:
        _require(w_post is None and gate is None and res_scale == 1.0, "w_post, gate and res_scale need y")
        _require(w_next is not None, "give y or w_next")
    return _NormResidual.apply(x, y, w_post, gate, w_next, float(res_scale), float(eps))


def moe_residual_block(x: Tensor, w_router: Tensor, w_gate_up: Tensor, w_down: Tensor, k: int,
                       w_pre: Tensor | None = None, w_post: Tensor | None = None, gate: Tensor | None = None,
                       res_scale: float = 1.0, w_next: Tensor | None = None, eps: float = 1e-6,
                       h: Tensor | None = None, **layer) -> tuple[Tensor, Tensor | None]:
    """moe_block with the norms and the residual around it: (z, h_next) of the
    residual stream x [T,d], z = res_scale x + gate N(moe_block(h); w_post),
    h_next = N(z; w_next), where h = N(x; w_pre), or is given (the last block's
    h_next).  `layer`: moe_block's options."""
    _require((w_pre is None) != (h is None), "give w_pre, or h from the block before")
    if h is None:
        x, h = norm_residual(x, w_next=w_pre, eps=eps)
    y = moe_block(h, w_router, w_gate_up, w_down, k, **layer)
    return norm_residual(x, y, w_post, gate, res_scale, w_next, eps)
