"""Python binding of the C ABI in include/moe.h (ctypes).

Argument marshalling only: tensors are checked (device, dtype, shape,
contiguity), their device pointers and torch's current HIP stream are handed
to the library, and a non-OK status raises.  Every step of the layer runs in
the library's HIP kernels; there is no fallback.  PyTorch supplies device
memory (outputs, workspace) and the stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from dataclasses import dataclass

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_mi355x.so")

MOE_F32, MOE_BF16 = 0, 1
PREC_NATIVE, PREC_FP8_BLOCK, PREC_MXFP8, PREC_FP8_BWD = 0, 1, 2, 3
OP_ROUTE, OP_FORWARD, OP_BACKWARD, OP_BACKWARD_RECOMPUTE = 0, 1, 2, 3
QUANT_ROWS, QUANT_WEIGHT, QUANT_WEIGHT_T = 0, 1, 2
DECODE_MAX_T = 256
GATE_NONE, GATE_CHANNEL, GATE_TOKEN = 0, 1, 2

_DT = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}
_TORCH = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16}
_WEIGHTS = {"native": 0, "fp8_block": 1, "mxfp8": 2, "mxfp4": 3}
_PREC = {"native": PREC_NATIVE, "fp8_block": PREC_FP8_BLOCK, "mxfp8": PREC_MXFP8, "fp8_bwd": PREC_FP8_BWD}


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int64), ("E", ctypes.c_int64),
                ("k", ctypes.c_int64), ("I", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("logits_dtype", ctypes.c_int32), ("precision", ctypes.c_int32),
                ("swiglu_limit", ctypes.c_float), ("flags", ctypes.c_int32)]


class MoeNormShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("gate_kind", ctypes.c_int32), ("res_scale", ctypes.c_float), ("eps", ctypes.c_float)]


class MoeRouting(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("topk_ids", ctypes.c_void_p),
                ("topk_w", ctypes.c_void_p), ("counts", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("row_of", ctypes.c_void_p),
                ("src_of", ctypes.c_void_p)]


class MoeKernelStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_int64),
                ("total_ms", ctypes.c_double)]


# exported entry points: (name, restype, argtypes)
_P = ctypes.c_void_p
_SIGS = [
    ("moe_workspace_bytes", ctypes.c_size_t, [ctypes.POINTER(MoeShape), ctypes.c_int]),
    ("moe_saved_bytes", ctypes.c_size_t, [ctypes.POINTER(MoeShape)]),
    ("moe_workspace_size", ctypes.c_int, [ctypes.POINTER(MoeShape), ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)]),
    ("moe_saved_size", ctypes.c_int, [ctypes.POINTER(MoeShape), ctypes.POINTER(ctypes.c_size_t)]),
    ("moe_route", ctypes.c_int, [ctypes.POINTER(MoeShape), ctypes.POINTER(MoeRouting), _P, ctypes.c_size_t, _P]),
    ("moe_route_noalloc", ctypes.c_int, [ctypes.POINTER(MoeShape), ctypes.POINTER(MoeRouting), _P]),
    ("moe_forward", ctypes.c_int, [ctypes.POINTER(MoeShape), _P, ctypes.POINTER(MoeRouting), _P, _P, _P, _P, _P,
                                   ctypes.c_size_t, _P]),
    ("moe_backward", ctypes.c_int, [ctypes.POINTER(MoeShape), _P, _P, ctypes.POINTER(MoeRouting), _P, _P, _P, _P,
                                    _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    ("moe_router_forward", ctypes.c_int, [ctypes.POINTER(MoeShape), _P, _P, _P, _P]),
    ("moe_router_workspace_size", ctypes.c_int, [ctypes.POINTER(MoeShape), ctypes.POINTER(ctypes.c_size_t)]),
    ("moe_router_backward", ctypes.c_int, [ctypes.POINTER(MoeShape), _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t,
                                           _P]),
    ("moe_saved8_size", ctypes.c_int, [ctypes.POINTER(MoeShape), ctypes.POINTER(ctypes.c_size_t)]),
    ("moe_workspace8_size", ctypes.c_int, [ctypes.POINTER(MoeShape), ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)]),
    ("moe_forward8", ctypes.c_int, [ctypes.POINTER(MoeShape), _P, ctypes.POINTER(MoeRouting), _P, _P, _P, _P, _P,
                                    ctypes.c_size_t, _P]),
    ("moe_backward8", ctypes.c_int, [ctypes.POINTER(MoeShape), _P, _P, ctypes.POINTER(MoeRouting), _P, _P, _P, _P,
                                     _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    ("moe_swiglu_save8", ctypes.c_int, [ctypes.POINTER(MoeShape), _P, ctypes.POINTER(MoeRouting), _P, _P, _P, _P]),
    ("moe_swiglu_backward8", ctypes.c_int, [ctypes.POINTER(MoeShape), _P, _P, _P, ctypes.POINTER(MoeRouting), _P, _P,
                                            _P, _P]),
    ("moe_decode_workspace_size", ctypes.c_int, [ctypes.POINTER(MoeShape), ctypes.POINTER(ctypes.c_size_t)]),
    ("moe_decode", ctypes.c_int, [ctypes.POINTER(MoeShape), ctypes.c_int, _P, ctypes.POINTER(MoeRouting), _P, _P, _P,
                                  _P, _P, _P, ctypes.c_size_t, _P]),
    ("moe_norm_forward", ctypes.c_int, [ctypes.POINTER(MoeNormShape)] + [_P] * 8),
    ("moe_norm_workspace_size", ctypes.c_int, [ctypes.POINTER(MoeNormShape), ctypes.POINTER(ctypes.c_size_t)]),
    ("moe_norm_backward", ctypes.c_int, [ctypes.POINTER(MoeNormShape)] + [_P] * 13 + [ctypes.c_size_t, _P]),
    ("moe_grouped_product", ctypes.c_int, [ctypes.POINTER(MoeShape), ctypes.c_int, _P, ctypes.c_int,
                                           ctypes.POINTER(MoeRouting), _P, _P, ctypes.c_int64, ctypes.c_int, _P, _P]),
    ("moe_permute", ctypes.c_int, [ctypes.POINTER(MoeShape), _P, ctypes.POINTER(MoeRouting), _P, _P]),
    ("moe_combine", ctypes.c_int, [ctypes.POINTER(MoeShape), _P, ctypes.POINTER(MoeRouting), _P, _P]),
    ("moe_quantize_fp8", ctypes.c_int, [ctypes.c_int, _P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _P, _P,
                                        _P]),
    ("moe_quantize_tokens_fp8", ctypes.c_int, [ctypes.POINTER(MoeShape), _P, ctypes.c_int64, ctypes.c_int,
                                               ctypes.POINTER(MoeRouting), _P, _P, _P, ctypes.c_size_t, _P]),
    ("moe_quantize_mxfp8", ctypes.c_int, [ctypes.c_int, _P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _P,
                                          _P, _P]),
    ("moe_quantize_mxfp4", ctypes.c_int, [_P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _P, _P, _P]),
    ("moe_quantize_tokens_mxfp8", ctypes.c_int, [ctypes.POINTER(MoeShape), _P, ctypes.c_int64, ctypes.c_int,
                                                 ctypes.POINTER(MoeRouting), _P, _P, _P, ctypes.c_size_t, _P]),
    ("moe_status_string", ctypes.c_char_p, [ctypes.c_int]),
    ("moe_last_error", ctypes.c_char_p, []),
    ("moe_profile_begin", ctypes.c_int, []),
    ("moe_profile_end", ctypes.c_int, [ctypes.POINTER(MoeKernelStat), ctypes.c_int, ctypes.POINTER(ctypes.c_int)]),
]

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded HIP library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"MoE HIP library not built ({LIB_PATH} missing): "
                               "run `python -m combine_top_route_amd.build`")
        l = ctypes.CDLL(LIB_PATH)
        for name, res, args in _SIGS:
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


class MoeError(RuntimeError):
    def __init__(self, call: str, status: int):
        l = lib()
        self.status = status
        super().__init__(f"{call}: {l.moe_status_string(status).decode()}: "
                         f"{l.moe_last_error().decode()}")


def _check(call: str, status: int):
    if status != 0:
        raise MoeError(call, status)


FLAG_PERSISTENT, FLAG_SKIP_MASKED = 1, 2


def make_shape(T, d, E, k, I, dtype=torch.bfloat16, logits_dtype=None, precision="native",
               swiglu_limit=0.0, persistent=False) -> MoeShape:
    """swiglu_limit > 0: the clamped SwiGLU with that limit; persistent: the
    bf16 GEMMs as persistent kernels (MOE_FLAG_PERSISTENT; see moe.h)."""
    logits_dtype = dtype if logits_dtype is None else logits_dtype
    return MoeShape(T, d, E, k, I, _DT[dtype], _DT[logits_dtype], _PREC[precision], float(swiglu_limit),
                    FLAG_PERSISTENT if persistent else 0)


def workspace_size(shape: MoeShape, op: int) -> int:
    n = lib().moe_workspace_bytes(ctypes.byref(shape), op)
    if n == 0:
        raise ValueError(f"moe_workspace_bytes: {lib().moe_last_error().decode()}")
    return n


def saved_size(shape: MoeShape) -> int:
    n = lib().moe_saved_bytes(ctypes.byref(shape))
    if n == 0:
        raise ValueError(f"moe_saved_bytes: {lib().moe_last_error().decode()}")
    return n


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device):
    """torch's current stream on a device, as the library takes it (the raw
    handle: building a torch.cuda.Stream object costs 2 us a call).  Refuses
    host memory: a CPU device has no index and would name the current GPU."""
    if device.type != "cuda":
        raise ValueError(f"tensors are on {device}; the kernels need a GPU's memory")
    return torch._C._cuda_getCurrentRawStream(
        torch.cuda.current_device() if device.index is None else device.index)


_HERE = contextlib.nullcontext()


def _on(device):
    """Context in which kernels launch on `device` (nothing to do, and nothing
    paid, when it is the current one).  Refuses host memory."""
    if device.type != "cuda":
        raise ValueError(f"tensors are on {device}; the kernels need a GPU's memory")
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


class _Entry:
    """An entry point that enqueues work, called with its tensors' device current
    and, as its last argument, torch's stream there.  Refuses host memory and
    raises on a status."""

    def __init__(self, name):
        self.name = name

    def __call__(self, device, *args):
        with _on(device):
            _check(self.name, getattr(lib(), self.name)(*args, _stream(device)))


_norm_forward, _norm_backward = _Entry("moe_norm_forward"), _Entry("moe_norm_backward")
_quantize_mxfp4, _grouped_product = _Entry("moe_quantize_mxfp4"), _Entry("moe_grouped_product")


def _need(t, name, shape, dtype, device):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


@dataclass
class Routing:
    """Routing tensors on the device (see moe_routing in include/moe.h)."""
    topk_ids: torch.Tensor
    topk_w: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    row_of: torch.Tensor
    src_of: torch.Tensor
    logits: torch.Tensor | None = None

    @staticmethod
    def empty(T, E, k, device, logits=None, topk_ids=None, topk_w=None) -> "Routing":
        i32 = dict(dtype=torch.int32, device=device)
        return Routing(
            topk_ids=torch.empty((T, k), **i32) if topk_ids is None else topk_ids,
            topk_w=torch.empty((T, k), dtype=torch.float32, device=device) if topk_w is None else topk_w,
            counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32),
            row_of=torch.empty(T * k, **i32), src_of=torch.empty(T * k, **i32), logits=logits)

    def on(self, device, *names) -> "Routing":
        """self, if the named tensors (those a call reads or writes) are on `device`."""
        for name in names:
            t = getattr(self, name)
            if t is not None and t.device != device:
                raise ValueError(f"routing.{name} is on {t.device}, expected {device}")
        return self

    def c(self) -> MoeRouting:
        return MoeRouting(_ptr(self.logits), _ptr(self.topk_ids), _ptr(self.topk_w), _ptr(self.counts),
                          _ptr(self.offsets), _ptr(self.row_of), _ptr(self.src_of))


class MoeLayer:
    """One layer shape with preallocated outputs and workspaces, so repeated
    calls (benchmarks, training loops) allocate nothing.  save=False: the
    forward keeps nothing and the backward recomputes H and Aw from x
    (activation checkpointing).  save8=True: the forward keeps H in 8 bits
    (moe_forward8, moe_backward8), about a third of the bytes."""

    def __init__(self, T, d, E, k, I, dtype=torch.bfloat16, logits_dtype=None,
                 precision="native", device="cuda", save=True, swiglu_limit=0.0, persistent=False,
                 save8=False):
        self.T, self.d, self.E, self.k, self.I = T, d, E, k, I
        self.dtype = dtype
        self.logits_dtype = dtype if logits_dtype is None else logits_dtype
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self.shape = make_shape(T, d, E, k, I, dtype, self.logits_dtype, precision, swiglu_limit, persistent)
        dev = self.device
        self.save8 = save8
        if save8:
            if not save:
                raise ValueError("save8 keeps a checkpoint; save=False keeps none")
            wf, wb = workspace8_size(self.shape, OP_FORWARD), workspace8_size(self.shape, OP_BACKWARD)
            ns = saved8_size(self.shape)
        else:
            wf = workspace_size(self.shape, OP_FORWARD)
            wb = workspace_size(self.shape, OP_BACKWARD if save else OP_BACKWARD_RECOMPUTE)
            ns = saved_size(self.shape) if save else 0
        self.ws_fwd = torch.empty(wf, dtype=torch.uint8, device=dev)
        self.ws_bwd = torch.empty(wb, dtype=torch.uint8, device=dev)
        self.saved = torch.empty(ns, dtype=torch.uint8, device=dev) if save else None
        self.out = torch.empty((T, d), dtype=dtype, device=dev)
        self.routing = Routing.empty(T, E, k, dev)
        self._topk = self.routing.topk_ids, self.routing.topk_w  # of the logits form
        self.dx = torch.empty((T, d), dtype=dtype, device=dev)
        self.dw_gate_up = torch.empty((E, 2 * I, d), dtype=dtype, device=dev)
        self.dw_down = torch.empty((E, d, I), dtype=dtype, device=dev)
        self.d_topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.dlogits = torch.empty((T, E), dtype=self.logits_dtype, device=dev)

    def saved_views(self):
        """(H [R,2I], A [R,I]) views of the saved buffer; with save8 its
        (codes [R,2I], scales [R,2 ceil(I/32)])."""
        R, I = self.T * self.k, self.I
        if self.save8:
            n, at, nb = R * 2 * I, -(-R * 2 * I // 256) * 256, 2 * -(-I // 32)
            return self.saved[:n].view(R, 2 * I), self.saved[at:at + R * nb].view(R, nb)
        flat = self.saved.view(self.dtype)
        return flat[:R * 2 * I].view(R, 2 * I), flat[R * 2 * I:].view(R, I)

    def forward(self, x, w_gate_up, w_down, logits=None, topk_ids=None, topk_w=None):
        T, d, E, k, I, dt, dev = self.T, self.d, self.E, self.k, self.I, self.dtype, self.device
        _need(x, "x", (T, d), dt, dev)
        _need(w_gate_up, "w_gate_up", (E, 2 * I, d), dt, dev)
        _need(w_down, "w_down", (E, d, I), dt, dev)
        r = self.routing
        if logits is not None:
            _need(logits, "logits", (T, E), self.logits_dtype, dev)
            r.logits = logits
            r.topk_ids, r.topk_w = self._topk
        else:
            _need(topk_ids, "topk_ids", (T, k), torch.int32, dev)
            _need(topk_w, "topk_w", (T, k), torch.float32, dev)
            r.logits = None
            r.topk_ids, r.topk_w = topk_ids, topk_w
        cr = r.c()
        name = "moe_forward8" if self.save8 else "moe_forward"
        with _on(dev):
            _check(name, getattr(lib(), name)(
                ctypes.byref(self.shape), _ptr(x), ctypes.byref(cr), _ptr(w_gate_up), _ptr(w_down),
                _ptr(self.out), _ptr(self.saved), _ptr(self.ws_fwd), self.ws_fwd.numel(), _stream(dev)))
        return self.out

    def backward(self, dout, x, w_gate_up, w_down, want_dlogits=True):
        T, d, E, I, dt, dev = self.T, self.d, self.E, self.I, self.dtype, self.device
        _need(dout, "dout", (T, d), dt, dev)
        _need(x, "x", (T, d), dt, dev)
        _need(w_gate_up, "w_gate_up", (E, 2 * I, d), dt, dev)
        _need(w_down, "w_down", (E, d, I), dt, dev)
        r = self.routing
        cr = r.c()
        dl = self.dlogits if (want_dlogits and r.logits is not None) else None
        name = "moe_backward8" if self.save8 else "moe_backward"
        with _on(dev):
            _check(name, getattr(lib(), name)(
                ctypes.byref(self.shape), _ptr(dout), _ptr(x), ctypes.byref(cr), _ptr(w_gate_up),
                _ptr(w_down), _ptr(self.saved), _ptr(self.dx), _ptr(self.dw_gate_up), _ptr(self.dw_down),
                _ptr(self.d_topk_w), _ptr(dl), _ptr(self.ws_bwd), self.ws_bwd.numel(), _stream(dev)))
        res = dict(dx=self.dx, dW_gate_up=self.dw_gate_up, dW_down=self.dw_down, d_topk_w=self.d_topk_w)
        if dl is not None:
            res["dlogits"] = dl
        return res


def _router_shape(x, w_router, logits_dtype) -> MoeShape:
    if x.dim() != 2 or w_router.dim() != 2 or w_router.shape[1] != x.shape[1]:
        raise ValueError(f"x must be [T, d] and w_router [E, d], got {tuple(x.shape)} and {tuple(w_router.shape)}")
    if x.dtype not in _DT or logits_dtype not in _DT:
        raise ValueError(f"x has dtype {x.dtype}, the logits {logits_dtype}, expected two of {tuple(_DT)}")
    _need(x, "x", x.shape, x.dtype, x.device)
    _need(w_router, "w_router", w_router.shape, x.dtype, x.device)
    return _shape_of(x.shape[0], x.shape[1], w_router.shape[0], 1, 8, x.dtype, logits_dtype, 0.0)


# The argument structs and sizes of recent calls: making one and asking for a
# size costs as much as a small kernel.
@functools.lru_cache(maxsize=256)
def _shape_of(T, d, E, k, I, dtype, logits_dtype, swiglu_limit):
    return make_shape(T, d, E, k, I, dtype, logits_dtype, swiglu_limit=swiglu_limit)


@functools.lru_cache(maxsize=256)
def _rows_shape(T, k, I, dtype, swiglu_limit):
    shape = make_shape(T, 8, max(k, 1), k, I, dtype, swiglu_limit=swiglu_limit)
    saved8_size(shape)  # refuses a bad T, k or I before anything is allocated
    return shape


@functools.lru_cache(maxsize=256)
def _router_workspace(T, d, E, dtype):
    return router_workspace_size(make_shape(T, d, E, 1, 8, dtype))


def router_workspace_size(shape: MoeShape) -> int:
    n = ctypes.c_size_t()
    _check("moe_router_workspace_size", lib().moe_router_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def router_logits(x, w_router, logits_dtype=torch.float32):
    """Router logits x w_router^T [T, E] (moe_router_forward in include/moe.h)
    of x [T, d] and w_router [E, d], both float32 or both bfloat16."""
    shape = _router_shape(x, w_router, logits_dtype)
    with _on(x.device):
        logits = torch.empty((x.shape[0], w_router.shape[0]), dtype=logits_dtype, device=x.device)
        _check("moe_router_forward", lib().moe_router_forward(ctypes.byref(shape), _ptr(x), _ptr(w_router),
                                                              _ptr(logits), _stream(x.device)))
    return logits


def router_backward(dlogits, x, w_router, dx_in=None):
    """(dx, dw_router) of the projection: dx = dx_in + dlogits w_router (dx_in
    None: zeros), dw_router = dlogits^T x (moe_router_backward)."""
    shape = _router_shape(x, w_router, dlogits.dtype)
    dev = x.device
    _need(dlogits, "dlogits", (x.shape[0], w_router.shape[0]), dlogits.dtype, dev)
    if dx_in is not None:
        _need(dx_in, "dx_in", x.shape, x.dtype, dev)
    n = _router_workspace(x.shape[0], x.shape[1], w_router.shape[0], x.dtype)
    with _on(dev):
        dx, dw = torch.empty_like(x), torch.empty_like(w_router)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        _check("moe_router_backward", lib().moe_router_backward(
            ctypes.byref(shape), _ptr(dlogits), _ptr(x), _ptr(w_router), _ptr(dx_in), _ptr(dx), _ptr(dw), _ptr(ws), n,
            _stream(dev)))
    return dx, dw


def saved8_size(shape: MoeShape) -> int:
    n = ctypes.c_size_t()
    _check("moe_saved8_size", lib().moe_saved8_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def workspace8_size(shape: MoeShape, op: int) -> int:
    n = ctypes.c_size_t()
    _check("moe_workspace8_size", lib().moe_workspace8_size(ctypes.byref(shape), op, ctypes.byref(n)))
    return n.value


def _row_args(rows, routing: Routing, T, k, name, width):
    """Checks of the checkpoint's row passes: rows [T*k, width]."""
    dev = rows.device
    if rows.dtype not in _DT:
        raise ValueError(f"{name} has dtype {rows.dtype}, expected one of {tuple(_DT)}")
    _need(rows, name, (T * k, width), rows.dtype, dev)
    if routing is not None:
        _need(routing.src_of, "src_of", (T * k,), torch.int32, dev)
        _need(routing.topk_w, "topk_w", (T, k), torch.float32, dev)
    return dev


def swiglu_save8(H, routing: Routing | None, T, k, swiglu_limit=0.0):
    """(Aw [T*k, I], codes uint8 [T*k, 2I], scales uint8 [T*k, 2 ceil(I/32)])
    of gate|up pre-activations H [T*k, 2I] in expert order (moe_swiglu_save8 in
    include/moe.h).  routing=None: the codes and scales alone (Aw is None)."""
    if H.dim() != 2 or H.shape[1] % 2:
        raise ValueError(f"H must be [T*k, 2I], got {tuple(H.shape)}")
    I = H.shape[1] // 2
    dev = _row_args(H, routing, T, k, "H", 2 * I)
    shape = _rows_shape(T, k, I, H.dtype, swiglu_limit)
    with _on(dev):
        aw = None if routing is None else torch.empty((T * k, I), dtype=H.dtype, device=dev)
        codes = torch.empty((T * k, 2 * I), dtype=torch.uint8, device=dev)
        scales = torch.empty((T * k, 2 * -(-I // 32)), dtype=torch.uint8, device=dev)
        cr = None if routing is None else ctypes.byref(routing.c())
        _check("moe_swiglu_save8", lib().moe_swiglu_save8(ctypes.byref(shape), _ptr(H), cr, _ptr(aw), _ptr(codes),
                                                          _ptr(scales), _stream(dev)))
    return aw, codes, scales


def swiglu_backward8(G, codes, scales, routing: Routing, T, k, swiglu_limit=0.0):
    """(dH [T*k, 2I], Aw [T*k, I], dw [T*k] float32) from G [T*k, I] and the
    codes and scales of swiglu_save8 (moe_swiglu_backward8)."""
    if G.dim() != 2:
        raise ValueError(f"G must be [T*k, I], got {tuple(G.shape)}")
    I = G.shape[1]
    dev = _row_args(G, routing, T, k, "G", I)
    _need(codes, "codes", (T * k, 2 * I), torch.uint8, dev)
    _need(scales, "scales", (T * k, 2 * -(-I // 32)), torch.uint8, dev)
    shape = _rows_shape(T, k, I, G.dtype, swiglu_limit)
    with _on(dev):
        dh = torch.empty((T * k, 2 * I), dtype=G.dtype, device=dev)
        aw = torch.empty((T * k, I), dtype=G.dtype, device=dev)
        dw = torch.empty(T * k, dtype=torch.float32, device=dev)
        cr = routing.c()
        _check("moe_swiglu_backward8", lib().moe_swiglu_backward8(
            ctypes.byref(shape), _ptr(G), _ptr(codes), _ptr(scales), ctypes.byref(cr), _ptr(dh), _ptr(aw), _ptr(dw),
            _stream(dev)))
    return dh, aw, dw


@functools.lru_cache(maxsize=256)
def _norm_shape(T, d, dtype, gate_kind, res_scale, eps):
    return MoeNormShape(T, d, _DT[dtype], gate_kind, res_scale, eps)


@functools.lru_cache(maxsize=256)
def _norm_workspace(T, d, dtype):
    return norm_workspace_size(MoeNormShape(T, d, _DT[dtype], GATE_NONE, 1.0, 1.0))


def norm_workspace_size(shape: MoeNormShape) -> int:
    n = ctypes.c_size_t()
    _check("moe_norm_workspace_size", lib().moe_norm_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def _norm_args(rows, name, w_post, gate, w_next, res_scale, eps):
    """Checks a norm's weights against rows [T, d]; its shape argument."""
    if rows.dim() != 2 or rows.dtype not in _DT:
        raise ValueError(f"{name} must be [T, d] of one of {tuple(_DT)}, got {tuple(rows.shape)} {rows.dtype}")
    T, d = rows.shape
    dt, dev = rows.dtype, rows.device
    _need(rows, name, (T, d), dt, dev)
    if w_post is not None:
        _need(w_post, "w_post", (d,), dt, dev)
    if w_next is not None:
        _need(w_next, "w_next", (d,), dt, dev)
    kind = GATE_NONE
    if gate is not None:
        kind = GATE_CHANNEL if gate.dim() == 1 else GATE_TOKEN
        _need(gate, "gate ([d] or [T, 1])", (d,) if kind == GATE_CHANNEL else (T, 1), dt, dev)
    return _norm_shape(T, d, dt, kind, float(res_scale), float(eps))


def norm_residual(x, y=None, w_post=None, gate=None, res_scale=1.0, w_next=None, eps=1e-6):
    """(z, h) of the residual stream x [T, d] and a block's output y
    (moe_norm_forward in include/moe.h): z = res_scale x + gate N(y; w_post), h
    = N(z; w_next), N(v; w) = v / sqrt(mean(v^2) + eps) w.  Without y z is x
    itself, without w_next h is None.  gate: [d], or [T, 1] for one per token.
    All in x's dtype."""
    shape = _norm_args(x, "x", w_post, gate, w_next, res_scale, eps)
    dev = x.device
    if y is not None:
        _need(y, "y", x.shape, x.dtype, dev)
    z = None if y is None else torch.empty_like(x)
    h = None if w_next is None else torch.empty_like(x)
    _norm_forward(dev, ctypes.byref(shape), _ptr(x), _ptr(y), _ptr(w_post), _ptr(gate), _ptr(w_next), _ptr(z), _ptr(h))
    return x if y is None else z, h


def norm_residual_backward(dz, dh, z, y=None, w_post=None, gate=None, res_scale=1.0, w_next=None, eps=1e-6):
    """Gradients of norm_residual from those of its z and h (dz or dh may be
    None; dh and w_next come together), at its z (x where there was no y) and y
    (moe_norm_backward): a dict of dx, dy (None without y), dw_post, dgate and
    dw_next (None where that weight is)."""
    if (dh is None) != (w_next is None):
        raise ValueError("give dh and w_next, or neither")
    shape = _norm_args(z, "z", w_post, gate, w_next, res_scale, eps)
    dev = z.device
    for name, t in (("dz", dz), ("dh", dh), ("y", y)):
        if t is not None:
            _need(t, name, z.shape, z.dtype, dev)
    n = _norm_workspace(z.shape[0], z.shape[1], z.dtype)
    out = {"dx": torch.empty_like(z)}
    for name, t in (("dy", y), ("dw_post", w_post), ("dgate", gate), ("dw_next", w_next)):
        out[name] = None if t is None else torch.empty_like(t)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _norm_backward(dev, ctypes.byref(shape), _ptr(dz), _ptr(dh), _ptr(z), _ptr(y), _ptr(w_post), _ptr(gate),
                   _ptr(w_next), _ptr(out["dx"]), _ptr(out["dy"]), _ptr(out["dw_post"]), _ptr(out["dgate"]),
                   _ptr(out["dw_next"]), _ptr(ws), n)
    return out


def decode_workspace_size(shape: MoeShape) -> int:
    n = ctypes.c_size_t()
    _check("moe_decode_workspace_size", lib().moe_decode_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def _weight_args(name, w, shape, dtype, weights, device):
    """Pointers of an expert weight [E, N, K] and of its scales: a tensor, or
    (coded formats) the (codes, scales) pair of quantize_fp8 / quantize_mxfp8
    with QUANT_WEIGHT, or of quantize_mxfp4."""
    if weights == "native":
        _need(w, name, shape, dtype, device)
        return _ptr(w), None
    if not isinstance(w, (tuple, list)) or len(w) != 2:
        raise ValueError(f"{name} must be a (codes, scales) pair for weights={weights!r}")
    E, N, K = shape
    _need(w[0], f"{name} codes", (E, N, K // 2) if weights == "mxfp4" else shape, torch.uint8, device)
    if weights == "fp8_block":
        _need(w[1], f"{name} scales", (E, N // 128, K // 128), torch.float32, device)
    else:
        _need(w[1], f"{name} scales", (E, N, K // 32), torch.uint8, device)
    return _ptr(w[0]), _ptr(w[1])


class MoeDecoder:
    """The layer for few tokens (moe_decode in include/moe.h), as a serving
    loop calls it: forward takes x [T, d] with any 1 <= T <= max_T, and outputs
    and workspace are allocated once, so calls allocate nothing and can be
    captured into a graph.  out, topk_ids and topk_w are views of the decoder's
    buffers and hold the last call's results; their rows from T on keep what
    they held.  Calls that overlap in time (streams, replayed graphs) need a
    decoder each.

    weights: "native" (tensors in dtype), or "fp8_block" / "mxfp8": (codes,
    scales) pairs from quantize_fp8 / quantize_mxfp8 with QUANT_WEIGHT, or
    "mxfp4": those of quantize_mxfp4.
    Routing by logits [T, E], or by topk_ids and topk_w [T, k]; an id outside
    [0, E) or a logit of -inf is an empty slot.  No gradient."""

    def __init__(self, max_T, d, E, k, I, dtype=torch.bfloat16, logits_dtype=None, weights="native",
                 device="cuda", swiglu_limit=0.0):
        if weights not in _WEIGHTS:
            raise ValueError(f"weights {weights!r} unknown")
        self.max_T, self.d, self.E, self.k, self.I, self.weights = max_T, d, E, k, I, weights
        self.dtype = dtype
        self.logits_dtype = dtype if logits_dtype is None else logits_dtype
        self.swiglu_limit = swiglu_limit
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        shape = make_shape(max_T, d, E, k, I, dtype, self.logits_dtype, "native", swiglu_limit)
        self.workspace = torch.empty(decode_workspace_size(shape), dtype=torch.uint8, device=dev)
        self._out = torch.empty((max_T, d), dtype=dtype, device=dev)
        self._ids = torch.empty((max_T, k), dtype=torch.int32, device=dev)
        self._w = torch.empty((max_T, k), dtype=torch.float32, device=dev)
        self._by_T = {}
        self.out, self.topk_ids, self.topk_w = self._out, self._ids, self._w

    def _views(self, T):
        """Shape argument and output views for T tokens (built once per T)."""
        v = self._by_T.get(T)
        if v is None:
            shape = make_shape(T, self.d, self.E, self.k, self.I, self.dtype, self.logits_dtype, "native",
                               self.swiglu_limit)
            v = self._by_T[T] = (shape, self._out[:T], self._ids[:T], self._w[:T])
        return v

    def forward(self, x, w_gate_up, w_down, logits=None, topk_ids=None, topk_w=None):
        E, d, I, dt, dev = self.E, self.d, self.I, self.dtype, self.device
        T = x.shape[0]
        if not 1 <= T <= self.max_T:
            raise ValueError(f"x has {T} tokens, this decoder takes 1 to {self.max_T}")
        _need(x, "x", (T, d), dt, dev)
        gu, gu_s = _weight_args("w_gate_up", w_gate_up, (E, 2 * I, d), dt, self.weights, dev)
        dn, dn_s = _weight_args("w_down", w_down, (E, d, I), dt, self.weights, dev)
        shape, out, ids, w = self._views(T)
        if logits is not None:
            if topk_ids is not None or topk_w is not None:
                raise ValueError("give logits, or topk_ids and topk_w, not both")
            _need(logits, "logits", (T, E), self.logits_dtype, dev)
        else:
            _need(topk_ids, "topk_ids", (T, self.k), torch.int32, dev)
            _need(topk_w, "topk_w", (T, self.k), torch.float32, dev)
            ids, w = topk_ids, topk_w
        routing = MoeRouting(_ptr(logits), _ptr(ids), _ptr(w), None, None, None, None)
        with _on(dev):
            _check("moe_decode", lib().moe_decode(
                ctypes.byref(shape), _WEIGHTS[self.weights], _ptr(x), ctypes.byref(routing), gu, gu_s, dn, dn_s,
                _ptr(out), _ptr(self.workspace), self.workspace.numel(), _stream(dev)))
        self.out, self.topk_ids, self.topk_w = out, ids, w
        return out


def route(logits, k):
    """Routing alone from router logits [T,E] (f32 or bf16)."""
    T, E = logits.shape
    dev = logits.device
    shape = make_shape(T, 8, E, k, 8, torch.bfloat16, logits.dtype)
    r = Routing.empty(T, E, k, dev, logits=logits)
    ws = torch.empty(workspace_size(shape, OP_ROUTE), dtype=torch.uint8, device=dev)
    cr = r.c()
    with _on(dev):
        _check("moe_route", lib().moe_route(ctypes.byref(shape), ctypes.byref(cr), _ptr(ws), ws.numel(),
                                             _stream(dev)))
    return r


def route_ids(topk_ids, topk_w, E):
    """Routing artefacts for given ids and weights (ids-in form)."""
    T, k = topk_ids.shape
    dev = topk_ids.device
    _need(topk_ids, "topk_ids", (T, k), torch.int32, dev)
    _need(topk_w, "topk_w", (T, k), torch.float32, dev)
    shape = make_shape(T, 8, E, k, 8, torch.bfloat16)
    r = Routing.empty(T, E, k, dev, topk_ids=topk_ids, topk_w=topk_w)
    ws = torch.empty(workspace_size(shape, OP_ROUTE), dtype=torch.uint8, device=dev)
    cr = r.c()
    with _on(dev):
        _check("moe_route", lib().moe_route(ctypes.byref(shape), ctypes.byref(cr), _ptr(ws), ws.numel(),
                                             _stream(dev)))
    return r


def route_noalloc(r: Routing, T, E, k, logits_dtype=torch.bfloat16):
    """moe_route_noalloc into the caller's routing tensors r (logits in when
    r.logits is set, else r.topk_ids / r.topk_w in); no workspace."""
    shape = make_shape(T, 8, E, k, 8, torch.bfloat16, logits_dtype)
    cr = r.on(r.counts.device, "logits", "topk_ids", "topk_w", "offsets", "row_of", "src_of").c()
    with _on(r.counts.device):
        _check("moe_route_noalloc", lib().moe_route_noalloc(ctypes.byref(shape), ctypes.byref(cr),
                                                             _stream(r.counts.device)))
    return r


def permute(x, routing: Routing, k, out=None):
    """Dispatch: xp [T*k, d] with xp[r] = x[src_of[r] / k] (into `out` when given)."""
    T, d = x.shape
    E = routing.counts.numel()
    shape = make_shape(T, d, E, k, 8, x.dtype)
    xp = torch.empty((T * k, d), dtype=x.dtype, device=x.device) if out is None else out
    _need(xp, "out", (T * k, d), x.dtype, x.device)
    cr = routing.on(x.device, "src_of", "row_of").c()
    with _on(x.device):
        _check("moe_permute", lib().moe_permute(ctypes.byref(shape), _ptr(x), ctypes.byref(cr), _ptr(xp),
                                                 _stream(x.device)))
    return xp


def combine(rows, routing: Routing, T, k, skip_masked=False):
    """out [T, d] of expert-sorted rows [T*k, d] (more are not read): each token's
    rows by their weights (moe_combine in include/moe.h).  skip_masked: slots
    whose logit (routing.logits) is -inf add nothing."""
    dev = rows.device
    if rows.dim() != 2 or rows.shape[0] < T * k or rows.dtype not in _DT or not rows.is_contiguous():
        raise ValueError(f"rows must be contiguous [T*k={T * k}, d] of one of {tuple(_DT)}, got {tuple(rows.shape)} "
                         f"{rows.dtype}")
    d = rows.shape[1]
    E = routing.counts.numel()
    cr = routing.on(dev, "row_of", "topk_w").c()
    shape = make_shape(T, d, E, k, 8, rows.dtype)
    if skip_masked:
        lg = routing.logits
        if lg is None or lg.dtype not in _DT:
            raise ValueError(f"skip_masked needs routing.logits, of one of {tuple(_DT)}")
        _need(lg, "routing.logits", (T, E), lg.dtype, dev)
        _need(routing.topk_ids, "routing.topk_ids", (T, k), torch.int32, dev)
        shape.logits_dtype = _DT[lg.dtype]
        shape.flags |= FLAG_SKIP_MASKED
    out = torch.empty((T, d), dtype=rows.dtype, device=dev)
    with _on(dev):
        _check("moe_combine", lib().moe_combine(ctypes.byref(shape), _ptr(rows), ctypes.byref(cr), _ptr(out),
                                                 _stream(dev)))
    return out


def grouped_product(x, weight, routing: Routing, T, k, gather=True, swiglu=False, swiglu_limit=0.0, out=None):
    """y [T*k, N] of expert-sorted rows times their experts' MXFP4 matrices
    (moe_grouped_product in include/moe.h): weight is the (codes [E, N, K/2],
    scales [E, N, K/32]) pair of quantize_mxfp4, the rows are x[src_of // k] of x
    [T, K], or without gather x [T*k, K] itself.  swiglu: weight holds N/2 gate
    rows, then N/2 up rows, and y is silu(g) u [T*k, N/2].  Rows behind the last
    expert's are left as they were (in `out` when given).  No gradient."""
    if not isinstance(weight, (tuple, list)) or len(weight) != 2 or weight[0].dim() != 3:
        raise ValueError("weight must be the (codes, scales) pair of quantize_mxfp4")
    if x.dim() != 2:
        raise ValueError(f"x must be [rows, K], got {tuple(x.shape)}")
    codes, scales = weight
    E, N, K = codes.shape[0], codes.shape[1], x.shape[1]
    dev, bf = x.device, torch.bfloat16
    _need(x, "x", (T if gather else T * k, K), bf, dev)
    _need(codes, "codes", (E, N, K // 2), torch.uint8, dev)
    _need(scales, "scales", (E, N, K // 32), torch.uint8, dev)
    _need(routing.offsets, "routing.offsets", (E + 1,), torch.int32, dev)
    if gather:
        _need(routing.src_of, "routing.src_of", (T * k,), torch.int32, dev)
    shape = _shape_of(T, K, E, k, 8, bf, bf, float(swiglu_limit))
    y = torch.empty((T * k, N // 2 if swiglu else N), dtype=bf, device=dev) if out is None else out
    _need(y, "out", (T * k, N // 2 if swiglu else N), bf, dev)
    cr = MoeRouting(None, None, None, None, _ptr(routing.offsets), None, _ptr(routing.src_of))
    _grouped_product(dev, ctypes.byref(shape), _WEIGHTS["mxfp4"], _ptr(x), int(gather), ctypes.byref(cr), _ptr(codes),
                     _ptr(scales), N, int(swiglu), _ptr(y))
    return y


def profile_begin():
    _check("moe_profile_begin", lib().moe_profile_begin())


def profile_end() -> dict:
    """{kernel name: (launches, total ms)} of the launches since profile_begin."""
    cap = 64
    arr = (MoeKernelStat * cap)()
    n = ctypes.c_int()
    _check("moe_profile_end", lib().moe_profile_end(arr, cap, ctypes.byref(n)))
    return {arr[i].name.decode(): (arr[i].launches, arr[i].total_ms) for i in range(min(n.value, cap))}


def quantize_fp8(src, kind=QUANT_ROWS):
    """e4m3 codes (uint8) and float32 scales of a bf16 tensor: kind
    QUANT_ROWS for [n0, n1] (1x128 blocks), QUANT_WEIGHT / QUANT_WEIGHT_T for
    [n0, n1, n2] (128x128 blocks, written as is or transposed)."""
    dev = src.device
    if src.dtype != torch.bfloat16 or not src.is_contiguous():
        raise ValueError("src must be a contiguous bf16 tensor")
    if kind == QUANT_ROWS:
        n0, n1 = src.shape
        n2 = 0
        q = torch.empty((n0, n1), dtype=torch.uint8, device=dev)
        s = torch.empty((n0, n1 // 128), dtype=torch.float32, device=dev)
    else:
        n0, n1, n2 = src.shape
        qs = (n0, n1, n2) if kind == QUANT_WEIGHT else (n0, n2, n1)
        q = torch.empty(qs, dtype=torch.uint8, device=dev)
        s = torch.empty((qs[0], qs[1] // 128, qs[2] // 128), dtype=torch.float32, device=dev)
    with _on(dev):
        _check("moe_quantize_fp8", lib().moe_quantize_fp8(kind, _ptr(src), n0, n1, n2, _ptr(q), _ptr(s),
                                                          _stream(dev)))
    return q, s


def quantize_tokens_fp8(src, routing: Routing, T, k, gather):
    """Token-block codes q [C, 128 nblk] and scales s [C, nblk] of a
    weight-gradient operand (see moe_quantize_tokens_fp8); nblk =
    ceil(T*k/128) + E."""
    dev = src.device
    C = src.shape[1]
    E = routing.counts.numel()
    shape = make_shape(T, C, E, k, 128, torch.bfloat16)
    nblk = -(-T * k // 128) + E
    q = torch.zeros((C, 128 * nblk), dtype=torch.uint8, device=dev)
    s = torch.zeros((C, nblk), dtype=torch.float32, device=dev)
    ws = torch.empty(workspace_size(shape, OP_ROUTE), dtype=torch.uint8, device=dev)
    cr = routing.on(dev, "offsets", *(["src_of"] if gather else [])).c()
    with _on(dev):
        _check("moe_quantize_tokens_fp8", lib().moe_quantize_tokens_fp8(
            ctypes.byref(shape), _ptr(src), C, 1 if gather else 0, ctypes.byref(cr), _ptr(q), _ptr(s), _ptr(ws),
            ws.numel(), _stream(dev)))
    return q, s


def quantize_mxfp8(src, kind=QUANT_ROWS):
    """MXFP8 e4m3 codes (uint8) and E8M0 scale bytes (uint8) of a bf16
    tensor: kind QUANT_ROWS for [n0, n1] (blocks of 32 along rows; s [n0,
    n1/32]), QUANT_WEIGHT for [n0, n1, n2] (blocks of 32 along rows; s [n0,
    n1, n2/32]), QUANT_WEIGHT_T (blocks of 32 down columns, written
    transposed; q [n0, n2, n1], s [n0, n2, n1/32])."""
    dev = src.device
    if src.dtype != torch.bfloat16 or not src.is_contiguous():
        raise ValueError("src must be a contiguous bf16 tensor")
    if kind == QUANT_ROWS:
        n0, n1 = src.shape
        n2 = 0
        qs = (n0, n1)
    else:
        n0, n1, n2 = src.shape
        qs = (n0, n1, n2) if kind == QUANT_WEIGHT else (n0, n2, n1)
    q = torch.empty(qs, dtype=torch.uint8, device=dev)
    s = torch.empty(qs[:-1] + (qs[-1] // 32,), dtype=torch.uint8, device=dev)
    with _on(dev):
        _check("moe_quantize_mxfp8", lib().moe_quantize_mxfp8(kind, _ptr(src), n0, n1, n2, _ptr(q), _ptr(s),
                                                              _stream(dev)))
    return q, s


def quantize_mxfp4(src):
    """MXFP4 codes [n0, n1, n2/2] (uint8, two e2m1 codes a byte, the even column
    low) and E8M0 scale bytes [n0, n1, n2/32] of bf16 weights [n0, n1, n2], for
    MoeDecoder(weights="mxfp4") and grouped_product (moe_quantize_mxfp4)."""
    dev = src.device
    if src.dtype != torch.bfloat16 or src.dim() != 3 or not src.is_contiguous():
        raise ValueError("src must be a contiguous bf16 tensor [n0, n1, n2]")
    n0, n1, n2 = src.shape
    q = torch.empty((n0, n1, n2 // 2), dtype=torch.uint8, device=dev)
    s = torch.empty((n0, n1, n2 // 32), dtype=torch.uint8, device=dev)
    _quantize_mxfp4(dev, _ptr(src), n0, n1, n2, _ptr(q), _ptr(s))
    return q, s


def quantize_tokens_mxfp8(src, routing: Routing, T, k, gather):
    """MXFP8 token-block codes q [C, 128 nblk] and scale bytes s [C, 4 nblk]
    of a weight-gradient operand (see moe_quantize_tokens_mxfp8)."""
    dev = src.device
    C = src.shape[1]
    E = routing.counts.numel()
    shape = make_shape(T, C, E, k, 128, torch.bfloat16)
    nblk = -(-T * k // 128) + E
    q = torch.zeros((C, 128 * nblk), dtype=torch.uint8, device=dev)
    s = torch.zeros((C, 4 * nblk), dtype=torch.uint8, device=dev)
    ws = torch.empty(workspace_size(shape, OP_ROUTE), dtype=torch.uint8, device=dev)
    cr = routing.on(dev, "offsets", *(["src_of"] if gather else [])).c()
    with _on(dev):
        _check("moe_quantize_tokens_mxfp8", lib().moe_quantize_tokens_mxfp8(
            ctypes.byref(shape), _ptr(src), C, 1 if gather else 0, ctypes.byref(cr), _ptr(q), _ptr(s), _ptr(ws),
            ws.numel(), _stream(dev)))
    return q, s
