"""Layer operators on torch tensors: the forward and backward passes whose gradients a ``MuonPlan`` steps on.

Everything runs in the HIP kernels behind the C ABI of ``include/muon_ops.h``;
this module checks arguments, allocates outputs and workspaces from torch's
caching allocator on the current stream, and ties the calls to autograd.

* ``linear``: act(x W + b) + residual, and ``expert_linear``, the same over rows
  grouped by expert with a weight [E, K, N];
* ``route``, ``dispatch``, ``combine``: entries sorted by expert, rows moved there
  and back with weights;
* ``dropout``: from a counter-based generator, the mask never stored.

Tensors are float32 or bfloat16, on one GPU, on the current torch stream.  Rows
may be strided; a tensor whose last dimension is not contiguous is copied
first.  The ``*_forward`` and ``*_backward`` functions are the same passes without
autograd, for code that captures them into a HIP graph: they take a tensor's value alone,
whether it requires a gradient or carries a tangent.  The others are differentiable
backwards, once; forward-mode differentiation raises, and so do tracers (``make_fx``,
``torch.jit.trace``), which cannot see the kernels.
"""

from __future__ import annotations

import ctypes
import math
import sys
from typing import NamedTuple

import torch
from torch.autograd import forward_ad

from .binding import MUON_BF16, MUON_F32, MUON_OK, MuonError, load_library, muon_last_error

MUON_ROUTE_MAX_EXPERTS = 1024
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
EXPORTED_OPS = ("muon_linear_workspace", "muon_linear_forward", "muon_linear_grad_act", "muon_linear_grad_input",
                "muon_linear_grad_weight", "muon_linear_backward", "muon_route_workspace", "muon_route", "muon_dispatch",
                "muon_dispatch_grad", "muon_combine", "muon_combine_grad", "muon_dropout")

_FORWARD, _BACKWARD = 0, 4


class LinearDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("w_layout", ctypes.c_int32), ("rows", ctypes.c_int64), ("k", ctypes.c_int64),
                ("n", ctypes.c_int64), ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64),
                ("w_stride", ctypes.c_int64), ("ldr", ctypes.c_int64), ("ldg", ctypes.c_int64)]


class MoveDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("experts", ctypes.c_int32), ("top", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("tokens", ctypes.c_int64), ("h", ctypes.c_int64),
                ("ldx", ctypes.c_int64), ("ldg", ctypes.c_int64), ("ldr", ctypes.c_int64)]


_ops = None


def load_ops():
    """libmuon.so with the signatures of include/muon_ops.h; raises if it is not built."""
    global _ops
    if _ops is not None:
        return _ops
    lib = load_library()
    P, I32, I64, U64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64
    D, M, UP = ctypes.POINTER(LinearDesc), ctypes.POINTER(MoveDesc), ctypes.POINTER(U64)
    sig = {
        "muon_linear_workspace": [D, I32, UP],
        "muon_linear_forward": [D, P, P, P, P, P, P, P, P, U64, P],
        "muon_linear_grad_act": [D, P, P, P, P, P, P, U64, P],
        "muon_linear_grad_input": [D, P, P, P, P, P, U64, P],
        "muon_linear_grad_weight": [D, P, P, P, P, P, U64, P],
        "muon_linear_backward": [D, P, P, P, P, P, P, P, P, P, U64, P],
        "muon_route_workspace": [I64, I32, UP],
        "muon_route": [P, I32, I64, I32, I32, P, P, P, P, U64, P],
        "muon_dispatch": [M, P, P, P, P, P],
        "muon_dispatch_grad": [M, P, P, P, P],
        "muon_combine": [M, P, P, P, P, P, P],
        "muon_combine_grad": [M, P, P, P, P, P, P, P, P],
        "muon_dropout": [I32, I64, P, P, P, ctypes.c_double, U64, U64, P, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    _ops = lib
    return lib


def _check(rc, where):
    if rc != MUON_OK:
        raise MuonError(rc, where, muon_last_error())


# ------------------------------------------------------------------ helpers


def _dtype(t, what):
    if t.dtype is torch.bfloat16:
        return MUON_BF16
    if t.dtype is torch.float32:
        return MUON_F32
    raise TypeError(f"{what} is {t.dtype}: float32 or bfloat16 is supported")


def _same(x, **others):
    for name, t in others.items():
        if t is None:
            continue
        if t.dtype is not x.dtype:
            raise TypeError(f"{name} is {t.dtype}, x is {x.dtype}")
        if t.device != x.device:
            raise ValueError(f"{name} is on {t.device}, x is on {x.device}")


def _gpu(t, what):
    if t.device.type != "cuda":
        raise ValueError(f"{what} must live on a GPU")


def _rows(t):
    """t with contiguous rows (last dimension of stride 1, no negative strides)."""
    return t if t.shape[-1] <= 1 or t.stride(-1) == 1 else t.contiguous()


def _ld(t):
    """Row stride of a 2-D tensor with contiguous rows."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _ptr(t):
    """The address of a tensor that may be left out.  Null means just that to the C functions, so a tensor that has
    no memory of its own (a wrapper subclass) must not pass for it."""
    if t is None:
        return None
    at = t.data_ptr()
    if not at and t.numel():
        raise ValueError(f"a {type(t).__name__} has no memory of its own: pass the tensor it wraps")
    return at


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


_jit_tracing, _modes, _key_on = torch._C._is_tracing, torch._C._len_torch_dispatch_stack, \
    torch._C._dispatch_tls_is_dispatch_key_included
_PRE_DISPATCH = torch._C.DispatchKey.PreDispatch


def _traced():
    """Whether torch.jit.trace or an fx tracer is recording.  An fx tracer is asked for only where some dispatch mode
    is on, which takes under a microsecond to see; other modes (a FLOP counter, say) are no tracers."""
    if _jit_tracing():
        return True
    if not (_modes() or _key_on(_PRE_DISPATCH)):
        return False
    tracer = sys.modules.get("torch.fx.experimental.proxy_tensor")
    return tracer is not None and tracer.get_proxy_mode() is not None


def _call(name, t, *args):
    """The C function on t's device and current stream."""
    if _traced():
        raise RuntimeError(f"{name} cannot be traced: a tracer would record its outputs' allocation alone")
    index = t.get_device()
    f = getattr(_ops or load_ops(), name)
    if index == torch.cuda.current_device():
        rc = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = f(*args, _raw_stream(index))
    if rc != MUON_OK:
        raise MuonError(rc, name, muon_last_error())


def _activation(name):
    if name not in ACTIVATIONS:
        raise ValueError(f"activation {name!r}: one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[name]


# ------------------------------------------------------------------ linear layers


class _Plan:
    """Descriptor and workspace sizes of a layer: what follows from shapes, strides and types alone."""

    def __init__(self, x, w, act, grouped):
        k, n = w.shape[-2:]
        groups = w.shape[0] if grouped else 0
        if w.stride(-1) == 1 and (k <= 1 or w.stride(-2) >= n):
            layout, ld = 0, w.stride(-2) if k > 1 else max(n, 1)
        else:
            layout, ld = 1, w.stride(-1) if n > 1 else max(k, 1)
        self.rows, self.k, self.n, self.groups, self.layout = x.shape[0], k, n, groups, layout
        self.y_shape, self.x_shape = (self.rows, n), (self.rows, k)
        self.db_shape = (groups, n) if grouped else (n,)
        lead = (groups,) if grouped else ()
        self.dw_shape = (*lead, k, n) if layout == 0 else (*lead, n, k)
        self.args = [_dtype(x, "x"), act, groups, layout, self.rows, k, n, _ld(x), ld, w.stride(0) if grouped else 0]
        self.descs = {}

    def get(self, op, ld):
        """(descriptor, workspace bytes) of one call whose residual or gradient rows are ld apart."""
        got = self.descs.get((op, ld))
        if got is None:
            d = LinearDesc(*self.args, ld, ld)
            need = ctypes.c_uint64(0)
            _check(load_ops().muon_linear_workspace(ctypes.byref(d), op, ctypes.byref(need)), "muon_linear_workspace")
            got = self.descs[(op, ld)] = (ctypes.byref(d), need.value)
        return got


_plans = {}


def _layout_ok(w):
    k, n = w.shape[-2:]
    return (w.stride(-1) == 1 and (k <= 1 or w.stride(-2) >= n)) or (w.stride(-2) == 1 and (n <= 1 or w.stride(-1) >= k))


def _plan(x, w, act, grouped):
    """The plan of x [rows, K] with contiguous rows and a weight with either of its last dimensions contiguous."""
    key = (x.shape, x.stride(), w.shape, w.stride(), x.dtype, act, grouped)
    p = _plans.get(key)
    if p is None:
        if len(_plans) >= 4096:
            _plans.clear()
        p = _plans[key] = _Plan(x, w, act, grouped)
    return p


def _workspace(size, x):
    return torch.empty(size, dtype=torch.uint8, device=x.device) if size else None


def _flat(t, cols):
    if t is None:
        return None
    return _rows(t if t.dim() == 2 else t.reshape(math.prod(t.shape[:-1]), cols))


def _check_linear(x, weight, bias, residual, offsets):
    grouped = offsets is not None
    if not x.is_cuda:
        raise ValueError("x must live on a GPU")
    _dtype(x, "x")
    if weight.dim() != (3 if grouped else 2):
        raise ValueError(f"weight has {weight.dim()} dimensions, expected {3 if grouped else 2}")
    if x.dim() < 1 or (grouped and x.dim() != 2):
        raise ValueError("x must be [rows, K]" if grouped else "x must have at least one dimension")
    k, n = weight.shape[-2:]
    if x.shape[-1] != k:
        raise ValueError(f"x has {x.shape[-1]} columns, the weight takes {k}")
    _same(x, weight=weight, bias=bias, residual=residual)
    want = (weight.shape[0], n) if grouped else (n,)
    if bias is not None and bias.shape != want:
        raise ValueError(f"bias has shape {tuple(bias.shape)}, expected {want}")
    if residual is not None and residual.shape != (*x.shape[:-1], n):
        raise ValueError(f"residual has shape {tuple(residual.shape)}, expected {(*x.shape[:-1], n)}")
    if grouped:
        e = weight.shape[0]
        if not 1 <= e <= 65535:
            raise ValueError(f"{e} experts: 1 to 65535 are supported")
        if offsets.dtype is not torch.int32 or offsets.shape != (e + 1,) or not offsets.is_contiguous():
            raise ValueError(f"offsets must be a contiguous int32 tensor of {e + 1} values")
        if offsets.device != x.device:
            raise ValueError(f"offsets is on {offsets.device}, x is on {x.device}")


def _forward(x, w, bias, residual, offsets, act, keep_z):
    """y and, where asked and the activation has a slope, z; x and residual 2-D with contiguous rows."""
    p = _plan(x, w, act, offsets is not None)
    d, size = p.get(_FORWARD, _ld(residual) if residual is not None else p.n)
    y = torch.empty(p.y_shape, dtype=x.dtype, device=x.device)
    z = torch.empty_like(y) if keep_z and act else None
    ws = _workspace(size, x)
    _call("muon_linear_forward", x, d, _ptr(offsets), x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(residual),
          y.data_ptr(), _ptr(z), _ptr(ws), size)
    return y, z


def _backward(p, dy, x, w, z, offsets, need_x, need_w, need_b):
    """dx, dw, db of plan p for dy [rows, N] with contiguous rows."""
    d, size = p.get(_BACKWARD, _ld(dy))
    dtype, dev = x.dtype, x.device
    dx = torch.empty(p.x_shape, dtype=dtype, device=dev) if need_x else None
    dw = torch.empty(p.dw_shape, dtype=dtype, device=dev) if need_w else None
    db = torch.empty(p.db_shape, dtype=dtype, device=dev) if need_b else None
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
    _call("muon_linear_backward", x, d, _ptr(offsets), x.data_ptr(), w.data_ptr(), _ptr(z), dy.data_ptr(), _ptr(dx),
          _ptr(dw), _ptr(db), _ptr(ws), size)
    if dw is not None and p.layout == 1:
        dw = dw.transpose(-1, -2)
    return dx, dw, db


def linear_forward(x, weight, bias=None, activation="none", residual=None, offsets=None, keep_z=False):
    """``linear`` (or, with ``offsets``, ``expert_linear``) without autograd.

    Returns (y, z); z, the value ahead of the activation, is None unless
    ``keep_z`` and the activation is not "none"."""
    act = _activation(activation)
    _check_linear(x, weight, bias, residual, offsets)
    return _prepared(x, weight, bias, residual, offsets, act, keep_z)[:2]


def _prepared(x, weight, bias, residual, offsets, act, keep_z):
    """The forward pass of checked arguments: y, z, and x and the weight as the kernels read them."""
    k, n = weight.shape[-2:]
    x2 = _flat(x, k)
    w = weight if _layout_ok(weight) else weight.contiguous()
    b = bias if bias is None or bias.is_contiguous() else bias.contiguous()
    y, z = _forward(x2, w, b, _flat(residual, n), offsets, act, keep_z)
    return y if x.dim() == 2 else y.view(*x.shape[:-1], n), z, x2, w


def linear_backward(dy, x, weight, z=None, activation="none", offsets=None, needs=(True, True, True)):
    """(dx, dW, db) of ``linear_forward`` for the gradient dy; needs: which of them are computed.

    z is what ``linear_forward(..., keep_z=True)`` returned (not used by "none").  The residual's gradient is dy."""
    act = _activation(activation)
    _check_linear(x, weight, None, dy, offsets)
    if act and (z is None or z.dtype is not x.dtype or z.device != x.device or not z.is_contiguous()
                or z.numel() != dy.numel()):
        raise ValueError("z must be the tensor that linear_forward(..., keep_z=True) returned")
    k, n = weight.shape[-2:]
    w = weight if _layout_ok(weight) else weight.contiguous()
    x2 = _flat(x, k)
    dx, dw, db = _backward(_plan(x2, w, act, offsets is not None), _flat(dy, n), x2, w, z, offsets, *needs)
    return None if dx is None else dx.view(x.shape), dw, db


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, offsets, act):
        y, z, x2, w = _prepared(x, weight, bias, residual, offsets, act, True)
        ctx.save_for_backward(x2, w, z, offsets)
        ctx.plan, ctx.x_shape = _plan(x2, w, act, offsets is not None), x.shape
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w, z, offsets = ctx.saved_tensors
        need_x, need_w, need_b, need_r = ctx.needs_input_grad[:4]
        dx = dw = db = None
        if need_x or need_w or need_b:
            dx, dw, db = _backward(ctx.plan, _flat(dy, w.shape[-1]), x, w, z, offsets, need_x, need_w, need_b)
            if dx is not None and len(ctx.x_shape) != 2:
                dx = dx.view(ctx.x_shape)
        return dx, dw, db, dy if need_r else None, None, None


def _tracked(*tensors):
    """Whether a call goes through its autograd function: for its gradient or, with forward-mode
    differentiation on, because torch refuses a tangent there (it would be dropped otherwise)."""
    if getattr(forward_ad, "_current_level", 0) >= 0:
        return True
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def linear(x, weight, bias=None, *, activation="none", residual=None):
    """act(x W + b) + residual.

    x [..., K], weight [K, N] (or the transposed view of a [N, K] tensor, read
    in place), bias [N], residual [..., N].  activation: "none", "relu", "silu",
    "gelu" or "gelu_tanh".  Differentiable in every tensor (once); for
    the gradient, z = x W + b is kept in x's type.

    bfloat16: y is rounded once, from float32.  With an activation the gradients are
    taken at the rounded z and from the gradient of z rounded to bfloat16, so dx and dW
    are about 1.4 times as far off as one rounding makes them, in the norm (2.4e-3
    against 1.7e-3); up to 64 rows (16 an expert on average in ``expert_linear``), and
    for "relu", they are not.  float32 tensors carry no such rounding."""
    if not _tracked(x, weight, bias, residual):
        return linear_forward(x, weight, bias, activation, residual)[0]
    _check_linear(x, weight, bias, residual, None)
    return _Linear.apply(x, weight, bias, residual, None, _activation(activation))


def expert_linear(x, weight, offsets, bias=None, *, activation="none"):
    """act(x_p W[e] + b[e]) for the rows p = offsets[e] .. offsets[e + 1] of every expert e.

    x [rows, K], weight [E, K, N] (its last two dimensions in either order in
    memory), offsets [E + 1] int32 on the GPU as ``route`` gives them, bias
    [E, N].  Rows past offsets[E] give zero and get a zero gradient.  The weight's
    gradient [E, K, N] is zero for an expert without rows."""
    if not _tracked(x, weight, bias):
        return linear_forward(x, weight, bias, activation, None, offsets)[0]
    _check_linear(x, weight, bias, None, offsets)
    return _Linear.apply(x, weight, bias, None, offsets, _activation(activation))


# ------------------------------------------------------------------ experts: there and back


class Routing(NamedTuple):
    """Entries (token, choice) sorted by expert.

    offsets [E + 1]: first sorted row of each expert, and the number routed;
    order [tokens * top]: flat entry of each sorted row, -1 past the routed ones;
    position [tokens, top]: sorted row of each entry, -1 where it is not routed.
    All int32 on the GPU."""
    offsets: torch.Tensor
    order: torch.Tensor
    position: torch.Tensor


_route_sizes = {}


def route(expert_ids, n_experts):
    """Sorts the entries of expert_ids [tokens, top] (int64 or int32) by expert, stably.

    An id outside [0, n_experts) (-1, say) is not routed."""
    _gpu(expert_ids, "expert_ids")
    if expert_ids.dim() != 2 or expert_ids.shape[1] < 1:
        raise ValueError("expert_ids must be [tokens, top] with top >= 1")
    if expert_ids.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"expert_ids is {expert_ids.dtype}: int64 or int32 is supported")
    ids = expert_ids.contiguous()
    tokens, top = ids.shape
    need = _route_sizes.get((tokens * top, n_experts))
    if need is None:
        got = ctypes.c_uint64(0)
        _check(load_ops().muon_route_workspace(tokens * top, n_experts, ctypes.byref(got)), "muon_route_workspace")
        if len(_route_sizes) >= 4096:
            _route_sizes.clear()
        need = _route_sizes[(tokens * top, n_experts)] = got.value
    # One allocation holds the three results and the workspace, each 16-byte aligned.
    e4, p4 = (n_experts + 1 + 3) // 4 * 4, (tokens * top + 3) // 4 * 4
    buf = torch.empty(e4 + 2 * p4 + need // 4, dtype=torch.int32, device=ids.device)
    at, end = buf.data_ptr(), tokens * top
    _call("muon_route", ids, ids.data_ptr(), ids.element_size(), tokens, top, n_experts, at, at + 4 * e4,
          at + 4 * (e4 + p4), at + 4 * (e4 + 2 * p4), need)
    return Routing(buf[:n_experts + 1], buf[e4:e4 + end], buf[e4 + p4:e4 + p4 + end].view(tokens, top))


def _check_routing(routing, t, rows, what):
    _gpu(t, what)
    _dtype(t, what)
    if t.dim() != 2:
        raise ValueError(f"{what} must have two dimensions")
    if t.device != routing.position.device:
        raise ValueError(f"{what} is on {t.device}, the routing is on {routing.position.device}")
    if t.shape[0] != rows:
        raise ValueError(f"{what} has {t.shape[0]} rows, expected {rows}")
    p, o = routing.position, routing.offsets
    if o.device != p.device:
        raise ValueError(f"the routing's offsets are on {o.device}, its positions on {p.device}")
    if p.dim() != 2 or p.dtype is not torch.int32 or o.dtype is not torch.int32 or not p.is_contiguous() \
            or not o.is_contiguous() or o.dim() != 1 or o.shape[0] < 2:
        raise ValueError("routing must be what route() returned")


def _dispatch(x, offsets, position):
    tokens, top = position.shape
    x = _rows(x)
    h = x.shape[1]
    d = MoveDesc(_dtype(x, "x"), offsets.shape[0] - 1, top, 0, tokens, h, _ld(x), h, h)
    xs = torch.empty((tokens * top, h), dtype=x.dtype, device=x.device)
    _call("muon_dispatch", x, ctypes.byref(d), offsets.data_ptr(), position.data_ptr(), x.data_ptr(), xs.data_ptr())
    return xs


def _dispatch_grad(dxs, offsets, position):
    tokens, top = position.shape
    dxs = _rows(dxs)
    h = dxs.shape[1]
    d = MoveDesc(_dtype(dxs, "dxs"), offsets.shape[0] - 1, top, 0, tokens, h, _ld(dxs), h, h)
    dx = torch.empty((tokens, h), dtype=dxs.dtype, device=dxs.device)
    _call("muon_dispatch_grad", dxs, ctypes.byref(d), position.data_ptr(), dxs.data_ptr(), dx.data_ptr())
    return dx


def dispatch_forward(x, routing):
    """``dispatch`` without autograd."""
    _check_routing(routing, x, routing.position.shape[0], "x")
    return _dispatch(x, routing.offsets, routing.position)


def dispatch_backward(dxs, routing):
    """dx of ``dispatch``: each token's sum over its rows of dxs."""
    _check_routing(routing, dxs, routing.position.numel(), "dxs")
    return _dispatch_grad(dxs, routing.offsets, routing.position)


def _check_weights(routing, weights):
    if weights.dtype is not torch.float32 or tuple(weights.shape) != tuple(routing.position.shape):
        raise ValueError(f"weights must be float32 of shape {tuple(routing.position.shape)}")
    if weights.device != routing.position.device:
        raise ValueError(f"weights is on {weights.device}, the routing is on {routing.position.device}")


def _combine(ys, offsets, position, weights, residual):
    tokens, top = position.shape
    ys, w = _rows(ys), weights.contiguous()
    h = ys.shape[1]
    residual = None if residual is None else _rows(residual)
    d = MoveDesc(_dtype(ys, "ys"), offsets.shape[0] - 1, top, 0, tokens, h, _ld(ys), h,
                 h if residual is None else _ld(residual))
    y = torch.empty((tokens, h), dtype=ys.dtype, device=ys.device)
    _call("muon_combine", ys, ctypes.byref(d), position.data_ptr(), w.data_ptr(), ys.data_ptr(), _ptr(residual),
          y.data_ptr())
    return y


def _combine_grad(dy, ys, offsets, position, weights, need_ys, need_w):
    tokens, top = position.shape
    dy, ys, w = _rows(dy), _rows(ys), weights.contiguous()
    h = ys.shape[1]
    d = MoveDesc(_dtype(ys, "ys"), offsets.shape[0] - 1, top, 0, tokens, h, _ld(ys), _ld(dy), h)
    dys = torch.empty((tokens * top, h), dtype=ys.dtype, device=ys.device) if need_ys else None
    dw = torch.empty((tokens, top), dtype=torch.float32, device=ys.device) if need_w else None
    _call("muon_combine_grad", ys, ctypes.byref(d), offsets.data_ptr(), position.data_ptr(), w.data_ptr(),
          ys.data_ptr(), dy.data_ptr(), _ptr(dys), _ptr(dw))
    return dys, dw


def _check_combine(ys, routing, weights, residual):
    _check_routing(routing, ys, routing.position.numel(), "ys")
    _check_weights(routing, weights)
    if residual is not None:
        _same(ys, residual=residual)
        want = (routing.position.shape[0], ys.shape[1])
        if residual.shape != want:
            raise ValueError(f"residual has shape {tuple(residual.shape)}, expected {want}")


def combine_forward(ys, routing, weights, residual=None):
    """``combine`` without autograd (weights float32)."""
    _check_combine(ys, routing, weights, residual)
    return _combine(ys, routing.offsets, routing.position, weights, residual)


def combine_backward(dy, ys, routing, weights, needs=(True, True)):
    """(dys, dweights) of ``combine``; needs: which of them are computed."""
    _check_routing(routing, dy, routing.position.shape[0], "dy")
    _check_routing(routing, ys, routing.position.numel(), "ys")
    _check_weights(routing, weights)
    _same(ys, dy=dy)
    if dy.shape[1] != ys.shape[1]:
        raise ValueError(f"dy has {dy.shape[1]} columns, ys has {ys.shape[1]}")
    return _combine_grad(dy, ys, routing.offsets, routing.position, weights, *needs)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, offsets, position):
        ctx.save_for_backward(offsets, position)
        return _dispatch(x, offsets, position)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dxs):
        return _dispatch_grad(dxs, *ctx.saved_tensors), None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, weights, residual, offsets, position):
        ctx.save_for_backward(ys, weights, offsets, position)
        return _combine(ys, offsets, position, weights, residual)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        ys, weights, offsets, position = ctx.saved_tensors
        need_ys, need_w, need_r = ctx.needs_input_grad[:3]
        dys = dw = None
        if need_ys or need_w:
            dys, dw = _combine_grad(dy, ys, offsets, position, weights, need_ys, need_w)
        return dys, dw, dy if need_r else None, None, None


def dispatch(x, routing):
    """Rows of x [tokens, H] in sorted order: xs[position[t][j]] = x[t], [tokens * top, H].

    Rows past the routed ones are zero.  Differentiable in x."""
    _check_routing(routing, x, routing.position.shape[0], "x")
    if not _tracked(x):
        return _dispatch(x, routing.offsets, routing.position)
    return _Dispatch.apply(x, routing.offsets, routing.position)


def combine(ys, routing, weights, residual=None):
    """y[t] = sum_j weights[t][j] ys[position[t][j]] (+ residual[t]), [tokens, H].

    Entries that were not routed add nothing.  weights [tokens, top] (bfloat16 is
    taken as float32).  Differentiable in ys, weights and residual."""
    if weights.dtype is torch.bfloat16:
        weights = weights.float()
    if not _tracked(ys, weights, residual):
        return combine_forward(ys, routing, weights, residual)
    _check_combine(ys, routing, weights, residual)
    return _Combine.apply(ys, weights, residual, routing.offsets, routing.position)


# ------------------------------------------------------------------ dropout


def dropout_forward(x, p, seed=0, offset=0, residual=None, state=None):
    """``dropout`` without autograd.  The gradient of x is the same call on dy without a residual."""
    _gpu(x, "x")
    code = _dtype(x, "x")
    if not 0.0 <= p < 1.0:
        raise ValueError(f"p is {p}: 0 <= p < 1 is supported")
    _same(x, residual=residual)
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, x {tuple(x.shape)}")
    if state is not None and (state.dtype is not torch.int64 or state.numel() != 2 or state.device != x.device
                              or not state.is_contiguous()):
        raise ValueError("state must be two contiguous int64 values on x's device: seed, offset")
    x = x.contiguous()
    residual = None if residual is None else residual.contiguous()
    y = torch.empty_like(x)
    _call("muon_dropout", x, code, x.numel(), x.data_ptr(), _ptr(residual), y.data_ptr(), p,
          seed & 0xFFFFFFFFFFFFFFFF, offset & 0xFFFFFFFFFFFFFFFF, _ptr(state))
    return y


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset, state):
        # A copy: the mask of the gradient is this pass's, whatever the caller writes into state later.
        ctx.state = None if state is None else state.clone()
        ctx.p, ctx.seed, ctx.offset = p, seed, offset
        return dropout_forward(x, p, seed, offset, residual, ctx.state)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        dx = dropout_forward(dy, ctx.p, ctx.seed, ctx.offset, None, ctx.state) if ctx.needs_input_grad[0] else None
        return dx, dy if ctx.needs_input_grad[1] else None, None, None, None, None


def dropout(x, p, *, seed=0, offset=0, residual=None, state=None):
    """x with each element zeroed with probability p and the others scaled by 1 / (1 - p), plus residual.

    p is taken to the nearest of 65536 steps; one that comes to 1 so is refused.  The mask follows from (seed,
    offset) and an element's flat index alone: calls that must differ get another
    seed or offset.  state: an int64 tensor [seed, offset] on the GPU used in
    their place, which a captured graph reads at every replay.  Differentiable
    in x and residual."""
    if not _tracked(x, residual):
        return dropout_forward(x, p, seed, offset, residual, state)
    return _Dropout.apply(x, residual, p, seed, offset, state)
