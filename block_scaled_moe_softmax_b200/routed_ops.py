"""The routed operators on torch tensors: routing and grouping, dispatch, linear, combine, and their
gradients (the ``moe_mx_*`` entry points of the same names in include/moe_mx.h).

    logits = linear(x, w_router, b_router, out_dtype=torch.float32)
    r = route_group(logits, top_k)
    h = linear(dispatch(x, r), w1, activation="swiglu", routing=r, preact=z)   # w1 [E, 2I, H]
    y = linear(h, w2, routing=r)                                               # w2 [E, H, I]
    out = combine(y, r)

    dy, dw, dlogits = combine_backward(dout, y, r, num_experts=E)
    dh, dw2, _ = linear_backward(dy, h, w2, routing=r)
    dg, dw1, _ = linear_backward(dh, g, w1, preact=z, activation="swiglu", routing=r)
    dx = dispatch_backward(dg, r)

Gradients are explicit calls, as everything in the library is: results carry no autograd history.  A call
on a tensor that requires a gradient, with autograd recording, warns (once a place); under
``torch.no_grad()`` it is silent.  Tensors are contiguous CUDA tensors of one device that start on 16 bytes
(MoeMxError else); a call is enqueued on ``stream`` (a torch.cuda.Stream or a raw handle; default: the current
stream of the tensors' device) and allocates only what it returns and its workspace, from torch's
allocator, as under ``with torch.cuda.stream(stream)``.  Wrong types, shapes or
devices raise TypeError or ValueError before anything is enqueued.  Output buffers may be passed in
(``out``, ``dy``, ``dx``); rows of grouped buffers that hold no pair (padding) are never written.

Every wait inside linear and linear_backward is bounded.  Calls return before their kernels run, so one whose
wait gives up (a GPU that stalls for seconds) leaves its result unfinished without an error there:
``check()`` waits for a stream and raises if that happened.  Call it where results leave the GPU anyway,
e.g. once a step.
"""
from __future__ import annotations

import functools
import warnings
from typing import NamedTuple

import torch

from . import moe_mx

_TYPES = {torch.bfloat16: moe_mx.MOE_MX_TYPE_BF16, torch.float32: moe_mx.MOE_MX_TYPE_F32,
          torch.float16: moe_mx.MOE_MX_TYPE_F16}
ACTIVATIONS = {"none": moe_mx.MOE_MX_LINEAR_NONE, "silu": moe_mx.MOE_MX_LINEAR_SILU,
               "gelu": moe_mx.MOE_MX_LINEAR_GELU, "swiglu": moe_mx.MOE_MX_LINEAR_SWIGLU}


class Routing(NamedTuple):
    """Where each (token, slot) pair goes, as route_group returns it."""
    topk_ids: torch.Tensor     # int32 [T, k] experts
    topk_w: torch.Tensor       # float32 [T, k] weights
    counts: torch.Tensor       # int32 [E] pairs of each expert
    pad_offsets: torch.Tensor  # int32 [E + 1] first grouped row of each expert
    pos_of_pair: torch.Tensor  # int32 [T * k] grouped row of each pair, -1: none
    rows: int                  # rows of the grouped buffers


def _tensor(t, name, device, dtype=None, shape=None):
    """t, checked: a contiguous tensor on CUDA device number ``device``, of the given type and shape."""
    # one test for the usual case: these checks are a good part of a small call's time on the host
    if (isinstance(t, torch.Tensor) and (dtype is None or t.dtype is dtype) and (shape is None or t.shape == shape)
            and t.is_contiguous() and t.get_device() == device):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has type {t.dtype}, not {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, not on {'the CPU' if device < 0 else f'cuda:{device}'}")


def _no_history(name, level=3):
    """Warns that a call's result is detached from an input that requires a gradient."""
    if torch.is_grad_enabled():
        warnings.warn(f"{name}: an input requires a gradient, but the result carries no autograd history; call "
                      "the gradient yourself, or under torch.no_grad() to say so", stacklevel=level)


def _device(t, name):
    """The number of t's CUDA device (-1 for a CPU tensor, which _on refuses)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    return t.get_device()


def _type(t, name):
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} has type {t.dtype}; bfloat16, float16 and float32 are supported")
    return code


def _on(t, device, stream):
    """The raw handle of the stream of a call on t's device."""
    if device < 0:
        raise ValueError(f"tensors must be on a CUDA device, not {t.device}")
    if stream is None:
        return _raw_stream(device)
    if isinstance(stream, int):
        return stream
    if stream.device_index != device:
        raise ValueError(f"stream is one of cuda:{stream.device_index}, the tensors are on cuda:{device}")
    return stream.cuda_stream


# The current stream's handle without a Stream object around it (2 us less a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _empty(shape, dtype, like, stream):
    """A new tensor of the call's stream: on another stream than the current one it comes from that
    stream's pool, since memory freed on the current stream may still be in use there."""
    if stream is None:
        return like.new_empty(*shape) if dtype is like.dtype else like.new_empty(*shape, dtype=dtype)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=like.device)
    with torch.cuda.stream(stream):
        return like.new_empty(*shape, dtype=dtype)


def _pairs(r: Routing, device):
    """(tokens, slots) of a routing whose weights and rows are checked."""
    _tensor(r.topk_w, "topk_w", device, torch.float32)
    shape = r.topk_w.shape
    if len(shape) != 2:
        raise ValueError("topk_w must be [tokens, slots]")
    T, k = shape
    _tensor(r.pos_of_pair, "pos_of_pair", device, torch.int32, (T * k,))
    return T, k


def _matrix(t, name, device, rows=None, dtype=None):
    """t as a checked [rows, columns] matrix; its columns."""
    shape = t.shape if isinstance(t, torch.Tensor) else None
    if shape is not None and (len(shape) != 2 or (rows is not None and shape[0] != rows)):
        raise ValueError(f"{name} has shape {tuple(shape)}, not [{'rows' if rows is None else rows}, columns]")
    _tensor(t, name, device, dtype)
    return shape[1]


def _out(out, shape, dtype, like, device, name, stream):
    if out is None:
        return _empty(shape, dtype, like, stream)
    return _tensor(out, name, device, dtype, shape)


def _call(name, *args):
    """The entry point of that name on raw arguments; raises MoeMxError."""
    code = getattr(moe_mx._lib or moe_mx.load_library(), name)(*args)
    if code:
        raise moe_mx.MoeMxError(code, moe_mx.moe_mx_last_error())


def _ptr(t):
    return None if t is None else t.data_ptr()


_linear_workspace = functools.lru_cache(1024)(moe_mx.moe_mx_linear_workspace)  # by sizes and types alone
_linear_backward_workspace = functools.lru_cache(1024)(moe_mx.moe_mx_linear_backward_workspace)


def max_grouped_rows(pairs: int, num_experts: int) -> int:
    """Rows that the grouped layout of so many pairs may take at most."""
    m = moe_mx.moe_mx_block_rows()
    return (pairs + min(pairs, num_experts) * (m - 1) + m - 1) // m * m


def route_group(router_logits: torch.Tensor, top_k: int, stream=None) -> Routing:
    """Softmax top-k routing of float32 logits [T, E] and the grouped layout of the pairs
    (moe_mx_route_group_noalloc, whose calls on one device share a scratch: order them)."""
    dev = _device(router_logits, "router_logits")
    E = _matrix(router_logits, "router_logits", dev, dtype=torch.float32)
    T = router_logits.shape[0]
    on = _on(router_logits, dev, stream)
    if router_logits.requires_grad:
        _no_history("route_group")
    rows = max_grouped_rows(T * top_k, E)
    new = lambda *shape, dtype=torch.int32: _empty(shape, dtype, router_logits, stream)  # noqa: E731
    ids, w = new(T, top_k), new(T, top_k, dtype=torch.float32)
    counts, pad, pos, pair = new(E), new(E + 1), new(T * top_k), new(rows)
    if T == 0:
        # on the call's stream, whose pool they are of
        with torch.cuda.stream(torch.cuda.ExternalStream(on, device=router_logits.device)):
            counts.zero_()
            pad.zero_()
    with torch.cuda.device(dev):
        moe_mx.moe_mx_route_group_noalloc(router_logits, T, E, top_k, ids, w, counts, pad, pair, pos, on)
    return Routing(ids, w, counts, pad, pos, rows)


def dispatch(x: torch.Tensor, routing: Routing, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Token rows x [T, H] at their pairs' grouped rows: [rows, H]; padding rows are not written."""
    dev = _device(x, "x")
    T, k = _pairs(routing, dev)
    H = _matrix(x, "x", dev, T)
    on = _on(x, dev, stream)
    code = _type(x, "x")
    if x.requires_grad:
        _no_history("dispatch")
    out = _out(out, (routing.rows, H), x.dtype, x, dev, "out", stream)
    _call("moe_mx_dispatch", x.data_ptr(), T, H, k, routing.pos_of_pair.data_ptr(), routing.rows, code, out.data_ptr(),
          on)
    return out


def _combine(grouped, routing, w, out_dtype, out, stream):
    dev = _device(grouped, "grouped")
    T, k = _pairs(routing, dev)
    H = _matrix(grouped, "grouped", dev, routing.rows)
    on = _on(grouped, dev, stream)
    code = _type(grouped, "grouped")
    if grouped.requires_grad or (w is not None and w.requires_grad):
        _no_history("dispatch_backward" if w is None else "combine", 4)
    if out is not None:
        out_dtype = out.dtype
    out = _out(out, (T, H), out_dtype or grouped.dtype, grouped, dev, "out", stream)
    _call("moe_mx_combine", grouped.data_ptr(), routing.rows, T, H, k, routing.pos_of_pair.data_ptr(), _ptr(w), code,
          _type(out, "out"), out.data_ptr(), on)
    return out


def combine(grouped: torch.Tensor, routing: Routing, out_dtype: torch.dtype | None = None,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The weighted sum of each token's grouped rows [rows, H]: [T, H]."""
    return _combine(grouped, routing, routing.topk_w, out_dtype, out, stream)


def dispatch_backward(dgrouped: torch.Tensor, routing: Routing, out_dtype: torch.dtype | None = None,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of dispatch: the plain sum of each token's grouped rows."""
    return _combine(dgrouped, routing, None, out_dtype, out, stream)


def combine_backward(dout: torch.Tensor, grouped: torch.Tensor, routing: Routing, num_experts: int = 0,
                     dy: torch.Tensor | None = None, stream=None):
    """Gradient of combine: (dgrouped [rows, H], dtopk_w [T, k], dlogits [T, num_experts] or None when
    num_experts is 0).  dlogits is the gradient through the router's softmax over the chosen logits."""
    dev = _device(dout, "dout")
    T, k = _pairs(routing, dev)
    H = _matrix(dout, "dout", dev, T)
    _tensor(grouped, "grouped", dev, None, (routing.rows, H))
    on = _on(dout, dev, stream)
    code, dout_code = _type(grouped, "grouped"), _type(dout, "dout")
    dy = _out(dy, (routing.rows, H), grouped.dtype, dout, dev, "dy", stream)
    w = routing.topk_w
    dw = _empty((T, k), torch.float32, w, stream)
    ids = dlogits = None
    if num_experts:
        ids = _tensor(routing.topk_ids, "topk_ids", dev, torch.int32, (T, k))
        dlogits = _empty((T, num_experts), torch.float32, w, stream)
    _call("moe_mx_combine_backward", dout.data_ptr(), grouped.data_ptr(), routing.rows, T, H, k,
          routing.pos_of_pair.data_ptr(), w.data_ptr(), _ptr(ids), num_experts, code, dout_code, dy.data_ptr(),
          dw.data_ptr(), _ptr(dlogits), on)
    return dy, dw, dlogits


def _linear_sizes(x, w, activation, routing, dev):
    """(experts, rows, N, K, activation, columns of out, counts, pad_offsets) of a linear call, its operands
    checked; raw pointers for the last two."""
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation {activation!r} is not one of {', '.join(ACTIVATIONS)}")
    K = _matrix(x, "x", dev)
    if x.dtype is not torch.bfloat16 and x.dtype is not torch.float16:
        raise TypeError(f"x has type {x.dtype}; bfloat16 and float16 are supported")
    _tensor(w, "w", dev, x.dtype)
    E = 0
    if routing is not None:
        E = _tensor(routing.counts, "counts", dev, torch.int32).numel()
        if E == 0:
            raise ValueError("the routing has no experts")
    shape = w.shape
    if len(shape) != (3 if E else 2) or shape[-1] != K or (E and shape[0] != E):
        raise ValueError(f"x {tuple(x.shape)} and w {tuple(shape)}: need [rows, K] and "
                         + (f"[{E}, N, K]" if E else "[N, K]"))
    rows, N = x.shape[0], shape[-2]
    counts = pad = None
    if E:
        if rows != routing.rows:
            raise ValueError(f"x has {rows} rows, the grouped layout {routing.rows}")
        counts = _tensor(routing.counts, "counts", dev, torch.int32, (E,)).data_ptr()
        pad = _tensor(routing.pad_offsets, "pad_offsets", dev, torch.int32, (E + 1,)).data_ptr()
    cols = N
    if activation == "swiglu":
        if N % 2:
            raise ValueError(f"swiglu needs an even number of weight rows, not {N}")
        cols = N // 2
    return E, rows, N, K, act, cols, counts, pad


def linear(x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None = None,
           residual: torch.Tensor | None = None, activation: str = "none", routing: Routing | None = None,
           out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
           preact: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """activation(x w^T + bias) + residual.  x [rows, K], w [N, K], bias float32 [N]; with ``routing`` the
    rows are grouped, w [E, N, K] and bias [E, N].  out and residual: [rows, N] ([rows, N/2] for
    swiglu) of x's type or float32; residual may be out itself.  A ``preact`` buffer [rows, N] receives
    x w^T + bias for linear_backward."""
    dev = _device(x, "x")
    E, rows, N, K, act, cols, counts, pad = _linear_sizes(x, w, activation, routing, dev)
    on = _on(x, dev, stream)
    if bias is not None:
        _tensor(bias, "bias", dev, torch.float32, (E, N) if E else (N,))
    if out is not None:
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = x.dtype if residual is None else residual.dtype
    if out_dtype is not x.dtype and out_dtype is not torch.float32:
        raise TypeError(f"out has type {out_dtype}; {x.dtype} (x's) and float32 are supported")
    out = _out(out, (rows, cols), out_dtype, x, dev, "out", stream)
    if residual is not None:
        _tensor(residual, "residual", dev, out_dtype, (rows, cols))
    if preact is not None:
        _tensor(preact, "preact", dev, x.dtype, (rows, N))
    if x.requires_grad or w.requires_grad or (bias is not None and bias.requires_grad) or \
            (residual is not None and residual.requires_grad):
        _no_history("linear")
    dt, ot = _type(x, "x"), _type(out, "out")
    need = _linear_workspace(E, rows, N, K, dt, act, ot)
    ws = _empty((need,), torch.uint8, x, stream) if need else None
    _call("moe_mx_linear", x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(residual), counts, pad, E, rows, N, K, dt, act,
          ot, out.data_ptr(), _ptr(preact), _ptr(ws), need, on)
    return out


def linear_backward(dout: torch.Tensor, x: torch.Tensor, w: torch.Tensor, preact: torch.Tensor | None = None,
                    activation: str = "none", routing: Routing | None = None, bias_grad: bool = False,
                    input_grad: bool = True, weight_grad: bool = True, dx: torch.Tensor | None = None,
                    dw: torch.Tensor | None = None, stream=None):
    """Gradient of linear: (dx, dw, dbias), None for those not asked for.  dout is of x's type or float32;
    preact as linear wrote it (for an activation).  The residual's gradient is dout."""
    dev = _device(x, "x")
    E, rows, N, K, act, cols, counts, pad = _linear_sizes(x, w, activation, routing, dev)
    on = _on(x, dev, stream)
    _tensor(dout, "dout", dev, None, (rows, cols))
    if dout.dtype is not x.dtype and dout.dtype is not torch.float32:
        raise TypeError(f"dout has type {dout.dtype}; {x.dtype} (x's) and float32 are supported")
    if act:
        _tensor(preact, "preact", dev, x.dtype, (rows, N))
    elif preact is not None:
        raise ValueError("preact is taken with an activation only")
    if not (input_grad or weight_grad or bias_grad):
        raise ValueError("no gradient is asked for")
    dt, gt = _type(x, "x"), _type(dout, "dout")
    dx = _out(dx, (rows, K), x.dtype, x, dev, "dx", stream) if input_grad else None
    dw = _out(dw, w.shape, x.dtype, x, dev, "dw", stream) if weight_grad else None
    db = _empty((E, N) if E else (N,), torch.float32, x, stream) if bias_grad else None
    need = _linear_backward_workspace(E, rows, N, K, dt, act, gt)
    ws = _empty((need,), torch.uint8, x, stream) if need else None
    _call("moe_mx_linear_backward", dout.data_ptr(), x.data_ptr(), w.data_ptr(), _ptr(preact), counts, pad, E, rows, N,
          K, dt, act, gt, _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws), need, on)
    return dx, dw, db


def check(device: torch.device | int | None = None, stream=None) -> None:
    """Wait for ``stream`` (default: the device's current one) and raise MoeMxError (code MOE_MX_ERR_TIMEOUT) if
    a linear or linear_backward of the device (default: the current one) left a result unfinished since the
    last check.  Later calls are not affected by one that failed."""
    dev = torch.device("cuda") if device is None else torch.device("cuda", device) if isinstance(device, int) else \
        torch.device(device)
    if dev.type != "cuda":
        raise ValueError(f"device must be a CUDA device, not {dev}")
    index = torch.cuda.current_device() if dev.index is None else dev.index
    if stream is None:
        stream = _raw_stream(index)
    _call("moe_mx_linear_status", index, stream if isinstance(stream, int) else stream.cuda_stream)
