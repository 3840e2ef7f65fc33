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

Gradients are explicit calls, as everything in the library is.  Tensors are contiguous CUDA tensors of
one device; a call is enqueued on ``stream`` (default: the tensors' device's current stream) and
allocates only what it returns and its workspace, from torch's allocator.  Wrong types, shapes or
devices raise TypeError or ValueError before anything is enqueued.  Output buffers may be passed in
(``out``, ``dy``, ``dx``); rows of grouped buffers that hold no pair (padding) are never written.
"""
from __future__ import annotations

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


def _tensor(t, name, like=None, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has type {t.dtype}, not {dtype}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, not {like.device}")
    return t


def _type(t, name):
    if t.dtype not in _TYPES:
        raise TypeError(f"{name} has type {t.dtype}; bfloat16, float16 and float32 are supported")
    return _TYPES[t.dtype]


def _on(t, stream):
    """The raw handle of the stream of a call on t's device."""
    if not t.is_cuda:
        raise ValueError(f"tensors must be on a CUDA device, not {t.device}")
    if stream is None:
        return torch.cuda.current_stream(t.device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _empty(shape, dtype, like, stream):
    """A new tensor that the call's stream uses first (the allocator learns of a stream of its own)."""
    t = torch.empty(shape, dtype=dtype, device=like.device)
    if isinstance(stream, torch.cuda.Stream):
        t.record_stream(stream)
    return t


def _pairs(r: Routing, like):
    T, k = r.topk_w.shape
    _tensor(r.topk_w, "topk_w", like, torch.float32)
    _tensor(r.pos_of_pair, "pos_of_pair", like, torch.int32, (T * k,))
    return T, k


def _out(out, shape, dtype, like, name, stream):
    if out is None:
        return _empty(shape, dtype, like, stream)
    return _tensor(out, name, like, dtype, shape)


def max_grouped_rows(pairs: int, num_experts: int) -> int:
    """Rows that the grouped layout of so many pairs may take at most."""
    m = moe_mx.moe_mx_block_rows()
    return (pairs + min(pairs, num_experts) * (m - 1) + m - 1) // m * m


def route_group(router_logits: torch.Tensor, top_k: int, stream=None) -> Routing:
    """Softmax top-k routing of float32 logits [T, E] and the grouped layout of the pairs
    (moe_mx_route_group_noalloc, whose calls on one device share a scratch: order them)."""
    _tensor(router_logits, "router_logits", dtype=torch.float32)
    if router_logits.dim() != 2:
        raise ValueError("router_logits must be [tokens, experts]")
    T, E = router_logits.shape
    on = _on(router_logits, stream)
    rows = max_grouped_rows(T * top_k, E)
    new = lambda *shape, dtype=torch.int32: _empty(shape, dtype, router_logits, stream)  # noqa: E731
    ids, w = new(T, top_k), new(T, top_k, dtype=torch.float32)
    counts, pad, pos, pair = new(E), new(E + 1), new(T * top_k), new(rows)
    if T == 0:
        counts.zero_()
        pad.zero_()
    with torch.cuda.device(router_logits.device):
        moe_mx.moe_mx_route_group_noalloc(router_logits, T, E, top_k, ids, w, counts, pad, pair, pos, on)
    return Routing(ids, w, counts, pad, pos, rows)


def dispatch(x: torch.Tensor, routing: Routing, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Token rows x [T, H] at their pairs' grouped rows: [rows, H]; padding rows are not written."""
    T, k = _pairs(routing, x)
    _tensor(x, "x", shape=(T, x.shape[-1]))
    on = _on(x, stream)
    out = _out(out, (routing.rows, x.shape[1]), x.dtype, x, "out", stream)
    moe_mx.moe_mx_dispatch(x, T, x.shape[1], k, routing.pos_of_pair, routing.rows, _type(x, "x"), out, on)
    return out


def _combine(grouped, routing, w, out_dtype, out, stream):
    T, k = _pairs(routing, grouped)
    _tensor(grouped, "grouped", shape=(routing.rows, grouped.shape[-1]))
    on = _on(grouped, stream)
    if out is not None:
        out_dtype = out.dtype
    out = _out(out, (T, grouped.shape[1]), out_dtype or grouped.dtype, grouped, "out", stream)
    moe_mx.moe_mx_combine(grouped, routing.rows, T, grouped.shape[1], k, routing.pos_of_pair, w,
                          _type(grouped, "grouped"), _type(out, "out"), out, on)
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
    T, k = _pairs(routing, dout)
    H = dout.shape[-1]
    _tensor(dout, "dout", shape=(T, H))
    _tensor(grouped, "grouped", dout, shape=(routing.rows, H))
    on = _on(dout, stream)
    dy = _out(dy, (routing.rows, H), grouped.dtype, dout, "dy", stream)
    dw = _empty((T, k), torch.float32, dout, stream)
    dlogits = None
    if num_experts:
        _tensor(routing.topk_ids, "topk_ids", dout, torch.int32, (T, k))
        dlogits = _empty((T, num_experts), torch.float32, dout, stream)
    moe_mx.moe_mx_combine_backward(dout, grouped, routing.rows, T, H, k, routing.pos_of_pair, routing.topk_w,
                                   routing.topk_ids, num_experts, _type(grouped, "grouped"), _type(dout, "dout"), dy,
                                   dw, dlogits, on)
    return dy, dw, dlogits


def _linear_sizes(x, w, activation, routing):
    """(experts, rows, N, K, activation, columns of out) of a linear call, its operands checked."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation {activation!r} is not one of {', '.join(ACTIVATIONS)}")
    _tensor(x, "x")
    _tensor(w, "w", x, x.dtype)
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"x has type {x.dtype}; bfloat16 and float16 are supported")
    E = 0 if routing is None else routing.counts.shape[0]
    if x.dim() != 2 or w.dim() != (3 if E else 2) or w.shape[-1] != x.shape[1] or (E and w.shape[0] != E):
        raise ValueError(f"x {tuple(x.shape)} and w {tuple(w.shape)}: need [rows, K] and "
                         + (f"[{E}, N, K]" if E else "[N, K]"))
    rows, K = x.shape
    N = w.shape[-2]
    if E:
        if rows != routing.rows:
            raise ValueError(f"x has {rows} rows, the grouped layout {routing.rows}")
        _tensor(routing.counts, "counts", x, torch.int32, (E,))
        _tensor(routing.pad_offsets, "pad_offsets", x, torch.int32, (E + 1,))
    if activation == "swiglu" and N % 2:
        raise ValueError(f"swiglu needs an even number of weight rows, not {N}")
    return E, rows, N, K, ACTIVATIONS[activation], N // 2 if activation == "swiglu" else N


def _segments(routing):
    return (None, None) if routing is None else (routing.counts, routing.pad_offsets)


def linear(x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None = None,
           residual: torch.Tensor | None = None, activation: str = "none", routing: Routing | None = None,
           out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
           preact: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """activation(x w^T + bias) + residual.  x [rows, K], w [N, K], bias float32 [N]; with ``routing`` the
    rows are grouped, w [E, N, K] and bias [E, N].  out and residual: [rows, N] ([rows, N/2] for
    swiglu) of x's type or float32; residual may be out itself.  A ``preact`` buffer [rows, N] receives
    x w^T + bias for linear_backward."""
    E, rows, N, K, act, cols = _linear_sizes(x, w, activation, routing)
    on = _on(x, stream)
    if bias is not None:
        _tensor(bias, "bias", x, torch.float32, (E, N) if E else (N,))
    if out is not None:
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = x.dtype if residual is None else residual.dtype
    out = _out(out, (rows, cols), out_dtype, x, "out", stream)
    if residual is not None:
        _tensor(residual, "residual", x, out_dtype, (rows, cols))
    if preact is not None:
        _tensor(preact, "preact", x, x.dtype, (rows, N))
    dt, ot = _type(x, "x"), _type(out, "out")
    need = moe_mx.moe_mx_linear_workspace(E, rows, N, K, dt, act, ot)
    ws = _empty(need, torch.uint8, x, stream) if need else None
    moe_mx.moe_mx_linear(x, w, bias, residual, *_segments(routing), E, rows, N, K, dt, act, ot, out, preact, ws, need,
                         on)
    return out


def linear_backward(dout: torch.Tensor, x: torch.Tensor, w: torch.Tensor, preact: torch.Tensor | None = None,
                    activation: str = "none", routing: Routing | None = None, bias_grad: bool = False,
                    input_grad: bool = True, weight_grad: bool = True, dx: torch.Tensor | None = None,
                    dw: torch.Tensor | None = None, stream=None):
    """Gradient of linear: (dx, dw, dbias), None for those not asked for.  dout is of x's type or float32;
    preact as linear wrote it (for an activation).  The residual's gradient is dout."""
    E, rows, N, K, act, cols = _linear_sizes(x, w, activation, routing)
    on = _on(x, stream)
    _tensor(dout, "dout", x, shape=(rows, cols))
    if activation != "none":
        _tensor(preact, "preact", x, x.dtype, (rows, N))
    elif preact is not None:
        raise ValueError("preact is taken with an activation only")
    if not (input_grad or weight_grad or bias_grad):
        raise ValueError("no gradient is asked for")
    dx = _out(dx, (rows, K), x.dtype, x, "dx", stream) if input_grad else None
    dw = _out(dw, tuple(w.shape), x.dtype, x, "dw", stream) if weight_grad else None
    db = _empty((E, N) if E else (N,), torch.float32, x, stream) if bias_grad else None
    dt, gt = _type(x, "x"), _type(dout, "dout")
    need = moe_mx.moe_mx_linear_backward_workspace(E, rows, N, K, dt, act, gt)
    ws = _empty(need, torch.uint8, x, stream) if need else None
    moe_mx.moe_mx_linear_backward(dout, x, w, preact, *_segments(routing), E, rows, N, K, dt, act, gt, dx, dw, db, ws,
                                  need, on)
    return dx, dw, db
