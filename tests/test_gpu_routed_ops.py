"""The routed operators (dispatch, combine, linear and their gradients) against plain float64 code."""
import math
import os
import subprocess
import sys
import warnings

import pytest
import torch

from block_scaled_moe_softmax_b200 import moe_mx
from tests import routed_ref as ref

ops = pytest.importorskip("block_scaled_moe_softmax_b200.routed_ops")
pytestmark = pytest.mark.gpu
BF, HF, F = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def rnd(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def untouched(buf, written, fill):
    """Rows of a grouped buffer that hold no pair keep the fill."""
    keep = torch.ones(buf.shape[0], dtype=torch.bool, device=buf.device)
    keep[written] = False
    assert torch.equal(buf[keep], torch.full_like(buf[keep], fill))


# ---------------------------------------------------------------- dispatch and combine
PERMUTE = [  # T, E, k, H, drop, hot
    (1, 1, 1, 8, 0.0, None), (1, 8, 2, 1, 0.0, None), (16, 8, 2, 256, 0.0, None), (7, 5, 3, 33, 0.3, None),
    (300, 60, 6, 1000, 0.1, None), (130, 4, 2, 130, 0.0, 1), (64, 40, 32, 72, 0.5, None), (3, 8, 2, 7168, 0.0, None),
    (5, 9, 9, 2056, 1.0, None),
]


@pytest.mark.parametrize("dtype", [BF, HF, F])
@pytest.mark.parametrize("T,E,k,H,drop,hot", PERMUTE)
def test_dispatch_copies_every_pair(T, E, k, H, drop, hot, dtype):
    r = ref.make_routing(T, E, k, 1, drop, hot)
    x = rnd((T, H), dtype, 2)
    out = torch.full((r.rows, H), 7.0, dtype=dtype, device="cuda")
    assert ops.dispatch(x, r, out=out) is out
    pos = r.pos_of_pair.long()
    tok = torch.arange(T * k, device="cuda") // k
    assert torch.equal(out[pos[pos >= 0]], x[tok[pos >= 0]])
    untouched(out, pos[pos >= 0], 7.0)


def _combine64(y, r, weighted):
    T, k = r.topk_w.shape
    pos = r.pos_of_pair.long().view(T, k)
    live = (pos >= 0)[..., None]
    rows = torch.where(live, y[pos.clamp(min=0)].to(ref.F64), 0.0)
    w = r.topk_w.to(ref.F64)[..., None] if weighted else 1.0
    return (rows * w).sum(1), (rows * w).abs().sum(1) * (k + 1) * 2.0 ** -23


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, F), (F, BF), (F, F), (BF, HF)])
@pytest.mark.parametrize("T,E,k,H,drop,hot", PERMUTE)
def test_combine_sums_every_pair(T, E, k, H, drop, hot, dtype, out, weighted):
    r = ref.make_routing(T, E, k, 3, drop, hot)
    y = torch.full((r.rows, H), math.nan, dtype=dtype, device="cuda")  # padding must not be read
    pos = r.pos_of_pair.long()
    y[pos[pos >= 0]] = rnd((int((pos >= 0).sum()), H), dtype, 4)
    got = (ops.combine if weighted else ops.dispatch_backward)(y, r, out_dtype=out)
    assert got.dtype == out
    ref.close(got, *_combine64(y, r, weighted), "combine")


@pytest.mark.parametrize("dtype,dout_t", [(BF, BF), (HF, F), (F, BF), (F, F)])
@pytest.mark.parametrize("T,E,k,H,drop,hot", PERMUTE)
def test_combine_backward(T, E, k, H, drop, hot, dtype, dout_t):
    r = ref.make_routing(T, E, k, 5, drop, hot)
    pos = r.pos_of_pair.long()
    live = pos[pos >= 0]
    y = torch.full((r.rows, H), math.nan, dtype=dtype, device="cuda")
    y[live] = rnd((len(live), H), dtype, 6)
    dout = rnd((T, H), dout_t, 7)
    dy = torch.full((r.rows, H), 7.0, dtype=dtype, device="cuda")
    got_dy, dw, dlogits = ops.combine_backward(dout, y, r, num_experts=E, dy=dy)
    assert got_dy is dy
    tok = torch.arange(T * k, device="cuda") // k
    d64, w64 = dout.to(ref.F64), r.topk_w.to(ref.F64)
    want = d64[tok] * w64.reshape(-1, 1)
    ref.close(dy[live], want[pos >= 0], want[pos >= 0].abs() * 2.0 ** -24, "dy")
    untouched(dy, live, 7.0)
    rows = torch.where((pos >= 0)[:, None], y[pos.clamp(min=0)].to(ref.F64), 0.0)
    prod = d64[tok] * rows
    want_dw, dw_b = prod.sum(1).view(T, k), prod.abs().sum(1).view(T, k) * (H + 2) * 2.0 ** -23
    ref.close(dw, want_dw, dw_b, "dw")
    # the softmax's gradient on what it is given: the bound follows dw's through the two sums
    g = w64 * (want_dw - (w64 * want_dw).sum(1, keepdim=True))
    size = want_dw.abs() + dw_b
    g_b = w64 * (dw_b + (w64 * dw_b).sum(1, keepdim=True) + (k + 4) * 2.0 ** -23 * (size + (w64 * size).sum(1, keepdim=True)))
    ids = r.topk_ids.long()
    zero = torch.zeros(T, E, dtype=ref.F64, device="cuda")
    ref.close(dlogits, zero.scatter_add(1, ids, g), zero.scatter_add(1, ids, g_b), "dlogits")
    assert torch.equal(dlogits[zero.scatter_add(1, ids, torch.ones_like(g)) == 0],
                       torch.zeros_like(dlogits[zero.scatter_add(1, ids, torch.ones_like(g)) == 0]))


def test_rows_and_ids_out_of_range_are_left_out():
    T, E, k, H = 4, 4, 2, 64
    r = ref.make_routing(T, E, k, 8)
    pos = r.pos_of_pair.clone()
    pos[0], pos[3] = r.rows, 2 ** 31 - 1  # behind the buffer
    bad = r._replace(pos_of_pair=pos)
    x = rnd((T, H), BF, 9)
    out = torch.zeros(r.rows, H, dtype=BF, device="cuda")
    ops.dispatch(x, bad, out=out)
    kept = [p for p in range(T * k) if p not in (0, 3)]
    want = torch.zeros_like(out)
    want[r.pos_of_pair.long()[kept]] = x[[p // k for p in kept]]
    assert torch.equal(out, want)
    dropped = pos.clone()
    dropped[[0, 3]] = -1
    ref.close(ops.combine(out, bad), *_combine64(out, r._replace(pos_of_pair=dropped), True), "combine")
    # a token that holds an expert twice, and ids outside the logits
    ids = r.topk_ids.clone()
    ids[0] = 2
    ids[1, 0], ids[2, 1] = -1, E
    dout = rnd((T, H), BF, 10)
    _, dw, dl = ops.combine_backward(dout, out, bad._replace(topk_ids=ids), num_experts=E)
    w = r.topk_w.to(ref.F64)
    g = w * (dw.to(ref.F64) - (w * dw.to(ref.F64)).sum(1, keepdim=True))
    want = torch.zeros(T, E, dtype=ref.F64, device="cuda")
    for t in range(T):
        for j in range(k):
            if 0 <= int(ids[t, j]) < E:
                want[t, int(ids[t, j])] += g[t, j]
    ref.close(dl, want, (w * dw.abs()).sum(1, keepdim=True) * 8 * 2.0 ** -23 + 0 * want, "dlogits")


# ---------------------------------------------------------------- linear
ACTS = ["none", "silu", "gelu", "swiglu"]
DENSE = [  # M, N, K
    (1, 1, 1), (1, 384, 512), (2, 10, 7), (16, 512, 1024), (17, 130, 200), (33, 64, 72), (64, 264, 136),
    (65, 130, 321), (127, 257, 96), (128, 128, 64), (129, 384, 640), (256, 512, 192), (300, 1000, 333),
    (515, 770, 264), (1024, 96, 2048),
]


def _linear_inputs(M, N, K, dtype, out, act, bias, residual, seed, E=0):
    cols = N // 2 if act == "swiglu" else N
    x = rnd((M, K), dtype, seed)
    w = rnd(((E,) if E else ()) + (N, K), dtype, seed + 1, K ** -0.5)
    b = rnd(((E,) if E else ()) + (N,), F, seed + 2) if bias else None
    res = rnd((M, cols), out, seed + 3) if residual else None
    return x, w, b, res, cols


def _check_linear(x, w, b, res, act, out, r=None, preact=True):
    rows, N = x.shape[0], w.shape[-2]
    pre = torch.full((rows, N), 7.0, dtype=x.dtype, device="cuda") if preact else None
    cols = N // 2 if act == "swiglu" else N
    buf = torch.full((rows, cols), 7.0, dtype=out, device="cuda")
    got = ops.linear(x, w, b, residual=res, activation=act, routing=r, out=buf, preact=pre)
    want, want_pre, bound, pre_bound = ref.linear64(x, w, b, res, act, r)
    ref.close(got, want, bound, "out")
    ref.close_norm(got, want, 1, "out")
    if preact:
        ref.close(pre, want_pre, pre_bound, "preact")
        ref.close_norm(pre, want_pre, 1, "preact")
    if r is not None:
        live = r.pos_of_pair.long()
        untouched(got, live[live >= 0], 7.0)
        if preact:
            untouched(pre, live[live >= 0], 7.0)


@pytest.mark.parametrize("M,N,K", DENSE)
@pytest.mark.parametrize("act,bias,residual,dtype,out", [
    ("none", False, False, BF, BF), ("none", True, True, BF, F), ("silu", True, False, HF, HF),
    ("gelu", False, True, BF, BF), ("swiglu", True, True, HF, F), ("swiglu", False, False, BF, BF)])
def test_linear_dense(M, N, K, act, bias, residual, dtype, out):
    N += N % 2 if act == "swiglu" else 0
    x, w, b, res, _ = _linear_inputs(M, N, K, dtype, out, act, bias, residual, 11)
    _check_linear(x, w, b, res, act, out)


FEW = [  # few rows: one launch, k shared by warps and the CTAs of a cluster
    (1, 384, 7168), (3, 40, 7168), (9, 34, 4104), (16, 10000, 1000), (8, 9480, 264), (5, 16, 8), (13, 130, 24),
    (16, 4096, 2056), (17, 384, 7168), (32, 130, 1000), (33, 258, 520), (64, 384, 7168), (50, 40, 72), (31, 1000, 2048),
]


@pytest.mark.parametrize("M,N,K", FEW)
@pytest.mark.parametrize("act,bias,residual,dtype,out", [
    ("none", True, True, BF, F), ("gelu", True, False, HF, HF), ("swiglu", True, True, BF, BF)])
def test_linear_few_rows(M, N, K, act, bias, residual, dtype, out):
    x, w, b, res, _ = _linear_inputs(M, N, K, dtype, out, act, bias, residual, 70)
    _check_linear(x, w, b, res, act, out)


def test_linear_few_rows_of_large_weights():
    """More weights than the few-row kernel takes: tiles of 32 tokens."""
    x, w, b, _, _ = _linear_inputs(9, 14400, 4096, BF, BF, "swiglu", True, False, 90)
    _check_linear(x, w, b, None, "swiglu", BF)


@pytest.mark.parametrize("M,N,K,act", [(1000, 384, 7168, "none"), (300, 264, 3000, "none"), (520, 256, 2048, "swiglu"),
                                       (40, 400, 7168, "silu"), (600, 34, 1040, "swiglu"), (16, 4096, 7168, "none"),
                                       (9, 1000, 20000, "none"), (30, 200, 9000, "swiglu")])
def test_linear_float32_outputs_keep_their_precision(M, N, K, act):
    """float32 outputs of long products.  The sum is kept in chains of 512 of k, 32 tensor-core additions that
    may truncate by 2^-23 of a running sum of norm sqrt(i / 32): 21.3 x 2^-23 = 2.5e-6 of a chain's norm at
    most, the same of the whole (chains add up in quadrature), and 14 rounding additions."""
    x, w, b, _, _ = _linear_inputs(M, N, K, BF, F, act, True, False, 71)
    got = ops.linear(x, w, b, activation=act, out_dtype=F)
    want, _, bound, _ = ref.linear64(x, w, b, None, act)
    ref.close(got, want, bound, "out")
    assert float((got.to(ref.F64) - want).norm() / want.norm()) <= 3e-6


GROUPED = [  # T, E, k, N, K, drop, hot
    (1, 1, 1, 64, 64, 0.0, None), (5, 6, 2, 40, 24, 0.0, None), (200, 3, 1, 96, 80, 0.2, None),
    (300, 8, 2, 256, 136, 0.0, 2), (700, 5, 2, 130, 70, 0.0, 0), (64, 40, 8, 264, 128, 0.3, None),
    (9, 6, 2, 66, 33, 1.0, None), (900, 4, 2, 320, 1100, 0.0, 1), (130, 7, 1, 34, 600, 0.0, None),
]


@pytest.mark.parametrize("T,E,k,N,K,drop,hot", GROUPED)
@pytest.mark.parametrize("act,bias,residual,dtype,out", [
    ("none", True, False, BF, BF), ("swiglu", True, False, BF, BF), ("gelu", False, True, HF, F),
    ("swiglu", True, True, HF, F)])
def test_linear_grouped(T, E, k, N, K, drop, hot, act, bias, residual, dtype, out):
    r = ref.make_routing(T, E, k, 12, drop, hot)
    x, w, b, res, _ = _linear_inputs(r.rows, N, K, dtype, out, act, bias, residual, 13, E)
    pos = r.pos_of_pair.long()
    pad = torch.ones(r.rows, dtype=torch.bool, device="cuda")
    pad[pos[pos >= 0]] = False
    x[pad] = math.nan  # padding must not reach a result
    _check_linear(x, w, b, res, act, out, r)


def _check_backward(dout, x, w, pre, act, r=None):
    dx = torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda")
    got = ops.linear_backward(dout, x, w, pre, act, r, bias_grad=True, dx=dx)
    want, bound = ref.linear_backward64(dout, x, w, pre, act, r)
    for name, g, a, b in zip(("dx", "dw", "db"), got, want, bound):
        ref.close(g, a, b, name)
    # one rounding of dz and one of the output
    ref.close_norm(got[0], want[0], 2, "dx")
    ref.close_norm(got[1], want[1], 2, "dw")
    if r is not None:
        live = r.pos_of_pair.long()
        untouched(dx, live[live >= 0], 7.0)
    return got


@pytest.mark.parametrize("M,N,K", DENSE)
@pytest.mark.parametrize("act,dtype,dout_t", [("none", BF, BF), ("none", BF, F), ("silu", HF, HF), ("gelu", BF, F),
                                              ("swiglu", BF, BF)])
def test_linear_backward_dense(M, N, K, act, dtype, dout_t):
    N += N % 2 if act == "swiglu" else 0
    x, w, _, _, cols = _linear_inputs(M, N, K, dtype, dout_t, act, False, False, 14)
    pre = rnd((M, N), dtype, 15) if act != "none" else None
    _check_backward(rnd((M, cols), dout_t, 16), x, w, pre, act)


@pytest.mark.parametrize("T,E,k,N,K,drop,hot", GROUPED)
@pytest.mark.parametrize("act,dtype,dout_t", [("none", BF, BF), ("swiglu", HF, HF), ("silu", BF, F)])
def test_linear_backward_grouped(T, E, k, N, K, drop, hot, act, dtype, dout_t):
    r = ref.make_routing(T, E, k, 17, drop, hot)
    x, w, _, _, cols = _linear_inputs(r.rows, N, K, dtype, dout_t, act, False, False, 18, E)
    pre = rnd((r.rows, N), dtype, 19) if act != "none" else None
    dout = rnd((r.rows, cols), dout_t, 20)
    pos = r.pos_of_pair.long()
    pad = torch.ones(r.rows, dtype=torch.bool, device="cuda")
    pad[pos[pos >= 0]] = False
    for t in (x, dout, pre):
        if t is not None:
            t[pad] = math.nan
    dx, dw, db = _check_backward(dout, x, w, pre, act, r)
    empty = r.counts == 0
    assert not dw[empty].abs().sum() and not db[empty].abs().sum()


@pytest.mark.parametrize("act", ACTS)
def test_linear_backward_against_differences(act):
    """<gradient, direction> against the float64 forward's central difference along the direction.  Each
    gradient element is off by at most its bound and its rounding; the difference quotient of step h by
    h^2 times a third derivative below 8 sum |terms| here."""
    M, N, K = 40, 48, 56
    x, w, b, _, cols = _linear_inputs(M, N, K, BF, BF, act, True, False, 21)
    v = rnd((M, cols), BF, 22)
    pre = torch.empty(M, N, dtype=BF, device="cuda")
    ops.linear(x, w, b, activation=act, preact=pre)
    dx, dw, db = ops.linear_backward(v, x, w, pre if act != "none" else None, act, bias_grad=True)
    f = lambda x_, w_, b_: (ref.act64(x_ @ w_.t() + b_, act) * v.to(ref.F64)).sum()  # noqa: E731
    x64, w64, b64 = x.to(ref.F64), w.to(ref.F64), b.to(ref.F64)
    # preact is rounded to bf16: act' moves by at most 1.1 (silu'', gelu'' < 0.8, swiglu's cross terms 1.1) z u
    z = x64 @ w64.t() + b64
    if act == "swiglu":
        g, up = z.chunk(2, -1)
        dz_move = torch.cat([v.abs() * (up.abs() * 0.8 * g.abs() + 1.1 * up.abs()), v.abs() * 1.1 * g.abs()], -1) * ref.u(BF)
    else:
        dz_move = v.abs() * 0.8 * z.abs() * ref.u(BF) if act != "none" else 0 * z
    _, (dxb, dwb, dbb) = ref.linear_backward64(v, x, w, pre if act != "none" else None, act)
    h = 1e-4
    for name, grad, bound, at, move in (
            ("dx", dx, dxb, 0, dz_move.to(ref.F64) @ w64.abs()),
            ("dw", dw, dwb, 1, dz_move.to(ref.F64).t() @ x64.abs()),
            ("db", db, dbb, 2, dz_move.to(ref.F64).sum(0))):
        d = rnd(grad.shape, F, 23 + at).to(ref.F64)
        args = [x64, w64, b64]
        lo, hi = list(args), list(args)
        lo[at], hi[at] = args[at] - h * d, args[at] + h * d
        want = float((f(*hi) - f(*lo)) / (2 * h))
        got = float((grad.to(ref.F64) * d).sum())
        tol = float(((bound + move + ref.u(grad.dtype) * grad.to(ref.F64).abs()) * d.abs()).sum())
        assert abs(got - want) <= tol + 1e-3, f"{name}: {got} against {want}, tolerance {tol}"


def test_no_tokens():
    r = ref.make_routing(1, 4, 1, 24, drop=1.0)
    empty = torch.empty(0, 64, dtype=BF, device="cuda")
    w = rnd((32, 64), BF, 25)
    assert ops.linear(empty, w).shape == (0, 32)
    dx, dw, db = ops.linear_backward(torch.empty(0, 32, dtype=BF, device="cuda"), empty, w, bias_grad=True,
                                     dw=torch.full_like(w, 7.0))
    assert dx.shape == (0, 64) and not dw.abs().sum() and not db.abs().sum()
    none = ops.route_group(torch.empty(0, 4, device="cuda"), 2)
    assert none.rows == 0 and ops.dispatch(empty, none).shape == (0, 64)
    assert ops.combine(torch.empty(0, 64, dtype=BF, device="cuda"), none).shape == (0, 64)
    # every pair left out: the combine writes zeros
    y = torch.full((r.rows, 64), math.nan, dtype=BF, device="cuda")
    assert not ops.combine(y, r).abs().sum()


def test_residual_in_place_and_infinities():
    x, w, b, res, _ = _linear_inputs(40, 64, 72, BF, BF, "none", True, True, 26)
    res[3, 5], res[4, 6] = math.inf, math.nan
    want = ops.linear(x, w, b, residual=res)
    got = ops.linear(x, w, b, residual=res, out=res)
    assert got is res and torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[~got.isnan()], want[~want.isnan()])
    assert math.isinf(float(got[3, 5])) and got.isnan().sum() == 1
    # a token with an infinity spoils its own row alone
    x[7, 0] = math.inf
    out = ops.linear(x, w, b)
    assert not out[7].isfinite().any() and out[:7].isfinite().all() and out[8:].isfinite().all()


@pytest.mark.parametrize("act", ACTS)
def test_far_activations_are_their_limits(act):
    """Activations and gradients at |z| of 1e2 and 1e30: the limits, no NaN from an overflowing power."""
    n = 8
    w = torch.eye(n, dtype=BF, device="cuda")
    x = torch.tensor([[1e2, -1e2, 1e30, -1e30, 1.0, 1.0, 1.0, 1.0]], dtype=BF, device="cuda")
    if act == "swiglu":
        w = torch.cat([w, w.flip(0)])
    pre = torch.empty(1, w.shape[0], dtype=BF, device="cuda")
    out = ops.linear(x, w, activation=act, preact=pre)
    assert out.isfinite().all()
    dx, _, _ = ops.linear_backward(torch.ones_like(out), x, w, pre if act != "none" else None, act)
    assert dx.isfinite().all()
    if act in ("silu", "gelu"):
        assert torch.equal(out[0, :4], x[0, :4].clamp(min=0)) and torch.equal(dx[0, :4].float(), torch.tensor([1., 0, 1, 0], device="cuda"))


# ---------------------------------------------------------------- together
def _stage_inputs(T=220, H=192, I=128, E=6, k=2):
    return dict(x=rnd((T, H), BF, 31), wr=rnd((E, H), BF, 32, H ** -0.5), br=rnd((E,), F, 33),
                w1=rnd((E, 2 * I, H), BF, 34, H ** -0.5), b1=rnd((E, 2 * I), F, 35), w2=rnd((E, H, I), BF, 36, I ** -0.5),
                dout=rnd((T, H), BF, 37)), k


def _layer(p, k):
    """One training pass of a routed layer of unquantised experts on a residual stream: outputs and gradients."""
    E = p["wr"].shape[0]
    logits = ops.linear(p["x"], p["wr"], p["br"], out_dtype=F)
    r = ops.route_group(logits, k)
    g = ops.dispatch(p["x"], r)
    z = torch.empty(r.rows, p["w1"].shape[1], dtype=BF, device="cuda")
    h = ops.linear(g, p["w1"], p["b1"], activation="swiglu", routing=r, preact=z)
    y = ops.linear(h, p["w2"], routing=r)
    out = ops.combine(y, r)
    dy, dw, dlogits = ops.combine_backward(p["dout"], y, r, num_experts=E)
    dh, dw2, _ = ops.linear_backward(dy, h, p["w2"], routing=r)
    dg, dw1, db1 = ops.linear_backward(dh, g, p["w1"], z, "swiglu", r, bias_grad=True)
    dxr, dwr, dbr = ops.linear_backward(dlogits, p["x"], p["wr"], bias_grad=True)
    dxe = ops.dispatch_backward(dg, r)
    return dict(logits=logits, out=out, dw1=dw1, db1=db1, dw2=dw2, dwr=dwr, dbr=dbr, dxr=dxr, dxe=dxe), r


def test_layer_and_its_gradients_together():
    """Against float64 autograd of the whole layer with the same selection.  Relative errors in norm: the
    values pass at most 8 roundings to bf16 in a row (x and w exact; g, z, h, y, dy, dh, dz, result),
    each at most u, and the sums in between do not enlarge a relative error in norm for these random
    operands by more than their condition, taken as 4."""
    p, k = _stage_inputs()
    got, r = _layer(p, k)
    T, E = got["logits"].shape
    leaf = {n: t.to(ref.F64).requires_grad_() for n, t in p.items() if n != "dout"}
    logits = leaf["x"] @ leaf["wr"].t() + leaf["br"]
    ids = r.topk_ids.long()
    # the selection is the given one; it is the top-k of these logits, within their rounding
    top = torch.topk(got["logits"], k, dim=1)
    assert torch.equal(top.indices.sort(1).values, ids.sort(1).values)
    w = torch.softmax(logits.gather(1, ids), 1)
    z = torch.einsum("th,enh->ten", leaf["x"], leaf["w1"]) + leaf["b1"]
    y = torch.einsum("tei,ehi->teh", ref.act64(z, "swiglu"), leaf["w2"])
    out = (y[torch.arange(T, device="cuda")[:, None], ids] * w[..., None]).sum(1)
    names = ["x", "wr", "br", "w1", "b1", "w2"]
    grads = dict(zip(names, torch.autograd.grad(out, [leaf[n] for n in names], p["dout"].to(ref.F64))))
    tol = 4 * 8 * ref.u(BF)
    for name, g, want in (("logits", got["logits"], logits), ("out", got["out"], out), ("w1", got["dw1"], grads["w1"]),
                          ("b1", got["db1"], grads["b1"]), ("w2", got["dw2"], grads["w2"]), ("wr", got["dwr"], grads["wr"]),
                          ("br", got["dbr"], grads["br"]), ("x", got["dxr"].to(ref.F64) + got["dxe"].to(ref.F64), grads["x"])):
        rel = float((g.to(ref.F64) - want.detach()).norm() / want.detach().norm())
        assert rel <= tol, f"{name}: relative error {rel:.2e}"


def test_layer_is_captured_replayed_and_repeats_its_bits():
    p, k = _stage_inputs(T=300, H=256)
    want, _ = _layer(p, k)
    again, _ = _layer(p, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _layer(p, k)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, _ = _layer(p, k)
    other = rnd(p["x"].shape, BF, 38)
    kept = p["x"].clone()
    for x in (other, kept):  # new inputs, then the first ones again
        p["x"].copy_(x)
        graph.replay()
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(again[name], want[name]), name
        assert torch.equal(got[name], want[name]), name


def test_two_streams_at_once():
    p, k = _stage_inputs(T=257)
    r = ref.make_routing(257, 6, 2, 39)
    jobs = [lambda s=s: ops.linear_backward(p["dout"], p["x"], rnd((192, 192), BF, s), rnd((257, 192), BF, s + 1), "silu",
                                            bias_grad=True) for s in (40, 50)]
    want = [[t.clone() for t in j()] for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        got = []
        for j, s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append(j())
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    assert r.rows > 0


def test_another_stream_is_used():
    """A call with stream= runs there: it sees what that stream wrote before."""
    s = torch.cuda.Stream()
    x = torch.zeros(64, 512, dtype=BF, device="cuda")
    w = rnd((32, 512), BF, 60)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        x.fill_(1.0)
    out = ops.linear(x, w, stream=s)
    s.synchronize()
    ref.close(out, *[a for i, a in enumerate(ref.linear64(torch.ones_like(x), w, None, None, "none")) if i in (0, 2)], "out")


def test_new_tensors_belong_to_the_calls_stream():
    """Memory freed on the current stream while its kernels still run is not handed to a call on another
    stream: the old tensor's late write would land in the call's result."""
    s = torch.cuda.Stream()
    x, w = rnd((256, 512), BF, 72), rnd((512, 512), BF, 73)
    want = ops.linear(x, w)
    torch.cuda.synchronize()
    for handle in (s, s.cuda_stream):
        old = torch.empty_like(want)
        torch.cuda._sleep(20_000_000)
        old.fill_(7.0)
        del old  # freed on the current stream, its fill still to come
        got = ops.linear(x, w, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_streams_forked_inside_a_capture():
    p, _ = _stage_inputs(T=270)
    w = rnd((192, 192), BF, 74)
    want = [ops.linear(p["x"], w, activation="silu"), ops.linear(p["dout"], w, activation="gelu")]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        x = p["x"] + 0  # a kernel of another library right before and after
        side.wait_stream(torch.cuda.current_stream())
        a = ops.linear(x, w, activation="silu")
        with torch.cuda.stream(side):
            b = ops.linear(p["dout"], w, activation="gelu") + 0
        torch.cuda.current_stream().wait_stream(side)
        c = a + 0
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c, want[0]) and torch.equal(b, want[1])
    assert moe_mx.moe_mx_linear_status(0) == moe_mx.MOE_MX_OK


def test_an_experts_weights_reach_its_own_rows_alone():
    """NaN weights of two experts, one without rows, between others: sizes off every tile and block."""
    E, N, K = 6, 66, 72
    r = ref.make_routing(150, E, 2, 75)
    x, w, b, _, _ = _linear_inputs(r.rows, N, K, BF, BF, "none", True, False, 76, E)
    want = ops.linear(x, w, b, routing=r)
    dout = rnd((r.rows, N), BF, 77)
    want_dx, _, _ = ops.linear_backward(dout, x, w, routing=r, weight_grad=False)
    empty = E // 3  # without rows
    bad = w.clone()
    bad[empty], bad[4] = math.nan, math.nan
    got = ops.linear(x, bad, b, routing=r)
    got_dx, _, _ = ops.linear_backward(dout, x, bad, routing=r, weight_grad=False)
    for e, lo, hi in ref.segments(r, r.rows):
        if e == 4:
            assert got[lo:hi].isnan().all() and got_dx[lo:hi].isnan().all()
        else:
            assert torch.equal(got[lo:hi], want[lo:hi]) and torch.equal(got_dx[lo:hi], want_dx[lo:hi])
    # a NaN row of one expert's x and dout stays out of the other experts' gradients
    want_dw, want_db = ops.linear_backward(dout, x, w, routing=r, bias_grad=True)[1:]
    lo = int(r.pad_offsets[4])
    x[lo], dout[lo] = math.nan, math.nan
    dw, db = ops.linear_backward(dout, x, w, routing=r, bias_grad=True)[1:]
    keep = [e for e in range(E) if e != 4]
    assert torch.equal(dw[keep], want_dw[keep]) and torch.equal(db[keep], want_db[keep])
    assert dw[4].isnan().all() and db[4].isnan().all()


def test_1024_experts():
    r = ref.make_routing(700, 1024, 3, 78)
    x, w, b, _, _ = _linear_inputs(r.rows, 40, 64, BF, BF, "silu", True, False, 79, 1024)
    _check_linear(x, w, b, None, "silu", BF, r)
    _check_backward(rnd((r.rows, 40), BF, 80), x, w, rnd((r.rows, 40), BF, 81), "silu", r)


def test_offsets_past_31_bits():
    """Grouped buffers, outputs and weights of more than 2^31 elements: rows at the far end."""
    T, k, H, E = 40000, 8, 7168, 16
    g = torch.Generator().manual_seed(82)
    ids = torch.argsort(torch.rand(T, E, generator=g), 1)[:, :k].cuda()
    logits = torch.full((T, E), -4.0, device="cuda").scatter_(1, ids, torch.arange(k, 0, -1, device="cuda").float().expand(T, k))
    r = ops.route_group(logits, k)
    assert r.rows * H > 2 ** 31
    x = rnd((T, H), BF, 83)
    y = ops.dispatch(x, r)
    pos = r.pos_of_pair.long()
    far = torch.topk(pos, 64).indices
    assert int(pos[far].min()) * H > 2 ** 31 and torch.equal(y[pos[far]], x[far // k])
    out = ops.combine(y, r)
    dy, dw, _ = ops.combine_backward(x, y, r, num_experts=E)
    tok = (far // k)[:8]
    ref.close(out[tok], x[tok].to(ref.F64), x[tok].to(ref.F64).abs() * (k + 4) * 2.0 ** -23, "combine")
    w = r.topk_w.reshape(-1)[far].to(ref.F64)[:, None]
    ref.close(dy[pos[far]], x[far // k].to(ref.F64) * w, (x[far // k].to(ref.F64) * w).abs() * 2.0 ** -24, "dy")
    sq = (x[tok].to(ref.F64) ** 2).sum(1, keepdim=True).expand(-1, k)
    ref.close(dw[tok], sq, sq * (H + 2) * 2.0 ** -23, "dw")
    del y, dy, out
    M, N, K = 300000, 7200, 64
    x, w = rnd((M, K), BF, 84), rnd((N, K), BF, 85)
    got = ops.linear(x, w)
    assert got.numel() > 2 ** 31
    want, _, bound, _ = ref.linear64(x[-300:], w, None, None, "none")
    ref.close(got[-300:], want, bound, "linear")
    dx, dw, _ = ops.linear_backward(got, x, w)
    (want, _, _), (bound, _, _) = ref.linear_backward64(got[-300:], x[-300:], w, None, "none")
    ref.close(dx[-300:], want, bound, "dx")
    del got, dx, dw
    E, N, K = 9, 32768, 8192
    r = ref.make_routing(20, E, 1, 86)
    w = torch.zeros(E, N, K, dtype=BF, device="cuda")
    assert w.numel() > 2 ** 31
    last = int(r.counts.nonzero().max())
    w[last, -64:] = rnd((64, K), BF, 87, K ** -0.5)
    x = rnd((r.rows, K), BF, 88)
    got = ops.linear(x, w, routing=r)
    lo, n = int(r.pad_offsets[last]), int(r.counts[last])
    want, _, bound, _ = ref.linear64(x[lo:lo + n], w[last, -64:].contiguous(), None, None, "none")
    ref.close(got[lo:lo + n, -64:], want, bound, "grouped")
    dout = rnd((r.rows, N), BF, 89)
    dw = ops.linear_backward(dout, x, w, routing=r)[1]
    want = dout[lo:lo + n, -64:].to(ref.F64).t() @ x[lo:lo + n].to(ref.F64)
    ref.close(dw[last, -64:], want, (n + 2) * 2.0 ** -23 * (dout[lo:lo + n, -64:].to(ref.F64).abs().t() @ x[lo:lo + n].to(ref.F64).abs()), "grouped dw")


def test_first_call_of_a_process_may_be_captured():
    code = """
import torch
from block_scaled_moe_softmax_b200 import routed_ops as ops
x = torch.ones(300, 128, dtype=torch.bfloat16, device='cuda')
w = torch.ones(64, 128, dtype=torch.bfloat16, device='cuda')
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = ops.linear(x, w)
    dx, dw, db = ops.linear_backward(y, x, w, bias_grad=True)
    z = ops.linear(x[:1], w, out_dtype=torch.float32)
g.replay()
torch.cuda.synchronize()
assert (y == 128).all() and (dx == 128 * 64).all() and (dw == 300 * 128).all() and (db == 300 * 128).all()
assert (z == 128).all()
print('captured')
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_routing_of_the_library_feeds_the_operators():
    T, E, k, H = 200, 32, 4, 128
    logits = rnd((T, E), F, 61)
    r = ops.route_group(logits, k)
    x = rnd((T, H), BF, 62)
    g = ops.dispatch(x, r)
    assert torch.equal(g[r.pos_of_pair.long()].view(T, k, H), x[:, None].expand(T, k, H))
    # weights sum to 1: combining copies of x gives x back, within the sum's and the output's rounding
    ref.close(ops.combine(g, r), x.to(ref.F64), x.to(ref.F64).abs() * (k + 4) * 2.0 ** -23, "round trip")


def test_errors_on_the_device_are_refused():
    x, w = rnd((8, 64), BF, 63), rnd((16, 64), BF, 64)
    with pytest.raises(ValueError, match="shape"):
        ops.linear(x, w, rnd((15,), F, 65))
    with pytest.raises(moe_mx.MoeMxError) as e:
        ops.linear(x, w, out=x.view(-1)[:128].view(8, 16))
    assert e.value.code == moe_mx.MOE_MX_ERR_INVALID_ARG and "overlap" in str(e.value)
    with pytest.raises(moe_mx.MoeMxError, match="aligned"):
        ops.linear(x.view(-1)[1:449].view(7, 64), w)
    with pytest.raises(moe_mx.MoeMxError, match="workspace"):
        moe_mx.moe_mx_linear_backward(rnd((8, 16), F, 66), x, w, None, None, None, 0, 8, 16, 64, 0, 0, 1,
                                      torch.empty_like(x), None, None, None, 0)


# ---------------------------------------------------------------- failure detection
def test_a_wait_that_gives_up_is_reported_and_harms_no_other_call():
    ops.check()
    x, w = rnd((300, 131072), BF, 100), rnd((264, 131072), BF, 101, 2.0 ** -8)
    want = ops.linear(x, w, activation="silu")  # waits of more than 100 us for its accumulators
    moe_mx.moe_mx_debug_linear_watchdog(0, 2000)  # a 2 ms wait on a flag nothing sets
    got = [ops.linear(x, w, activation="silu") for _ in range(3)]  # the word is set by now
    with pytest.raises(moe_mx.MoeMxError) as e:
        ops.check()
    assert e.value.code == moe_mx.MOE_MX_ERR_TIMEOUT
    for t in got:
        assert torch.equal(t, want)
    ops.check()  # read and cleared
    s = torch.cuda.Stream()
    moe_mx.moe_mx_debug_linear_watchdog(0, 2000, s)
    with pytest.raises(moe_mx.MoeMxError):
        ops.check("cuda:0", s)
    ops.check(0, s.cuda_stream)
    assert moe_mx.moe_mx_linear_status(0) == moe_mx.MOE_MX_OK


# ---------------------------------------------------------------- long sums
def _positive(shape, dtype, seed, mean):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(shape, generator=g, device="cuda").add_(0.5).mul_(mean)).to(dtype)


def _ends(n, m=64):
    return torch.arange(n, device="cuda") if n <= 2 * m else torch.cat([torch.arange(m), torch.arange(n - m, n)]).cuda()


def _unbiased(got, want, factor=1):
    """16-bit outputs of a long sum of one sign.  The tensor core truncates each addition of 16 products by
    less than 2^-22 of the sum it leaves; a chain of 8192 (float16: 512 additions to a growing sum) is short by
    at most 2^-13, one of 65536 (bf16) by 2^-10, and by half of that where the sum grows evenly: u / 8.  Chains are
    joined in float32 and the result is rounded once, by u at most and by nothing in the mean of n values but
    4 u / sqrt(n).  factor: how often the sum enters the output."""
    rel = (got.to(ref.F64) - want) / want
    u = ref.u(got.dtype)
    assert float(rel.abs().max()) <= u + factor * u / 4 + 2.0 ** -18, f"{float(rel.abs().max()):.2e}"
    assert abs(float(rel.mean())) <= factor * u / 8 + 4 * u / rel.numel() ** 0.5, f"mean {float(rel.mean()):.2e}"


LONG = [  # M, N, K, act, bias and residual, preact: one round of tiles, so that k is not split
    (40, 18944, 33280, "none", False, False), (40, 18944, 33280, "silu", True, True),
    (200, 9471, 33281, "none", True, True), (33, 18944, 33280, "swiglu", False, True),
    (9472, 512, 33280, "none", False, False), (9472, 512, 33280, "silu", True, True),
    (9472, 511, 33280, "gelu", True, False), (9472, 512, 33280, "swiglu", True, True),
    (12544, 576, 33280, "none", True, True), (18944, 128, 33280, "none", False, False),
    (18944, 126, 33280, "swiglu", False, True), (4, 40, 1 << 20, "none", True, False),
]


@pytest.mark.parametrize("M,N,K,act,more,preact", LONG)
def test_long_sums_of_16_bit_outputs(M, N, K, act, more, preact):
    x, w = _positive((M, K), HF, 110, 0.05), _positive((N, K), HF, 111, 20 / (0.05 * K))
    cols = N // 2 if act == "swiglu" else N
    b = rnd((N,), F, 112) if more else None
    res = rnd((M, cols), HF, 113) if more else None
    pre = torch.empty(M, N, dtype=HF, device="cuda") if preact else None
    got = ops.linear(x, w, b, residual=res, activation=act, preact=pre)
    rows, at = _ends(M), _ends(cols)
    wat = torch.cat([at, at + cols]) if act == "swiglu" else at
    z = x[rows].to(ref.F64) @ w[wat].to(ref.F64).t()
    if more:
        z = z + b[wat].to(ref.F64)
    want = ref.act64(z, act)
    if more:
        want = want + res[rows][:, at].to(ref.F64)
    _unbiased(got[rows][:, at], want, 2 if act == "swiglu" else 1)
    if preact:
        _unbiased(pre[rows][:, wat], z)


@pytest.mark.parametrize("M,N,K,dtype", [
    (40, 33280, 18944, HF), (9472, 33280, 512, HF), (18944, 33280, 120, HF), (300000, 2048, 2304, HF),
    (150000, 9472, 128, HF), (200000, 130, 70, HF), (600000, 2048, 2304, BF)])
def test_long_sums_of_gradients(M, N, K, dtype):
    d, x = _positive((M, N), dtype, 114, 0.3), _positive((M, K), dtype, 115, 2000.0 / (0.3 * M))
    w = _positive((N, K), dtype, 116, 2000.0 / (0.3 * N))
    dx, dw, _ = ops.linear_backward(d, x, w)
    rows, at, n = _ends(M), _ends(K), _ends(N)
    _unbiased(dx[rows][:, at], d[rows].to(ref.F64) @ w[:, at].to(ref.F64))
    _unbiased(dw[n][:, at], d[:, n].to(ref.F64).t() @ x[:, at].to(ref.F64))


def test_long_sums_of_one_experts_gradients():
    """All rows at one of several experts: the depth of dw is known on the device alone."""
    T, E, N, K = 70000, 3, 264, 136
    r = ref.make_routing(T, E, 1, 117, hot=2)
    d, x = _positive((r.rows, N), HF, 118, 0.3), _positive((r.rows, K), HF, 119, 2000.0 / (0.3 * T))
    w = rnd((E, N, K), HF, 120)
    _, dw, db = ops.linear_backward(d, x, w, routing=r, bias_grad=True)
    lo, n = int(r.pad_offsets[2]), int(r.counts[2])
    assert n == T
    _unbiased(dw[2], d[lo:lo + n].to(ref.F64).t() @ x[lo:lo + n].to(ref.F64))
    assert not dw[:2].abs().sum() and not db[:2].abs().sum()


# ---------------------------------------------------------------- float32 gradients of float16 operands
@pytest.mark.parametrize("size,act", [(1e-7, "none"), (1e-6, "swiglu"), (3e-9, "silu"), (1e6, "none"), (2e5, "gelu"),
                                      (1e-40, "none")])
@pytest.mark.parametrize("M,N,K", [(1000, 384, 264), (130, 66, 70), (3, 40, 24)])
def test_float32_gradients_outside_float16s_range(M, N, K, size, act):
    """x and w of a size that brings dx and dw into float16's range; two roundings, of dz and of the result."""
    back = min(1 / size, 2.0 ** 12) if size < 1 else max(1 / size, 2.0 ** -13)
    x, w = rnd((M, K), HF, 130, back), rnd((N, K), HF, 131, back)
    cols = N // 2 if act == "swiglu" else N
    d = rnd((M, cols), F, 132, size)
    pre = rnd((M, N), HF, 133) if act != "none" else None
    dx, dw, db = ops.linear_backward(d, x, w, pre, act, bias_grad=True)
    want, _ = ref.linear_backward64(d, x, w, pre, act)
    small = 2.0 ** -25  # half a subnormal step of the results
    for g, t, name in ((dx, want[0], "dx"), (dw, want[1], "dw")):
        assert g.isfinite().all(), name
        err = float((g.to(ref.F64) - t).norm())
        tol = (math.sqrt(2) * ref.u(HF) + 2.0 ** -16) * float(t.norm()) + small * t.numel() ** 0.5
        assert err <= tol, f"{name}: {err / float(t.norm()):.2e}"
    rel = float((db.to(ref.F64) - want[2]).norm() / want[2].norm())
    assert rel <= (2.0 ** -16 if size > 1e-38 else 1e-4), f"db: {rel:.2e}"  # float32 itself is subnormal there


def test_float32_gradients_of_experts_of_different_sizes():
    """Each expert's gradients are scaled by its own largest value; an infinity or NaN in one row spoils that
    row of dx and its expert's dw alone, and no finite value near it."""
    T, E, N, K = 500, 6, 136, 200
    r = ref.make_routing(T, E, 2, 140)
    d = rnd((r.rows, N), F, 141)
    x, w = rnd((r.rows, K), HF, 142), rnd((E, N, K), HF, 143)
    pad = torch.ones(r.rows, dtype=torch.bool, device="cuda")
    for e, lo, hi in ref.segments(r, r.rows):
        size = 10.0 ** (3 * (e - 3))  # 1e-9 .. 1e6
        d[lo:hi] *= size
        x[lo:hi] *= min(max(1 / size, 2.0 ** -13), 2.0 ** 12)
        w[e] *= min(max(1 / size, 2.0 ** -13), 2.0 ** 12)
        pad[lo:hi] = False
    d[pad], x[pad] = math.nan, math.nan
    def check(dx, dw, skip=None):
        (tx, tw, _), _ = ref.linear_backward64(d, x, w, None, "none", r)
        for e, lo, hi in ref.segments(r, r.rows):
            if hi == lo:
                continue
            rows = [i for i in range(lo, hi) if i != skip]
            for g, t in ((dx[rows], tx[rows]), (dw[e], tw[e])):
                if not t.isfinite().all():
                    continue
                tol = (math.sqrt(2) * ref.u(HF) + 2.0 ** -16) * float(t.norm()) + 2.0 ** -25 * t.numel() ** 0.5
                assert float((g.to(ref.F64) - t).norm()) <= tol, e
    dx, dw, _ = ops.linear_backward(d, x, w, routing=r)
    again = ops.linear_backward(d, x, w, routing=r)
    assert torch.equal(dx[~pad], again[0][~pad]) and torch.equal(dw, again[1])
    check(dx, dw)
    lo = int(r.pad_offsets[4])
    d[lo, 0] = math.inf
    dx, dw, _ = ops.linear_backward(d, x, w, routing=r)
    check(dx, dw, lo)
    assert not dx[lo].isfinite().any() and not dw[4, 0].isfinite().any() and dw[4, 1:].isfinite().all()


def test_float32_gradients_of_rows_of_different_sizes():
    """Rows of one segment 2^20 apart keep their relative precision."""
    M, N, K = 64, 256, 128
    d = rnd((M, N), F, 150, 1e-3) * 2.0 ** -(torch.arange(M, device="cuda") % 21)[:, None]
    x, w = rnd((M, K), HF, 151), rnd((N, K), HF, 152, 1000.0)
    dx = ops.linear_backward(d, x, w, weight_grad=False)[0]
    want = d.to(ref.F64) @ w.to(ref.F64)
    err, size = (dx.to(ref.F64) - want).norm(dim=1), want.norm(dim=1)
    assert bool((err <= (math.sqrt(2) * ref.u(HF) + 2.0 ** -16) * size + 2.0 ** -25 * K ** 0.5).all())


def test_outputs_over_any_input_are_refused():
    M, N, K, E, k = 4, 64, 68, 4, 2
    x, w, b = rnd((M, K), BF, 160), rnd((N, K), BF, 161), rnd((M, N), F, 162)
    with pytest.raises(moe_mx.MoeMxError, match="overlap"):
        ops.linear(x, w, b[0], out=b)
    with pytest.raises(moe_mx.MoeMxError, match="overlap"):
        ops.linear(x, w, b[0], preact=b.view(-1).view(BF)[:M * N].view(M, N))
    need = moe_mx.moe_mx_linear_workspace(0, M, N, K, 0, 0, 0)
    assert need > 0
    big = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for name in ("x", "w", "out"):
        t = {"x": x, "w": w, "out": torch.empty(M, N, dtype=BF, device="cuda")}
        t[name] = big
        with pytest.raises(moe_mx.MoeMxError, match="workspace.*overlap"):
            moe_mx.moe_mx_linear(t["x"], t["w"], None, None, None, None, 0, M, N, K, 0, 0, 0, t["out"], None, big, need)
    need = moe_mx.moe_mx_linear_backward_workspace(0, M, N, K, 0, 0, 0)
    big, dw = torch.zeros(need, dtype=torch.uint8, device="cuda"), torch.empty_like(w)
    d = rnd((M, N), BF, 163)
    for args in ((big, x, w, None, dw), (d, x, big, torch.empty_like(x), None), (d, x, w, None, big)):
        with pytest.raises(moe_mx.MoeMxError, match="workspace.*overlap"):
            moe_mx.moe_mx_linear_backward(*args[:3], None, None, None, 0, M, N, K, 0, 0, 0, args[3], args[4], None, big, need)
    # the routing of the permutes
    r = ref.make_routing(M, E, k, 164)
    buf = torch.zeros(r.rows, 8, dtype=F, device="cuda")
    xs = rnd((M, 8), F, 165)
    with pytest.raises(moe_mx.MoeMxError, match="overlap"):
        ops.dispatch(xs, r._replace(pos_of_pair=buf.view(torch.int32).view(-1)[:M * k]), out=buf)
    with pytest.raises(moe_mx.MoeMxError, match="overlap"):
        ops.combine(rnd((r.rows, 8), F, 166), r._replace(topk_w=buf.view(-1)[:M * k].view(M, k)), out=buf[:M])
    with pytest.raises(moe_mx.MoeMxError, match="overlap"):
        ops.combine_backward(xs, rnd((r.rows, 8), F, 167), r._replace(topk_w=buf.view(-1)[:M * k].view(M, k)), dy=buf)
    assert not buf.any() and not big.any()
    # out may be the residual itself, and what a call does not touch may lie anywhere
    ops.linear(x, w, residual=d, out=d)
    ops.combine_backward(xs, rnd((r.rows, 8), F, 168), r, dy=buf)
    y = rnd((r.rows, 8), F, 169)
    want = ops.combine_backward(xs, y, r)
    both = r.topk_w.clone()
    moe_mx.moe_mx_combine_backward(xs, y, r.rows, M, 8, k, r.pos_of_pair, both, None, 0, 1, 1, None, both, None)
    assert torch.equal(both, want[1])
    moe_mx.moe_mx_combine_backward(xs, y, r.rows, M, 8, k, r.pos_of_pair, r.topk_w, None, 0, 1, 1, y, None, None)
    assert torch.equal(y[r.pos_of_pair.long()], want[0][r.pos_of_pair.long()])


def test_results_without_history_are_announced():
    r = ref.make_routing(8, 4, 2, 170)
    x, w, b = rnd((8, 64), BF, 171), rnd((32, 64), BF, 172), rnd((32,), F, 173)
    logits, g = rnd((8, 4), F, 174), rnd((r.rows, 64), BF, 175)
    calls = [("linear", lambda: ops.linear(x, w, b), x), ("linear", lambda: ops.linear(x, w, b), w),
             ("linear", lambda: ops.linear(x, w, b), b), ("dispatch", lambda: ops.dispatch(x, r), x),
             ("combine", lambda: ops.combine(g, r), g), ("combine", lambda: ops.combine(g, r), r.topk_w),
             ("route_group", lambda: ops.route_group(logits, 2), logits)]
    for name, call, leaf in calls:
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            want = call()  # nothing requires a gradient
            leaf.requires_grad_()
            with torch.no_grad():
                call()
        with pytest.warns(UserWarning, match=f"{name}.*no autograd history") as seen:
            got = call()
        assert seen[0].filename == __file__
        leaf.requires_grad_(False)
        if name != "dispatch":  # whose padding rows are not written
            got, want = (got.pos_of_pair, want.pos_of_pair) if name == "route_group" else (got, want)
            assert torch.equal(got, want) and not got.requires_grad


def test_types_that_do_not_go_together_are_type_errors():
    x, w = rnd((8, 64), BF, 180), rnd((16, 64), BF, 181)
    for kw in (dict(out_dtype=HF), dict(out=rnd((8, 16), HF, 182)), dict(residual=rnd((8, 16), HF, 183)),
               dict(out_dtype=torch.float64)):
        with pytest.raises(TypeError, match="out has type"):
            ops.linear(x, w, **kw)
    with pytest.raises(TypeError, match="dout has type"):
        ops.linear_backward(rnd((8, 16), HF, 184), x, w)


def test_the_binding_makes_the_same_calls():
    """The entry points by their names, on raw arguments, against routed_ops."""
    T, E, k, H, N = 50, 6, 2, 72, 40
    r = ref.make_routing(T, E, k, 190)
    x, w, b = rnd((T, H), BF, 191), rnd((E, N, H), BF, 192), rnd((E, N), F, 193)
    live = r.pos_of_pair.long()
    g = torch.zeros(r.rows, H, dtype=BF, device="cuda")
    moe_mx.moe_mx_dispatch(x, T, H, k, r.pos_of_pair, r.rows, 0, g)
    assert torch.equal(g[live], ops.dispatch(x, r)[live])
    y, z = torch.zeros(r.rows, N, dtype=F, device="cuda"), torch.zeros(r.rows, N, dtype=BF, device="cuda")
    need = moe_mx.moe_mx_linear_workspace(E, r.rows, N, H, 0, moe_mx.MOE_MX_LINEAR_SILU, 1)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    moe_mx.moe_mx_linear(g, w, b, None, r.counts, r.pad_offsets, E, r.rows, N, H, 0, moe_mx.MOE_MX_LINEAR_SILU, 1, y, z,
                         ws, need)
    want_z = torch.zeros_like(z)
    assert torch.equal(y[live], ops.linear(g, w, b, activation="silu", routing=r, out_dtype=F, preact=want_z)[live])
    assert torch.equal(z, want_z)
    out = torch.empty(T, N, dtype=BF, device="cuda")
    moe_mx.moe_mx_combine(y, r.rows, T, N, k, r.pos_of_pair, r.topk_w, 1, 0, out)
    assert torch.equal(out, ops.combine(y, r, out_dtype=BF))
    dy, dw, dl = torch.zeros_like(y), torch.empty(T, k, device="cuda"), torch.empty(T, E, device="cuda")
    moe_mx.moe_mx_combine_backward(out, y, r.rows, T, N, k, r.pos_of_pair, r.topk_w, r.topk_ids, E, 1, 0, dy, dw, dl)
    want = ops.combine_backward(out, y, r, num_experts=E)
    assert torch.equal(dy[live], want[0][live]) and torch.equal(dw, want[1]) and torch.equal(dl, want[2])
    need = moe_mx.moe_mx_linear_backward_workspace(E, r.rows, N, H, 0, moe_mx.MOE_MX_LINEAR_SILU, 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    dx, dwt, db = torch.zeros_like(g), torch.empty_like(w), torch.empty_like(b)
    moe_mx.moe_mx_linear_backward(dy, g, w, z, r.counts, r.pad_offsets, E, r.rows, N, H, 0, moe_mx.MOE_MX_LINEAR_SILU, 1,
                                  dx, dwt, db, ws, need)
    want = ops.linear_backward(dy, g, w, z, "silu", r, bias_grad=True)
    assert torch.equal(dx[live], want[0][live]) and torch.equal(dwt, want[1]) and torch.equal(db, want[2])


# ---------------------------------------------------------------- float32 outputs, each held to its own sums
@pytest.mark.parametrize("M,N,K,act,chain", [
    (16, 4096, 7168, "none", 8), (8, 4096, 7168, "swiglu", 8), (1, 384, 7168, "none", 8), (9, 1000, 20000, "none", 8),
    (24, 1024, 5000, "none", 16), (50, 1000, 2048, "none", 16), (16, 2048, 20000, "swiglu", 8),
    (64, 2048, 1984, "none", 16)])
def test_few_rows_in_float32_keep_short_chains(M, N, K, act, chain):
    """Few rows: a warp sums at most 256 of k, 16 additions of 16 products, in one tensor-core chain, and longer
    slices in chains of 128 (8 additions) or 64.  An addition truncates by half a step in the mean, 2^-24 of the
    running sum at most; the running sums r_1 .. r_n of a chain of n random additions correlate as min(i, j), so
    that the chain is off by sqrt(sum min(i, j) / n) = sqrt((n + 1) (2 n + 1) / 6) such parts of its norm, and the
    whole by the same of its own.  Joining at most 64 chains of a warp, 8 warps and 8 CTAs: 80 roundings
    of 2^-24 / sqrt(3) of a growing sum.  The last case has more multiplications (260 M) than the few-row kernel
    takes: a tile product in 8 splits of 4 blocks, 16 additions too."""
    plan = moe_mx.moe_mx_debug_linear_plan(0, 0, M, N, K, 0, ops.ACTIVATIONS[act], 1)
    assert plan == ((256, 64, 8, 0) if (M, N, K) == (64, 2048, 1984) else (0, 0, 0, 0))
    x, w, b, _, _ = _linear_inputs(M, N, K, BF, F, act, True, False, 200)
    got = ops.linear(x, w, b, activation=act, out_dtype=F)
    want = ref.linear64(x, w, b, None, act)[0]
    tol = 2.0 ** -24 * math.sqrt((chain + 1) * (2 * chain + 1) / 6 + 80 / 3 / 2)
    tol *= math.sqrt(2) if act == "swiglu" else 1  # two such sums in each output
    rel = float((got.to(ref.F64) - want).norm() / want.norm())
    assert rel <= tol, f"{rel:.2e} of {tol:.2e}"


def test_layer_outputs_each_to_their_own_roundings():
    """As test_layer_and_its_gradients_together, each result to the number of its roundings in a row (each at most
    u, independent: sqrt(n) u in norm): out h, y, out; dw2 dy, h, dw2; dw1 dy, dh, z, dz, dw1; db1 dy, dh, z; the
    router's through y (h, y), dz and the result, with a condition of 2 for the difference in the softmax's
    gradient; dx all of dw1's and dg, and the sum's.  float32 logits: one chain of 12 additions."""
    p, k = _stage_inputs()
    got, r = _layer(p, k)
    leaf = {n: t.to(ref.F64).requires_grad_() for n, t in p.items() if n != "dout"}
    logits = leaf["x"] @ leaf["wr"].t() + leaf["br"]
    ids = r.topk_ids.long()
    w = torch.softmax(logits.gather(1, ids), 1)
    z = torch.einsum("th,enh->ten", leaf["x"], leaf["w1"]) + leaf["b1"]
    y = torch.einsum("tei,ehi->teh", ref.act64(z, "swiglu"), leaf["w2"])
    out = (y[torch.arange(ids.shape[0], device="cuda")[:, None], ids] * w[..., None]).sum(1)
    names = ["x", "wr", "br", "w1", "b1", "w2"]
    grads = dict(zip(names, torch.autograd.grad(out, [leaf[n] for n in names], p["dout"].to(ref.F64))))
    u = ref.u(BF)
    for name, g, want, tol in (
            ("logits", got["logits"], logits, 2.0 ** -24 * math.sqrt(13 * 25 / 6 + 2)),
            ("out", got["out"], out, math.sqrt(3) * u), ("w2", got["dw2"], grads["w2"], math.sqrt(3) * u),
            ("w1", got["dw1"], grads["w1"], math.sqrt(5) * u), ("b1", got["db1"], grads["b1"], math.sqrt(3) * u),
            ("wr", got["dwr"], grads["wr"], 2 * math.sqrt(4) * u), ("br", got["dbr"], grads["br"], 2 * math.sqrt(2) * u),
            ("x", got["dxr"].to(ref.F64) + got["dxe"].to(ref.F64), grads["x"], math.sqrt(8) * u)):
        rel = float((g.to(ref.F64) - want.detach()).norm() / want.detach().norm())
        assert rel <= tol, f"{name}: relative error {rel:.2e} of {tol:.2e}"


def test_no_tokens_on_another_stream():
    """counts and pad_offsets are zeroed on the call's stream: zeros from another could come before a write still
    to come to the memory they got."""
    s, E = torch.cuda.Stream(), 4096 // 4 - 1  # both in blocks of one size
    torch.cuda.synchronize()
    for handle in (s, s.cuda_stream):
        with torch.cuda.stream(s):
            old = [torch.empty(E + i % 2, dtype=torch.int32, device="cuda") for i in range(12)]
            torch.cuda._sleep(20_000_000)
            for t in old:
                t.fill_(7)
            del t, old  # freed on s, their fills still to come
        r = ops.route_group(torch.empty(0, E, device="cuda"), 2, stream=handle)
        torch.cuda.synchronize()
        assert not r.counts.any() and not r.pad_offsets.any()
    r = ops.route_group(torch.empty(0, E, device="cuda"), 2, stream=0)  # the default stream by its handle
    assert not r.counts.any() and not r.pad_offsets.any()
    x = rnd((4, 72), BF, 210)
    assert torch.equal(ops.linear(x, x, stream=0), ops.linear(x, x))


@pytest.mark.parametrize("dtype", [BF, F])
def test_a_shard_that_no_pair_goes_to(dtype):
    """A grouped layout of no rows: nothing is moved, sums and gradients are zero."""
    T, E, k, H = 5, 4, 2, 40
    i32 = lambda *s, v=0: torch.full(s, v, dtype=torch.int32, device="cuda")  # noqa: E731
    r = ops.Routing(i32(T, k), torch.rand(T, k, device="cuda"), i32(E), i32(E + 1), i32(T * k, v=-1), 0)
    x, none = rnd((T, H), dtype, 220), torch.empty(0, H, dtype=dtype, device="cuda")
    assert ops.dispatch(x, r).shape == (0, H)
    for out in (ops.combine(none, r), ops.dispatch_backward(none, r)):
        assert out.shape == (T, H) and not out.any()
    dy, dw, dlogits = ops.combine_backward(x, none, r, num_experts=E)
    assert dy.shape == (0, H) and not dw.any() and not dlogits.any()
    if dtype == BF:
        w = rnd((E, 24, H), BF, 221)
        assert ops.linear(none, w, routing=r).shape == (0, 24)
        dx, dw, db = ops.linear_backward(none.new_empty(0, 24), none, w, routing=r, bias_grad=True)
        assert dx.shape == (0, H) and not dw.any() and not db.any()
