"""Plain float64 definitions of the routed operators, and the error bounds their outputs are held to.

Bounds count roundings (u = eps / 2 is half a step of a type): an output rounded once to type t
is off by u_t |value|; a float32 sum of n products, in any order and even if every addition
truncates, by n 2^-23 sum |products|; a value computed in float32 from an activation by a few
ulp, taken as 2^-20 of it (exp to 2 ulp with an argument error of |z| 2^-24, |z| <= 8 here).
"""
import math

import torch

F64 = torch.float64


def u(t):
    return torch.finfo(t).eps / 2


def make_routing(T, E, k, seed, drop=0.0, hot=None, device="cuda"):
    """A Routing of random distinct experts: each token k of E; `drop` of the pairs left out (-1);
    `hot`: an expert that every token takes; experts E//3 and (if 8 or more) E - 1 are never taken when k
    allows it, so that empty segments occur inside and at the end."""
    from block_scaled_moe_softmax_b200.routed_ops import Routing, max_grouped_rows
    g = torch.Generator().manual_seed(seed)
    score = torch.rand(T, E, generator=g)
    if k <= E - 2:
        score[:, E // 3] = -1
        if E >= 8:
            score[:, E - 1] = -1
    if hot is not None:
        score[:, hot] = 2
    ids = torch.argsort(score, 1, descending=True)[:, :k].contiguous()
    w = torch.softmax(torch.randn(T, k, generator=g), 1)
    flat = ids.reshape(-1).clone()
    if drop:
        flat[torch.rand(T * k, generator=g) < drop] = -1
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    pad = torch.zeros(E + 1, dtype=torch.long)
    pad[1:] = torch.cumsum((counts + 127) // 128 * 128, 0)
    pos = torch.full((T * k,), -1, dtype=torch.long)
    nxt = pad[:-1].clone()
    for p, e in enumerate(flat.tolist()):
        if e >= 0:
            pos[p] = nxt[e]
            nxt[e] += 1
    i32 = lambda t: t.to(torch.int32).to(device).contiguous()  # noqa: E731
    return Routing(i32(ids), w.to(device), i32(counts), i32(pad), i32(pos), max_grouped_rows(T * k, E))


def segments(r, rows):
    """(expert, first row, end) of each segment; a dense call is one."""
    if r is None:
        return [(0, 0, rows)]
    pad, counts = r.pad_offsets.tolist(), r.counts.tolist()
    return [(e, pad[e], pad[e] + counts[e]) for e in range(len(counts))]


def act64(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "swiglu":
        g, up = z.chunk(2, -1)
        return g * torch.sigmoid(g) * up
    return z


def act_grad64(d, z, act):
    """d * act'(z) (both halves for swiglu), from the formulas."""
    if act == "none":
        return d
    if act == "silu":
        q = torch.sigmoid(z)
        return d * (q + z * q * (1 - q))
    if act == "gelu":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z ** 3))
        return d * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z))
    g, up = z.chunk(2, -1)
    q = torch.sigmoid(g)
    return torch.cat([d * up * (q + g * q * (1 - q)), d * g * q], -1)


def linear64(x, w, bias, residual, act, r=None):
    """(out, preact, bound on |out - exact| before its rounding, the same of preact); rows without a
    pair are NaN."""
    rows, N = x.shape[0], w.shape[-2]
    cols = N // 2 if act == "swiglu" else N
    nan = lambda n: torch.full((rows, n), math.nan, dtype=F64, device=x.device)  # noqa: E731
    out, pre, out_b, pre_b = nan(cols), nan(N), nan(cols), nan(N)
    for e, lo, hi in segments(r, rows):
        xe = x[lo:hi].to(F64)
        we = (w if r is None else w[e]).to(F64)
        z = xe @ we.t()
        zb = (x.shape[1] + 2) * 2.0 ** -23 * (xe.abs() @ we.abs().t())
        if bias is not None:
            b = (bias if r is None else bias[e]).to(F64)
            z = z + b
            zb = zb + 2.0 ** -23 * (b.abs() + z.abs())
        pre[lo:hi], pre_b[lo:hi] = z, zb
        a = act64(z, act)
        # |act'| <= 1.13 for silu and gelu; for swiglu each half scales the other's error
        if act == "swiglu":
            g, up = z.chunk(2, -1)
            gb, ub = zb.chunk(2, -1)
            ab = 1.13 * gb * (up.abs() + ub) + ub * (g.abs() + gb)
        else:
            ab = zb * (1.13 if act != "none" else 1)
        ab = ab + (2.0 ** -20 * a.abs() if act != "none" else 0)
        if residual is not None:
            res = residual[lo:hi].to(F64)
            a = a + res
            ab = ab + 2.0 ** -23 * (a.abs() + res.abs())
        out[lo:hi], out_b[lo:hi] = a, ab
    return out, pre, out_b, pre_b


def linear_backward64(dout, x, w, pre, act, r=None):
    """(dx, dw, db) and bounds on their errors before the outputs' rounding.  dz is off by u of the
    operands' type (its one rounding) and 2^-18 of |dout| (|1| + |z|)-sized terms of act' (cancellation in
    act' leaves an absolute error of a few 2^-24 times its terms)."""
    t = x.dtype
    rows, K = x.shape
    N = w.shape[-2]
    E = 1 if r is None else w.shape[0]
    dx = torch.full((rows, K), math.nan, dtype=F64, device=x.device)
    dxb = dx.clone()
    dw = torch.zeros(E, N, K, dtype=F64, device=x.device)
    dwb, db, dbb = dw.clone(), dw[..., 0].clone(), dw[..., 0].clone()
    for e, lo, hi in segments(r, rows):
        d, xe = dout[lo:hi].to(F64), x[lo:hi].to(F64)
        we = (w if r is None else w[e]).to(F64)
        z = pre[lo:hi].to(F64) if pre is not None else None
        dz = act_grad64(d, z, act)
        err0 = torch.zeros_like(dz)
        if act == "swiglu":
            g, up = z.chunk(2, -1)
            err0 = 2.0 ** -18 * torch.cat([d.abs() * up.abs() * (1 + g.abs()), d.abs() * g.abs()], -1)
        elif act != "none":
            err0 = 2.0 ** -18 * d.abs() * (1 + z.abs()) ** 3
        dzb = err0 + u(t) * dz.abs() * (act != "none" or dout.dtype != t)
        if t == torch.float16:
            dzb = dzb + 2.0 ** -25  # half a subnormal step
        n, m = N + 2, hi - lo + 2
        dx[lo:hi] = dz @ we
        dxb[lo:hi] = dzb @ we.abs() + n * 2.0 ** -23 * ((dz.abs() + dzb) @ we.abs())
        dw[e] = dz.t() @ xe
        dwb[e] = dzb.t() @ xe.abs() + m * 2.0 ** -23 * ((dz.abs() + dzb).t() @ xe.abs())
        db[e] = dz.sum(0)
        dbb[e] = err0.sum(0) + m * 2.0 ** -23 * dz.abs().sum(0)
    if r is None:
        dw, dwb, db, dbb = dw[0], dwb[0], db[0], dbb[0]
    return (dx, dw, db), (dxb, dwb, dbb)


def close(got, want, bound, tag=""):
    """got (rounded once to its type) against want; where want is NaN got is not compared."""
    live = ~torch.isnan(want)
    g, w, b = got.to(F64)[live], want[live], (bound if torch.is_tensor(bound) else torch.full_like(want, bound))[live]
    tol = b + u(got.dtype) * (w.abs() + b) + torch.finfo(got.dtype).smallest_normal * u(got.dtype) * 2
    bad = ~((g - w).abs() <= tol)
    assert not bad.any(), (f"{tag}: {int(bad.sum())} of {bad.numel()} values off, the worst by "
                           f"{float(((g - w).abs() / tol).nan_to_num(math.inf).max()):.2f} of the bound")


def close_norm(got, want, roundings, tag=""):
    """Relative 2-norm error: independent roundings of at most u each add up to sqrt(roundings) u; a
    float32 sum's error (below 2^-16 in norm for the lengths tested) comes on top."""
    live = ~torch.isnan(want)
    g, w = got.to(F64)[live], want[live]
    if not w.numel() or not w.abs().max():
        assert not g.numel() or not g.abs().max(), tag
        return
    rel = float((g - w).norm() / w.norm())
    assert rel <= math.sqrt(roundings) * u(got.dtype) + 2.0 ** -16, f"{tag}: relative error {rel:.2e}"
