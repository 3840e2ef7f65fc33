"""Cases of the routed operators: linear, linear_backward, dispatch, combine and combine_backward.

Every case is one pass through one operator, in its plain form (elementary torch operations in
float32) or, with ``own`` set, through block_scaled_moe_softmax_b200.routed_ops.  Rows sorted by
expert live in the library's grouped layout: expert e's rows start at pad_offsets[e], a multiple of
128, and the rows behind its counts[e] pairs are padding, which no operator reads or writes (the
output buffers of such cases are made once, zeroed, and kept by the caller).
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------- cases
def _linear(name, op, M, K, N, dtype="bf16", out="bf16", act="none", bias=True, residual=False, preact=False,
            E=0, top_k=0):
    """M tokens of K features, N weight rows; E > 0: the tokens' top_k pairs sorted over E experts."""
    return dict(name=name, op=op, M=M, K=K, N=N, dtype=dtype, out=out, act=act, bias=bias, residual=residual,
                preact=preact, E=E, top_k=top_k)


def _rows(name, op, M, H, E, top_k, dtype="bf16", out="bf16", weighted=True):
    return dict(name=name, op=op, M=M, H=H, E=E, top_k=top_k, dtype=dtype, out=out, weighted=weighted)


def listed():
    return [
        # the router's logits of one decoded token: the smallest product, latency counts
        _linear("router_t1", "linear", 1, 7168, 384, out="f32"),
        # the router's logits of a prefill
        _linear("router_prefill", "linear", 8192, 7168, 384, out="f32"),
        # an unquantised shared expert's second product of a prefill, added to the residual stream
        _linear("shared_fc2_prefill", "linear", 8192, 2048, 7168, residual=True),
        # unquantised experts' first product with SwiGLU in training (64 experts of the prefill shape);
        # the products before the activation are kept for the backward pass
        _linear("experts_fc1", "linear", 2048, 7168, 4096, act="swiglu", bias=False, preact=True, E=64, top_k=8),
        # the router's gradients in training: float32 gradients of the logits
        _linear("router_backward", "linear_backward", 4096, 7168, 384, out="f32"),
        # gradients of small ragged experts in float16
        _linear("experts_backward", "linear_backward", 1000, 1408, 2816, dtype="f16", out="f16", act="swiglu", E=16,
                top_k=4),
        # one decode step of a tiny layer: the smallest copy
        _rows("dispatch_tiny", "dispatch", 16, 256, 8, 2),
        # a prefill's rows sorted over 384 experts
        _rows("dispatch_prefill", "dispatch", 8192, 7168, 384, 8),
        # a batched decode's float32 expert outputs summed back to bf16 tokens
        _rows("combine_decode", "combine", 256, 7168, 384, 8, dtype="f32"),
        # a long prefill of the smaller layer
        _rows("combine_prefill", "combine", 16384, 4096, 128, 8),
        # odd sizes: 333 tokens of 1000 features in float16
        _rows("combine_backward_odd", "combine_backward", 333, 1000, 60, 6, dtype="f16", out="f16"),
        # a training step's gradients through the combine, its weights and the router's softmax
        _rows("combine_backward_large", "combine_backward", 8192, 7168, 384, 8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "dispatch", "combine", "combine_backward"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op in ("linear", "linear_backward"):
        act = rng.choice(["none", "none", "silu", "gelu", "swiglu"])
        E = rng.choice([0, 0, _log(rng, 2, 64)])
        M = _log(rng, 1 if op == "linear" else 16, 8192 if E == 0 else 2048)
        K = _log(rng, 64, 7168)
        N = _log(rng, 16, 4096)
        if rng.random() < 0.7:  # most models' sizes are multiples of 64
            K, N = max(64, K // 64 * 64), max(64, N // 64 * 64)
        if act == "swiglu":
            N += N % 2
        out = rng.choice([dtype, dtype, "f32"])
        return _linear(None, op, M, K, N, dtype, out, act, rng.random() < 0.6,
                       op == "linear" and act != "swiglu" and rng.random() < 0.4,
                       op == "linear_backward" or rng.random() < 0.3, E,
                       rng.randint(1, min(E, 8)) if E else 0) | {"name": ""}
    dtype = rng.choice([dtype, dtype, "f32"])
    E = _log(rng, 4, 384)
    H = _log(rng, 64, 7168)
    if rng.random() < 0.7:
        H = max(64, H // 64 * 64)
    out = dtype if op == "dispatch" else rng.choice([dtype, "bf16", "f32"])
    M = _log(rng, 1, 4096)
    return _rows("", op, M, H, E, rng.randint(1, min(E, 8)), dtype, out, op != "combine" or rng.random() < 0.7)


# ---------------------------------------------------------------- inputs
def _routing(M, E, top_k, gen):
    """top_k distinct experts of each token, unevenly loaded, and the grouped layout of the pairs."""
    dev = "cuda"
    skew = torch.randn(E, generator=gen, device=dev) * 0.5
    logits = torch.randn(M, E, generator=gen, device=dev) + skew
    top, ids = torch.topk(logits, top_k, dim=1)
    P = M * top_k
    flat = ids.reshape(-1)
    counts = torch.bincount(flat, minlength=E)
    pad = (counts + 127) // 128 * 128
    pad_offsets = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    pad_offsets[1:] = torch.cumsum(pad, 0)
    order = torch.argsort(flat, stable=True)
    starts = torch.cumsum(counts, 0) - counts
    pos = torch.empty(P, dtype=torch.int64, device=dev)
    pos[order] = pad_offsets[flat[order]] + torch.arange(P, device=dev) - starts[flat[order]]
    rows = (P + min(P, E) * 127 + 127) // 128 * 128
    return dict(topk_ids=ids.to(torch.int32), topk_w=torch.softmax(top, 1), counts=counts.to(torch.int32),
                pad_offsets=pad_offsets.to(torch.int32), pos_of_pair=pos.to(torch.int32), rows=rows,
                most=int(counts.max()))


def _normal(shape, dtype, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=_DTYPES[dtype]) * scale).to(_DTYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    dt, E, M = c["dtype"], c["E"], c["M"]
    s = {"case": c}
    if E:
        s["routing"] = r = _routing(M, E, c["top_k"], gen)
    if c["op"] in ("linear", "linear_backward"):
        K, N = c["K"], c["N"]
        No = N // 2 if c["act"] == "swiglu" else N
        rows = r["rows"] if E else M
        lead = (E,) if E else ()
        s["w"] = _normal(lead + (N, K), dt, gen, K ** -0.5)
        s["bias"] = torch.randn(lead + (N,), generator=gen, device="cuda") * 0.1 if c["bias"] else None
        s["x"] = _spread(_normal((M, K), dt, gen), r) if E else _normal((M, K), dt, gen)
        out = _DTYPES[c["out"]]
        if c["op"] == "linear":
            s["residual"] = _normal((rows, No), c["out"], gen) if c["residual"] else None
            s["out"] = torch.zeros(rows, No, dtype=out, device="cuda")
            s["preact"] = torch.zeros(rows, N, dtype=_DTYPES[dt], device="cuda") if c["preact"] else None
        else:
            z = _normal((rows, N), dt, gen)
            s["preact"] = z if c["act"] != "none" else None
            s["dout"] = _normal((rows, No), c["out"], gen)
            s["dx"] = torch.zeros(rows, K, dtype=_DTYPES[dt], device="cuda")
        return s
    H = c["H"]
    if c["op"] == "dispatch":
        s["x"] = _normal((M, H), dt, gen)
        s["out"] = torch.zeros(r["rows"], H, dtype=_DTYPES[dt], device="cuda")
    else:
        s["y"] = _normal((r["rows"], H), dt, gen)
        if c["op"] == "combine_backward":
            s["dout"] = _normal((M, H), c["out"], gen)
            s["dy"] = torch.zeros(r["rows"], H, dtype=_DTYPES[dt], device="cuda")
    return s


def _spread(x, r):
    """Token rows at their pairs' grouped rows (padding rows zero)."""
    out = torch.zeros(r["rows"], x.shape[1], dtype=x.dtype, device=x.device)
    k = r["topk_ids"].shape[1]
    out[r["pos_of_pair"].long()] = x.repeat_interleave(k, 0)
    return out


# ---------------------------------------------------------------- the operators
def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        return _own(op, c, s)
    return {"linear": _plain_linear, "linear_backward": _plain_linear_backward, "dispatch": _plain_dispatch,
            "combine": _plain_combine, "combine_backward": _plain_combine_backward}[op](c, s)


def _own(op, c, s):
    from block_scaled_moe_softmax_b200 import routed_ops as ops
    r = None
    if c["E"]:
        d = s["routing"]
        r = ops.Routing(d["topk_ids"], d["topk_w"], d["counts"], d["pad_offsets"], d["pos_of_pair"], d["rows"])
    if op == "linear":
        out = ops.linear(s["x"], s["w"], s["bias"], residual=s["residual"], activation=c["act"], routing=r,
                         out=s["out"], preact=s["preact"])
        return [out] if s["preact"] is None else [out, s["preact"]]
    if op == "linear_backward":
        dx, dw, db = ops.linear_backward(s["dout"], s["x"], s["w"], preact=s["preact"], activation=c["act"],
                                         routing=r, bias_grad=c["bias"], dx=s["dx"])
        return [dx, dw] if db is None else [dx, dw, db]
    if op == "dispatch":
        return [ops.dispatch(s["x"], r, out=s["out"])]
    if op == "combine":
        if c["weighted"]:
            return [ops.combine(s["y"], r, out_dtype=_DTYPES[c["out"]])]
        return [ops.dispatch_backward(s["y"], r, out_dtype=_DTYPES[c["out"]])]
    return list(ops.combine_backward(s["dout"], s["y"], r, num_experts=c["E"], dy=s["dy"]))


def _blocks(r, E):
    """Grouped row of each slot of an [E, most] block of rows, and whether it holds a pair."""
    slot = torch.arange(r["most"], device="cuda")
    return r["pad_offsets"][:E, None].long() + slot, slot < r["counts"][:, None]


def _act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "swiglu":
        g, u = z.chunk(2, -1)
        return g * torch.sigmoid(g) * u
    return z


def _act_backward(d, z, act):
    if act == "silu":
        q = torch.sigmoid(z)
        return d * (q * (1 + z * (1 - q)))
    if act == "gelu":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return d * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z))
    if act == "swiglu":
        g, u = z.chunk(2, -1)
        q = torch.sigmoid(g)
        return torch.cat([d * u * (q * (1 + g * (1 - q))), d * g * q], -1)
    return d


def _plain_linear(c, s):
    E, w = c["E"], s["w"].float()
    bias = s["bias"]
    if E:
        at, live = _blocks(s["routing"], E)
        at = torch.where(live, at, 0)
        z = torch.bmm(s["x"].float()[at], w.transpose(1, 2))
        if bias is not None:
            z = z + bias[:, None]
        a = _act(z, c["act"])
        rows = at[live]
        out, pre = torch.zeros_like(s["out"]), None
        if s["residual"] is not None:
            out[rows] = (a[live] + s["residual"][rows].float()).to(out.dtype)
        else:
            out[rows] = a[live].to(out.dtype)
        if s["preact"] is not None:
            pre = torch.zeros_like(s["preact"])
            pre[rows] = z[live].to(pre.dtype)
        return [out] if pre is None else [out, pre]
    z = s["x"].float() @ w.t()
    if bias is not None:
        z = z + bias
    a = _act(z, c["act"])
    if s["residual"] is not None:
        a = a + s["residual"].float()
    out = a.to(s["out"].dtype)
    return [out] if s["preact"] is None else [out, z.to(s["preact"].dtype)]


def _plain_linear_backward(c, s):
    E, w, dt = c["E"], s["w"].float(), s["w"].dtype
    d = s["dout"].float()
    dz = _act_backward(d, None if s["preact"] is None else s["preact"].float(), c["act"])
    if E:
        at, live = _blocks(s["routing"], E)
        at = torch.where(live, at, 0)
        dzb = dz[at] * live[..., None]
        dxb = torch.bmm(dzb, w)
        dw = torch.bmm(dzb.transpose(1, 2), s["x"].float()[at]).to(dt)
        dx = torch.zeros_like(s["dx"])
        dx[at[live]] = dxb[live].to(dt)
        return [dx, dw, dzb.sum(1)] if c["bias"] else [dx, dw]
    dx, dw = (dz @ w).to(dt), (dz.t() @ s["x"].float()).to(dt)
    return [dx, dw, dz.sum(0)] if c["bias"] else [dx, dw]


def _plain_dispatch(c, s):
    r = s["routing"]
    out = torch.zeros_like(s["out"])
    out[r["pos_of_pair"].long()] = s["x"].repeat_interleave(c["top_k"], 0)
    return [out]


def _plain_combine(c, s):
    r = s["routing"]
    y = s["y"][r["pos_of_pair"].long()].float().view(c["M"], c["top_k"], -1)
    if c["weighted"]:
        y = y * r["topk_w"][..., None]
    return [y.sum(1).to(_DTYPES[c["out"]])]


def _plain_combine_backward(c, s):
    r = s["routing"]
    pos, w = r["pos_of_pair"].long(), r["topk_w"]
    y = s["y"][pos].float().view(c["M"], c["top_k"], -1)
    d = s["dout"].float()[:, None]
    dy = torch.zeros_like(s["dy"])
    dy[pos] = (d * w[..., None]).to(dy.dtype).view(-1, c["H"])
    dw = (d * y).sum(2)
    g = w * (dw - (w * dw).sum(1, keepdim=True))
    dlogits = torch.zeros(c["M"], c["E"], device="cuda").scatter_(1, r["topk_ids"].long(), g)
    return [dy, dw, dlogits]


# ---------------------------------------------------------------- work
def work(case):
    c = case
    b, ob, P = _BYTES[c["dtype"]], _BYTES[c["out"]], c["M"] * max(1, c["top_k"])
    E, M = c["E"], c["M"]
    if c["op"] in ("linear", "linear_backward"):
        K, N = c["K"], c["N"]
        No = N // 2 if c["act"] == "swiglu" else N
        hit = min(E, P) if E else 1
        if c["op"] == "linear":
            bytes_ = (P * K + hit * N * K) * b + P * No * ob * (2 if c["residual"] else 1)
            bytes_ += 4 * hit * N * c["bias"] + (P * N * b if c["preact"] else 0)
            return {"bytes": bytes_, "flops": 2 * P * N * K}
        n = E if E else 1
        bytes_ = P * No * ob + (2 * P * K + (hit + n) * N * K) * b + 4 * n * N * c["bias"]
        bytes_ += P * N * b if c["act"] != "none" else 0
        return {"bytes": bytes_, "flops": 4 * P * N * K}
    H = c["H"]
    if c["op"] == "dispatch":
        return {"bytes": (M + P) * H * b + 4 * P, "flops": 0}
    if c["op"] == "combine":
        return {"bytes": P * H * b + M * H * ob + P * (8 if c["weighted"] else 4), "flops": 2 * P * H}
    return {"bytes": 2 * P * H * b + M * H * ob + 16 * P + 4 * M * E, "flops": 3 * P * H}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    r = s.get("routing")
    f = torch.float64

    def product():
        E = c["E"]
        n = s["w"].shape[-2]
        starts = r["pad_offsets"].tolist() if E else [0]
        counts = r["counts"].tolist() if E else [c["M"]]
        rows = r["rows"] if E else c["M"]
        no = n // 2 if c["act"] == "swiglu" else n
        back = c["op"] == "linear_backward"
        out = torch.zeros(rows, c["K"] if back else no, dtype=f, device="cuda")
        second = torch.zeros(max(E, 1), n, c["K"], dtype=f, device="cuda") if back else \
            torch.zeros(rows, n, dtype=f, device="cuda")
        db = torch.zeros(max(E, 1), n, dtype=f, device="cuda")
        for e, (lo, m) in enumerate(zip(starts, counts)):
            x = s["x"][lo:lo + m].to(f)
            w = (s["w"][e] if E else s["w"]).to(f)
            if not back:
                z = x @ w.t()
                if s["bias"] is not None:
                    z += (s["bias"][e] if E else s["bias"]).to(f)
                second[lo:lo + m] = z
                a = _exact_act(z, c["act"])
                if s["residual"] is not None:
                    a = a + s["residual"][lo:lo + m].to(f)
                out[lo:lo + m] = a
                continue
            d = s["dout"][lo:lo + m].to(f)
            if c["act"] != "none":
                with torch.enable_grad():
                    z = s["preact"][lo:lo + m].to(f).requires_grad_()
                    d = torch.autograd.grad(_exact_act(z, c["act"]), z, d)[0]
            out[lo:lo + m] = d @ w
            second[e] = d.t() @ x
            db[e] = d.sum(0)
        if back:
            if not E:
                second, db = second[0], db[0]
            return [out, second, db] if c["bias"] else [out, second]
        return [out, second] if s["preact"] is not None else [out]

    if c["op"] in ("linear", "linear_backward"):
        return product()
    pos, k = r["pos_of_pair"].long(), c["top_k"]
    if c["op"] == "dispatch":
        out = torch.zeros(r["rows"], c["H"], dtype=f, device="cuda")
        for j in range(k):
            out.index_copy_(0, pos[j::k], s["x"].to(f))
        return [out]
    w = r["topk_w"].to(f)
    if c["op"] == "combine":
        out = torch.zeros(c["M"], c["H"], dtype=f, device="cuda")
        for j in range(k):
            row = s["y"][pos[j::k]].to(f)
            out += row * w[:, j:j + 1] if c["weighted"] else row
        return [out]
    d = s["dout"].to(f)
    dy = torch.zeros(r["rows"], c["H"], dtype=f, device="cuda")
    dw = torch.empty(c["M"], k, dtype=f, device="cuda")
    for j in range(k):
        dy.index_copy_(0, pos[j::k], d * w[:, j:j + 1])
        dw[:, j] = torch.einsum("th,th->t", d, s["y"][pos[j::k]].to(f))
    # the weights are softmax over the chosen logits: J = diag(w) - w w^T
    jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
    g = torch.einsum("tij,tj->ti", jac, dw)
    dlogits = torch.zeros(c["M"], c["E"], dtype=f, device="cuda")
    dlogits.scatter_add_(1, r["topk_ids"].long(), g)
    return [dy, dw, dlogits]


def _exact_act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        return z / (1 + torch.exp(-2 * u))
    if act == "swiglu":
        h = z.shape[1] // 2
        return z[:, :h] / (1 + torch.exp(-z[:, :h])) * z[:, h:]
    return z
