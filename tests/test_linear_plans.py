"""Every instance of the tile product, at sizes of more tiles than the card has SM pairs: which plan a size gets
(on the host), and that product against plain float64 code (on a GPU).  A pair then takes a second and third
tile: the accumulators' parity over chains, residuals loaded ahead, tiles found by each warp or ahead of it."""
import pytest
import torch

from block_scaled_moe_softmax_b200 import moe_mx
from block_scaled_moe_softmax_b200 import routed_ops as ops
from tests import routed_ref as ref

BF, HF, F = torch.bfloat16, torch.float16, torch.float32
PAIRS = 74

# M, N, K, type, out, activation, bias, residual, preact; columns of a tile, tokens of one (0: 256 rows), splits, sum
FORWARD = [
    # 256 columns: one 16-bit output in lines, with every part of the epilogue, ragged columns, float32, SwiGLU
    (5000, 4104, 576, BF, BF, "none", False, False, False, (256, 0, 1, 0)),
    (5000, 4104, 576, HF, HF, "silu", True, False, False, (256, 0, 1, 0)),
    (5000, 4104, 576, BF, BF, "gelu", True, True, True, (256, 0, 1, 0)),
    (5000, 4097, 577, HF, HF, "silu", True, True, True, (256, 0, 1, 0)),
    (5000, 4104, 320, BF, F, "gelu", True, True, False, (256, 0, 1, 0)),
    (5000, 4096, 576, BF, BF, "swiglu", False, False, True, (256, 0, 1, 0)),
    (5000, 4102, 576, HF, HF, "swiglu", True, True, True, (256, 0, 1, 0)),
    (5000, 4102, 512, BF, F, "swiglu", True, True, False, (256, 0, 1, 0)),
    (2048, 2560, 14336, BF, BF, "gelu", True, True, True, (256, 0, 3, 0)),
    (2048, 2560, 14336, HF, HF, "swiglu", True, False, True, (256, 0, 3, 0)),
    # 192 columns
    (3000, 2048, 700, BF, BF, "none", False, False, False, (192, 0, 1, 0)),
    (3000, 2048, 700, HF, HF, "silu", True, True, True, (192, 0, 1, 0)),
    (3000, 2050, 700, BF, BF, "gelu", True, True, True, (192, 0, 1, 0)),
    (3000, 2048, 500, BF, F, "none", True, True, True, (192, 0, 1, 0)),
    # the same with chains summed in registers
    (20000, 384, 1096, BF, F, "none", True, False, False, (192, 0, 1, 1)),
    (20000, 384, 1096, HF, F, "silu", True, True, True, (192, 0, 1, 1)),
    (5000, 4101, 577, BF, F, "gelu", True, True, True, (192, 0, 1, 1)),
    # 128 columns
    (30000, 128, 300, HF, HF, "none", True, False, False, (128, 0, 1, 0)),
    (30000, 128, 300, BF, BF, "gelu", True, True, True, (128, 0, 1, 0)),
    (30000, 126, 300, BF, BF, "swiglu", True, True, True, (128, 0, 1, 0)),
    (30000, 128, 600, HF, F, "silu", True, True, True, (128, 0, 1, 1)),
    (5000, 4096, 576, BF, F, "swiglu", True, True, True, (128, 0, 1, 1)),
    (5000, 4102, 576, HF, F, "swiglu", False, False, False, (128, 0, 1, 1)),
    # tiles of tokens
    (200, 20000, 576, BF, BF, "silu", True, False, False, (256, 224, 1, 0)),
    (300, 12000, 576, BF, BF, "gelu", True, True, True, (256, 128, 1, 0)),
    (200, 20001, 577, HF, HF, "none", True, True, True, (256, 224, 1, 0)),
    (200, 20000, 576, BF, BF, "swiglu", True, True, True, (256, 224, 1, 0)),
    (200, 20000, 576, BF, F, "silu", True, True, True, (256, 128, 1, 1)),
    (200, 20000, 576, HF, F, "swiglu", True, True, True, (256, 128, 1, 1)),
]

# M, N, K, type, dout's type, activation, which gradient has more tiles than pairs; its plan
BACKWARD = [
    (20000, 384, 1096, BF, F, "none", 1, (256, 0, 1, 0)), (20000, 384, 1095, HF, F, "silu", 1, (256, 0, 1, 0)),
    (20000, 96, 72, HF, HF, "silu", 1, (128, 0, 1, 0)), (200, 576, 20000, BF, BF, "gelu", 1, (256, 224, 1, 0)),
    (20000, 9000, 136, BF, BF, "none", 1, (256, 0, 3, 0)), (20000, 9000, 72, BF, BF, "none", 1, (128, 0, 3, 0)),
    (1000, 4104, 4104, BF, BF, "swiglu", 2, (256, 0, 1, 0)), (1000, 4102, 4101, HF, F, "gelu", 2, (256, 0, 1, 0)),
    (1000, 20000, 96, BF, BF, "silu", 2, (128, 0, 1, 0)), (8000, 2056, 1096, HF, HF, "none", 2, (256, 0, 3, 0)),
]

# T, E, k, N, K, type, out, activation; columns and tokens of a tile, sum
GROUPED = [
    (3000, 8, 2, 1056, 600, BF, BF, "swiglu", (256, 256, 1, 0)), (3000, 8, 2, 1056, 600, HF, F, "swiglu", (256, 256, 1, 1)),
    (3000, 8, 2, 1030, 600, BF, BF, "swiglu", (128, 0, 1, 0)), (3000, 8, 2, 1030, 600, HF, F, "swiglu", (128, 0, 1, 1)),
    (3000, 8, 2, 1056, 600, BF, F, "gelu", (256, 256, 1, 1)), (3000, 8, 2, 1101, 601, HF, HF, "silu", (256, 256, 1, 0)),
    (16, 384, 8, 512, 1024, BF, BF, "swiglu", (256, 256, 1, 0)), (700, 384, 8, 264, 520, BF, F, "none", (256, 256, 1, 1)),
]
_TYPE = {BF: moe_mx.MOE_MX_TYPE_BF16, HF: moe_mx.MOE_MX_TYPE_F16, F: moe_mx.MOE_MX_TYPE_F32}


def _plan(which, E, M, N, K, dtype, act, io):
    return moe_mx.moe_mx_debug_linear_plan(which, E, M, N, K, _TYPE[dtype], ops.ACTIVATIONS[act], _TYPE[io])


def _tiles(plan, rows, cols):
    bn, tok, splits, _ = plan
    return (-(-rows // tok) * -(-cols // 256) if tok else -(-rows // 256) * -(-cols // bn)) * splits


def test_these_sizes_get_these_plans():
    for M, N, K, dtype, out, act, _, _, _, plan in FORWARD:
        assert _plan(0, 0, M, N, K, dtype, act, out) == plan, (M, N, K, act)
        assert _tiles(plan, M, N) > PAIRS
    for M, N, K, dtype, dout, act, which, plan in BACKWARD:
        assert _plan(which, 0, M, N, K, dtype, act, dout) == plan, (M, N, K, act)
        assert _tiles(plan, *((M, K) if which == 1 else (N, K))) > PAIRS
    for T, E, k, N, K, dtype, out, act, plan in GROUPED:
        assert _plan(0, E, ops.max_grouped_rows(T * k, E), N, K, dtype, act, out) == plan, (E, N, K, act)


def test_every_width_order_and_sum_is_among_them():
    forward = {(p[0], p[1] > 0, p[3]) for *_, p in FORWARD}
    assert forward == {(256, False, 0), (192, False, 0), (192, False, 1), (128, False, 0), (128, False, 1), (256, True, 0),
                       (256, True, 1)}
    assert {(w, p[0], p[1] > 0) for *_, w, p in BACKWARD} == {(1, 256, False), (1, 128, False), (1, 256, True),
                                                               (2, 256, False), (2, 128, False)}
    assert {(p[0], p[3]) for *_, p in GROUPED} == {(256, 0), (256, 1), (128, 0), (128, 1)}


def test_the_plan_getter_refuses():
    for args in ((3, 0, 8, 16, 64, 0, 0, 0), (0, -1, 8, 16, 64, 0, 0, 0), (0, 0, 8, 16, 64, 0, 9, 0), (1, 0, 8, 15, 64, 0, 3, 0)):
        with pytest.raises(moe_mx.MoeMxError) as e:
            moe_mx.moe_mx_debug_linear_plan(*args)
        assert e.value.code == moe_mx.MOE_MX_ERR_INVALID_ARG


def _rnd(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _check(x, w, b, res, act, out, preact, r=None):
    rows, N = x.shape[0], w.shape[-2]
    cols = N // 2 if act == "swiglu" else N
    buf = torch.full((rows, cols), 7.0, dtype=out, device="cuda")
    pre = torch.full((rows, N), 7.0, dtype=x.dtype, device="cuda") if preact else None
    ops.linear(x, w, b, residual=res, activation=act, routing=r, out=buf, preact=pre)
    want, want_pre, bound, pre_bound = ref.linear64(x, w, b, res, act, r)
    ref.close(buf, want, bound, "out")
    ref.close_norm(buf, want, 1, "out")
    if preact:
        ref.close(pre, want_pre, pre_bound, "preact")
        ref.close_norm(pre, want_pre, 1, "preact")
    if r is not None:  # padding rows keep what they held
        pad = want[:, 0].isnan()
        assert bool((buf[pad] == 7.0).all()) and (not preact or bool((pre[pad] == 7.0).all()))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,dtype,out,act,bias,residual,preact,plan", FORWARD)
def test_forward_of_many_tiles(M, N, K, dtype, out, act, bias, residual, preact, plan):
    x, w = _rnd((M, K), dtype, 1), _rnd((N, K), dtype, 2, K ** -0.5)
    b = _rnd((N,), F, 3) if bias else None
    res = _rnd((M, N // 2 if act == "swiglu" else N), out, 4) if residual else None
    _check(x, w, b, res, act, out, preact)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,dtype,dout,act,which,plan", BACKWARD)
def test_gradients_of_many_tiles(M, N, K, dtype, dout, act, which, plan):
    x, w = _rnd((M, K), dtype, 5), _rnd((N, K), dtype, 6, K ** -0.5)
    d = _rnd((M, N // 2 if act == "swiglu" else N), dout, 7)
    pre = _rnd((M, N), dtype, 8) if act != "none" else None
    got = ops.linear_backward(d, x, w, pre, act, bias_grad=True)
    want, bound = ref.linear_backward64(d, x, w, pre, act)
    for name, g, a, e in zip(("dx", "dw", "db"), got, want, bound):
        ref.close(g, a, e, name)
    ref.close_norm(got[0], want[0], 2, "dx")
    ref.close_norm(got[1], want[1], 2, "dw")


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,N,K,dtype,out,act,plan", GROUPED)
def test_grouped_products_of_many_tiles(T, E, k, N, K, dtype, out, act, plan):
    r = ref.make_routing(T, E, k, 9)
    cols = N // 2 if act == "swiglu" else N
    assert sum(-(-c // 256) for c in r.counts.tolist()) * -(-cols // (128 if act == "swiglu" else 256)) > PAIRS
    x, w = _rnd((r.rows, K), dtype, 10), _rnd((E, N, K), dtype, 11, K ** -0.5)
    _check(x, w, _rnd((E, N), F, 12), _rnd((r.rows, cols), out, 13), act, out, True, r)
    d, pre = _rnd((r.rows, cols), dtype, 14), _rnd((r.rows, N), dtype, 15)
    pre = pre if act != "none" else None
    dx = torch.full_like(x, 7.0)
    got = ops.linear_backward(d, x, w, pre, act, r, bias_grad=True, dx=dx)
    want, bound = ref.linear_backward64(d, x, w, pre, act, r)
    for name, g, a, e in zip(("dx", "dw", "db"), got, want, bound):
        ref.close(g, a, e, name)
    ref.close_norm(got[0], want[0], 2, "dx")
    ref.close_norm(got[1], want[1], 2, "dw")
    assert bool((dx[want[0][:, 0].isnan()] == 7.0).all())
