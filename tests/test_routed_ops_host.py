"""Refusals of the routed operators, on the host: nothing here reaches a device."""
import ctypes
import types

import pytest
import torch

from block_scaled_moe_softmax_b200 import moe_mx
from block_scaled_moe_softmax_b200 import routed_ops as ops

BAD = moe_mx.MOE_MX_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    return moe_mx.load_library()


def _err():
    return moe_mx.moe_mx_last_error()


@pytest.mark.parametrize("T,H,k,rows,dtype,word", [
    (-1, 64, 2, 128, 0, "num_tokens"), (4, 0, 2, 128, 0, "hidden"), (4, (1 << 20) + 1, 2, 128, 0, "hidden"),
    (4, 64, 0, 128, 0, "top_k"), (4, 64, 33, 128, 0, "top_k"), (4, 64, 2, -1, 0, "rows"),
    (4, 64, 2, 1 << 31, 0, "rows"), (4, 64, 2, 128, 3, "dtype"), (4, 64, 2, 128, 0, "device pointer")])
def test_permutes_refuse(lib, T, H, k, rows, dtype, word):
    assert lib.moe_mx_dispatch(None, T, H, k, None, rows, dtype, None, None) == BAD and word in _err()
    assert lib.moe_mx_combine(None, rows, T, H, k, None, None, dtype, 0, None, None) == BAD and word in _err()
    keep = ctypes.create_string_buffer(64)
    assert lib.moe_mx_combine_backward(None, None, rows, T, H, k, None, None, None, 0, dtype, 0,
                                       ctypes.addressof(keep), None, None, None) == BAD and word in _err()


def test_combine_backward_refuses(lib):
    f = lib.moe_mx_combine_backward
    keep = ctypes.create_string_buffer(64)
    p = ctypes.addressof(keep)
    assert f(None, None, 128, 4, 64, 2, None, None, None, 0, 0, 0, None, None, None, None) == BAD and "none of" in _err()
    assert f(None, None, 128, 4, 64, 2, None, None, None, 0, 0, 0, None, None, p, None) == BAD and "num_experts" in _err()
    assert f(None, None, 128, 4, 64, 2, None, None, None, 1025, 0, 0, None, None, p, None) == BAD
    assert f(None, None, 128, 4, 64, 2, None, None, None, 0, 0, 9, p, None, None, None) == BAD and "dout_dtype" in _err()
    assert f(p, None, 128, 4, 64, 2, None, None, None, 0, 0, 0, p, None, None, None) == BAD and "device pointer" in _err()


@pytest.mark.parametrize("E,rows,N,K,dtype,act,io,word", [
    (-1, 8, 16, 64, 0, 0, 0, "num_experts"), (1025, 8, 16, 64, 0, 0, 0, "num_experts"), (0, -1, 16, 64, 0, 0, 0, "rows"),
    (0, 1 << 31, 16, 64, 0, 0, 0, "rows"), (0, 8, 0, 64, 0, 0, 0, "N="), (0, 8, 16, 0, 0, 0, 0, "K="),
    (0, 8, (1 << 20) + 1, 64, 0, 0, 0, "N="), (0, 8, 16, 64, 1, 0, 1, "dtype"), (0, 8, 16, 64, 0, 0, 2, "dtype"),
    (0, 8, 16, 64, 0, 4, 0, "activation"), (0, 8, 16, 64, 0, -1, 0, "activation"), (0, 8, 15, 64, 0, 3, 0, "even")])
def test_linear_refuses(lib, E, rows, N, K, dtype, act, io, word):
    assert lib.moe_mx_linear(*[None] * 6, E, rows, N, K, dtype, act, io, None, None, None, 0, None) == BAD and word in _err()
    assert lib.moe_mx_linear_backward(*[None] * 6, E, rows, N, K, dtype, act, io, None, None, None, None, 0,
                                      None) == BAD and word in _err()
    assert lib.moe_mx_linear_workspace(E, rows, N, K, dtype, act, io) == BAD and word in _err()
    assert lib.moe_mx_linear_backward_workspace(E, rows, N, K, dtype, act, io) == BAD and word in _err()


def test_linear_refuses_pointers(lib):
    keep = ctypes.create_string_buffer(4096)
    p = ctypes.addressof(keep)  # host memory
    assert lib.moe_mx_linear(p, p, None, None, None, None, 0, 8, 16, 64, 0, 0, 0, p, None, None, 0, None) == BAD
    assert "device pointer" in _err()
    assert lib.moe_mx_linear_backward(p, p, p, None, None, None, 0, 8, 16, 64, 0, 0, 0, None, None, None, None, 0,
                                      None) == BAD and "none of" in _err()
    assert lib.moe_mx_linear_backward(p, p, p, None, None, None, 0, 8, 16, 64, 0, 1, 0, p, None, None, None, 0,
                                      None) == BAD and "preact" in _err()
    # nothing to do is no error
    assert lib.moe_mx_linear(None, None, None, None, None, None, 0, 0, 16, 64, 0, 0, 0, None, None, None, 0, None) == 0
    assert lib.moe_mx_dispatch(None, 0, 64, 2, None, 128, 0, None, None) == 0


def test_workspace_covers_the_largest_calls(lib):
    for E, rows, N, K in ((0, 1, 1, 1), (0, 8192, 384, 7168), (64, 24576, 4096, 7168), (1024, (1 << 31) - 1025, 128, 64)):
        assert lib.moe_mx_linear_workspace(E, rows, N, K, 0, 0, 0) >= 0
        assert lib.moe_mx_linear_backward_workspace(E, rows, N, K, 0, 1, 0) >= 2 * rows * N


def test_status_refuses_a_device_that_is_not_there(lib):
    assert lib.moe_mx_linear_status(-1, None) in (BAD, moe_mx.MOE_MX_ERR_CUDA)
    assert lib.moe_mx_linear_status(1 << 20, None) in (BAD, moe_mx.MOE_MX_ERR_CUDA)


def test_workspace_of_no_rows_is_no_error(lib):
    for E in (0, 4):
        assert lib.moe_mx_linear_workspace(E, 0, 32, 64, 0, 0, 0) >= 0
        assert lib.moe_mx_linear_backward_workspace(E, 0, 32, 64, 0, 0, 0) >= 0


def _cpu_routing(T=4, k=2, E=4):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    return ops.Routing(i(T, k), torch.ones(T, k), i(E), i(E + 1), i(T * k), ops.max_grouped_rows(T * k, E))


def test_wrappers_refuse_types_shapes_and_devices():
    r = _cpu_routing()
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        ops.dispatch(x, r)
    with pytest.raises(ValueError, match="CUDA device"):
        ops.linear(x, w)
    with pytest.raises(ValueError, match="CUDA device"):
        ops.route_group(torch.zeros(4, 8), 2)
    with pytest.raises(TypeError, match="float32"):
        ops.route_group(x, 2)
    with pytest.raises(ValueError, match="shape"):
        ops.dispatch(x[:3], r)
    with pytest.raises(ValueError, match="contiguous"):
        ops.dispatch(torch.zeros(64, 4).t(), r)
    with pytest.raises(ValueError, match="shape"):
        ops.combine(x, r)
    with pytest.raises(ValueError, match="shape"):
        ops.combine_backward(x, x, r)
    with pytest.raises(TypeError):
        ops.linear(x, w.float())
    with pytest.raises(TypeError, match="supported"):
        ops.linear(x.float(), w.float())
    with pytest.raises(ValueError, match="activation"):
        ops.linear(x, w, activation="relu6")
    with pytest.raises(ValueError, match="need"):
        ops.linear(x, torch.zeros(16, 65, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="need"):
        ops.linear(x, w, routing=r)
    with pytest.raises(ValueError, match="rows"):
        ops.linear(x, torch.zeros(4, 16, 64, dtype=torch.bfloat16), routing=r)
    with pytest.raises(ValueError, match="even"):
        ops.linear(x, w[:15], activation="swiglu")


def test_grouped_rows_bound_is_the_librarys():
    for pairs, experts in ((0, 4), (1, 4), (8, 4), (500, 384)):
        hit = min(pairs, experts)
        assert ops.max_grouped_rows(pairs, experts) == -(-(pairs + hit * 127) // 128) * 128


def test_watchdog_and_check_refuse(lib):
    for us in (0, -1, 10000001):
        assert lib.moe_mx_debug_linear_watchdog(0, us, None) == BAD and "timeout_us" in _err()
    assert lib.moe_mx_debug_linear_watchdog(-1, 1000, None) in (BAD, moe_mx.MOE_MX_ERR_CUDA)
    with pytest.raises(ValueError, match="CUDA device"):
        ops.check("cpu")


def test_products_of_2_to_the_31_values_are_not_split(lib):
    """The sum of a split product's planes counts values in 32 bits: none of that size has planes."""
    for M, N in ((1 << 15, 1 << 16), ((1 << 15) + 1, 1 << 16), (74 * 256 + 1, 116000), ((1 << 20) + 3, 2049)):
        for K in (1 << 13, 1 << 17, 1 << 20):
            assert M * N >= 1 << 31
            assert lib.moe_mx_linear_workspace(0, M, N, K, 0, 0, 0) < 4 * M * N
    assert lib.moe_mx_linear_workspace(0, 2048, 2560, 14336, 0, 0, 0) >= 2 * 4 * 2048 * 2560  # split, in 240 tiles


def test_wrappers_refuse_an_empty_routing_and_other_devices_streams():
    r = _cpu_routing()
    x = torch.zeros(r.rows, 64, dtype=torch.bfloat16)
    none = r._replace(counts=torch.zeros(0, dtype=torch.int32), pad_offsets=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="no experts"):  # not a dense product over the padding too
        ops.linear(x, torch.zeros(16, 64, dtype=torch.bfloat16), routing=none)
    with pytest.raises(TypeError, match="counts"):
        ops.linear(x, torch.zeros(4, 16, 64, dtype=torch.bfloat16), routing=r._replace(counts=[1, 2, 3, 4]))
    other = types.SimpleNamespace(cuda_stream=1, device_index=1)
    with pytest.raises(ValueError, match="stream"):
        ops._on(x, 0, other)
    assert ops._on(x, 1, other) == 1
