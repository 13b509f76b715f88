"""The entry points of 4-bit weights and of layers of experts on the CPU: what
they refuse before anything touches a device, in the library and in the
binding."""
import ctypes as C
import os

import pytest


@pytest.fixture(scope="module")
def dq():
    import dynamic_quantized_gemm_amd as dq
    from dynamic_quantized_gemm_amd import build

    if not os.path.exists(dq.LIB_PATH):
        build.build()
    dq.load()
    return dq


def test_w4_init_refuses(dq):
    lib = dq.load()

    def init(e=1, n=64, k=256, g=64, x=dq.DQ_BF16, s=dq.DQ_F32, y=dq.DQ_BF16, rows=8):
        h = C.c_void_p()
        rc = lib.dq_w4_init(C.byref(h), e, n, k, g, x, s, y, 0, rows)
        assert h.value is None and dq.dqip_last_error()
        return rc

    for name in ("e", "n", "k", "rows"):
        assert init(**{name: 0}) == dq.DQ_ERR_ARG
        assert init(**{name: -3}) == dq.DQ_ERR_ARG
    for g in (0, -128, 1, 16, 48, 96, 192 - 1, 200):
        assert init(g=g) == dq.DQ_ERR_ARG
    for name in ("x", "s", "y"):
        for t in (dq.DQ_I8, dq.DQ_U8, 9, -1):
            assert init(**{name: t}) == dq.DQ_ERR_TYPE
    assert init(e=dq.DQ_W4_EXPERTS_MAX + 1) == dq.DQ_ERR_RANGE
    assert init(n=dq.DQ_W4_N_MAX + 1) == dq.DQ_ERR_RANGE
    assert init(k=dq.DQ_W4_K_MAX + 1) == dq.DQ_ERR_RANGE
    assert init(rows=dq.DQ_W4_ROWS_MAX + 1) == dq.DQ_ERR_RANGE
    assert init(n=2 ** 62) == dq.DQ_ERR_RANGE
    assert lib.dq_w4_init(None, 1, 64, 256, 64, 1, 0, 1, 0, 8) == dq.DQ_ERR_ARG


def test_moe_init_refuses(dq):
    lib = dq.load()

    def init(t=16, e=8, k=2, type=dq.DQ_F32, scoring=0, scale=1.0):
        h = C.c_void_p()
        rc = lib.dq_moe_init(C.byref(h), t, e, k, type, scoring, 1, scale)
        assert h.value is None and dq.dqip_last_error()
        return rc

    for name in ("t", "e", "k"):
        assert init(**{name: 0}) == dq.DQ_ERR_ARG
        assert init(**{name: -1}) == dq.DQ_ERR_ARG
    assert init(k=9) == dq.DQ_ERR_ARG
    assert init(type=dq.DQ_I8) == dq.DQ_ERR_TYPE
    assert init(scoring=2) == dq.DQ_ERR_ARG
    for s in (float("inf"), float("nan")):
        assert init(scale=s) == dq.DQ_ERR_ARG
    assert init(e=dq.DQ_MOE_EXPERTS_MAX + 1) == dq.DQ_ERR_RANGE
    assert init(e=100, k=dq.DQ_MOE_TOP_K_MAX + 1) == dq.DQ_ERR_RANGE
    assert init(t=dq.DQ_MOE_TOKENS_MAX + 1) == dq.DQ_ERR_RANGE
    assert lib.dq_moe_init(None, 16, 8, 2, 0, 0, 1, 1.0) == dq.DQ_ERR_ARG


def test_calls_without_a_context(dq):
    lib = dq.load()
    assert lib.dq_w4_set_w(None, 1, 1, None, None, None) == dq.DQ_ERR_STATE
    assert lib.dq_w4_forward(None, 1, 1, 1, 1, None) == dq.DQ_ERR_STATE
    assert lib.dq_w4_forward_grouped(None, 1, 1, 1, 1, 1, None, 1, None) == dq.DQ_ERR_STATE
    assert lib.dq_moe_route(None, 1, 1, 1, 1, 1, 1, 1, 1, None) == dq.DQ_ERR_STATE
    assert lib.dq_moe_combine(None, 1, 1, 1, 1, 0, 1, 1, None, 0, 1, None) == dq.DQ_ERR_STATE
    assert lib.dq_w4_info(None) is None and lib.dq_moe_info(None) is None
    lib.dq_w4_release(None)
    lib.dq_moe_release(None)
    import torch

    t = torch.zeros((1, 1))
    for call in (lambda: dq.dq_w4_set_w(0, t, t), lambda: dq.dq_w4_forward(0, t, t),
                 lambda: dq.dq_w4_forward_grouped(0, t, t, t), lambda: dq.dq_moe_route(0, t, t, t, t, t, t),
                 lambda: dq.dq_moe_combine(0, t, t, t, t)):
        with pytest.raises(dq.DQError) as e:
            call()
        assert e.value.status == dq.DQ_ERR_STATE


class _Fake:
    """A context's sizes in the binding, without a device."""

    def __init__(self, table, value):
        self.table, self.value = table, value

    def __enter__(self):
        self.table[1] = self.value
        return 1

    def __exit__(self, *a):
        self.table.pop(1, None)


def test_binding_refuses_tensors_on_the_host_and_shapes(dq):
    import torch
    from dynamic_quantized_gemm_amd import _binding as B

    def refused(status, call):
        with pytest.raises(dq.DQError) as e:
            call()
        assert e.value.status == status, e.value

    f = torch.zeros
    with _Fake(B._W4_DIMS, (2, 8, 16, 8, 1, dq.DQ_F32, dq.DQ_F32, dq.DQ_F32)) as h:
        refused(dq.DQ_ERR_ARG, lambda: dq.dq_w4_set_w(h, f((2, 8, 8), dtype=torch.uint8), f((2, 8, 1))))
        refused(dq.DQ_ERR_TYPE, lambda: dq.dq_w4_set_w(h, f((2, 8, 8)), f((2, 8, 1))))
        refused(dq.DQ_ERR_ARG, lambda: dq.dq_w4_forward(h, f((3, 16)), f((3, 8))))
        refused(dq.DQ_ERR_ARG, lambda: dq.dq_w4_forward(h, f((3, 17)), f((3, 8))))
        refused(dq.DQ_ERR_ARG, lambda: dq.dq_w4_forward(h, f((3, 2, 16)), f((3, 8))))
        refused(dq.DQ_ERR_ARG, lambda: dq.dq_w4_forward_grouped(h, f((3, 16)), f((3,), dtype=torch.int32), f((3, 8))))
    with _Fake(B._MOE_DIMS, (8, 2, dq.DQ_F32)) as h:
        i = torch.zeros((4, 2), dtype=torch.int32)
        refused(dq.DQ_ERR_ARG, lambda: dq.dq_moe_route(h, f((4, 8)), i, f((4, 2)), i, i, i))
        refused(dq.DQ_ERR_ARG, lambda: dq.dq_moe_route(h, f((4, 9)), i, f((4, 2)), i, i, i))
        refused(dq.DQ_ERR_ARG, lambda: dq.dq_moe_combine(h, f((8, 5)), f((4, 2)), i, f((4, 5))))
        refused(dq.DQ_ERR_ARG, lambda: dq.dq_moe_combine(h, f((8, 6)), f((4, 2)), i, f((4, 5))))
        refused(dq.DQ_ERR_TYPE, lambda: dq.dq_moe_combine(h, f((8, 5), dtype=torch.float64), f((4, 2)), i, f((4, 5))))
