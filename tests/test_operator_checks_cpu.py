"""Checks of the routers', products' and layer's arguments that need no GPU: sizes at the edge of an
int, a router's choice as a layer takes it, options that would be ignored."""
import ctypes as C
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    from expert_offload_fp4_b200 import build
    build.build()
    import expert_offload_fp4_b200 as mod
    return mod


def test_sizes_at_the_edge_of_an_int_are_refused(m):
    L, E = m._lib.load(), m._lib
    buf = (C.c_uint8 * 4096)()
    p = (C.addressof(buf) + 255) // 256 * 256
    c = C.byref(E.RouteChoice(1, 0, 1, 1, 1, 1, 1.0))

    def refused(what, rc):
        assert rc == E.MOE_EINVAL and what in L.moe_last_error(), (rc, L.moe_last_error())

    for big in (2 ** 31 - 1, 2 ** 31 - 8, 2 ** 30 + 1):
        refused(b"T must be at most", L.moe_route_select(p, E.MOE_F32, 1, None, big, 1, c, p, p, None))
        refused(b"T must be at most", L.moe_route_grouped(p, p, None, big, 8, 1, c, p, p, p, 1 << 62, None))
        assert L.moe_route_grouped_workspace_bytes(big, 16) == 0
    for big in (2 ** 31 - 8, 2 ** 30 + 8):
        refused(b"H must", L.moe_route_grouped(p, p, None, 1, big, 1, c, p, p, p, 1 << 62, None))
    assert L.moe_route_grouped_workspace_bytes(2 ** 30, 16) > 0
    st = (C.c_int * 1)()
    for K in (2 ** 31 - 32, 2 ** 31 - 256):
        w = E.Fp4WeightDesc(p, p, 1.0, 64, K, E.MOE_NVFP4)
        refused(b"K too large", L.moe_fp4_linear(C.byref(w), p, E.MOE_BF16, 1 << 40, 1, None, 0, p + 2048, E.MOE_BF16, 64, st, None))
        refused(b"K too large", L.moe_fp4_swiglu(C.byref(w), C.byref(w), p, E.MOE_BF16, 1 << 40, 1, p + 2048, 64, st, None))
