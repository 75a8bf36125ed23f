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


def test_a_routed_layer_checks_the_choice_it_is_given(m):
    """idx and w are inputs here: an int64 idx, as torch.topk gives, or another k is not read as int32 [T, k]."""
    called = []
    pool = SimpleNamespace(k=2, E=8, H=256, handle=None,
                           lib=SimpleNamespace(moe_decode_layer_routed=lambda *a: called.append(a) or 0))
    x = torch.zeros((3, 256), dtype=torch.bfloat16)
    idx, w = torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2))
    cs = SimpleNamespace(cuda_stream=1)
    for what, bad in [("idx", dict(idx=idx.long())), ("idx", dict(idx=idx[:2])), ("idx", dict(idx=torch.zeros((3, 4), dtype=torch.int32))),
                      ("idx", dict(idx=torch.zeros((3, 4), dtype=torch.int32)[:, ::2])), ("w must", dict(w=w.double())),
                      ("w must", dict(w=w.bfloat16())), ("w must", dict(w=w[:, :1])), ("w must", dict(w=torch.zeros((2, 3)).t())),
                      ("CUDA device", {})]:
        a = dict(idx=idx, w=w) | bad
        with pytest.raises(ValueError, match=what):
            m.decode_layer_routed(pool, 0, x, a["idx"], a["w"], None, None, None, None, copy_stream=cs, stream=cs)
    assert not called


def test_a_layer_with_a_router_of_its_own_refuses_renormalize(m):
    """renormalize belongs to moe_route's gate; a GroupedRouting has its own."""
    pool = SimpleNamespace(k=2, E=8, H=256, max_tokens=4)
    for r in (0, 1):
        with pytest.raises(ValueError, match="renormalize"):
            m.DecodeLayer(pool, 2, device="cpu", router=m.GroupedRouting(), renormalize=r)
