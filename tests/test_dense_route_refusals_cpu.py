"""Refusals of the grouped router and the 4-bit products: wrong shapes, types,
strides, options and devices are errors before anything is launched (CPU only)."""
import ctypes as C

import numpy as np
import pytest
import torch

from route_reference import choose


@pytest.fixture(scope="module")
def m():
    from expert_offload_fp4_b200 import build
    build.build()
    import expert_offload_fp4_b200 as mod
    return mod


GOOD = dict(k=2, score=1, n_group=4, topk_group=2, group_top=2, renormalize=1, scale=1.0)


def choice(m, **kw):
    d = dict(GOOD, **kw)
    return m._lib.RouteChoice(d["k"], d["score"], d["n_group"], d["topk_group"], d["group_top"], d["renormalize"],
                              d["scale"])


def test_route_calls_refuse_bad_options(m):
    L, E = m._lib.load(), m._lib
    buf = (C.c_uint8 * 256)()
    p = C.c_void_p((C.addressof(buf) + 15) // 16 * 16)
    ws = L.moe_route_grouped_workspace_bytes(4, 16)
    assert ws > 0 and L.moe_route_grouped_workspace_bytes(0, 16) == 0 and L.moe_route_grouped_workspace_bytes(1, 0) == 0

    def both(expect, T=4, En=16, **kw):
        c = C.byref(choice(m, **kw))
        assert L.moe_route_grouped(p, p, None, T, 256, En, c, p, p, p, 1 << 30, None) == E.MOE_EINVAL
        assert expect in L.moe_last_error(), L.moe_last_error()
        assert L.moe_route_select(p, E.MOE_F32, En, None, T, En, c, p, p, None) == E.MOE_EINVAL
        assert expect in L.moe_last_error()

    both(b"T > 0", T=0)
    both(b"T > 0", T=-1)
    both(b"E <= 1024", En=2048)
    both(b"k <= 32", k=0)
    both(b"k <= 32", k=33)
    both(b"score", score=2)
    both(b"n_group", n_group=0)
    both(b"n_group", n_group=5)
    both(b"n_group", n_group=64, En=128)
    both(b"topk_group", topk_group=0)
    both(b"topk_group", topk_group=5)
    both(b"kept groups", k=9)
    both(b"group_top", group_top=0)
    both(b"group_top", group_top=3)
    both(b"renormalize", renormalize=2)
    for s in (0.0, -1.0, float("inf"), float("nan")):
        both(b"scale", scale=s)
    g = C.byref(choice(m))
    odd = C.c_void_p(p.value | 2)
    for args, expect in [
            ((None, p, None, 4, 256, 16, g, p, p, p, ws), b"null"), ((p, None, None, 4, 256, 16, g, p, p, p, ws), b"null"),
            ((p, p, None, 4, 256, 16, g, None, p, p, ws), b"null"), ((p, p, None, 4, 256, 16, g, p, None, p, ws), b"null"),
            ((p, p, None, 4, 256, 16, None, p, p, p, ws), b"null"), ((p, p, None, 4, 257, 16, g, p, p, p, ws), b"H must"),
            ((p, p, None, 4, 0, 16, g, p, p, p, ws), b"H must"), ((odd, p, None, 4, 256, 16, g, p, p, p, ws), b"aligned"),
            ((p, odd, None, 4, 256, 16, g, p, p, p, ws), b"aligned"),
            ((p, p, None, 4, 256, 16, g, p, p, p, ws - 1), b"workspace"),
            ((p, p, None, 4, 256, 16, g, p, p, None, ws), b"workspace"),
            ((p, p, None, 4, 256, 16, g, p, p, odd, ws), b"aligned")]:
        assert L.moe_route_grouped(*args, None) == E.MOE_EINVAL and expect in L.moe_last_error(), (args, L.moe_last_error())
    for args, expect in [
            ((None, E.MOE_F32, 16, None, 4, 16, g, p, p), b"null"), ((p, 2, 16, None, 4, 16, g, p, p), b"bf16 or fp32"),
            ((p, E.MOE_F32, 15, None, 4, 16, g, p, p), b"stride"), ((odd, E.MOE_F32, 16, None, 4, 16, g, p, p), b"aligned")]:
        assert L.moe_route_select(*args, None) == E.MOE_EINVAL and expect in L.moe_last_error(), (args, L.moe_last_error())


def test_fp4_calls_refuse_bad_arguments(m):
    L, E = m._lib.load(), m._lib
    buf = (C.c_uint8 * 256)()
    p = (C.addressof(buf) + 15) // 16 * 16

    def weight(**kw):
        d = dict(codes=p, scales=p, tensor_scale=1.0, N=64, K=64, fmt=E.MOE_NVFP4)
        d.update(kw)
        return E.Fp4WeightDesc(d["codes"], d["scales"], d["tensor_scale"], d["N"], d["K"], d["fmt"])

    def linear(expect, w=None, x=p, xt=0, ldx=64, T=2, add=None, lda=64, y=p, yt=0, ldy=64, st=p):
        w = weight() if w is None else w
        assert L.moe_fp4_linear(C.byref(w), x, xt, ldx, T, add, lda, y, yt, ldy, st, None) == E.MOE_EINVAL
        assert expect in L.moe_last_error(), L.moe_last_error()

    linear(b"null", weight(codes=None))
    linear(b"null", weight(scales=None))
    linear(b"format", weight(fmt=7))
    linear(b"multiple of 32", weight(K=48))
    linear(b"multiple of 32", weight(K=0))
    linear(b"N > 0", weight(N=0))
    linear(b"aligned", weight(codes=p + 4))
    linear(b"T must", T=0)
    linear(b"T must", T=17)
    big = (C.c_uint8 * 4096)()
    q = (C.addressof(big) + 15) // 16 * 16
    linear(b"y overlaps x", x=q, y=q + 64)
    linear(b"y overlaps x", x=q, y=q + 2 * 64 * 2 - 2)
    linear(b"y overlaps add", x=q, y=q + 512, add=q + 512 + 2)
    linear(b"y overlaps add", x=q, y=q + 512, add=q + 512, lda=66)
    linear(b"K too large", weight(K=131072 + 32), T=1, ldx=1 << 20)
    linear(b"K too large", weight(K=16416), T=15, ldx=1 << 20)
    linear(b"N too large", weight(N=(1 << 30) + 1))
    linear(b"null x", x=None)
    linear(b"null y", y=None)
    linear(b"null status", st=None)
    linear(b"type", xt=2)
    linear(b"type", yt=-1)
    linear(b"stride", ldx=63)
    linear(b"stride", ldy=63)
    linear(b"stride", add=p, lda=1)
    linear(b"aligned", x=p + 2)
    linear(b"aligned", ldx=66)
    linear(b"aligned", y=p + 1)
    linear(b"aligned", add=p + 2, yt=1)

    def swiglu(expect, g=None, u=None, x=p, ldx=64, T=2, h=p, ldh=64, st=p):
        g, u = g or weight(), u or weight()
        assert L.moe_fp4_swiglu(C.byref(g), C.byref(u), x, 0, ldx, T, h, ldh, st, None) == E.MOE_EINVAL
        assert expect in L.moe_last_error(), L.moe_last_error()

    swiglu(b"h overlaps x", x=q, h=q + 128)
    swiglu(b"one shape", u=weight(N=65))
    swiglu(b"one shape", u=weight(K=96))
    swiglu(b"one shape", u=weight(fmt=E.MOE_MXFP4))
    swiglu(b"T must", T=17)
    swiglu(b"null h", h=None)
    swiglu(b"aligned", h=p + 2)
    swiglu(b"aligned", x=p + 8)
    swiglu(b"stride", ldh=10)
    swiglu(b"null status", st=None)


def test_python_checks_need_no_gpu(m):
    bf = torch.zeros((3, 64), dtype=torch.bfloat16)
    idx, w = torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2))
    ws = torch.zeros(4096, dtype=torch.uint8)
    wr = torch.zeros((16, 64), dtype=torch.bfloat16)

    def refused(match, fn, *a, **kw):
        with pytest.raises(ValueError, match=match):
            fn(*a, **kw)

    refused("contiguous bfloat16", m.route_grouped, bf.float(), wr, idx, w, ws)
    refused("contiguous bfloat16", m.route_grouped, bf, wr[:, ::2], idx, w, ws)
    refused("contiguous bfloat16", m.route_grouped, bf[:, :32], wr[:, :32], idx, w, ws)
    refused("idx", m.route_grouped, bf, wr, idx.long(), w, ws)
    refused("idx", m.route_grouped, bf, wr, idx[:2], w, ws)
    refused("w must", m.route_grouped, bf, wr, idx, w[:, :1], ws)
    refused("bias", m.route_grouped, bf, wr, idx, w, ws, bias=torch.zeros(15))
    refused("bias", m.route_grouped, bf, wr, idx, w, ws, bias=torch.zeros(16, dtype=torch.bfloat16))
    refused("CUDA device", m.route_grouped, bf, wr, idx, w, ws)
    refused("score", m.route_select, torch.zeros((3, 16)), idx, w, score="tanh")
    refused("logits", m.route_select, torch.zeros((3, 16), dtype=torch.float16), idx, w)
    refused("contiguous rows", m.route_select, torch.zeros((3, 32))[:, ::2], idx, w)
    refused("CUDA device", m.route_select, torch.zeros((3, 16)), idx, w)

    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    refused("fmt", m.FP4Weight, u8(4, 16), u8(4, 1), "int4")
    refused("uint8", m.FP4Weight, u8(4, 16).int(), u8(4, 1), "mxfp4")
    refused("multiple of 32", m.FP4Weight, u8(4, 8), u8(4, 1), "mxfp4")
    refused("scales", m.FP4Weight, u8(4, 16), u8(4, 1), "nvfp4")
    refused("CUDA device", m.FP4Weight, u8(4, 16), u8(4, 2), "nvfp4")


def test_reference_choice_on_a_hand_worked_token():
    """Groups {0,1}, {2,3}, {4,5}: scores .5 each way, bias moves the choice, not the weight."""
    l = np.log(np.array([[0.6, 0.1, 0.5, 0.45, 0.3, 0.2]]) / (1 - np.array([[0.6, 0.1, 0.5, 0.45, 0.3, 0.2]])))
    i, w = choose(l, 2, n_group=3, topk_group=1, group_top=2)
    assert i.tolist() == [[2, 3]]                       # .95 beats .7 and .5
    np.testing.assert_allclose(w, [[0.5 / 0.95, 0.45 / 0.95]], rtol=1e-12)
    i, w = choose(l, 2, n_group=3, topk_group=1, group_top=1, renormalize=False, scale=2.0)
    assert i.tolist() == [[0, 1]]
    np.testing.assert_allclose(w, [[1.2, 0.2]], rtol=1e-12)
    i, w = choose(l, 2, bias=[0, 0, 0, 0, 1.0, 0], renormalize=False)
    assert i.tolist() == [[4, 0]]
    np.testing.assert_allclose(w, [[0.3, 0.6]], rtol=1e-12)


def test_shared_expert_and_routed_layer_refusals(m):
    from types import SimpleNamespace as N
    g = N(N=64, K=128, fmt="nvfp4")
    assert m.SharedExpert(g, g, N(N=128, K=64, fmt="mxfp4")).I == 64
    for bad in (N(N=64, K=96, fmt="nvfp4"), N(N=64, K=128, fmt="mxfp4")):
        with pytest.raises(ValueError, match="one shape and format"):
            m.SharedExpert(g, bad, N(N=128, K=64, fmt="nvfp4"))
    with pytest.raises(ValueError, match="down"):
        m.SharedExpert(g, g, N(N=64, K=128, fmt="nvfp4"))
    L, E = m._lib.load(), m._lib
    buf = (C.c_uint8 * 64)()
    p, s1 = C.cast(buf, C.c_void_p), C.c_void_p(0x1000)
    call = lambda pool, stream, cs: L.moe_decode_layer_routed(pool, 0, p, 1, p, p, p, p, p, p, None, None, None, 1,
                                                              stream, cs)
    assert call(None, None, s1) == E.MOE_EINVAL and b"null pool" in L.moe_last_error()
    assert call(p, s1, s1) == E.MOE_EINVAL and b"copy_stream" in L.moe_last_error()
    assert call(p, s1, None) == E.MOE_EINVAL and b"copy_stream" in L.moe_last_error()


@pytest.mark.parametrize("E", [1, 64, 160, 300, 1024])
def test_grouped_workspace_serves_fewer_tokens(E):
    from expert_offload_fp4_b200 import _lib
    size = _lib.load().moe_route_grouped_workspace_bytes
    sizes = [size(T, E) for T in [*range(1, 300), *range(300, 25000, 97)]]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
