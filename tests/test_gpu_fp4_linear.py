"""The 4-bit products (moe_fp4_linear, moe_fp4_swiglu) against the dequantised
product in 64 bits.

Error bound of one output, with S = sum |x||w|: every product is exact; the sum of K
of them is formed in fp32 from partial sums of at most 64, so at most K/64 + 40
roundings of at most 2^-23 S each (2^-23, not 2^-24: the tensor core may truncate);
x enters to 2^-22 of its largest element in the row; the result is rounded once to
y's type.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    from expert_offload_fp4_b200 import build
    build.build()
    import expert_offload_fp4_b200 as mod
    return mod


def weight(m, N, K, fmt, seed, ts=0.75):
    """Random codes and scales (on the device) and the dequantised matrix in float64."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    if fmt == "mxfp4":
        scales = rng.integers(110, 122, (N, K // 32), dtype=np.uint8)
    else:
        scales = rng.integers(0x00, 0x50, (N, K // 16), dtype=np.uint8)
    W = oracle.dequant(fmt, codes, scales, 1.0).astype(np.float64) * (float(np.float32(ts)) if fmt == "nvfp4" else 1)
    return m.FP4Weight(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), fmt, ts), W


def acts(T, K, dtype, seed, spread=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, K), generator=g)
    if spread:
        x = x * torch.exp2(torch.randint(-12, 4, (T, K), generator=g).float())
    return x.to(dtype)


def bound(x, W, K, dtype, ref):
    xa, Wa = x.double().abs().numpy(), np.abs(W)
    S = xa @ Wa.T
    b = (K / 64 + 40) * 2.0 ** -23 * S + 2.0 ** -22 * xa.max(1, initial=0)[:, None] * Wa.sum(1)[None, :]
    return b + (np.abs(ref) + b) * (torch.finfo(dtype).eps / 2) + 1e-40


def run_linear(m, x, Wq, ydtype, add=None, status=None, **kw):
    y = torch.full((x.shape[0], Wq.N), float("nan"), dtype=ydtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.fp4_linear(x.cuda(), Wq, y, st, add=None if add is None else add.cuda(), **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    return y.cpu()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,N,K", [
    (1, 1, 32), (1, 127, 64), (2, 128, 96), (3, 129, 2080), (4, 4096, 512), (5, 300, 256), (7, 1000, 992),
    (8, 2048, 768), (9, 640, 4096), (11, 257, 1056), (15, 513, 8192), (16, 2051, 2048), (16, 130, 288),
    (1, 20011, 1024), (1, 4096, 4096), (13, 20000, 320), (1, 257, 16416), (16, 70, 16384)])
@pytest.mark.parametrize("xd,yd", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32)])
def test_linear_matches_dequantised_product(m, fmt, T, N, K, xd, yd):
    Wq, W = weight(m, N, K, fmt, N + K)
    x = acts(T, K, xd, T + K)
    ref = x.double().numpy() @ W.T
    got = run_linear(m, x, Wq, yd).double().numpy()
    assert np.all(np.abs(got - ref) <= bound(x, W, K, yd, ref))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("xd", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 6])
def test_linear_on_activations_of_wide_range(m, fmt, xd, T):
    Wq, W = weight(m, 384, 1024, fmt, 5)
    x = acts(T, 1024, xd, 6, spread=True)
    x[0, 7] = 3000.0
    ref = x.double().numpy() @ W.T
    got = run_linear(m, x, Wq, torch.float32).double().numpy()
    assert np.all(np.abs(got - ref) <= bound(x, W, 1024, torch.float32, ref))


@pytest.mark.parametrize("scale", [2.0 ** 100, 2.0 ** -100, 2.0 ** -130])
def test_linear_on_very_large_and_very_small_activations(m, scale):
    Wq, W = weight(m, 200, 512, "nvfp4", 7)
    x = (acts(3, 512, torch.float32, 8).double() * scale).float()
    ref = x.double().numpy() @ W.T
    got = run_linear(m, x, Wq, torch.float32).double().numpy()
    # below fp32's normal range a result is rounded to a multiple of 2^-149
    assert np.all(np.abs(got - ref) <= bound(x, W, 512, torch.float32, ref) + 2.0 ** -140)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_zero_rows_of_x_and_zero_weights_give_zero(m, fmt):
    Wq, W = weight(m, 200, 288, fmt, 9)
    x = acts(4, 288, torch.bfloat16, 10)
    x[2] = 0
    got = run_linear(m, x, Wq, torch.float32)
    assert torch.all(got[2] == 0)
    zero = m.FP4Weight(torch.zeros_like(Wq.codes), Wq.scales, fmt, 0.75)
    assert torch.all(run_linear(m, x, zero, torch.float32) == 0)


@pytest.mark.parametrize("T", [1, 5])
def test_nonfinite_activations_stay_in_their_row(m, T):
    """A NaN or infinite element makes its own row's outputs non-finite, no other's."""
    Wq, _ = weight(m, 300, 512, "nvfp4", 11)
    x = acts(T + 2, 512, torch.bfloat16, 12)
    clean = run_linear(m, x, Wq, torch.float32)
    x[1, 77] = float("nan")
    x[2, 5] = float("inf")
    got = run_linear(m, x, Wq, torch.float32)
    keep = [t for t in range(T + 2) if t not in (1, 2)]
    assert torch.equal(got[keep], clean[keep])
    assert not torch.isfinite(got[1]).any()
    assert not torch.isfinite(got[2]).any()


@pytest.mark.parametrize("yd", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("in_place", [False, True])
def test_add_strides_and_untouched_columns(m, yd, in_place):
    T, N, K = 6, 515, 320
    Wq, W = weight(m, N, K, "mxfp4", 13)
    xbuf = acts(T, K + 64, torch.bfloat16, 14).cuda()
    ybuf = torch.full((T, N + 3), 7.0, dtype=yd, device="cuda")
    abuf = acts(T, N + 10, yd, 15).cuda()
    x, y, add = xbuf[:, 8:8 + K], ybuf[:, 1:1 + N], abuf[:, 3:3 + N]
    if in_place:
        y.copy_(add)
        add_arg = y
    else:
        add_arg = add
    ref = add.double().cpu().numpy() + x.double().cpu().numpy() @ W.T
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.fp4_linear(x, Wq, y, st, add=add_arg)
    torch.cuda.synchronize()
    b = bound(x.cpu(), W, K, yd, ref) + np.abs(add.double().cpu().numpy()) * 2.0 ** -24
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= b)
    assert torch.all(ybuf[:, 0] == 7.0) and torch.all(ybuf[:, N + 1:] == 7.0)


def test_rows_of_a_larger_matrix(m):
    """A slice of rows of a weight: scales that start at odd addresses."""
    full, W = weight(m, 400, 288, "nvfp4", 16)
    lo = 37
    part = m.FP4Weight(full.codes[lo:lo + 200], full.scales[lo:lo + 200], "nvfp4", 0.75)
    x = acts(3, 288, torch.bfloat16, 17)
    whole = run_linear(m, x, full, torch.float32)
    assert torch.equal(run_linear(m, x, part, torch.float32), whole[:, lo:lo + 200])


def test_result_does_not_depend_on_the_other_tokens_and_repeats(m):
    Wq, _ = weight(m, 700, 2048, "nvfp4", 18)
    x = acts(16, 2048, torch.bfloat16, 19)
    whole = run_linear(m, x, Wq, torch.float32)
    assert torch.equal(whole, run_linear(m, x, Wq, torch.float32))


@pytest.mark.parametrize("T", [1, 5])
def test_codes_beyond_32_bit_offsets(m, T):
    """4.3 GB of codes; rows spread over them, the last ones included."""
    N, K, yd = 2 ** 20 + 77, 8192, torch.float32
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.randint(0x20, 0x50, (N, K // 16), dtype=torch.uint8, device="cuda")
    x = acts(T, K, torch.bfloat16, 40)
    got = run_linear(m, x, m.FP4Weight(codes, scales, "nvfp4", 0.75), yd).double().numpy()
    rows = torch.cat([torch.arange(0, N, 20011), torch.arange(N - 80, N)])
    at = rows.cuda()
    W = oracle.dequant("nvfp4", codes[at].cpu().numpy(), scales[at].cpu().numpy(), 1.0).astype(np.float64) * 0.75
    ref = x.double().numpy() @ W.T
    assert np.all(np.abs(got[:, rows.numpy()] - ref) <= bound(x, W, K, yd, ref))
    assert np.all(np.isfinite(got))


@pytest.mark.parametrize("T,shapes", [(4, [(4000, 1024), (3001, 2048)]), (16, [(4096, 1024), (4096, 1024)]),
                                      (16, [(2048, 512), (6000, 2048)]), (12, [(512, 2048), (512, 2048)])])
def test_calls_on_two_streams_at_once(m, T, shapes):
    mats = [weight(m, N, K, fmt, 50)[0] for (N, K), fmt in zip(shapes, ("nvfp4", "mxfp4"))]
    xs = [acts(T, Wq.K, torch.bfloat16, 52 + i).cuda() for i, Wq in enumerate(mats)]
    alone = [run_linear(m, x, Wq, torch.float32) for x, Wq in zip(xs, mats)]
    streams = [torch.cuda.Stream() for _ in mats]
    ys = [torch.empty((20, T, Wq.N), device="cuda") for Wq in mats]
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for r in range(20):
        for i, s in enumerate(streams):
            m.fp4_linear(xs[i], mats[i], ys[i][r], st[i:i + 1], stream=s)
    torch.cuda.synchronize()
    assert not st.any()
    for i in range(2):
        assert all(torch.equal(y.cpu(), alone[i]) for y in ys[i])


# ------------------------------------------------------------------ the gated pair

@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,I,H", [(1, 1, 32), (1, 768, 2048), (3, 65, 96), (4, 2048, 4096), (8, 130, 1056),
                                   (16, 768, 2048), (7, 6000, 512), (16, 200, 8192)])
@pytest.mark.parametrize("xd", [torch.bfloat16, torch.float32])
def test_swiglu_matches_reference(m, fmt, T, I, H, xd):
    Gq, G = weight(m, I, H, fmt, I + H)
    Uq, U = weight(m, I, H, fmt, I + H + 1, ts=1.5)
    x = acts(T, H, xd, T) * 0.25
    xd64 = x.double().numpy()
    g, u = xd64 @ G.T, xd64 @ U.T
    sg = 1.0 / (1.0 + np.exp(-np.clip(g, -700, 700)))
    ref = g * sg * u
    h = torch.full((T, I), float("nan"), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.fp4_swiglu(x.cuda(), Gq, Uq, h, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    # |d silu/dg| <= 1.1; the sigmoid itself to 2^-21 relative of its value (exp's argument
    # rounded to fp32: |g| 2^-24, at most 2^-17 where it still matters)
    bg, bu = bound(x, G, H, torch.float32, g), bound(x, U, H, torch.float32, u)
    silu = np.abs(g * sg)
    b = 1.1 * bg * (np.abs(u) + bu) + silu * bu + silu * np.abs(u) * (2.0 ** -21 + np.abs(g) * 2.0 ** -23) + 1e-37
    assert np.all(np.abs(h.double().cpu().numpy() - ref) <= b)


def test_shared_expert_run_and_graph_replay(m):
    """SwiGLU, down projection and the sum with another result, as a decode step uses
    them: eager, then captured and replayed on new inputs."""
    T, H, I = 4, 1024, 384
    Gq, G = weight(m, I, H, "nvfp4", 20, ts=0.01)
    Uq, U = weight(m, I, H, "nvfp4", 21, ts=0.01)
    Dq, D = weight(m, H, I, "nvfp4", 22, ts=0.01)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, h = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, I), device="cuda")
    routed, y = torch.zeros_like(x), torch.zeros_like(x)

    def step():
        m.fp4_swiglu(x, Gq, Uq, h, st)
        m.fp4_linear(h, Dq, y, st, add=routed)

    def check():
        torch.cuda.synchronize()
        xd = x.double().cpu().numpy()
        g, u = xd @ G.T, xd @ U.T
        hd = g / (1 + np.exp(-g)) * u
        ref = routed.double().cpu().numpy() + hd @ D.T
        hb = 1.1 * bound(x.cpu(), G, H, torch.float32, g) * (np.abs(u) + 1) + np.abs(g) * bound(
            x.cpu(), U, H, torch.float32, u) + np.abs(hd) * 2.0 ** -18
        b = hb @ np.abs(D).T + bound(torch.from_numpy(hd), D, I, torch.bfloat16, ref)
        b = b + np.abs(routed.double().cpu().numpy()) * 2.0 ** -24
        assert np.all(np.abs(y.double().cpu().numpy() - ref) <= b)
        assert int(st.item()) == 0

    x.copy_(acts(T, H, torch.bfloat16, 23)); routed.copy_(acts(T, H, torch.bfloat16, 24))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for seed in (25, 26):
        x.copy_(acts(T, H, torch.bfloat16, seed)); routed.copy_(acts(T, H, torch.bfloat16, seed + 10))
        y.zero_()
        graph.replay()
        check()
