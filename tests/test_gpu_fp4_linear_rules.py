"""What the 4-bit products' documentation allows and takes for granted: every K * T up to the
limit, operands that share a buffer but no byte, tokens that do not see one another."""
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


def weight(m, N, K, fmt, seed):
    """Random codes and scales (on the device) and the dequantised matrix in float64."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    if fmt == "mxfp4":
        scales = rng.integers(110, 122, (N, K // 32), dtype=np.uint8)
    else:
        scales = rng.integers(0x00, 0x50, (N, K // 16), dtype=np.uint8)
    W = oracle.dequant(fmt, codes, scales, 1.0).astype(np.float64)
    return m.FP4Weight(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), fmt), W


def acts(T, K, seed, dtype=torch.bfloat16):
    return torch.randn((T, K), generator=torch.Generator().manual_seed(seed)).to(dtype)


def bound(x, W, K, dtype, ref):
    """S = sum |x||w|: at most K/64 + 40 roundings of 2^-23 S, x to 2^-22 of its row's largest element,
    one rounding to the result's type."""
    xa, Wa = x.double().abs().numpy(), np.abs(W)
    b = (K / 64 + 40) * 2.0 ** -23 * (xa @ Wa.T) + 2.0 ** -22 * xa.max(1)[:, None] * Wa.sum(1)[None, :]
    return b + (np.abs(ref) + b) * (torch.finfo(dtype).eps / 2) + 1e-40


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def limit(T):
    """The largest K of T tokens: K * T, K rounded up to 256 and T to even, is at most 262144."""
    return 262144 // (T + T % 2) // 256 * 256


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T", range(1, 17))
def test_the_largest_k_of_every_token_count(m, fmt, T):
    K, N = limit(T), 70
    Wq, W = weight(m, N, K, fmt, T)
    x = acts(T, K, T)
    y, st = torch.full((T, N), float("nan"), device="cuda"), status()
    m.fp4_linear(x.cuda(), Wq, y, st)
    torch.cuda.synchronize()
    ref = x.double().numpy() @ W.T
    assert int(st.item()) == 0
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= bound(x, W, K, torch.float32, ref))
    with pytest.raises(m._lib.MoeError, match="K too large"):
        big = m.FP4Weight(torch.zeros((1, K // 2 + 16), dtype=torch.uint8, device="cuda"),
                          torch.zeros((1, K // 32 + 1), dtype=torch.uint8, device="cuda"), "mxfp4")
        m.fp4_linear(torch.zeros((T, K + 32), dtype=torch.bfloat16, device="cuda"), big,
                     torch.zeros((T, 1), device="cuda"), st)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,K", [(9, 24608), (10, 25600), (11, 20512), (12, 21760), (5, 43040), (6, 43264), (13, 18464),
                                 (14, 18688)])
@pytest.mark.parametrize("xd", [torch.bfloat16, torch.float32])
def test_k_near_the_limit(m, fmt, T, K, xd):
    (Gq, G), (Uq, U) = weight(m, 133, K, fmt, T), weight(m, 133, K, fmt, T + 50)
    x = acts(T, K, K, xd)
    y, st = torch.full((T, 133), float("nan"), dtype=torch.bfloat16, device="cuda"), status()
    m.fp4_linear(x.cuda(), Gq, y, st)
    h = torch.full((T, 133), float("nan"), device="cuda")
    m.fp4_swiglu((x * 2.0 ** -9).cuda(), Gq, Uq, h, st)
    torch.cuda.synchronize()
    ref = x.double().numpy() @ G.T
    assert int(st.item()) == 0
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= bound(x, G, K, torch.bfloat16, ref))
    xs = x * 2.0 ** -9
    g, u = ref * 2.0 ** -9, x.double().numpy() @ U.T * 2.0 ** -9
    sg = 1.0 / (1.0 + np.exp(-np.clip(g, -700, 700)))
    bg, bu = bound(xs, G, K, torch.float32, g), bound(xs, U, K, torch.float32, u)
    silu = np.abs(g * sg)
    # |d silu/dg| <= 1.1; the sigmoid to 2^-21 of its value and its argument's rounding
    b = 1.1 * bg * (np.abs(u) + bu) + silu * bu + silu * np.abs(u) * (2.0 ** -21 + np.abs(g) * 2.0 ** -23) + 1e-37
    assert np.all(np.abs(h.double().cpu().numpy() - g * sg * u) <= b)


# ------------------------------------------------------------------ operands in one buffer

@pytest.mark.parametrize("T", [2, 16])
@pytest.mark.parametrize("yd", [torch.bfloat16, torch.float32])
def test_column_slices_of_one_buffer(m, T, yd):
    """x, add and y beside one another in the rows of one buffer; the columns between stay."""
    N, K = 320, 256
    Wq, W = weight(m, N, K, "nvfp4", 1)
    buf = torch.randn((T, K + 8 + 2 * N + 8), generator=torch.Generator().manual_seed(T)).to(yd).cuda()
    before = buf.clone()
    x, add, y = buf[:, :K], buf[:, K + 8:K + 8 + N], buf[:, K + 8 + N:K + 8 + 2 * N]
    st = status()
    m.fp4_linear(x, Wq, y, st, add=add)
    torch.cuda.synchronize()
    xc, ac = before[:, :K].cpu(), before[:, K + 8:K + 8 + N].double().cpu().numpy()
    ref = xc.double().numpy() @ W.T + ac
    got = y.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= bound(xc, W, K, yd, ref) + np.abs(ac) * 2.0 ** -24)
    assert torch.equal(buf[:, :K + 8 + N], before[:, :K + 8 + N]) and torch.equal(buf[:, K + 8 + 2 * N:], before[:, K + 8 + 2 * N:])
    assert int(st.item()) == 0


def test_rows_dealt_out_in_turn_share_a_buffer(m):
    """Rows of x and y alternate: their spans cross, their bytes do not."""
    T, K = 5, 512
    Wq, W = weight(m, K, K, "mxfp4", 2)
    buf = acts(2 * T, K, 3).cuda()
    x, y = buf[0::2], buf[1::2]
    xc, st = x.cpu(), status()
    m.fp4_linear(x, Wq, y, st)
    torch.cuda.synchronize()
    ref = xc.double().numpy() @ W.T
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= bound(xc, W, K, torch.bfloat16, ref))
    assert torch.equal(x.cpu(), xc)


def test_operands_that_do_share_bytes_are_refused(m):
    T, K = 4, 256
    Wq, _ = weight(m, K, K, "nvfp4", 4)
    buf, st = torch.zeros((T + 1, 2 * K), dtype=torch.bfloat16, device="cuda"), status()
    flat = buf.view(-1)
    x = buf[:T, :K]
    for y in (buf[:T, K - 2:2 * K - 2], buf[:T, 8:K + 8], flat[2 * K - 8:2 * K - 8 + T * 2 * K].view(T, 2 * K)[:, :K],
              flat[K + 2:K + 2 + 3 * (2 * K - 64) + K].as_strided((T, K), (2 * K - 64, 1))):
        with pytest.raises(m._lib.MoeError, match="y overlaps x"):
            m.fp4_linear(x, Wq, y, st)
        with pytest.raises(m._lib.MoeError, match="y overlaps add"):
            m.fp4_linear(torch.zeros((T, K), dtype=torch.bfloat16, device="cuda"), Wq, y, st, add=x)


# ------------------------------------------------------------------ tokens on their own

@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,N,K", [(2, 200, 512), (5, 700, 2048), (16, 1000, 4096)])
def test_a_token_does_not_see_the_others(m, fmt, T, N, K):
    """The same token at the same place among others, huge, tiny, zero and NaN ones included: the same bits."""
    Wq, _ = weight(m, N, K, fmt, 5)
    x = acts(T, K, 6)
    out = []
    for i, s in enumerate((1.0, 2.0 ** 90, 2.0 ** -90, 0.0, float("nan"))):
        other = (acts(T, K, 7 + i).float() * s).bfloat16()
        other[T // 2] = x[T // 2]
        y, st = torch.empty((T, N), device="cuda"), status()
        m.fp4_linear(other.cuda(), Wq, y, st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        out.append(y[T // 2].cpu())
    assert all(torch.equal(o, out[0]) for o in out) and torch.isfinite(out[0]).all()
