"""Where the grouped router's fp32 values say less than its 64-bit choice needs: scores that tie
though their logits differ, sums that the tensor cores cut, squares below fp32's range, NaN rows.
Against the 64-bit reference: indices equal."""
import numpy as np
import pytest
import torch

from route_reference import choose

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    from expert_offload_fp4_b200 import build
    build.build()
    import expert_offload_fp4_b200 as mod
    return mod


def grouped(m, x, wr, b, k, **kw):
    T, E = x.shape[0], wr.shape[0]
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), dtype=torch.float32, device="cuda")
    ws = torch.zeros(m.route_grouped_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    m.route_grouped(x.cuda(), wr.cuda(), idx, w, ws, bias=None if b is None else b.cuda(), **kw)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy()


def select(m, logits, b, k, **kw):
    T = logits.shape[0]
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), dtype=torch.float32, device="cuda")
    m.route_select(logits.cuda(), idx, w, bias=None if b is None else b.cuda(), **kw)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy()


# ------------------------------------------------------------------ NaN rows of W_r

def test_a_nan_row_does_not_hide_the_largest_row(m):
    """Expert 9 is large and its products cancel (its sum errs by more than its distance to expert 10);
    expert `nan` is NaN, at every place in turn."""
    T, H, E = 64, 128, 64
    g = torch.Generator().manual_seed(4)
    r = torch.randn((T, 60), generator=g)
    x = torch.zeros((T, H))
    x[:, 0] = 1.0
    x[:, 1:61], x[:, 64:124] = r, r
    u = torch.randn(60, generator=g) * 1000
    wr = torch.randn((E, H), generator=g) * 0.01
    wr[9] = 0
    wr[9, 0], wr[9, 1:61], wr[9, 64:124] = 3.0, u, -u
    wr[10] = 0
    wr[10, 0], wr[10, 62] = 3.0, 2.0 ** -12
    x[:, 62] = torch.where(torch.arange(T) % 2 == 0, 1.0, -1.0)
    x = x.bfloat16()
    for nan in range(E):
        w = wr.bfloat16()
        w[nan] = float("nan")
        kw = dict(score="sigmoid")
        gi, gw = grouped(m, x, w, None, 4, **kw)
        ri, rw = choose(x.double().numpy() @ w.double().numpy().T, 4, **kw)
        assert np.array_equal(gi, ri), nan


@pytest.mark.parametrize("T", [3, 70])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_bias_ranks_last_and_keeps_the_score_as_weight(m, T, score):
    g = torch.Generator().manual_seed(5)
    x, wr = torch.randn((T, 256), generator=g).bfloat16(), (torch.randn((24, 256), generator=g) * 0.05).bfloat16()
    b = (torch.rand(24, generator=g) - 0.5) * 0.2
    b[[1, 2, 5, 6, 7]] = float("nan")
    for kw in (dict(score=score), dict(score=score, n_group=4, topk_group=2, group_top=2, renormalize=False)):
        k = 12
        gi, gw = grouped(m, x, wr, b, k, **kw)
        l = x.double().numpy() @ wr.double().numpy().T
        ri, rw = choose(l, k, bias=b.numpy(), **kw)
        assert np.array_equal(gi, ri)
        # logits of more than 32 tokens: 2^-17 |x| |W_e|, four times that in a renormalised weight
        dl = 2.0 ** -17 * np.linalg.norm(x.double().numpy(), axis=1)[:, None] * float(wr.double().norm(dim=1).max())
        assert np.all(np.abs(gw - rw) <= rw * (4 * dl + 2.0 ** -23))


# ------------------------------------------------------------------ what the tensor cores cut

@pytest.mark.parametrize("H,at", [(128, 5), (2048, 700)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_choice_when_a_token_and_a_row_share_one_large_channel(m, H, at, sign):
    """A product of 300 in an MMA's sum cuts every product below 2^-17 (25 bits below the largest's
    exponent): row 0's 127 others, of just less, are lost, and 2^-10 with them."""
    T, E = 40, 4
    x = torch.zeros((T, H))
    lo = at // 128 * 128
    x[:, lo:lo + 128] = 1.0
    x[:, at] = 300.0
    wr = torch.zeros((E, H))
    wr[0, lo:lo + 128] = sign * 1.9921875 * 2.0 ** -18
    wr[1, lo + 127] = sign * 1.5 * 2.0 ** -11
    wr[3, lo + 126] = sign * 1.25 * 2.0 ** -11
    wr[:, at] = 1.0
    x, wr = x.bfloat16(), wr.bfloat16()
    l = x.double().numpy() @ wr.double().numpy().T
    for kw in (dict(score="softmax"), dict(score="softmax", n_group=2, topk_group=1, group_top=1)):
        for b in (None, torch.zeros(E)):
            assert np.array_equal(grouped(m, x, wr, b, 2, **kw)[0], choose(l, 2, **kw)[0])


@pytest.mark.parametrize("H", [128, 1000, 4096])
@pytest.mark.parametrize("outlier", [1.0, 40.0, 3000.0])
def test_choice_between_close_rows_of_tokens_with_outliers(m, H, outlier):
    """Channels that are large in x and in W_r; rows in fours that differ in their smallest elements."""
    g = torch.Generator().manual_seed(H)
    T, E = 300, 32
    x, wr = torch.randn((T, H), generator=g).abs(), torch.randn((E, H), generator=g).abs() * 0.5 / H ** 0.5
    x[:, 3] *= outlier
    wr[:, 3] = 8.0 / outlier
    x, wr = x.bfloat16(), wr.bfloat16()
    for e in range(0, E, 4):
        for j in range(1, 4):
            wr[e + j] = wr[e]
            hit = torch.rand(H, generator=g) < 0.5
            hit[3] = False
            # a neighbouring bf16 value
            wr[e + j, hit] = (wr[e + j, hit].view(torch.int16) + (1 if j % 2 else -1)).view(torch.bfloat16)
    xd, wd = x.double().numpy(), wr.double().numpy()
    l = np.stack([(xd * row).sum(1) for row in wd], 1)
    for kw in (dict(score="softmax"), dict(score="sigmoid", n_group=8, topk_group=3, group_top=2)):
        assert np.array_equal(grouped(m, x, wr, None, 6, **kw)[0], choose(l, 6, **kw)[0])


# ------------------------------------------------------------------ squares out of range

@pytest.mark.parametrize("ex,ew", [(0, 0), (60, 50), (68, 63), (-50, -60), (-63, -68), (-40, -75)])
def test_choice_of_tokens_whose_squares_leave_the_range(m, ex, ew):
    """Tokens times 2^-ex and rows times 2^ew.  A token and the rows share one large channel; row 0's
    127 other products are small enough to be lost beside it, row 1's is not, and row 0 is the larger."""
    T, E, H = 40, 4, 128
    x, wr = torch.full((T, H), 2.0 ** -8), torch.zeros((E, H))
    x[:, 5] = 1.171875
    wr[0] = 1.9921875 * 2.0 ** -18
    wr[1, 127] = 1.5 * 2.0 ** -11
    wr[3, 126] = 1.25 * 2.0 ** -11
    wr[:, 5] = 1.0
    xs, ws = (x.double() * 2.0 ** -ex).bfloat16(), (wr.double() * 2.0 ** ew).bfloat16()
    l = xs.double().numpy() @ ws.double().numpy().T
    assert np.array_equal(l, (x.double().numpy() @ wr.double().numpy().T) * 2.0 ** (ew - ex))
    kw = dict(score="softmax")
    assert np.array_equal(grouped(m, xs, ws, None, 2, **kw)[0], choose(l, 2, **kw)[0])


def test_zero_and_tiny_tokens_among_others(m):
    """Rows of a padded batch, tokens of the smallest elements and of one element."""
    T, E, H = 130, 40, 264
    g = torch.Generator().manual_seed(6)
    x, wr = torch.randn((T, H), generator=g), torch.randn((E, H), generator=g) * 0.1
    x[::3] = 0
    x[1::6] = 0
    x[1::6, 7] = 2.0 ** -133
    x[5] *= 2.0 ** -126
    x[8] = -0.0
    wr[20:] = wr[:20]
    x, wr = x.bfloat16(), wr.bfloat16()
    xd, wd = x.double().numpy(), wr.double().numpy()
    l = np.stack([(xd * row).sum(1) for row in wd], 1)
    for b in (None, torch.linspace(-0.1, 0.1, E)):
        for kw in (dict(score="sigmoid"), dict(score="softmax", n_group=8, topk_group=3, group_top=2, renormalize=False)):
            gi, _ = grouped(m, x, wr, b, 6, **kw)
            assert np.array_equal(gi, choose(l, 6, bias=None if b is None else b.numpy(), **kw)[0])


# ------------------------------------------------------------------ scores that tie

TIES = [dict(), dict(n_group=4, topk_group=2, group_top=1)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kw", TIES)
@pytest.mark.parametrize("top", [0.0, 3.0, 15.0])
@pytest.mark.parametrize("E", [8, 64])
def test_select_ties_are_those_of_the_scores(m, score, kw, top, E):
    """Logits near 0 that differ by less than a score's rounding: the lower index, with a bias of
    zeros as without one."""
    rng = np.random.default_rng(E)
    rows = np.zeros((40, E), np.float32)
    rows[0, :7] = [1e-20, 2e-20, 3e-20, 0, 0, 0, 5e-20]
    for t in range(1, 40):
        rows[t] = rng.standard_normal(E) * 10.0 ** rng.choice([-30, -28, -26, -7, -5, -4], E)
        rows[t, rng.integers(0, E, 3)] = 0
    if top:
        rows[:, E - 2] = top
    l = torch.from_numpy(rows)
    ri, rw = choose(l.double().numpy(), 3, score=score, **kw)
    for b in (None, torch.zeros(E)):
        gi, gw = select(m, l, b, 3, score=score, **kw)
        assert np.array_equal(gi, ri)
        assert np.all(np.abs(gw - rw) <= rw * 2.0 ** -23)
    assert ri[0].tolist()[:2] != [6, 2]


@pytest.mark.parametrize("T", [1, 20, 33, 300])
@pytest.mark.parametrize("kw", TIES)
def test_ties_of_scores_of_exact_logits(m, T, kw):
    """Logits from x and W_r: 1e-20 steps beside a largest of 3, and 6e-11 steps at 15, where a
    sigmoid has no bits for them."""
    E, H = 16, 64
    x = torch.zeros((T, H))
    x[:, 0], x[:, 1], x[:, 2] = 2.0 ** -40, 2.0 ** -17, 1.0
    near = torch.zeros((E, H))
    near[:, 0] = 2.0 ** -27 * torch.arange(E).flip(0)
    near[9, 2] = 3.0
    high = torch.zeros((E, H))
    high[:, 1] = 2.0 ** -17 * torch.arange(E)
    high[:, 2] = 15.0
    for wr, scores in ((near, ("softmax", "sigmoid")), (high, ("sigmoid",))):
        x, wr = x.bfloat16(), wr.bfloat16()
        l = x.double().numpy() @ wr.double().numpy().T
        for score in scores:
            for b in (None, torch.zeros(E)):
                assert np.array_equal(grouped(m, x, wr, b, 5, score=score, **kw)[0], choose(l, 5, score=score, **kw)[0])


# ------------------------------------------------------------------ weights of few tokens

@pytest.mark.parametrize("T,H,E,k,kw,with_bias", [
    (1, 4096, 256, 6, dict(score="sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5), True),
    (3, 2048, 128, 8, dict(score="softmax", renormalize=False, scale=16.0), False),
    (8, 264, 20, 3, dict(score="softmax", n_group=5, topk_group=2, group_top=2), True),
    (32, 4096, 384, 8, dict(score="sigmoid", renormalize=False), True),
    (17, 512, 1024, 32, dict(score="softmax", n_group=32, topk_group=9, group_top=1), True)])
def test_weights_of_few_tokens_are_rounded_once(m, T, H, E, k, kw, with_bias):
    """Up to 32 tokens the logits are fp64 sums of exact products, off by less than 2^-40 of 1 here; a weight
    is one rounding (2^-24) from the 64-bit one."""
    g = torch.Generator().manual_seed(T + E)
    x, wr = torch.randn((T, H), generator=g).bfloat16(), (torch.randn((E, H), generator=g) * 0.9 / H ** 0.5).bfloat16()
    b = (torch.rand(E, generator=g) - 0.5) * 0.2 if with_bias else None
    gi, gw = grouped(m, x, wr, b, k, **kw)
    ri, rw = choose(x.double().numpy() @ wr.double().numpy().T, k, bias=None if b is None else b.numpy(), **kw)
    assert np.array_equal(gi, ri)
    assert np.all(np.abs(gw - rw) <= rw * (2.0 ** -24 + 2.0 ** -38))
