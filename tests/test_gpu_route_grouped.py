"""The grouped router (moe_route_grouped, moe_route_select) against a 64-bit
reference: indices equal, weights within the rounding they are allowed.

Weights from given logits are computed in fp64 and rounded once: 2^-24 relative.
From x, a logit may carry an error of DL = 2^-17 |x| |W_e| (fp32 partial sums of a
few hundred exact products each); a score's relative error is then at most 2 DL and
a renormalised weight's 4 DL.
"""
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


def inputs(T, H, E, seed, sigma=0.02):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H), generator=g).bfloat16()
    wr = (torch.randn((E, H), generator=g) * sigma * (2048 / H) ** 0.5).bfloat16()
    b = (torch.rand(E, generator=g) - 0.5) * 0.2
    return x, wr, b


def run_grouped(m, x, wr, b, k, ws=None, stream=None, **kw):
    T, E = x.shape[0], wr.shape[0]
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), dtype=torch.float32, device="cuda")
    if ws is None:
        ws = torch.zeros(m.route_grouped_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    m.route_grouped(x.cuda(), wr.cuda(), idx, w, ws, bias=None if b is None else b.cuda(), stream=stream, **kw)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy()


def check_grouped(x, wr, b, k, got, **kw):
    xd, wd = x.double().numpy(), wr.double().numpy()
    ri, rw = choose(xd @ wd.T, k, bias=None if b is None else b.numpy(), **kw)
    assert np.array_equal(got[0], ri)
    dl = 2.0 ** -17 * np.linalg.norm(xd, axis=1)[:, None] * np.linalg.norm(wd, axis=1).max()
    assert np.all(np.abs(got[1] - rw) <= rw * (4 * dl + 2.0 ** -24) + 1e-45)


CASES = [
    # T, H, E, k, options
    (1, 4096, 256, 6, dict(score="sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5), True),
    (1, 8, 1, 1, dict(score="softmax"), False),
    (2, 264, 20, 3, dict(score="sigmoid", n_group=5, topk_group=2, group_top=2), True),
    (3, 2048, 128, 8, dict(score="softmax", renormalize=False, scale=16.0), False),
    (5, 256, 16, 2, dict(score="softmax", n_group=4, topk_group=1, group_top=1), True),
    (8, 2048, 128, 8, dict(score="softmax"), False),
    (9, 1032, 96, 32, dict(score="sigmoid", n_group=3, topk_group=1, group_top=2), True),
    (16, 4096, 256, 8, dict(score="sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5), True),
    (17, 512, 1024, 8, dict(score="softmax", n_group=32, topk_group=5, group_top=1), True),
    (33, 2048, 130, 7, dict(score="sigmoid", renormalize=False), True),
    (64, 4096, 256, 8, dict(score="sigmoid", n_group=8, topk_group=8, group_top=2), True),
    (127, 136, 160, 6, dict(score="softmax", n_group=8, topk_group=3, group_top=1, renormalize=False), False),
    (128, 2048, 128, 8, dict(score="softmax", n_group=8, topk_group=3, group_top=1), False),
    (129, 2048, 256, 8, dict(score="sigmoid", n_group=8, topk_group=4, group_top=2), True),
    (300, 5120, 384, 8, dict(score="sigmoid"), True),
    (385, 4096, 1000, 6, dict(score="softmax", n_group=4, topk_group=2, group_top=2), True),
    (2048, 2048, 128, 8, dict(score="softmax"), False),
    (4100, 4096, 256, 8, dict(score="sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5), True),
]


@pytest.mark.parametrize("T,H,E,k,opt,with_bias", CASES)
def test_grouped_router_matches_reference(m, T, H, E, k, opt, with_bias):
    x, wr, b = inputs(T, H, E, T * 7 + E)
    b = b if with_bias else None
    check_grouped(x, wr, b, k, run_grouped(m, x, wr, b, k, **opt), **opt)


@pytest.mark.parametrize("T", [1, 7, 16, 200, 1030])
def test_choice_between_experts_that_fp32_sums_cannot_tell_apart(m, T):
    """Rows of W_r in sets that differ by one small product: logits 1e-9 apart."""
    H, E, k = 2048, 64, 8
    x, wr, _ = inputs(T, H, E, 3)
    x[:, 100] = 2.0 ** -14
    for e in range(0, E, 4):
        for j in range(1, 4):
            wr[e + j] = wr[e]
        wr[e:e + 4, 100] = torch.tensor([2.0 ** -16, 2.0 ** -15, 0.0, 2.0 ** -15])
    for opt in (dict(score="softmax"), dict(score="sigmoid", n_group=4, topk_group=2, group_top=2)):
        check_grouped(x, wr, None, k, run_grouped(m, x, wr, None, k, **opt), **opt)


# near: groups that are near-copies of group 0 (the rest are independent), one of them an exact copy
CLOSE_GROUPS = [
    # E, n_group, topk_group, group_top, near, score, with_bias
    (256, 8, 4, 2, 5, "sigmoid", True),
    (256, 8, 4, 2, 8, "sigmoid", True),
    (128, 8, 3, 1, 4, "softmax", False),
    (96, 4, 2, 2, 3, "softmax", False),
    (160, 32, 20, 2, 32, "sigmoid", False),
    (64, 4, 1, 1, 4, "sigmoid", True),
    (48, 3, 2, 2, 3, "softmax", True),
    (12, 6, 3, 2, 6, "softmax", True),
]


def near_copies(rows, gs, near, rng, step, share):
    """rows [E, n] with groups 1 .. near - 1 replaced by group 0 with a share of its elements changed
    by step(values), the last of them left equal to it."""
    for g in range(1, near):
        part = rows[:gs].copy()
        if g + 1 < near:
            hit = rng.random(part.shape) < share
            part[hit] = step(part[hit])
        rows[g * gs:(g + 1) * gs] = part
    return rows


@pytest.mark.parametrize("T", [1, 9, 32, 33, 700])
@pytest.mark.parametrize("E,n_group,topk_group,group_top,near,score,with_bias", CLOSE_GROUPS)
def test_choice_between_groups_that_fp32_sums_cannot_tell_apart(m, T, E, n_group, topk_group, group_top, near, score, with_bias):
    H, gs, rng = 512, E // n_group, np.random.default_rng(T + E)
    x, wr, b = inputs(T, H, E, 31 * T + E)
    # a neighbouring bf16 value: 2^-8 of an element
    step = lambda v: (v.view(np.uint32) + np.uint32(0x10000)).view(np.float32)
    wr = torch.from_numpy(near_copies(wr.float().numpy().copy(), gs, near, rng, step, 0.02)).bfloat16()
    if with_bias:
        b = torch.from_numpy(near_copies(b.numpy().copy()[:, None], gs, near, rng, lambda v: v + np.float32(1e-6), 0.3)[:, 0].copy())
    else:
        b = None
    k = min(8, topk_group * gs)
    kw = dict(score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)
    got = run_grouped(m, x, wr, b, k, **kw)
    # (expert by expert in one order, so that equal rows have equal logits)
    xd, wd = x.double().numpy(), wr.double().numpy()
    logits = np.stack([(xd * row).sum(1) for row in wd], 1)
    ri, rw = choose(logits, k, bias=None if b is None else b.numpy(), **kw)
    assert np.array_equal(got[0], ri)
    dl = 2.0 ** -17 * np.linalg.norm(xd, axis=1)[:, None] * np.linalg.norm(wd, axis=1).max()
    assert np.all(np.abs(got[1] - rw) <= rw * (4 * dl + 2.0 ** -24) + 1e-45)


@pytest.mark.parametrize("T", [1, 333])
@pytest.mark.parametrize("E,n_group,topk_group,group_top,near,score,with_bias", CLOSE_GROUPS)
def test_select_between_close_groups(m, T, E, n_group, topk_group, group_top, near, score, with_bias):
    gs, rng = E // n_group, np.random.default_rng(T + E)
    l = rng.standard_normal((T, E)).astype(np.float32)
    step = lambda v: np.nextafter(v, np.float32(9.0))
    for t in range(T):
        near_copies(l[t][:, None], gs, near, rng, step, 0.5)
    b = None
    if with_bias:
        b = near_copies(((rng.random(E, np.float32) - 0.5) * 0.2)[:, None], gs, near, rng, step, 0.5)[:, 0].copy()
    k = min(8, topk_group * gs)
    kw = dict(score=score, n_group=n_group, topk_group=topk_group, group_top=group_top)
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    m.route_select(torch.from_numpy(l).cuda(), idx, w, bias=None if b is None else torch.from_numpy(b).cuda(), **kw)
    ri, rw = choose(l.astype(np.float64), k, bias=b, **kw)
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert np.all(np.abs(w.cpu().numpy() - rw) <= rw * 2.0 ** -23 + 1e-45)


@pytest.mark.parametrize("T", [1, 5, 140])
def test_equal_experts_and_zero_tokens_go_to_the_lower_index(m, T):
    x, wr, _ = inputs(T, 256, 32, 5)
    wr[16:] = wr[:16]
    x[T // 2] = 0
    for opt in (dict(score="softmax"), dict(score="sigmoid", n_group=4, topk_group=2, group_top=2)):
        check_grouped(x, wr, None, 6, run_grouped(m, x, wr, None, 6, **opt), **opt)


@pytest.mark.parametrize("T", [1, 3, 150])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts(m, T, score):
    """bias -inf: some experts, whole groups, all but one, all."""
    x, wr, b = inputs(T, 512, 32, 6)
    kw = dict(score=score, n_group=4, topk_group=2, group_top=2)
    for mask in (range(0, 32, 3), range(0, 16), range(0, 31), range(32)):
        bb = b.clone()
        bb[list(mask)] = -float("inf")
        got = run_grouped(m, x, wr, bb, 5, **kw)
        check_grouped(x, wr, bb, 5, got, **kw)
        assert np.all(got[1][np.isin(got[0], list(mask))] == 0)


@pytest.mark.parametrize("T", [2, 130])
def test_nan_token_leaves_the_others_alone_and_its_indices_valid(m, T):
    x, wr, b = inputs(T, 256, 64, 8)
    kw = dict(score="sigmoid", n_group=8, topk_group=3, group_top=2)
    clean = run_grouped(m, x, wr, b, 4, **kw)
    x[1] = float("nan")
    got = run_grouped(m, x, wr, b, 4, **kw)
    keep = np.arange(T) != 1
    assert np.array_equal(got[0][keep], clean[0][keep]) and np.array_equal(got[1][keep], clean[1][keep])
    assert got[0][1].tolist() == [0, 1, 2, 3] and np.all(np.isnan(got[1][1]))


@pytest.mark.parametrize("T", [1, 4, 160])
def test_large_and_tiny_values(m, T):
    """Logits far beyond exp's range, subnormal inputs, and one infinite bias."""
    x, wr, b = inputs(T, 256, 32, 9)
    b[7] = float("inf")
    for s in (2.0 ** 60, 2.0 ** -60, 2.0 ** -126):
        xs = (x.float() * s).bfloat16()
        for score in ("softmax", "sigmoid"):
            l = xs.double().numpy() @ wr.double().numpy().T
            got = run_grouped(m, xs, wr, b, 4, score=score, renormalize=False)
            ri, rw = choose(l, 4, score=score, bias=b.numpy(), renormalize=False)
            assert np.array_equal(got[0], ri), s
            assert np.all(got[0][:, 0] == 7)


def test_choice_does_not_depend_on_the_batch(m):
    x, wr, b = inputs(600, 2048, 256, 10)
    kw = dict(score="sigmoid", n_group=8, topk_group=4, group_top=2)
    whole = run_grouped(m, x, wr, b, 8, **kw)
    for lo, hi in ((0, 1), (17, 33), (100, 180), (599, 600)):
        part = run_grouped(m, x[lo:hi], wr, b, 8, **kw)
        assert np.array_equal(part[0], whole[0][lo:hi])


@pytest.mark.parametrize("T", [3, 32, 90])
def test_calls_on_two_streams_at_once(m, T):
    kw = dict(n_group=8, topk_group=4, group_top=2)
    cases = [inputs(T, 1024, 128, 60 + i) for i in range(2)]
    alone = [run_grouped(m, x, wr, b, 6, **kw) for x, wr, b in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    on = [[t.cuda() for t in c] for c in cases]
    ws = [torch.zeros(m.route_grouped_workspace_bytes(T, 128), dtype=torch.uint8, device="cuda") for _ in cases]
    idx = torch.zeros((2, 20, T, 6), dtype=torch.int32, device="cuda")
    w = torch.zeros((2, 20, T, 6), device="cuda")
    torch.cuda.synchronize()
    for r in range(20):
        for i, s in enumerate(streams):
            m.route_grouped(on[i][0], on[i][1], idx[i, r], w[i, r], ws[i], bias=on[i][2], stream=s, **kw)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(np.array_equal(a, alone[i][0]) for a in idx[i].cpu().numpy())
        assert all(np.array_equal(a, alone[i][1]) for a in w[i].cpu().numpy())


@pytest.mark.parametrize("T", [33, 129])
@pytest.mark.parametrize("H,E,k", [(8, 5, 2), (16, 1024, 32), (72, 33, 4), (200, 257, 9)])
def test_short_rows_and_odd_expert_counts_of_a_prompt(m, T, H, E, k):
    x, wr, b = inputs(T, H, E, H + E)
    check_grouped(x, wr, b, k, run_grouped(m, x, wr, b, k))


@pytest.mark.parametrize("T", [1, 40, 520])
def test_workspace_is_left_ready_and_graphs_replay(m, T):
    x, wr, b = inputs(T, 1024, 128, 11)
    x2 = inputs(T, 1024, 128, 12)[0]
    kw = dict(score="sigmoid", n_group=8, topk_group=4, group_top=2)
    want = [run_grouped(m, v, wr, b, 8, **kw) for v in (x, x2)]
    ws = torch.zeros(m.route_grouped_workspace_bytes(T, 128), dtype=torch.uint8, device="cuda")
    for v, r in ((x, want[0]), (x2, want[1]), (x, want[0])):
        got = run_grouped(m, v, wr, b, 8, ws=ws, **kw)
        assert np.array_equal(got[0], r[0]) and np.array_equal(got[1], r[1])
    xd, wd, bd = x.cuda(), wr.cuda(), b.cuda()
    idx = torch.zeros((T, 8), dtype=torch.int32, device="cuda")
    w = torch.zeros((T, 8), device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        m.route_grouped(xd, wd, idx, w, ws, bias=bd, **kw)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        m.route_grouped(xd, wd, idx, w, ws, bias=bd, **kw)
    for v, r in ((x2, want[1]), (x, want[0])):
        xd.copy_(v)
        idx.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(idx.cpu().numpy(), r[0]) and np.array_equal(w.cpu().numpy(), r[1])


# ------------------------------------------------------------------ the choice alone

def run_select(m, logits, b, k, **kw):
    T = logits.shape[0]
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), dtype=torch.float32, device="cuda")
    m.route_select(logits, idx, w, bias=None if b is None else b.cuda(), **kw)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy()


def check_select(logits, b, k, got, **kw):
    ri, rw = choose(logits.double().cpu().numpy(), k, bias=None if b is None else b.numpy(), **kw)
    assert np.array_equal(got[0], ri)
    ok = np.abs(got[1] - rw) <= np.abs(rw) * 2.0 ** -24 * (1 + 2.0 ** -20) + 2.0 ** -150
    assert np.all(ok | (np.isnan(got[1]) & np.isnan(rw)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,pad,opt", [
    (1, 1, 1, 0, dict(score="softmax")),
    (1, 256, 8, 0, dict(score="sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5)),
    (5, 33, 32, 1, dict(score="softmax", renormalize=False)),
    (70, 160, 6, 8, dict(score="softmax", n_group=8, topk_group=3, group_top=1, scale=16.0)),
    (1001, 128, 8, 3, dict(score="sigmoid", n_group=32, topk_group=6, group_top=2)),
    (300, 1024, 20, 0, dict(score="softmax", n_group=2, topk_group=1, group_top=2)),
    (37, 993, 9, 5, dict(score="sigmoid", n_group=3, topk_group=2, group_top=2)),
])
@pytest.mark.parametrize("with_bias", [False, True])
def test_select_matches_reference(m, dtype, T, E, k, pad, opt, with_bias):
    g = torch.Generator().manual_seed(T + E)
    full = torch.randn((T, E + pad), generator=g).to(dtype)
    b = (torch.rand(E, generator=g) - 0.5) * 0.2 if with_bias else None
    logits = full.cuda()[:, :E]
    check_select(logits, b, k, run_select(m, logits, b, k, **opt), **opt)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n_group,topk_group", [(1, 1), (4, 2)])
def test_select_masked_infinite_and_nan_logits(m, score, n_group, topk_group):
    inf, lowest = float("inf"), torch.finfo(torch.float32).min
    rows = torch.randn((12, 24), generator=torch.Generator().manual_seed(2))
    rows[1, ::2] = -inf
    rows[2] = -inf
    rows[3, :23] = -inf
    rows[4] = lowest
    rows[5, 3:] = lowest
    rows[6, 5] = float("nan")
    rows[7] = float("nan")
    rows[8, 4] = inf
    rows[9, 2] = -inf
    rows[9, 3] = float("nan")
    rows[10, :] = 0.0
    rows[11, :] = torch.linspace(-800, 800, 24)
    b = (torch.rand(24, generator=torch.Generator().manual_seed(3)) - 0.5) * 0.2
    for bias in (None, b):
        for renorm in (True, False):
            kw = dict(score=score, n_group=n_group, topk_group=topk_group, group_top=2, renormalize=renorm)
            check_select(rows.cuda(), bias, 5, run_select(m, rows.cuda(), bias, 5, **kw), **kw)


def test_select_on_another_stream(m):
    logits = torch.randn((50, 64), device="cuda")
    idx = torch.zeros((50, 4), dtype=torch.int32, device="cuda")
    w = torch.zeros((50, 4), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    m.route_select(logits, idx, w, score="softmax", stream=s)
    s.synchronize()
    check_select(logits, None, 4, (idx.cpu().numpy(), w.cpu().numpy()), score="softmax")
