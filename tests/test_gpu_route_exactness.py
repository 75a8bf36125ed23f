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
