"""A decode layer with the grouped router and a shared expert, as a decode step uses
them: against the 64-bit choice, the oracle's experts and the dequantised shared
expert in float64.  Tolerance as for every decode layer: 2e-2 of the output's rms."""
import numpy as np
import pytest
import torch

import oracle
from route_reference import choose
from synthetic import gen, workloads as W

pytestmark = pytest.mark.gpu
TOL = 2e-2


@pytest.fixture(scope="module")
def m():
    from expert_offload_fp4_b200 import build
    build.build()
    import expert_offload_fp4_b200 as mod
    return mod


def workload(fmt, H, I, E, k, L):
    return W.Workload(name="grouped", H=H, I=I, E=E, k=k, L=L, fmt=fmt, seed=31, batches=(1,), steps=4, zipf_s=0.0,
                      weight_recipe="normal" if fmt == W.NVFP4 else "uniform", exp_range=(-6, -2))


def bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def f64(bits):
    return gen.bf16_bits_to_f32(bits).astype(np.float64)


def matrix(m, rows, K, fmt, seed, sigma):
    """A 4-bit matrix of about N(0, sigma) entries and its float64 values."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (rows, K // 2), dtype=np.uint8)
    rms = 2.99                                  # of the 16 E2M1 values
    if fmt == "mxfp4":
        scales = np.full((rows, K // 32), 127 + int(round(np.log2(sigma / rms))), np.uint8)
        ts = 1.0
    else:
        scales = rng.integers(0x34, 0x3C, (rows, K // 16), dtype=np.uint8)     # 0.75 to 1.4
        ts = sigma / rms
    values = oracle.dequant(fmt, codes, scales, 1.0).astype(np.float64) * float(np.float32(ts))
    return m.FP4Weight(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), fmt, ts), values


@pytest.mark.parametrize("fmt,H,I,E,k,S,T", [("nvfp4", 512, 256, 16, 3, 12, 4), ("mxfp4", 256, 512, 24, 4, 24, 1),
                                             ("nvfp4", 768, 256, 16, 2, 16, 13)])
@pytest.mark.parametrize("native", [True, False])
def test_layer_with_grouped_router_and_shared_expert(m, fmt, H, I, E, k, S, T, native):
    w = workload(fmt, H, I, E, k, 2)
    routing = m.GroupedRouting(score="sigmoid", n_group=4, topk_group=2, group_top=2, renormalize=True, scale=2.5)
    pool = m.Pool(H, I, E, k, 2, fmt, S, max_tokens=T)
    experts = {(l, e): gen.expert_weights(w, l, e) for l in range(2) for e in range(E)}
    for (l, e), t in experts.items():
        pool.load_expert(l, e, t)
    Is = 320
    (Gq, G), (Uq, U) = matrix(m, Is, H, fmt, 1, 0.05), matrix(m, Is, H, fmt, 2, 0.05)
    Dq, D = matrix(m, H, Is, fmt, 3, 0.05)
    shared = m.SharedExpert(Gq, Uq, Dq)
    lo = m.DecodeLayer(pool, T, router=routing)
    if not native:
        lo.ffn_events = []
    try:
        for step in range(2):
            for l in range(2):
                x, wr = gen.activations(w, l, step, T), gen.router_weight(w, l)
                b = (np.random.default_rng(l).random(E).astype(np.float32) - 0.5) * 0.2
                y = lo(l, bf16(x), bf16(wr), torch.from_numpy(b).cuda(), shared=shared)
                torch.cuda.synchronize()
                assert int(lo.status.item()) == 0
                idx, wt = choose(f64(x) @ f64(wr).T, k, score="sigmoid", bias=b, n_group=4, topk_group=2, group_top=2,
                                 scale=2.5)
                assert np.array_equal(lo.idx.cpu().numpy(), idx)
                ex = {e: experts[(l, e)] for e in sorted(set(idx.ravel().tolist()))}
                routed, _ = oracle.moe_decode(fmt, H, I, E, x, idx, wt.astype(np.float32), ex)
                g, u = f64(x) @ G.T, f64(x) @ U.T
                ref = routed.astype(np.float64) + (g / (1 + np.exp(-g)) * u) @ D.T
                rms = float(np.sqrt(np.mean(ref ** 2)))
                assert np.max(np.abs(y.double().cpu().numpy() - ref)) <= TOL * rms
    finally:
        pool.close()


def test_routed_call_refuses_a_shared_copy_stream_and_matches_the_routing_call(m):
    """moe_decode_layer_routed on moe_route's own idx and w gives moe_decode_layer's bits."""
    w = workload("nvfp4", 512, 256, 16, 2, 1)
    T = 3
    pool = m.Pool(w.H, w.I, w.E, w.k, 1, w.fmt, 16, max_tokens=T)
    try:
        for e in range(w.E):
            pool.load_expert(0, e, gen.expert_weights(w, 0, e))
        lo = m.DecodeLayer(pool, T)
        x, wr = bf16(gen.activations(w, 0, 0, T)), bf16(gen.router_weight(w, 0))
        want = lo(0, x, wr, None).clone()
        torch.cuda.synchronize()
        lo.y.zero_()
        m.decode_layer_routed(pool, 0, x, lo.idx, lo.w, lo.slot_of, lo.y_part, lo.y, lo.status, lookup=lo.lookup,
                              copy_stream=lo.copy_stream)
        torch.cuda.synchronize()
        assert int(lo.status.item()) == 0 and torch.equal(lo.y, want)
        with pytest.raises(ValueError, match="copy_stream"):
            m.decode_layer_routed(pool, 0, x, lo.idx, lo.w, lo.slot_of, lo.y_part, lo.y, lo.status)
        with pytest.raises(ValueError, match="H differs"):
            Gq, _ = matrix(m, 64, 256, "nvfp4", 4, 0.05)
            Dq, _ = matrix(m, 256, 64, "nvfp4", 5, 0.05)
            lo(0, x, wr, None, shared=m.SharedExpert(Gq, Gq, Dq))
    finally:
        pool.close()


def test_prompt_through_grouped_router_and_prefill(m):
    """A prompt: grouped router, lookup, prefill FFN and combine, with the same choice and
    weights given to the oracle token by token."""
    w = workload("nvfp4", 512, 256, 16, 2, 1)
    T = 160
    pool = m.Pool(w.H, w.I, w.E, w.k, 1, w.fmt, 16, max_tokens=16)
    try:
        experts = {e: gen.expert_weights(w, 0, e) for e in range(w.E)}
        for e, t in experts.items():
            pool.load_expert(0, e, t)
        x, wr = gen.activations(w, 0, 0, T), gen.router_weight(w, 0)
        kw = dict(score="softmax", n_group=4, topk_group=3, group_top=1)
        idx = torch.empty((T, w.k), dtype=torch.int32, device="cuda")
        wt = torch.empty((T, w.k), device="cuda")
        ws = torch.zeros(m.route_grouped_workspace_bytes(T, w.E), dtype=torch.uint8, device="cuda")
        m.route_grouped(bf16(x), bf16(wr), idx, wt, ws, **kw)
        slot = torch.empty_like(idx)
        lk = m.slot_lookup(pool, 0, idx, slot)
        cs = torch.cuda.Stream()
        m.stream_misses(pool, 0, lk, cs)
        cs.synchronize()
        y_part = torch.empty((T, w.k, w.H), device="cuda")
        y = torch.empty((T, w.H), dtype=torch.bfloat16, device="cuda")
        pws = torch.empty(m.prefill_workspace_bytes(pool, T), dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        m.prefill_ffn(pool, 0, bf16(x), idx, wt, slot, y_part, pws, status)
        m.combine(y_part, y)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        ri, rw = choose(f64(x) @ f64(wr).T, w.k, **kw)
        assert np.array_equal(idx.cpu().numpy(), ri)
        got = y.double().cpu().numpy()
        for t in range(0, T, 13):
            ref, _ = oracle.moe_prefill_token(w.H, w.I, w.E, x[t], ri[t], rw[t].astype(np.float32), experts)
            rms = float(np.sqrt(np.mean(np.asarray(ref, np.float64) ** 2)))
            assert np.max(np.abs(got[t] - ref)) <= TOL * rms
    finally:
        pool.close()
