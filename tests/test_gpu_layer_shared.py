"""Products and routers between decode FFNs as a program chains them: results that pass from one
kernel to another while the next is already starting, on other streams, in reused buffers."""
import numpy as np
import pytest
import torch

from synthetic import gen, workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    from expert_offload_fp4_b200 import build
    build.build()
    import expert_offload_fp4_b200 as mod
    return mod


def workload(H, I, E, k, L):
    return W.Workload(name="chain", H=H, I=I, E=E, k=k, L=L, fmt=W.NVFP4, seed=33, batches=(1,), steps=4, zipf_s=0.0,
                      weight_recipe="normal", exp_range=(-6, -2))


def bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def full_pool(m, w, T):
    """A pool whose slots hold every expert of every layer, and a layer's buffers."""
    pool = m.Pool(w.H, w.I, w.E, w.k, w.L, w.fmt, w.L * w.E, max_tokens=T)
    for l in range(w.L):
        for e in range(w.E):
            pool.load_expert(l, e, gen.expert_weights(w, l, e))
    lo = m.DecodeLayer(pool, T)
    idx = torch.arange(w.E, dtype=torch.int32, device="cuda").view(-1, w.k)
    slot = torch.empty_like(idx)
    for l in range(w.L):
        m.stream_misses(pool, l, m.slot_lookup(pool, l, idx, slot), lo.copy_stream)
    torch.cuda.synchronize()
    return pool, lo


def matrix(m, rows, K, seed, sigma=0.05):
    """A 4-bit matrix of about N(0, sigma) entries."""
    rng = np.random.default_rng(seed)
    codes = torch.from_numpy(rng.integers(0, 256, (rows, K // 2), dtype=np.uint8)).cuda()
    scales = torch.from_numpy(rng.integers(0x34, 0x3C, (rows, K // 16), dtype=np.uint8)).cuda()
    return m.FP4Weight(codes, scales, "nvfp4", sigma / 2.99)


@pytest.mark.parametrize("between", ["swiglu", "linear", "route", "route_small", "route_large", "select"])
def test_resident_layers_with_another_kernel_between(m, between):
    """A layer's y is the next layer's x, with a kernel between them that does not write it: the next
    layer's early read of x finds y complete, whatever the kernel between lets start when."""
    T, w = 4, workload(512, 256, 16, 2, 2)
    pool, lo = full_pool(m, w, T)
    try:
        wr = [bf16(gen.router_weight(w, l)) for l in range(2)]
        gate, up, head = matrix(m, 64, w.H, 1), matrix(m, 64, w.H, 2), matrix(m, 48, w.H, 3)
        h, logits = torch.empty((T, 64), device="cuda"), torch.empty((T, 48), device="cuda")
        many = torch.randn((40, w.H), device="cuda").bfloat16()
        n = 40 if between == "route_large" else T
        idx, wt = torch.empty((n, 2), dtype=torch.int32, device="cuda"), torch.empty((n, 2), device="cuda")
        ws = torch.zeros(m.route_grouped_workspace_bytes(40, w.E), dtype=torch.uint8, device="cuda")
        ws0 = torch.zeros(m.route_workspace_bytes(T, w.E), dtype=torch.uint8, device="cuda")
        given = torch.randn((T, w.E), device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")

        def layer(l, x, y):
            m.decode_resident(pool, l, x.view(1, T, w.H), [wr[l]], None, 1, lo.idx, lo.w, lo.slot_of, lo.y_part,
                              y.view(1, T, w.H), st)

        def kernel(y):
            if between == "swiglu":
                m.fp4_swiglu(y, gate, up, h, st)
            elif between == "linear":
                m.fp4_linear(y, head, logits, st)
            elif between == "route":
                m.route(y, wr[1], None, 2, 1, idx, wt, ws0)
            elif between == "route_small":
                m.route_grouped(y, wr[1], idx, wt, ws)
            elif between == "route_large":
                m.route_grouped(many, wr[1], idx, wt, ws)
            else:
                m.route_select(given, idx, wt)

        xs = [bf16(gen.activations(w, 0, s, T)) for s in range(20)]
        want = []
        for x in xs:
            y0, y1 = torch.empty_like(x), torch.empty_like(x)
            layer(0, x, y0)
            torch.cuda.synchronize()
            layer(1, y0, y1)
            torch.cuda.synchronize()
            want.append(y1)
        y0 = torch.zeros_like(xs[0])
        got = [torch.empty_like(x) for x in xs]
        for x, y1 in zip(xs, got):
            layer(0, x, y0)
            kernel(y0)
            layer(1, y0, y1)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    finally:
        pool.close()


def shared_expert(m, H, I, seed):
    return m.SharedExpert(matrix(m, I, H, seed), matrix(m, I, H, seed + 1), matrix(m, H, I, seed + 2))


def test_shared_expert_of_a_layer_on_another_stream(m):
    """The scratch for h is allocated inside the call.  Memory that the current stream has freed but is
    still to write belongs to that stream, not to the layer's."""
    T, w, I = 4, workload(512, 256, 16, 2, 1), 4096
    pool, lo = full_pool(m, w, T)
    try:
        sh, wr = shared_expert(m, w.H, I, 4), bf16(gen.router_weight(w, 0))
        x = bf16(gen.activations(w, 0, 0, T))
        want = lo(0, x, wr, None, shared=sh).clone()
        torch.cuda.synchronize()
        other = torch.cuda.Stream()
        for i in range(3):
            fresh = m.DecodeLayer(pool, T)
            torch.cuda.synchronize()
            # on the current stream: a long wait, then writes to blocks of h's size, which are free for
            # later work of that stream from here on
            old = [torch.empty(T * I, device="cuda") for _ in range(8)]
            torch.cuda._sleep(20_000_000)
            for t in old:
                t.fill_(float("nan"))
            at = {t.data_ptr() for t in old}
            del old, t
            got = fresh(0, x, wr, None, stream=other, shared=sh)
            assert fresh._h[-1].data_ptr() not in at
            other.synchronize()
            torch.cuda.synchronize()
            assert int(fresh.status.item()) == 0 and torch.equal(got, want)
    finally:
        pool.close()


@pytest.mark.parametrize("native", [True, False])
@pytest.mark.parametrize("grouped", [True, False])
def test_a_layer_takes_the_buffer_it_returned(m, native, grouped):
    """y of one call as x of the next, with a shared expert: the same bits as from a copy of y."""
    T, w = 4, workload(512, 256, 16, 2, 3)
    pool, _ = full_pool(m, w, T)
    try:
        routing = m.GroupedRouting(n_group=4, topk_group=2, group_top=2) if grouped else None
        lo = m.DecodeLayer(pool, T, router=routing)
        if not native:
            lo.ffn_events = []
        sh, wr = shared_expert(m, w.H, 320, 7), [bf16(gen.router_weight(w, l)) for l in range(w.L)]
        x = bf16(gen.activations(w, 0, 0, T))
        want = [x]
        for l in range(w.L):
            want.append(lo(l, want[-1], wr[l], None, shared=sh).clone())
            torch.cuda.synchronize()
        y = x
        for l in range(w.L):
            y = lo(l, y, wr[l], None, shared=sh)
            assert torch.equal(y, want[l + 1])
        for l in range(w.L):
            y = lo(l, x if l == 0 else y, wr[l], None, shared=sh)
        assert torch.equal(y, want[-1]) and int(lo.status.item()) == 0
    finally:
        pool.close()
