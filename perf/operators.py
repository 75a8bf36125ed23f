"""What is measured of the routing and 4-bit product operators.

`listed()` names the cases, `draw(rng)` draws more of the same ranges, `prepare`
makes a case's inputs, `run` makes one pass: with `own` set, through the
library's entry points (route_grouped, route_select, fp4_linear, fp4_swiglu),
otherwise as elementary torch operations.  `exact` is the operators' definition
in 64 bits, written apart from the plain form.
"""
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"mxfp4": 32, "nvfp4": 16}
# tensor scale of weights drawn from N(0, 0.02): largest of many draws over 6 * 448
NVFP4_TENSOR_SCALE = float(np.float32(5.5 * 0.02 / (6.0 * 448.0)))


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token of the 284B-shaped layer, scored as large expert counts are:
        # sigmoid, a selection bias, 4 of 8 groups by their two best experts
        dict(name="route_t1_sigmoid", op="route", T=1, H=4096, E=256, k=6, score="sigmoid", bias=True,
             n_group=8, topk_group=4, group_top=2, renormalize=True, scale=2.5),
        # a decode batch of the 35B-shaped layer, plain softmax scores
        dict(name="route_t8_softmax", op="route", T=8, H=2048, E=128, k=8, score="softmax", bias=False,
             n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0),
        # its 2048-token prompt, groups by their best expert, weights not renormalised
        dict(name="route_prompt", op="route", T=2048, H=2048, E=128, k=8, score="softmax", bias=False,
             n_group=8, topk_group=3, group_top=1, renormalize=False, scale=16.0),
        # a long prompt chunk of the 284B-shaped layer
        dict(name="route_long", op="route", T=8192, H=4096, E=256, k=8, score="sigmoid", bias=True,
             n_group=8, topk_group=4, group_top=2, renormalize=True, scale=2.5),
        # logits a program already has: a decode batch, and a ragged prompt in bf16
        dict(name="select_t16", op="select", T=16, E=256, k=8, dtype="fp32", pad=0, score="sigmoid", bias=True,
             n_group=8, topk_group=4, group_top=2, renormalize=True, scale=2.5),
        dict(name="select_ragged", op="select", T=4093, E=160, k=6, dtype="bf16", pad=8, score="softmax",
             bias=False, n_group=8, topk_group=3, group_top=1, renormalize=False, scale=16.0),
        # a projection of the 284B-shaped layer's width, one token, added to a residual
        dict(name="linear_t1_square", op="linear", T=1, N=4096, K=4096, fmt="mxfp4", x="bf16", y="bf16",
             add=True),
        # odd output and block counts, three tokens, fp32 in and out
        dict(name="linear_t3_ragged", op="linear", T=3, N=5003, K=2080, fmt="nvfp4", x="fp32", y="fp32",
             add=False),
        # the output head over a large vocabulary, one token and a full decode batch
        dict(name="linear_t1_head", op="linear", T=1, N=131072, K=4096, fmt="nvfp4", x="bf16", y="fp32",
             add=False),
        dict(name="linear_t16_head", op="linear", T=16, N=100003, K=4096, fmt="mxfp4", x="bf16", y="fp32",
             add=False),
        # the always-active expert beside the routed ones: SwiGLU, down, plus their result
        dict(name="shared_t1", op="shared", T=1, H=2048, I=768, fmt="nvfp4"),
        dict(name="shared_t8", op="shared", T=8, H=4096, I=2048, fmt="mxfp4"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_choice(rng, case):
    """Scores, groups and weights of a router over E = n_group * size experts."""
    n_group = rng.choice([1, 1, 2, 4, 8, 8])
    size = _log_int(rng, 8, 256 // n_group if n_group > 2 else 128)
    topk_group = rng.randint(1, n_group)
    group_top = rng.choice([1, 2])
    case.update(E=n_group * size, n_group=n_group, topk_group=topk_group, group_top=group_top,
                k=rng.randint(1, min(8, topk_group * size)), score=rng.choice(["sigmoid", "softmax"]),
                bias=rng.random() < 0.5, renormalize=rng.random() < 0.5, scale=rng.choice([1.0, 2.5, 16.0]))
    return case


def draw(rng):
    op = rng.choice(["route", "route", "select", "linear", "linear", "shared"])
    if op == "route":
        return _draw_choice(rng, dict(op=op, T=_log_int(rng, 1, 8192), H=256 * _log_int(rng, 1, 16)))
    if op == "select":
        return _draw_choice(rng, dict(op=op, T=_log_int(rng, 1, 8192), dtype=rng.choice(["fp32", "bf16"]),
                                      pad=rng.choice([0, 1, 8])))
    fmt = rng.choice(["mxfp4", "nvfp4"])
    if op == "shared":
        return dict(op=op, T=rng.randint(1, 16), H=32 * _log_int(rng, 8, 128), I=32 * _log_int(rng, 2, 64),
                    fmt=fmt)
    K = 32 * _log_int(rng, 4, 256)
    return dict(op=op, T=rng.randint(1, 16), N=_log_int(rng, 60, min(131072, 100003 * 4096 // K)), K=K, fmt=fmt,
                x=rng.choice(["bf16", "bf16", "fp32"]), y=rng.choice(["bf16", "fp32"]),
                add=rng.random() < 0.5)


def work(case):
    T, op = case["T"], case["op"]
    width = {"bf16": 2, "fp32": 4}
    if op == "route":
        H, E, k = case["H"], case["E"], case["k"]
        return {"bytes": (T + E) * H * 2 + (E * 4 if case["bias"] else 0) + T * k * 8, "flops": 2 * T * H * E}
    if op == "select":
        E, k = case["E"], case["k"]
        return {"bytes": T * E * width[case["dtype"]] + (E * 4 if case["bias"] else 0) + T * k * 8,
                "flops": 4 * T * E}
    per = 0.5 + 1.0 / BLOCK[case["fmt"]]
    if op == "linear":
        N, K = case["N"], case["K"]
        return {"bytes": int(N * K * per) + T * K * width[case["x"]]
                + T * N * width[case["y"]] * (2 if case["add"] else 1), "flops": 2 * T * N * K}
    H, I = case["H"], case["I"]
    return {"bytes": int(3 * H * I * per) + T * H * 2 * 3 + T * I * 4, "flops": 6 * T * H * I}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _weight(g, rows, K, fmt):
    """Codes [rows, K/2], block scales [rows, K/bs] and the tensor scale.  MXFP4:
    uniform codes, exponents -10 to -6; NVFP4: N(0, 0.02) weights, quantised."""
    if fmt == "mxfp4":
        codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda", generator=g)
        scales = torch.randint(117, 122, (rows, K // 32), dtype=torch.uint8, device="cuda", generator=g)
        return codes, scales, 1.0
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, K // 16), dtype=torch.uint8, device="cuda")
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    step = max(1, (1 << 26) // K)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        v = torch.randn((n, K // 16, 16), device="cuda", generator=g) * 0.02
        s8 = (v.abs().amax(2) / (6.0 * NVFP4_TENSOR_SCALE)).clamp_(2.0 ** -6, 448.0).to(torch.float8_e4m3fn)
        scales[r:r + n] = s8.view(torch.uint8)
        q = v / (s8.float() * NVFP4_TENSOR_SCALE).unsqueeze(2)
        c = torch.bucketize(q.abs(), mid, out_int32=True).to(torch.uint8) | ((q < 0).to(torch.uint8) << 3)
        c = c.view(n, K // 2, 2)
        codes[r:r + n] = c[..., 0] | (c[..., 1] << 4)
    return codes, scales, NVFP4_TENSOR_SCALE


_DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _router_out(case, st):
    T, E, k = case["T"], case["E"], case["k"]
    st["idx"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
    st["w"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
    st["keys"] = dict(score=case["score"], n_group=case["n_group"], topk_group=case["topk_group"],
                      group_top=case["group_top"], renormalize=case["renormalize"], scale=case["scale"])


def prepare(case, seed):
    g = _gen(seed)
    op, T = case["op"], case["T"]
    st = dict(case=case)
    randn = lambda *s: torch.randn(s, device="cuda", generator=g)
    if op in ("route", "select"):
        E = case["E"]
        st["bias"] = (torch.rand(E, device="cuda", generator=g) - 0.5) * 0.2 if case["bias"] else None
        _router_out(case, st)
        if op == "route":
            st["x"] = randn(T, case["H"]).bfloat16()
            st["wr"] = (randn(E, case["H"]) * 0.02).bfloat16()
            if own:
                import expert_offload_fp4_b200 as m
                st["ws"] = torch.zeros(m.route_grouped_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
        else:
            st["logits"] = randn(T, E + case["pad"]).to(_DTYPE[case["dtype"]])[:, :E]
        return st
    fmt = case["fmt"]
    if op == "linear":
        weights = {"W": _weight(g, case["N"], case["K"], fmt)}
        st["x"] = randn(T, case["K"]).to(_DTYPE[case["x"]])
        st["add"] = randn(T, case["N"]).to(_DTYPE[case["y"]]) if case["add"] else None
        st["y"] = torch.empty((T, case["N"]), dtype=_DTYPE[case["y"]], device="cuda")
    else:
        H, I = case["H"], case["I"]
        weights = {"gate": _weight(g, I, H, fmt), "up": _weight(g, I, H, fmt), "down": _weight(g, H, I, fmt)}
        st["x"] = randn(T, H).bfloat16()
        st["routed"] = randn(T, H).bfloat16()
        st["h"] = torch.empty((T, I), dtype=torch.float32, device="cuda")
        st["y"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    st["weights"] = weights
    if own:
        import expert_offload_fp4_b200 as m
        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        for name, (codes, scales, ts) in weights.items():
            st[name] = m.FP4Weight(codes, scales, fmt, ts)
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    if own:
        return _run_own(case["op"], st)
    if case["op"] == "route":
        # neighbouring selection values are often closer than fp32 sums tell apart
        return _plain_select(st["x"].double() @ st["wr"].double().t(), st["bias"], case)
    if case["op"] == "select":
        return _plain_select(st["logits"].double(), st["bias"], case)
    if case["op"] == "linear":
        y = st["x"].float() @ _plain_weight(st["weights"]["W"]).t()
        if st["add"] is not None:
            y = y + st["add"].float()
        return y.to(st["y"].dtype)
    x = st["x"].float()
    gate, up = x @ _plain_weight(st["weights"]["gate"]).t(), x @ _plain_weight(st["weights"]["up"]).t()
    h = gate / (1.0 + torch.exp(-gate)) * up
    y = st["routed"].float() + h @ _plain_weight(st["weights"]["down"]).t()
    return h, y.bfloat16()


def _run_own(op, st):
    import expert_offload_fp4_b200 as m
    if op == "route":
        m.route_grouped(st["x"], st["wr"], st["idx"], st["w"], st["ws"], bias=st["bias"], **st["keys"])
        return st["idx"], st["w"]
    if op == "select":
        m.route_select(st["logits"], st["idx"], st["w"], bias=st["bias"], **st["keys"])
        return st["idx"], st["w"]
    if op == "linear":
        m.fp4_linear(st["x"], st["W"], st["y"], st["status"], add=st["add"])
        return st["y"]
    m.fp4_swiglu(st["x"], st["gate"], st["up"], st["h"], st["status"])
    m.fp4_linear(st["h"], st["down"], st["y"], st["status"], add=st["routed"])
    return st["h"], st["y"]


def _plain_weight(weight):
    codes, scales, ts = weight
    rows, K = codes.shape[0], codes.shape[1] * 2
    nib = torch.stack((codes & 15, codes >> 4), 2).view(rows, K)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = table[nib.int()]
    bs = K // scales.shape[1]
    s = torch.exp2(scales.float() - 127.0) if bs == 32 else scales.view(torch.float8_e4m3fn).float()
    return (v.view(rows, K // bs, bs) * s.unsqueeze(2)).view(rows, K) * ts


def _plain_select(logits, bias, case):
    T, E = logits.shape
    G, k = case["n_group"], case["k"]
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-logits))
    else:
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        s = e / e.sum(1, keepdim=True)
    c = s if bias is None else s + bias.double()
    if G > 1:
        top = torch.sort(c.view(T, G, E // G), dim=2, descending=True).values[..., :case["group_top"]].sum(2)
        kept = torch.sort(top, dim=1, descending=True, stable=True).indices[:, :case["topk_group"]]
        mask = torch.zeros((T, G), dtype=torch.bool, device=c.device).scatter_(1, kept, True)
        c = c.masked_fill(~mask.repeat_interleave(E // G, 1), -math.inf)
    idx = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(s, 1, idx)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return idx.int(), (w * case["scale"]).float()


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_weight(codes, scales, ts, fmt):
    half = np.array(E2M1)
    pair = np.concatenate((half, -half))
    lut = torch.from_numpy(np.stack((np.tile(pair, 16), np.repeat(pair, 16)), 1)).to(codes.device)
    w = lut[codes.long()].flatten(1)
    b = scales.long()
    if fmt == "mxfp4":
        s = torch.ldexp(torch.ones_like(b, dtype=torch.float64), b - 127)
    else:
        ex, man = (b >> 3) & 15, (b & 7).double()
        s = torch.where(ex == 0, man / 512.0, torch.ldexp(1.0 + man / 8.0, ex - 7))
    return w * s.repeat_interleave(BLOCK[fmt], 1) * ts


def _exact_product(x, weight, fmt):
    codes, scales, ts = weight
    rows, K = codes.shape[0], codes.shape[1] * 2
    out = torch.empty((x.shape[0], rows), dtype=torch.float64, device=x.device)
    step = max(1, (1 << 26) // K)
    for r in range(0, rows, step):
        out[:, r:r + step] = x @ _exact_weight(codes[r:r + step], scales[r:r + step], ts, fmt).t()
    return out


def _exact_choice(logits, bias, case):
    """Row by row from the definition: explicit keys, sorted by (-value, index)."""
    l = logits.cpu().numpy()
    T, E = l.shape
    if case["score"] == "sigmoid":
        s = np.where(l >= 0, 1.0 / (1.0 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1.0 + np.exp(-np.abs(l))))
    else:
        d = l - l.max(1)[:, None]
        s = np.exp(d - np.log(np.exp(d).sum(1))[:, None])
    c = s + (0.0 if bias is None else bias.double().cpu().numpy())
    size, m = E // case["n_group"], case["group_top"]
    group = np.partition(c.reshape(T, -1, size), size - m, 2)[..., size - m:].sum(2)
    idx = np.empty((T, case["k"]), np.int32)
    for t in range(T):
        keep = np.lexsort((np.arange(group.shape[1]), -group[t]))[:case["topk_group"]]
        cand = np.sort(np.concatenate([np.arange(q * size, (q + 1) * size) for q in keep]))
        idx[t] = cand[np.lexsort((cand, -c[t, cand]))[:case["k"]]]
    w = np.take_along_axis(s, idx.astype(np.int64), 1)
    if case["renormalize"]:
        w = w / w.sum(1, keepdims=True)
    return torch.from_numpy(idx).to(logits.device), torch.from_numpy(w * case["scale"]).to(logits.device)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "route":
        x, wr = st["x"].double(), st["wr"].double()
        return _exact_choice(torch.stack([x @ row for row in wr], 1), st["bias"], case)
    if case["op"] == "select":
        return _exact_choice(st["logits"].double(), st["bias"], case)
    if case["op"] == "linear":
        y = _exact_product(st["x"].double(), st["weights"]["W"], case["fmt"])
        return y if st["add"] is None else y + st["add"].double()
    x = st["x"].double()
    gate = _exact_product(x, st["weights"]["gate"], case["fmt"])
    h = gate * torch.sigmoid(gate) * _exact_product(x, st["weights"]["up"], case["fmt"])
    return h, st["routed"].double() + _exact_product(h, st["weights"]["down"], case["fmt"])
