"""Routers and products called from several threads at once, their first calls included."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

RUN = """
import threading
import torch
import expert_offload_fp4_b200 as m

shapes = [(1, 64), (6, 200), (40, 96), (300, 1024)]
cases = []
for i, (T, E) in enumerate(shapes * 2):
    g = torch.Generator(device="cuda").manual_seed(i % len(shapes))
    x = torch.randn((T, 512), device="cuda", generator=g).bfloat16()
    wr = (torch.randn((E, 512), device="cuda", generator=g) * 0.05).bfloat16()
    codes = torch.randint(0, 256, (E, 256), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(110, 122, (E, 16), dtype=torch.uint8, device="cuda", generator=g)
    cases.append(dict(x=x, wr=wr, W=m.FP4Weight(codes, scales, "mxfp4"), idx=torch.empty((T, 4), dtype=torch.int32, device="cuda"),
                      w=torch.empty((T, 4), device="cuda"), y=torch.empty((min(T, 16), E), device="cuda"),
                      ws=torch.zeros(m.route_grouped_workspace_bytes(T, E), dtype=torch.uint8, device="cuda"),
                      st=torch.zeros(1, dtype=torch.int32, device="cuda"), stream=torch.cuda.Stream()))
torch.cuda.synchronize()
start, errors = threading.Barrier(len(cases)), []


def work(c):
    try:
        start.wait()
        for _ in range(10):
            m.route_grouped(c["x"], c["wr"], c["idx"], c["w"], c["ws"], stream=c["stream"])
            m.fp4_linear(c["x"][:16], c["W"], c["y"], c["st"], stream=c["stream"])
    except Exception as e:
        errors.append(e)


threads = [threading.Thread(target=work, args=(c,)) for c in cases]
for t in threads:
    t.start()
for t in threads:
    t.join()
torch.cuda.synchronize()
assert not errors, errors
half = len(shapes)
for a, b in zip(cases[:half], cases[half:]):
    assert int(a["st"].item()) == 0 and int(b["st"].item()) == 0
    for k in ("idx", "w", "y"):
        assert torch.equal(a[k], b[k]), k
    l = a["x"].double() @ a["wr"].double().t()
    assert torch.equal(a["idx"].long(), l.topk(4, 1).indices)
print("threads ok")
"""

FIRST = """
import threading
import torch
import expert_offload_fp4_b200 as m

x, wr = torch.randn((40, 256), device="cuda").bfloat16(), torch.randn((16, 256), device="cuda").bfloat16()
W = m.FP4Weight(torch.zeros((64, 128), dtype=torch.uint8, device="cuda"), torch.zeros((64, 8), dtype=torch.uint8, device="cuda"), "mxfp4")
idx, w = torch.empty((40, 2), dtype=torch.int32, device="cuda"), torch.empty((40, 2), device="cuda")
ws = torch.zeros(m.route_grouped_workspace_bytes(40, 16), dtype=torch.uint8, device="cuda")
y, st = torch.empty((8, 64), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
calls = dict(route=lambda: m.route_grouped(x, wr, idx, w, ws), linear=lambda: m.fp4_linear(x[:8], W, y, st),
             swiglu=lambda: m.fp4_swiglu(x[:8], W, W, y, st))
errors = []


def work(f):
    try:
        f()
    except Exception as e:
        errors.append(e)


for f in calls.values():
    t = threading.Thread(target=work, args=(f,))
    t.start()
    t.join()
torch.cuda.synchronize()
assert not errors, errors
print("threads ok")
"""


@pytest.mark.parametrize("run", [FIRST, RUN], ids=["a_thread_for_each_call", "eight_threads"])
def test_calls_from_fresh_threads(run):
    from expert_offload_fp4_b200 import build
    build.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", run], cwd=root, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, PYTHONPATH=root))
    assert r.returncode == 0 and "threads ok" in r.stdout, r.stdout + r.stderr
