"""GPU test, in a process of its own, of attention over a paged cache whose first call stands in a graph's capture: two graphs,
one for each of its kernels, share the workspace that the capture made, replayed in turn and after it was freed and made anew."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BODY = """
import sys
sys.path.insert(0, "tests")
import torch as t
import gemm_rocmfp4_dequant_gb300 as rf4
import paged_util as pu
few = pu.Paged([1, 1], [5000, 77], 2, 64, 16, 0, seed=1)
many = pu.Paged([150, 40], [5000, 77], 2, 64, 16, 0, seed=2)
qs = [p.queries(8, t.float16) for p in (few, many)]
outs = [t.zeros(q.shape, dtype=t.float16, device="cuda") for q in qs]
rf4.cache_read(few.cache, rows=few.m)  # the shared workspace: never in a capture
t.cuda.synchronize()
free = t.cuda.mem_get_info()[0]
graphs = []
for p, q, out in zip((few, many), qs, outs):
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        rf4.paged_attention(q, p.cache, 0.125, out=out)
    graphs.append(graph)
assert free - t.cuda.mem_get_info()[0] >= 50 << 20
for i in (0, 1, 0, 0, 1):
    outs[i].zero_()
    graphs[i].replay()
want = []
for p, q, out in zip((few, many), qs, outs):
    ref, tol = p.attention(q, 0.125)
    assert bool(((out.double() - ref).abs() <= tol + pu.rounding(ref, t.float16) * (1 + 2.0 ** -6)).all())
    want.append(out.clone())
del graphs
t.cuda.synchronize()
rf4.load().rocmfp4_shutdown()
for p, q, w in zip((few, many), qs, want):
    assert t.equal(rf4.paged_attention(q, p.cache, 0.125), w)
assert rf4.device_error_bits() == 0
print("done")
"""


def test_first_call_in_a_capture():
    import __graft_entry__
    __graft_entry__.build()
    r = subprocess.run([sys.executable, "-c", BODY], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("done"), r.stdout[-2000:] + r.stderr[-2000:]
