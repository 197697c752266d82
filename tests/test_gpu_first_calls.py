"""GPU tests, each in a process of its own, of what the first call of an entry point sets up: the products do not take the
mixture of experts' workspace, and a first call may stand in a graph's capture once any entry point has run."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
START = """
import torch as t
import gemm_rocmfp4_dequant_gb300 as rf4
K, I, E = 256, 256, 4
g = t.Generator(device="cuda")
g.manual_seed(0)
X = t.randn(2, K, generator=g, device="cuda").half()
W = rf4.quantize(t.randn(64, K, generator=g, device="cuda").half())
router = t.randn(E, K, generator=g, device="cuda")
gu = t.randint(0, 24, (E * 2 * I * rf4.row_bytes(K, 0),), generator=g, device="cuda", dtype=t.uint8)
dn = t.randint(0, 24, (E * K * rf4.row_bytes(I, 0),), generator=g, device="cuda", dtype=t.uint8)
Y = t.zeros(2, K, device="cuda")
ids, probs = t.zeros(2, 2, dtype=t.int32, device="cuda"), t.zeros(2, 2, device="cuda")
y = t.zeros(2, K, device="cuda").half()
w = t.ones(K, device="cuda")
rf4.gemm(W, X, 64, K)
t.cuda.synchronize()
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def run(body):
    r = subprocess.run([sys.executable, "-c", START + body], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("done"), r.stdout[-2000:] + r.stderr[-2000:]


def test_workspace_of_the_experts_comes_with_their_first_call():
    run("""
free = t.cuda.mem_get_info()[0]
rf4.moe(X, router, gu, dn, I, 2, Y=Y, ids=ids, probs=probs)
t.cuda.synchronize()
after = t.cuda.mem_get_info()[0]
assert free - after >= 36 << 20, (free, after)
first = Y.clone()
free = t.cuda.mem_get_info()[0]
rf4.moe(X, router, gu, dn, I, 2, Y=Y, ids=ids, probs=probs)
t.cuda.synchronize()
assert t.cuda.mem_get_info()[0] == free and t.equal(first, Y)
rf4.load().rocmfp4_shutdown()
Y.zero_()
rf4.moe(X, router, gu, dn, I, 2, Y=Y, ids=ids, probs=probs)
assert t.equal(first, Y) and rf4.device_error_bits() == 0
print("done")
""")


def test_first_calls_in_a_capture():
    run("""
graph = t.cuda.CUDAGraph()
with t.cuda.graph(graph):
    rf4.add_rmsnorm(X, w, y=y)
    rf4.moe(y, router, gu, dn, I, 2, Y=Y, ids=ids, probs=probs)
graph.replay()
t.cuda.synchronize()
want = rf4.moe(rf4.add_rmsnorm(X, w, dtype=t.float16).y, router, gu, dn, I, 2)
assert t.equal(want[0], Y) and t.equal(want[1], ids) and float(Y.abs().max()) > 0 and rf4.device_error_bits() == 0
print("done")
""")
