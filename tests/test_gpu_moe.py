"""GPU tests of rocmfp4_moe against the layer in 64 bits on exactly dequantised weights.

Tolerance, from the arithmetic (u = 2^-24): a product of a row is a sum of exact products (at most 11 significant bits by
11, both exact in fp32) or, for the down product, of products rounded once; a lane adds at most 8 terms a chain, two
chains, two halves, K / 32 / 4 blocks and 5 shuffles: for these K at most 8 + 3 + 64 + 5 additions, so a sum is off by at
most 80 u of the sum of its terms' magnitudes.  With a = |Wg| |x| and b = |Wu| |x|, and |SiLU'| <= 1.1, |SiLU(g)| <= |g|,
    |dh| <= 88 u a |u| + 80 u |SiLU(g)| b + 16 u |h|        (expf, a division and two products)
    |dY| <= sum_j p_j (|Wd| |dh_j| + 80 u |Wd| |h_j|) + (dp / p + 20 u) sum_j p_j |Wd| |h_j|,
dp / p <= 2 dl + 2^-20 for a logit's error dl = 40 u sum |r x| (512 threads: at most 8 terms each at these K, then 5 + 16).
The whole output is held to relative L2 error 1e-5 as well, the bar of every product here.  Experts and their order are
exact: the inputs are checked to have no two logits nearer than their errors.
"""
import numpy as np
import pytest

import gemm_rocmfp4_dequant_gb300 as rf4
from gpu_util import REL_L2, torch

pytestmark = pytest.mark.gpu

DUAL, FAST = rf4.DUAL, rf4.FAST
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    assert rf4.device_error_bits() == 0


def blocks(t, rows, k, variant, g, low=0, high=24):
    bb = 18 if variant == DUAL else 17
    w = t.randint(0, 256, (rows, k // 32, bb), generator=g, device="cuda", dtype=t.uint8)
    w[..., 16:] = t.randint(low, high, w[..., 16:].shape, generator=g, device="cuda", dtype=t.uint8)
    return w.view(-1)


def make(M, E, k, K, I, variant, act, rtype, seed):
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    X = t.randn(M, K, generator=g, device="cuda").to(t.float16 if act == 0 else t.bfloat16)
    router = (t.randn(E, K, generator=g, device="cuda") * (2 / K ** 0.5)).to(rtype)
    return X, router, blocks(t, E * 2 * I, K, variant, g), blocks(t, E * K, I, variant, g)


def reference(X, router, Wgu, Wd, I, k, variant, route, scale):
    """(Y, its error bound, ids, probs) in 64 bits."""
    t = torch()
    M, K = X.shape
    E = router.shape[0]
    x, r = X.double(), router.double()
    logits = x @ r.T
    order = t.argsort(-logits, dim=1, stable=True)
    dl = 40 * U * (x.abs() @ r.abs().T).amax(1)
    ranked = logits.gather(1, order)
    for m in range(M):
        if E > k:
            assert float((ranked[m, :k] - ranked[m, 1:k + 1]).min()) > 2 * float(dl[m]), "inputs with a tie"
    ids = order[:, :k]
    best = ranked[:, :k]
    if route == rf4.ROUTE_SOFTMAX:
        p = t.softmax(logits, 1).gather(1, ids)
    elif route == rf4.ROUTE_SOFTMAX_TOPK:
        p = t.softmax(best, 1)
    else:
        p = t.sigmoid(best)
        p = p / p.sum(1, keepdim=True)
    p = p * scale
    gu = rf4.dequant(Wgu, E * 2 * I, K, variant).view(E, 2 * I, K)
    dn = rf4.dequant(Wd, E * K, I, variant).view(E, K, I)
    Y, bound = t.zeros(M, K, dtype=t.float64, device="cuda"), t.zeros(M, K, dtype=t.float64, device="cuda")
    for m in range(M):
        for j in range(k):
            w, d = gu[ids[m, j]].double(), dn[ids[m, j]].double()
            both, mag = w @ x[m], w.abs() @ x[m].abs()
            g, u = both[:I], both[I:]
            s = g * t.sigmoid(g)
            h = s * u
            dh = 88 * U * mag[:I] * u.abs() + 80 * U * s.abs() * mag[I:] + 16 * U * h.abs()
            whole = d.abs() @ h.abs()
            Y[m] += p[m, j] * (d @ h)
            bound[m] += p[m, j].abs() * (d.abs() @ dh + (100 * U + 2 * dl[m] + 2.0 ** -20) * whole)
    return Y, bound, ids, p


def run_and_check(M, E, k, K, I, variant, act, route=rf4.ROUTE_SOFTMAX_TOPK, scale=1.0, rtype=None, seed=0):
    t = torch()
    X, router, Wgu, Wd = make(M, E, k, K, I, variant, act, rtype or t.bfloat16, seed)
    Y, ids, probs = rf4.moe(X, router, Wgu, Wd, I, k, variant, route, scale)
    ref, bound, rids, rp = reference(X, router, Wgu, Wd, I, k, variant, route, scale)
    assert t.equal(ids.long(), rids)
    assert float(((probs.double() - rp).abs() / rp.abs()).max()) < 2e-5
    err = (Y.double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    assert float(err.norm() / ref.norm()) <= REL_L2
    again = rf4.moe(X, router, Wgu, Wd, I, k, variant, route, scale)
    assert all(t.equal(a, b) for a, b in zip((Y, ids, probs), again))


# K, I: whole rows and parts of rows per stage, all lane counts, rows of odd block counts, unaligned rows
SHAPES = [(1, 4, 2, 256, 256), (1, 8, 2, 512, 512), (3, 6, 3, 32, 32), (2, 5, 1, 64, 96), (5, 7, 4, 160, 224), (8, 16, 4, 1024, 768),
          (4, 3, 3, 2048, 96), (13, 10, 3, 1056, 352), (32, 8, 2, 512, 544), (2, 4, 2, 5120, 1536), (1, 2, 1, 7168, 64), (3, 4, 2, 128, 6144)]


@pytest.mark.parametrize("variant", [DUAL, FAST])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_matches_definition(shape, act, variant):
    run_and_check(*SHAPES[shape], variant, act, route=shape % 3, scale=(1.0, 2.5)[shape % 2], seed=100 + shape)


@pytest.mark.parametrize("variant", [DUAL, FAST])
@pytest.mark.parametrize("shape", [(8, 16, 4, 2560, 1536), (6, 12, 6, 512, 2048), (5, 24, 5, 96, 4096), (4, 20, 5, 2464, 1568)])
def test_tile_counts(shape, variant):
    """Output rows that do not deal out evenly over the SMs, and fewer tiles than SMs."""
    run_and_check(*shape, variant, 0, seed=200)


@pytest.mark.parametrize("rtype", ["float32", "float16"])
def test_router_types_and_many_experts(rtype):
    t = torch()
    run_and_check(2, 300, 16, 256, 64, DUAL, 0, rtype=getattr(t, rtype), seed=7)
    run_and_check(9, 512, 8, 512, 32, FAST, 1, rtype=getattr(t, rtype), route=rf4.ROUTE_SIGMOID, seed=8)


def test_every_token_to_every_expert():
    for M in (1, 2, 31, 32):
        run_and_check(M, 3, 3, 256, 128, DUAL, 0, route=rf4.ROUTE_SOFTMAX, seed=M)


def test_every_code_and_scale():
    """Each code byte under every finite scale byte: one token, one expert, K = I = 32 and weights that leave one product
    at a time; sums of a few exact terms agree to fp32 rounding."""
    t = torch()
    for variant in (DUAL, FAST):
        bb = 18 if variant == DUAL else 17
        E, I, K = 127, 32, 32
        Wgu = t.zeros(E, 2 * I, 1, bb, dtype=t.uint8, device="cuda")
        q = t.arange(256, device="cuda", dtype=t.uint8).view(16, 16)
        Wgu[:, :16, 0, :16] = q  # gate rows 0..15: all code bytes, 16 to a row
        Wgu[:, 16:32, 0, :16] = q.flip(0)
        Wgu[:, I:, 0, :16] = 0x11  # up rows: ones
        Wgu[..., 16:] = t.arange(E, device="cuda", dtype=t.uint8)[:, None, None, None]
        Wgu[:, I:, 0, 16:] = 0x40
        Wd = t.zeros(E, K, 1, bb, dtype=t.uint8, device="cuda")
        for n in range(16):  # output n: 1.0 * h[n]
            Wd[:, n, 0, n] = 0x01
            Wd[:, 16 + n, 0, n] = 0x10
        Wd[..., 16:] = 0x40
        X = (2.0 ** t.randint(-3, 3, (32, K), device="cuda").float()).half()
        for part in range(0, E, 32):
            n = min(32, E - part)
            router = t.zeros(E, K, device="cuda")
            x = X[:n].clone()
            # token m chooses expert part + m: a router row that only that token reaches
            x[:, :] = x[0]
            for m in range(n):
                one = router.clone()
                one[part + m] = 1.0
                Y, ids, probs = rf4.moe(x[m:m + 1], one, Wgu.view(-1), Wd.view(-1), I, 1, variant)
                assert int(ids) == part + m and float(probs) == 1.0
                w = rf4.dequant(Wgu[part + m].reshape(-1), 2 * I, K, variant).double()
                both = w @ x[m].double()
                g, u = both[:I], both[I:]
                want = g * t.sigmoid(g) * u
                mag = w.abs() @ x[m].double().abs()
                assert bool(((Y[0].double() - want).abs() <= 40 * U * (mag[:I] * u.abs() + want.abs()) + 1e-30).all())


def test_large_hidden_values():
    """Hidden values far beyond fp16's range keep fp32 accuracy."""
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(5)
    M, E, k, K, I = 3, 4, 2, 512, 256
    X, router, _, _ = make(M, E, k, K, I, DUAL, 1, t.bfloat16, 3)
    X = X * 64
    Wgu, Wd = blocks(t, E * 2 * I, K, DUAL, g, 64, 100), blocks(t, E * K, I, DUAL, g, 64, 100)
    Y, ids, probs = rf4.moe(X, router / 64, Wgu, Wd, I, k, DUAL)
    ref, bound, rids, rp = reference(X, router / 64, Wgu, Wd, I, k, DUAL, 1, 1.0)
    assert t.equal(ids.long(), rids) and float(ref.abs().max()) > 1e9
    assert float((Y.double() - ref).norm() / ref.norm()) <= REL_L2 and bool(((Y.double() - ref).abs() <= bound).all())


def test_ties_and_odd_logits():
    """Equal logits go to the lowest index; NaN orders last; a token's NaN does not reach another token."""
    t = torch()
    X, router, Wgu, Wd = make(4, 6, 2, 256, 64, DUAL, 0, t.bfloat16, 11)
    Y, ids, probs = rf4.moe(X, t.zeros_like(router), Wgu, Wd, 64, 3, DUAL)
    assert ids.tolist() == [[0, 1, 2]] * 4 and bool((probs - 1 / 3).abs().max() < 1e-6)
    want = rf4.moe(X, router, Wgu, Wd, 64, 2, DUAL)
    Xn = X.clone()
    Xn[2, 7] = float("nan")
    got = rf4.moe(Xn, router, Wgu, Wd, 64, 2, DUAL)
    keep = [0, 1, 3]
    assert all(t.equal(a[keep], b[keep]) for a, b in zip(got, want)) and bool(got[0][2].isnan().all())
    assert got[1][2].tolist() == [0, 1]
    r = router.clone()
    r[:, :] = 0
    r[3, :] = float("nan")
    assert 3 not in rf4.moe(X, r, Wgu, Wd, 64, 5, DUAL)[1].flatten().tolist()


def test_writes_stay_inside_and_inputs_untouched():
    t = torch()
    M, E, k, K, I = 3, 5, 2, 96, 160
    X, router, Wgu, Wd = make(M, E, k, K, I, FAST, 0, t.bfloat16, 21)
    keep = [v.clone() for v in (X, router, Wgu, Wd)]
    big = t.full((M * K + 64,), 7.0, device="cuda")
    ids, probs = t.full((M + 2, k), 99, dtype=t.int32, device="cuda"), t.full((M + 2, k), 7.0, device="cuda")
    rf4.moe(X, router, Wgu, Wd, I, k, FAST, Y=big[32:32 + M * K].view(M, K), ids=ids[1:1 + M], probs=probs[1:1 + M])
    assert bool((big[:32] == 7).all()) and bool((big[32 + M * K:] == 7).all())
    assert ids[0].tolist() == [99, 99] and ids[-1].tolist() == [99, 99] and probs[0].tolist() == [7, 7] and probs[-1].tolist() == [7, 7]
    assert all(t.equal(a, b) for a, b in zip(keep, (X, router, Wgu, Wd)))


def test_graph_capture_and_back_to_back():
    """Replays and eager calls on one stream share the workspace and its barrier counters."""
    t = torch()
    a = make(2, 8, 2, 512, 256, DUAL, 0, t.bfloat16, 31)
    b = make(5, 12, 3, 1024, 96, FAST, 1, t.bfloat16, 32)
    wa, wb = rf4.moe(*a, 256, 2, DUAL), rf4.moe(*b, 96, 3, FAST)
    out = tuple(t.empty_like(o) for o in wa)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        rf4.moe(*a, 256, 2, DUAL, Y=out[0], ids=out[1], probs=out[2])
    for _ in range(20):
        graph.replay()
        got = rf4.moe(*b, 96, 3, FAST)
    t.cuda.synchronize()
    assert all(t.equal(x, y) for x, y in zip(out, wa)) and all(t.equal(x, y) for x, y in zip(got, wb))


def test_refusals():
    t = torch()
    X, router, Wgu, Wd = make(2, 4, 2, 64, 64, DUAL, 0, t.bfloat16, 41)
    with pytest.raises(rf4.RocmFP4Error):
        rf4.moe(X, router, Wgu, Wd, 64, 5)
    with pytest.raises(rf4.RocmFP4Error):
        rf4.moe(X, router.double(), Wgu, Wd, 64, 2)
    with pytest.raises(TypeError):
        rf4.moe(X.float(), router, Wgu, Wd, 64, 2)
    with pytest.raises(ValueError):
        rf4.moe(X, router, Wgu[:-18], Wd, 64, 2)
    with pytest.raises(ValueError):
        rf4.moe(X, router[:, :32], Wgu, Wd, 64, 2)
    with pytest.raises(ValueError):
        rf4.moe(X, router, Wgu, Wd, 64, 2, Y=t.empty(2, 32, device="cuda"))
    assert rf4.moe(X[:0], router, Wgu, Wd, 64, 2)[0].shape == (0, 64)
    assert np.isfinite(rf4.moe(X[0], router, Wgu, Wd, 64, 2)[0].cpu().numpy()).all()
