"""GPU tests of rocmfp4_moe with many experts and many tokens together, against the layer in 64 bits.

Activations are small integers and router weights multiples of 1/32, so that logits are exact in fp32 whatever the order of the
sum (below 2^24 units) and the choice is exact too, ties included (lowest expert first).  The tolerance is that of the layer's
other tests: a product's sum is off by at most 80 u (u = 2^-24) of the sum of its terms' magnitudes, with a = |Wg| |x|,
b = |Wu| |x|, |SiLU'| <= 1.1 and |SiLU(g)| <= |g|
    |dh| <= 88 u a |u| + 80 u |SiLU(g)| b + 16 u |h|,   |dY| <= sum_j p_j (|Wd| |dh_j| + (100 u + 2^-20) |Wd| |h_j|),
and the whole output's relative L2 error is at most 1e-5."""
import pytest

import gemm_rocmfp4_dequant_gb300 as rf4
from gpu_util import REL_L2, torch
from test_gpu_moe import blocks

pytestmark = pytest.mark.gpu

DUAL, FAST = rf4.DUAL, rf4.FAST
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    assert rf4.device_error_bits() == 0


def make(M, E, K, I, variant, act, seed):
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    X = t.randint(-4, 5, (M, K), generator=g, device="cuda").to(t.float16 if act == 0 else t.bfloat16)
    router = (t.randint(-16, 17, (E, K), generator=g, device="cuda") / 32.0).to(t.bfloat16)
    return X, router, blocks(t, E * 2 * I, K, variant, g), blocks(t, E * K, I, variant, g)


def run_and_check(M, E, k, K, I, variant, act, route, seed):
    t = torch()
    X, router, Wgu, Wd = make(M, E, K, I, variant, act, seed)
    Y, ids, probs = rf4.moe(X, router, Wgu, Wd, I, k, variant, route)
    logits = X.double() @ router.double().T
    order = t.argsort(-logits, dim=1, stable=True)[:, :k]
    assert t.equal(ids.long(), order)
    best = logits.gather(1, order)
    if route == rf4.ROUTE_SOFTMAX:
        p = t.softmax(logits, 1).gather(1, order)
    elif route == rf4.ROUTE_SOFTMAX_TOPK:
        p = t.softmax(best, 1)
    else:
        p = t.sigmoid(best)
        p = p / p.sum(1, keepdim=True)
    assert bool(((probs.double() - p).abs() <= 2e-5 * p + 1e-37).all())
    rows_gu, rows_dn = Wgu.view(E, -1), Wd.view(E, -1)
    ref, bound = (t.zeros(M, K, dtype=t.float64, device="cuda") for _ in range(2))
    for e in t.unique(order).tolist():
        m, j = t.nonzero(order == e, as_tuple=True)
        w, d = rf4.dequant(rows_gu[e], 2 * I, K, variant).double(), rf4.dequant(rows_dn[e], K, I, variant).double()
        both, mag = X[m].double() @ w.T, X[m].double().abs() @ w.abs().T
        g, u = both[:, :I], both[:, I:]
        s = g * t.sigmoid(g)
        h = s * u
        dh = 88 * U * mag[:, :I] * u.abs() + 80 * U * s.abs() * mag[:, I:] + 16 * U * h.abs()
        pj = p[m, j][:, None]
        ref.index_add_(0, m, pj * (h @ d.T))
        bound.index_add_(0, m, pj * ((dh + (100 * U + 2.0 ** -20) * h.abs()) @ d.abs().T))
    err = (Y.double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    assert float(err.norm() / ref.norm()) <= REL_L2


@pytest.mark.parametrize("variant", [DUAL, FAST])
@pytest.mark.parametrize("K,I", [(512, 512), (96, 160)])
@pytest.mark.parametrize("M,E,k", [(13, 410, 8), (16, 512, 8), (16, 497, 2), (17, 413, 8), (20, 512, 16), (21, 281, 8), (24, 384, 8), (32, 298, 8),
                                   (32, 384, 6), (32, 512, 1), (32, 512, 8), (32, 512, 16), (31, 511, 10)])
def test_many_experts_and_tokens(M, E, k, K, I, variant):
    """Aligned and unaligned rows; the selection's room is larger than the ring."""
    run_and_check(M, E, k, K, I, variant, (M + k) % 2, (M + E) % 3, seed=M * 1000 + E)


@pytest.mark.parametrize("variant", [DUAL, FAST])
@pytest.mark.parametrize("M", [9, 16, 17, 24, 32])
def test_rings_of_few_stages(M, variant):
    """The copies' ring has one or two stages at these tokens; several spans a row."""
    run_and_check(M, 64, 8, 1536, 1024, variant, M % 2, rf4.ROUTE_SOFTMAX_TOPK, seed=M)
    run_and_check(M, 40, 6, 1056, 352, variant, 1 - M % 2, rf4.ROUTE_SIGMOID, seed=M + 50)


def test_all_logits_equal():
    """Every expert is a candidate for every token."""
    t = torch()
    X, _, Wgu, Wd = make(32, 512, 64, 64, DUAL, 0, 1)
    _, ids, probs = rf4.moe(X, t.zeros(512, 64, device="cuda"), Wgu, Wd, 64, 16, DUAL)
    assert bool((ids == t.arange(16, device="cuda")).all()) and bool((probs == 1 / 16).all())


@pytest.mark.parametrize("variant", [DUAL, FAST])
def test_matrices_past_31_bits(variant):
    """Matrices of more than 2^31 bytes: the last experts' rows lie past 32-bit offsets."""
    t = torch()
    M, E, k, K, I = 3, 160, 2, 7168, 2048
    X, router, Wgu, Wd = make(M, E, K, I, variant, 0, 77)
    assert Wgu.numel() > 1 << 31
    router[:] = 0
    router[E - 1, :] = X[0].bfloat16() / 64
    router[E - 2, :] = X[1].bfloat16() / 64
    router[0, :] = X[2].bfloat16() / 64
    Y, ids, probs = rf4.moe(X, router, Wgu, Wd, I, k, variant)
    logits = X.double() @ router.double().T
    order = t.argsort(-logits, dim=1, stable=True)[:, :k]
    assert t.equal(ids.long(), order) and ids[:, 0].tolist() == [E - 1, E - 2, 0]
    p = t.softmax(logits.gather(1, order), 1)
    for m in range(M):
        ref = t.zeros(K, dtype=t.float64, device="cuda")
        for j, e in enumerate(order[m].tolist()):
            both = rf4.dequant(Wgu.view(E, -1)[e], 2 * I, K, variant).double() @ X[m].double()
            h = both[:I] * t.sigmoid(both[:I]) * both[I:]
            ref += p[m, j] * (rf4.dequant(Wd.view(E, -1)[e], K, I, variant).double() @ h)
        assert float((Y[m].double() - ref).norm() / ref.norm()) <= REL_L2
