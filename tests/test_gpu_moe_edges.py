"""GPU tests of rocmfp4_moe at the ends of its arithmetic: sigmoid weights of very small logits, hidden values beyond fp32."""
import math

import pytest

import gemm_rocmfp4_dequant_gb300 as rf4
from gpu_util import REL_L2, torch
from test_gpu_moe import blocks

pytestmark = pytest.mark.gpu

DUAL, FAST = rf4.DUAL, rf4.FAST


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()
    yield
    assert rf4.device_error_bits() == 0


def layer(X, ids, p, Wgu, Wd, E, K, I, variant):
    """The chosen experts' products in 64 bits."""
    t = torch()
    ref = t.zeros(X.shape[0], K, dtype=t.float64, device="cuda")
    for m in range(X.shape[0]):
        for e, w in zip(ids[m].tolist(), p[m]):
            both = rf4.dequant(Wgu.view(E, -1)[e], 2 * I, K, variant).double() @ X[m].double()
            h = both[:I] * t.sigmoid(both[:I]) * both[I:]
            ref[m] += w * (rf4.dequant(Wd.view(E, -1)[e], K, I, variant).double() @ h)
    return ref


@pytest.mark.parametrize("low", [1, 20, 80, 88, 90, 100, 200, 255])
def test_sigmoid_weights_of_very_small_logits(low):
    """p = sigmoid(l) / sum of the chosen sigmoids is finite for every finite logit: for l far below 0 a softmax of l.

    Logits are exact: -(low + e) for the first token, twice that for the second, 1 + e above it for the third.  Each weight
    takes an exp() of a rounded argument below 8 (2^-21), one below 1 and three roundings: below 2^-19 of itself."""
    t = torch()
    E, k, K, I = 8, 5, 64, 64
    g = t.Generator(device="cuda")
    g.manual_seed(low)
    X = t.ones(3, K, dtype=t.float16, device="cuda")
    X[1] = 2.0
    X[2] = -0.5
    router = (-(low + t.arange(E, device="cuda").float()) / K)[:, None].expand(E, K).contiguous()
    Wgu, Wd = blocks(t, E * 2 * I, K, DUAL, g), blocks(t, E * K, I, DUAL, g)
    Y, ids, probs = rf4.moe(X, router, Wgu, Wd, I, k, DUAL, rf4.ROUTE_SIGMOID, 1.5)
    logits = X.double() @ router.double().T
    best, order = t.sort(logits, dim=1, descending=True, stable=True)
    assert t.equal(ids.long(), order[:, :k])
    best = best[:, :k]
    # sigmoid(l) = exp(l - top) exp(top) / (1 + exp(l)), of which exp(top) cancels
    p = t.where(best < 0, t.exp(best - best[:, :1]) / (1 + t.exp(best)), t.sigmoid(best))
    p = 1.5 * p / p.sum(1, keepdim=True)
    assert bool(((probs.double() - p).abs() <= 2.0 ** -19 * p).all())
    ref = layer(X, ids, p, Wgu, Wd, E, K, I, DUAL)
    assert float((Y.double() - ref).norm() / ref.norm()) <= REL_L2


def test_sigmoid_weight_of_minus_infinity():
    """A masked expert that is chosen all the same has weight 0 next to finite logits."""
    t = torch()
    E, K, I = 4, 64, 32
    g = t.Generator(device="cuda")
    g.manual_seed(1)
    X = t.ones(1, K, dtype=t.float16, device="cuda")
    router = (-(120.0 + t.arange(E, device="cuda").float()) / K)[:, None].expand(E, K).contiguous()
    router[2] = -math.inf
    Wgu, Wd = blocks(t, E * 2 * I, K, FAST, g), blocks(t, E * K, I, FAST, g)
    Y, ids, probs = rf4.moe(X, router, Wgu, Wd, I, E, FAST, rf4.ROUTE_SIGMOID)
    assert ids.tolist() == [[0, 1, 3, 2]] and float(probs[0, 3]) == 0.0
    p = t.softmax(t.tensor([0.0, -1.0, -3.0], dtype=t.float64, device="cuda"), 0)
    assert bool(((probs[0, :3].double() - p).abs() <= 2.0 ** -19 * p).all()) and bool(Y.isfinite().all())


@pytest.mark.parametrize("variant", [DUAL, FAST])
@pytest.mark.parametrize("K,I", [(512, 512), (96, 64)])
@pytest.mark.parametrize("sign", [1, -1])
def test_infinite_hidden_value(K, I, variant, sign):
    """h[0] = SiLU(2^71) * 2^71 is beyond fp32, h[1] = 2^100 beyond fp16 with the opposite sign in every output: outputs are
    infinite with the sign of h[0]'s weight, and NaN where that weight is 0; a second expert adds finite values, and the other
    tokens are as without the first."""
    t = torch()
    E, bb = 2, 18 if variant == DUAL else 17
    g = t.Generator(device="cuda")
    g.manual_seed(K)
    X = t.randn(3, K, generator=g, device="cuda").bfloat16()
    X[0] = 0.0
    X[0, 0] = 2.0 ** 60
    router = t.zeros(E, K, device="cuda")
    Wgu, Wd = blocks(t, E * 2 * I, K, variant, g).view(E, 2, I, K // 32, bb), blocks(t, E * K, I, variant, g).view(E, K, I // 32, bb)
    Wgu[0] = 0  # expert 0: byte 0's low nibble is column 0
    Wgu[0, :, 0, 0, 0] = 7  # 10 * 224
    Wgu[0, :, 0, 0, 16:] = 0x7E
    Wgu[0, :, 1, 0, 0] = 1  # 2^-10
    Wgu[0, :, 1, 0, 16:] = 1
    if sign < 0:
        Wgu[0, 1, :2, 0, 0] += 8
    Wd[0] = 0
    Wd[0, :, :, 16:] = 0x40
    n = t.arange(K, device="cuda")
    Wd[0, :, 0, 0] = t.where(n % 3 == 0, 1, t.where(n % 3 == 1, 9, 0)).to(t.uint8)  # 1, -1, 0
    Wd[0, :, 0, 1] = t.where(n % 3 == 0, 15, 7).to(t.uint8)                        # -10, 10
    args = (router, Wgu.reshape(-1), Wd.reshape(-1), I, 2, variant)
    Y, ids, probs = rf4.moe(X, *args)
    assert ids.tolist() == [[0, 1]] * 3 and bool((probs == 0.5).all())
    inf = float("inf")
    assert bool((Y[0, n % 3 == 0] == sign * inf).all()) and bool((Y[0, n % 3 == 1] == -sign * inf).all()) and bool(Y[0, n % 3 == 2].isnan().all())
    assert bool(Y[1:].isfinite().all()) and t.equal(Y[1:], rf4.moe(X[1:].clone(), *args)[0])


@pytest.mark.parametrize("variant", [DUAL, FAST])
def test_infinite_hidden_values_of_both_signs(variant):
    """Infinite hidden values of opposite signs: NaN where both have a weight, infinite where the products' signs agree."""
    t = torch()
    K = I = 32
    bb = 18 if variant == DUAL else 17
    X = t.zeros(1, K, device="cuda").bfloat16()
    X[0, 0] = 2.0 ** 60
    Wgu, Wd = t.zeros(2, I, 1, bb, dtype=t.uint8, device="cuda"), t.zeros(K, 1, bb, dtype=t.uint8, device="cuda")
    Wgu[:, :2, 0, 0] = 7
    Wgu[1, 1, 0, 0] = 15
    Wgu[..., 16:] = 0x7E
    Wd[..., 16:] = 0x40
    Wd[:16, 0, 0], Wd[:16, 0, 1] = 1, 1   # inf - inf
    Wd[16:, 0, 0], Wd[16:, 0, 1] = 1, 9   # inf + inf
    Y, _, _ = rf4.moe(X, t.zeros(1, K, device="cuda"), Wgu.view(-1), Wd.view(-1), I, 1, variant)
    assert bool(Y[0, :16].isnan().all()) and bool((Y[0, 16:] == float("inf")).all())
