"""GPU test of the decode-step example: each stage of each step against its definition in 64 bits, on the inputs that the
stage was given (rounded activations among them), so that no rounding of an earlier stage enters the comparison.

Every product, the attention and the experts are held to relative L2 error 1e-5, the bar of every product here; a norm's
fp16 output to 2^-11 (fp16's rounding) and 2^-18 of itself, and the residual's fp32 sum to 2^-23."""
import importlib.util
import os

import pytest

import gemm_rocmfp4_dequant_gb300 as rf4
from gpu_util import REL_L2, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    yield m
    assert rf4.device_error_bits() == 0


def near(got, want, rel=REL_L2):
    assert float((got.double() - want).norm() / want.norm()) <= rel


def check_norm(y, h, w):
    want = h / (h * h).mean(1, keepdim=True).add(1e-6).sqrt() * w.double()
    assert bool(((y.double() - want).abs() <= (2.0 ** -11 + 2.0 ** -18) * want.abs() + 2.0 ** -25).all())


def test_steps_match_definitions(example):
    t = torch()
    c = example.Config(layers=2, width=512, heads=8, kv_heads=2, head=64, experts=6, top_k=2, hidden=256, vocab=1000, tokens=32, batch=3)
    d = example.Decoder(c, seed=4)
    tokens = t.tensor([5, 17, 999], device="cuda")
    G = c.heads // c.kv_heads
    for n in range(3):
        r = d.step(tokens)
        stream, x = d.embedding[tokens].double(), None
        for i, (w, s) in enumerate(zip(d.layers, r["layers"])):
            h = stream if x is None else x.double() + stream
            check_norm(s["normed"], h, w["norm1"])
            near(s["qkv"], s["normed"].double() @ rf4.dequant(w["qkv"], s["qkv"].shape[1], c.width).double().T)
            K, V = (rf4.dequant(d.cache[i, j].reshape(-1), c.batch * c.kv_heads * c.tokens, c.head).double().view(c.batch, c.kv_heads, c.tokens, c.head)[:, :, :n + 1]
                    for j in (0, 1))
            q = s["q"].double().view(c.batch, c.kv_heads, G, c.head)
            p = t.softmax(q @ K.transpose(2, 3) * c.head ** -0.5, -1)
            near(s["attention"], (p @ V).view(c.batch, c.heads, c.head))
            near(s["o"], s["attention"].half().double().view(c.batch, -1) @ rf4.dequant(w["o"], c.width, c.heads * c.head).double().T)
            h2 = s["o"].double() + h.float().double()
            assert bool(((s["residual"].double() - h2).abs() <= 2.0 ** -23 * h2.abs() + 2.0 ** -23 * h.abs()).all())
            check_norm(s["moe_in"], h2, w["norm2"])
            b = s["moe_in"].double()
            best, ids = t.topk(b @ w["router"].double().T, c.top_k, dim=1)
            assert t.equal(s["ids"].long(), ids)
            gu = rf4.dequant(w["gate_up"], c.experts * 2 * c.hidden, c.width).double().view(c.experts, 2 * c.hidden, c.width)
            dn = rf4.dequant(w["down"], c.experts * c.width, c.hidden).double().view(c.experts, c.width, c.hidden)
            want = t.zeros_like(b)
            for m in range(c.batch):
                for p_, e in zip(t.softmax(best[m], 0), ids[m]):
                    both = gu[e] @ b[m]
                    g, u = both[:c.hidden], both[c.hidden:]
                    want[m] += p_ * (dn[e] @ (g * t.sigmoid(g) * u))
            near(s["moe"], want)
            stream, x = s["residual"].double(), s["moe"]
        check_norm(r["final"], x.double() + stream, d.norm)
        near(r["logits"], r["final"].double() @ rf4.dequant(d.head, c.vocab, c.width).double().T)
        logp = t.log_softmax(r["logits"].double(), 1)
        assert t.equal(r["next"].long(), r["logits"].argmax(1)) and t.equal(r["top_ids"][:, 0], r["next"])
        assert float((r["logprob"].double() - logp.amax(1)).abs().max()) <= 2.0 ** -16 * 4
        assert float((r["entropy"].double() + (logp.exp() * logp).sum(1)).abs().max()) <= 2.0 ** -16 * 16
        tokens = r["next"].long()
    assert d.length == 3


def test_full_cache_is_refused(example):
    c = example.Config(layers=1, width=256, heads=4, kv_heads=1, head=64, experts=2, top_k=1, hidden=256, vocab=64, tokens=32, batch=1)
    d = example.Decoder(c)
    d.length = 32
    with pytest.raises(ValueError):
        d.step(torch().zeros(1, dtype=torch().int64, device="cuda"))
