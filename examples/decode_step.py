"""A mixture-of-experts decoder taking single-token steps on ROCmFP4 weights.

    python examples/decode_step.py [--layers 4] [--batch 2] [--steps 8]

Every layer is

    residual, RMS norm -> fused QKV product -> K and V rows quantised into the ROCmFP4 cache -> decode attention
    -> O product -> residual, RMS norm -> mixture of experts,

and behind the last one come the final norm, the head's product and the log probabilities of the tokens that were
chosen.  Weights are random; no positions are encoded.
"""
import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_rocmfp4_dequant_gb300 as rf4  # noqa: E402


@dataclass
class Config:
    layers: int = 4
    width: int = 2048
    heads: int = 16
    kv_heads: int = 4
    head: int = 64
    experts: int = 32
    top_k: int = 4
    hidden: int = 768
    vocab: int = 32000
    tokens: int = 256  # room of the cache, a multiple of 32
    batch: int = 2
    top_n: int = 5


class Decoder:
    """Weights, cache and buffers; ``step`` runs one token of every sequence and returns its outputs by name."""

    def __init__(self, c: Config, seed: int = 0):
        self.c = c
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def dense(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).half()

        def packed(rows, k):
            return rf4.quantize(dense(rows, k, scale=k ** -0.5))

        qkv = (c.heads + 2 * c.kv_heads) * c.head
        self.layers = [dict(
            norm1=1 + dense(c.width, scale=0.1), qkv=packed(qkv, c.width), o=packed(c.width, c.heads * c.head),
            norm2=1 + dense(c.width, scale=0.1), router=dense(c.experts, c.width, scale=2 * c.width ** -0.5),
            gate_up=packed(c.experts * 2 * c.hidden, c.width), down=packed(c.experts * c.width, c.hidden)) for _ in range(c.layers)]
        self.norm = 1 + dense(c.width, scale=0.1)
        self.head = packed(c.vocab, c.width)
        self.embedding = dense(c.vocab, c.width)
        self.row = rf4.row_bytes(c.head, rf4.DUAL)
        cache = (c.layers, 2, c.batch, c.kv_heads, c.tokens, self.row)
        self.cache = torch.zeros(cache, dtype=torch.uint8, device="cuda")
        self.length = 0

    def _append(self, layer: int, k, v):
        """The new token's K and V rows (fp16 [batch, kv_heads, head]) into the cache: one row of blocks each."""
        c, t = self.c, self.length
        for which, rows in enumerate((k, v)):
            blocks = rf4.quantize(rows.reshape(c.batch * c.kv_heads, c.head))
            self.cache[layer, which, :, :, t].copy_(blocks.view(c.batch, c.kv_heads, self.row))

    def step(self, tokens):
        """tokens: int64 [batch] -> what the step computed, the chosen next tokens and their log probabilities among it."""
        c = self.c
        if self.length >= c.tokens:
            raise ValueError("the cache is full")
        out = []
        lens = torch.full((c.batch,), self.length + 1, dtype=torch.int32, device="cuda")
        residual = self.embedding[tokens].float()
        x = None  # what the previous block adds to the residual stream
        for i, w in enumerate(self.layers):
            if x is None:
                a = rf4.add_rmsnorm(residual, w["norm1"]).y
            else:
                a, residual, _, _ = rf4.add_rmsnorm(x, w["norm1"], residual=residual)
            qkv = rf4.gemm(w["qkv"], a, (c.heads + 2 * c.kv_heads) * c.head, c.width)
            q, k, v = qkv.half().view(c.batch, -1, c.head).split((c.heads, c.kv_heads, c.kv_heads), dim=1)
            self._append(i, k, v)
            att = rf4.decode_attention(q.contiguous(), self.cache[i, 0], self.cache[i, 1], lens, c.kv_heads, c.tokens, c.head ** -0.5)
            o = rf4.gemm(w["o"], att.half().view(c.batch, -1), c.width, c.heads * c.head)
            b, residual, _, _ = rf4.add_rmsnorm(o, w["norm2"], residual=residual)
            x, ids, probs = rf4.moe(b, w["router"], w["gate_up"], w["down"], c.hidden, c.top_k)
            out.append(dict(normed=a, qkv=qkv, q=q, attention=att, o=o, residual=residual.clone(), moe_in=b, moe=x, ids=ids, probs=probs))
        f, residual, _, _ = rf4.add_rmsnorm(x, self.norm, residual=residual)
        logits = rf4.gemm(self.head, f, c.vocab, c.width)
        best = logits.argmax(1).int()
        logprob, entropy, top_ids, top = rf4.logprobs(logits, best, top_n=c.top_n)
        self.length += 1
        return dict(layers=out, final=f, residual=residual, logits=logits, next=best, logprob=logprob, entropy=entropy, top_ids=top_ids, top=top)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name in ("layers", "batch"):
        ap.add_argument("--" + name, type=int, default=getattr(Config, name))
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    d = Decoder(Config(layers=a.layers, batch=a.batch))
    tokens = torch.arange(a.batch, device="cuda")
    for n in range(a.steps):
        r = d.step(tokens)
        tokens = r["next"].long()
        print(f"step {n}: tokens {tokens.tolist()}, log probabilities {[round(v, 3) for v in r['logprob'].tolist()]}, "
              f"entropy {[round(v, 3) for v in r['entropy'].tolist()]}")
    print(f"kernels launched {rf4.launch_count()}, error bits {rf4.device_error_bits()}")


if __name__ == "__main__":
    main()
