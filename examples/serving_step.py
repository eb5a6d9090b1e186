#!/usr/bin/env python3
"""Speculative decoding end to end on a small random model: prompts through
prompt attention into the paged cache, then steps of k drafts whose k+1 target
rows come from attention over the cache and are verified by rejection sampling.

  python examples/serving_step.py [--steps 8] [--k 7] [--cache bf16|e4m3] [--temperature 0.7]

Per step and layer the new tokens' keys and values are appended and attended
to; the rejected ones are dropped by lowering the sequences' lengths.  Prints
the accepted length of every step.
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from speculative_decoding_verification_68_gb300 import SpecAttention, SpecVerifier  # noqa: E402


class Model:
    """A target of `layers` attention layers without feed-forward parts, and a
    draft that sees only the last token; random weights, bf16."""

    def __init__(self, vocab=4096, q_heads=8, kv_heads=2, head_dim=64, layers=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.hq, self.hkv, self.d, self.layers = vocab, q_heads, kv_heads, head_dim, layers
        width = q_heads * head_dim

        def weight(rows, cols, scale=1.0):
            return (torch.randn((rows, cols), generator=g, device="cuda") * scale * rows ** -0.5).bfloat16()

        self.embed = torch.randn((vocab, width), generator=g, device="cuda").bfloat16()
        self.qkv = [weight(width, (q_heads + 2 * kv_heads) * head_dim) for _ in range(layers)]
        self.out = [weight(width, width) for _ in range(layers)]
        self.head = weight(width, vocab, 3.0)

    def project(self, x, layer):
        """q, k and v [n, heads, head_dim]: slices of one tensor."""
        fused = (x @ self.qkv[layer]).view(x.shape[0], -1, self.d)
        return fused.split([self.hq, self.hkv, self.hkv], 1)

    def forward(self, tokens, attention):
        """Logits of packed tokens; attention(layer, q, k, v) gives [n, q_heads, head_dim]."""
        x = self.embed[tokens]
        for layer in range(self.layers):
            q, k, v = self.project(x, layer)
            x = x + attention(layer, q, k, v).flatten(1) @ self.out[layer]
        return x @ self.head

    def draft_logits(self, tokens):
        return self.embed[tokens] @ self.head


class Server:
    def __init__(self, model: Model, max_seqs: int, max_tokens: int, k: int, cache=torch.bfloat16, page_size=16):
        self.model, self.k, self.max_seqs, self.page_size = model, k, max_seqs, page_size
        self.attn = SpecAttention(model.hq, model.hkv, model.d, max_seqs)
        self.verifier = SpecVerifier(max_seqs, k, model.vocab, torch.bfloat16)
        pages = -(-max_tokens // page_size)
        self.pools = [self.attn.alloc_pool(max_seqs * pages, page_size, cache) for _ in range(model.layers)]
        self.table = torch.randperm(max_seqs * pages, device="cuda").int().view(max_seqs, pages)
        self.kv_len = torch.zeros(max_seqs, dtype=torch.int32, device="cuda")       # tokens in the cache
        self.step_cu = torch.arange(0, max_seqs * (k + 1) + 1, k + 1, dtype=torch.int32, device="cuda")

    def prefill(self, prompts):
        """Runs the prompts (lists of tokens); their last tokens' next ones are greedy."""
        lengths = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
        cu = torch.nn.functional.pad(lengths.cumsum(0), (1, 0)).int()
        tokens = torch.tensor([t for p in prompts for t in p], device="cuda")
        self.kv_len, self.longest = lengths, max(len(p) for p in prompts)

        def attention(layer, q, k, v):
            self.attn.append(self.pools[layer], k, v, cu, lengths, self.table)
            return self.attn.prompt(q, k, v, cu)["out"]

        logits = self.model.forward(tokens, attention)
        self.last = logits[cu[1:].long() - 1].argmax(-1)
        return self.last

    def step(self, temperature, generator=None):
        """One step for every sequence; returns tokens [B, k+1] (-1 past the accepted ones and the drawn one) and tau."""
        B, k = self.max_seqs, self.k
        uniforms = torch.rand((B, k + 1), generator=generator, device="cuda")
        drafts, rows, last = [], [], self.last
        for _ in range(k):
            logits = self.model.draft_logits(last)
            greedy = logits.argmax(-1)
            p = torch.softmax(logits.float() / temperature.clamp_min(1e-3)[:, None], -1)
            last = torch.where(temperature > 0, torch.multinomial(p, 1, generator=generator)[:, 0], greedy)
            drafts.append(last)
            rows.append(logits)
        drafts = torch.stack(drafts, 1)
        tokens = torch.cat([self.last[:, None], drafts], 1).flatten()
        length, self.longest = self.kv_len + k + 1, self.longest + k + 1         # on the device, and a bound here

        def attention(layer, q, key, v):
            self.attn.append(self.pools[layer], key, v, self.step_cu, length, self.table)
            return self.attn.attend(self.pools[layer], q, self.step_cu, length, self.table, max_kv=self.longest)["out"]

        target = self.model.forward(tokens, attention).view(B, k + 1, -1)
        out = self.verifier.verify(target, torch.stack(rows, 1), drafts.int(), temperature, uniforms)
        tau = out["tau"]
        self.kv_len = self.kv_len + tau + 1                      # the rejected drafts leave the cache
        self.last = out["tokens"].gather(1, tau.long()[:, None])[:, 0].long()
        return out["tokens"], tau


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--k", type=int, default=7)
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--temperature", type=float, default=0.7)
    a = ap.parse_args()
    generator = torch.Generator(device="cuda").manual_seed(1)
    model = Model()
    prompts = [torch.randint(model.vocab, (5 + 37 * b,)).tolist() for b in range(a.seqs)]
    server = Server(model, a.seqs, max(map(len, prompts)) + (a.steps + 1) * (a.k + 1), a.k,
                    torch.bfloat16 if a.cache == "bf16" else torch.float8_e4m3fn)
    server.prefill(prompts)
    temperature = torch.full((a.seqs,), a.temperature, device="cuda")
    for step in range(a.steps):
        _, tau = server.step(temperature, generator)
        print(f"step {step}: accepted {tau.tolist()}, cached {server.kv_len.tolist()}")
    assert server.attn.get_error() == 0 and server.verifier.get_error() == (0, 0)


if __name__ == "__main__":
    main()
