"""Speculative decoding with every operator of a decode step, on a small model
with random weights: K-quant matvecs, rotary positions, a quantised paged
cache, attention of a tree of drafts over it, verification, and the accepted
drafts moved up in the cache.

    python examples/speculative_decode.py [--fmt q8] [--tokens 128] [--temperature 0]

Drafts come from the text so far (what followed the last token before): a
chain of its successors, and a second branch with the successor before that.
With temperature 0 the tokens are those of decoding one at a time.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quant_quantized_matvec_gb300 as kq  # noqa: E402
from quant_quantized_matvec_gb300 import synth  # noqa: E402


class Model:
    """Embedding, `layers` of attention and a gated feed-forward block, and a
    head over the vocabulary.  K-quant weights; f32 activations.  (Random
    Q6_K weights have no mean; of the others' only the feed-forward block has
    any, or every token would be the same.)"""

    def __init__(self, layers=2, hidden=512, heads=8, kv_heads=2, dim=64, ffn=1024, vocab=1003,
                 fmt=kq.KV_Q8, length=4096, mix=0.1):
        self.hidden, self.heads, self.kv_heads, self.dim, self.vocab = hidden, heads, kv_heads, dim, vocab
        self.mix = mix  # small: the next token hangs mostly on the last, and text repeats itself

        def weight(f, rows, cols, label):
            w = synth.kquant_matrix(f, rows, cols, f"speculative/{label}")
            return f, torch.from_numpy(w.reshape(-1)).cuda(), rows, cols

        self.embed = weight(kq.Q6_K, vocab, hidden, "embed")
        self.head = weight(kq.Q6_K, vocab, hidden, "head")
        self.layers = [dict(
            q=weight(kq.Q6_K, heads * dim, hidden, f"q{i}"),
            k=weight(kq.Q6_K, kv_heads * dim, hidden, f"k{i}"),
            v=weight(kq.Q6_K, kv_heads * dim, hidden, f"v{i}"),
            o=weight(kq.Q6_K, hidden, heads * dim, f"o{i}"),
            gate=weight(kq.Q4_K, ffn, hidden, f"gate{i}"),
            up=weight(kq.Q5_K, ffn, hidden, f"up{i}"),
            down=weight(kq.Q6_K, hidden, ffn, f"down{i}")) for i in range(layers)]
        self.table = kq.rope_table(length, dim, base=10000.0, scaling="linear", factor=2.0)
        pages = length // kq.KV_PAGE
        self.caches = [kq.KVCache(fmt, kv_heads, dim, pages) for _ in range(layers)]
        # one sequence, its pages in the pool's order
        self.pages = torch.arange(pages, dtype=torch.int32, device="cuda")[None]

    def batch(self, ctx, n):
        """The sequence with ctx committed tokens and n new ones."""
        return kq.KVBatch(torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                          torch.tensor([ctx], dtype=torch.int32, device="cuda"), self.pages, n, n)

    @staticmethod
    def _norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    @staticmethod
    def _set(x, *weights):
        """Several projections of x in one launch."""
        ys = [torch.empty(x.shape[0], w[2], device="cuda") for w in weights]
        kq.matvec_set([(*w, x, y) for w, y in zip(weights, ys)])
        return ys

    def forward(self, tokens, positions, batch, mask):
        """Logits [n, vocab] after each of the new tokens, whose keys and
        values go into the caches."""
        n = tokens.numel()
        x = self._norm(kq.dequant_rows(*self.embed, tokens))
        for w, cache in zip(self.layers, self.caches):
            q, k, v = self._set(self._norm(x), w["q"], w["k"], w["v"])
            q = kq.rope(q.view(n, self.heads, self.dim), positions, self.table)
            kq.kv_append(cache, batch, k.view(n, self.kv_heads, self.dim),
                         v.view(n, self.kv_heads, self.dim), positions, self.table)
            y = kq.tree_attention(cache, batch, q, mask).view(n, -1)
            x = x + self.mix * self._norm(kq.matvec(*w["o"], y))
            gate, up = self._set(self._norm(x), w["gate"], w["up"])
            x = x + self.mix * self._norm(kq.matvec(*w["down"], torch.nn.functional.silu(gate) * up))
        return kq.matvec(*self.head, self._norm(x))


def distribution(logits, temperature):
    if temperature > 0:
        return torch.softmax(logits / temperature, -1)
    return torch.zeros_like(logits).scatter_(-1, logits.argmax(-1, keepdim=True), 1.0)


def drafts(text, depth, most=16):
    """Tokens and parents of a tree whose node 0 is the text's last token: the
    chain of what followed each token the last time, and of the time before."""
    last, before = {}, {}
    for a, b in zip(text, text[1:]):
        if last.get(a) != b:
            before[a] = last.get(a)
        last[a] = b
    tokens, parents = [text[-1]], [-1]
    for first in (last, before):
        at, t = 0, first.get(text[-1])
        while t is not None and len(tokens) < min(most, 1 + depth * (1 if first is last else 2)):
            tokens.append(t)
            parents.append(at)
            at, t = len(tokens) - 1, last.get(t)
    return tokens, parents


def generate(model, prompt, count, depth=6, temperature=0.0, seed=0):
    """`count` tokens after the prompt, and how many each step gave.  depth 0:
    one token at a time."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    text, ctx, steps = list(prompt), 0, []
    for i in range(0, len(prompt) - 1, 16):  # the prompt but its last token
        part = prompt[i:min(i + 16, len(prompt) - 1)]
        pos = torch.arange(ctx, ctx + len(part), dtype=torch.int32, device="cuda")
        model.forward(torch.tensor(part, dtype=torch.int32, device="cuda"), pos,
                      model.batch(ctx, len(part)), None)
        ctx += len(part)
    while len(text) < len(prompt) + count:
        tokens, parents = drafts(text, depth) if depth else ([text[-1]], [-1])
        n = len(tokens)
        at = [0] * n
        for i in range(1, n):
            at[i] = at[parents[i]] + 1
        dev = {k: torch.tensor(v, dtype=torch.int32, device="cuda")
               for k, v in dict(tokens=tokens, parents=parents, pos=[ctx + d for d in at]).items()}
        mask = torch.tensor(kq.tree_mask(parents), dtype=torch.int64, device="cuda")
        batch = model.batch(ctx, n)
        p = distribution(model.forward(dev["tokens"], dev["pos"], batch, mask), temperature)
        u, u_next = (torch.rand(m, generator=gen, device="cuda") for m in (n, 1))
        path, got, token = kq.verify_tree(batch.start, dev["tokens"], dev["parents"], p, None, u,
                                          u_next, n)
        for cache in model.caches:
            kq.kv_move(cache, batch, path, got)
        kept = path[:int(got)].tolist()
        text += [tokens[i] for i in kept[1:]] + [int(token)]
        ctx += len(kept)
        steps.append(len(kept))
    return text[len(prompt):len(prompt) + count], steps


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--fmt", choices=("f16", "q8", "q4"), default="q8")
    ap.add_argument("--tokens", type=int, default=128)
    ap.add_argument("--temperature", type=float, default=0.0)
    a = ap.parse_args()
    model = Model(fmt=getattr(kq, "KV_" + a.fmt.upper()))
    prompt = [(7 * i * i + 3) % model.vocab for i in range(40)]
    text, steps = generate(model, prompt, a.tokens, temperature=a.temperature)
    print("tokens:", text)
    print(f"{len(text)} tokens in {len(steps)} steps, {sum(steps) / len(steps):.2f} a step")


if __name__ == "__main__":
    main()
