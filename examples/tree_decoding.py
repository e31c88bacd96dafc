"""Sampled decoding with drafted token trees, end to end on random weights.

A small decoder (Q4_0 matrices) runs one batched forward over the trees of two
sequences a step, with the library's operators for everything that touches
weights, cache or vocabulary:

    draft      a tree a sequence from a bigram table (siblings drawn without
               replacement)
    forward    Matrix.verify for the projections, PagedCache.attend for the
               attention: every node sees the cached rows and its ancestors
    verify     verify_sample walks each tree by rejection sampling
    commit     PagedCache.commit moves the accepted branch behind the cached rows

At the end one sequence is forked and both go on from the same prefix.

    python examples/tree_decoding.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decode_verification_qmm_gb300 as q  # noqa: E402

LAYERS, HIDDEN, HEADS, KV_HEADS, HEAD_DIM, MLP, VOCAB = 2, 512, 8, 4, 64, 1024, 1000


class Model:
    """Random weights of a decoder; `sharp` scales its scores."""

    def __init__(self, seed=0, sharp=6.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def matrix(n, k, sigma):
            w = torch.randn(n, k, generator=g, device="cuda") * sigma
            return q.Matrix(q.QMM_FMT_Q4_0, q.quantize_q4_0(w), n, k)

        qkv = (HEADS + 2 * KV_HEADS) * HEAD_DIM
        self.embed = torch.randn(VOCAB, HIDDEN, generator=g, device="cuda")
        self.layers = [dict(qkv=matrix(qkv, HIDDEN, HIDDEN ** -0.5), out=matrix(HIDDEN, HEADS * HEAD_DIM, 0.04),
                            up=matrix(2 * MLP, HIDDEN, HIDDEN ** -0.5), down=matrix(HIDDEN, MLP, 0.03))
                       for _ in range(LAYERS)]
        self.head = matrix(VOCAB, HIDDEN, sharp * HIDDEN ** -0.5)
        # the drafter: the target's own scores without its layers, and some noise
        bigram = self.norm(self.embed) @ (self.head.dequantize().t())
        self.bigram = bigram + torch.randn(VOCAB, VOCAB, generator=g, device="cuda")
        self.freq = 10000.0 ** (-torch.arange(0, HEAD_DIM, 2, device="cuda") / HEAD_DIM)

    @staticmethod
    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def rotate(self, x, positions):
        a = positions[..., None, None] * self.freq
        c, s = a.cos(), a.sin()
        x, y = x[..., ::2], x[..., 1::2]
        return torch.stack([x * c - y * s, x * s + y * c], -1).flatten(-2)

    def forward(self, cache, tokens, depths, table, lens, mask):
        """Scores [B, T, V] after every node of tokens [B, T]."""
        B, T = tokens.shape
        x = self.embed[tokens.long()].view(B * T, HIDDEN)
        positions = (lens[:, None] + depths).float()
        for i, w in enumerate(self.layers):
            qkv = w["qkv"].verify(self.norm(x).bfloat16()).view(B, T, -1, HEAD_DIM)
            qk = self.rotate(qkv[:, :, :HEADS + KV_HEADS], positions)
            x_q, x_k = qk[:, :, :HEADS].bfloat16(), qk[:, :, HEADS:].bfloat16()
            att, _ = cache.attend(i, x_q, x_k, qkv[:, :, HEADS + KV_HEADS:].bfloat16(), table, lens, mask=mask)
            x = x + w["out"].verify(att.view(B * T, -1))
            up = w["up"].verify(self.norm(x).bfloat16())
            x = x + w["down"].verify((torch.nn.functional.silu(up[:, :MLP]) * up[:, MLP:]).bfloat16())
        return self.head.verify(self.norm(x).bfloat16()).view(B, T, VOCAB)


class Decoder:
    """Sequences that are decoded together, a tree of nodes a step."""

    # node 0 is the last committed token; two branches from it, the first goes on
    PARENTS = [-1, 0, 0, 1, 1, 2, 3, 6]

    def __init__(self, model, nodes=8, pages=64, temperature=1.0, seed=1):
        self.model, self.temperature = model, temperature
        self.cache = q.PagedCache(LAYERS, pages, 16, HEADS, KV_HEADS, HEAD_DIM, max_batch=2)
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.parents = self.PARENTS[:nodes]
        self.accepted = self.steps = 0

    def start(self, prompt):
        """A sequence with all of the prompt but its last token in the cache."""
        seq = self.cache.new_sequence()
        seq.tokens = list(prompt)
        body = seq.tokens[:-1]
        for at in range(0, len(body), 16):  # chains of up to 16 rows, what one verify call takes
            part = torch.tensor([body[at:at + 16]], dtype=torch.int32, device="cuda")
            self.cache.reserve([seq], part.shape[1])
            table, lens = self.cache.tables([seq])
            self.model.forward(self.cache, part, torch.arange(part.shape[1], device="cuda")[None], table, lens, None)
            self.cache.advance([seq], [part.shape[1]])
        return seq

    def draft(self, seqs):
        """Tokens [B, T] of the trees and the drafter's scores after each node."""
        B, T = len(seqs), len(self.parents)
        tokens = torch.zeros(B, T, dtype=torch.int32, device="cuda")
        scores = torch.zeros(B, T, VOCAB, device="cuda")
        tokens[:, 0] = torch.tensor([s.tokens[-1] for s in seqs], device="cuda")
        for i in range(T):
            scores[:, i] = self.model.bigram[tokens[:, i].long()]
            kids = [c for c in range(T) if self.parents[c] == i]
            if kids:
                noise = torch.empty(B, VOCAB, device="cuda").exponential_(generator=self.g)
                order = (scores[:, i] / self.temperature - noise.log()).topk(len(kids), 1).indices
                tokens[:, kids] = order.to(torch.int32)
        return tokens, scores

    def step(self, seqs):
        """One forward over the sequences' trees; 1 to depth + 1 tokens each."""
        B, T = len(seqs), len(self.parents)
        cache = self.cache
        cache.reserve(seqs, T)
        table, lens = cache.tables(seqs)
        parents = torch.tensor([self.parents] * B, dtype=torch.int32)
        depths = [0]
        for p in self.parents[1:]:
            depths.append(depths[p] + 1)
        tokens, drafted = self.draft(seqs)
        scores = self.model.forward(cache, tokens, torch.tensor([depths] * B, device="cuda"), table, lens,
                                    q.tree_mask(parents).cuda())
        accept, path = q.verify_sample(
            scores, drafted, tokens, torch.rand(B, T, generator=self.g, device="cuda"),
            torch.empty(B, VOCAB, device="cuda").exponential_(generator=self.g), parents=parents.cuda(),
            temperature=torch.full((B,), self.temperature, device="cuda"))
        cache.commit(table, lens, path, accept)
        # the host learns what was kept
        kept, walk, tokens = accept.tolist(), path.tolist(), tokens.tolist()
        for b, s in enumerate(seqs):
            k, last = kept[b]
            s.tokens += [tokens[b][n] for n in walk[b][:k]] + [last]
            self.accepted += k
            self.steps += 1
        cache.advance(seqs, [k + 1 for k, _ in kept])

    def fork(self, seq):
        other = self.cache.fork(seq)
        other.tokens = list(seq.tokens)
        return other

    def check(self):
        for status in [self.cache.sync_status()] + [w.sync_status() for layer in self.model.layers
                                                    for w in layer.values()]:
            if status != q.QMM_OK:
                raise RuntimeError(q.qmm_strerror(status))


def main():
    model = Model()
    d = Decoder(model)
    seqs = [d.start(range(5, 45)), d.start([7, 1, 3])]
    for _ in range(20):
        d.step(seqs)
    d.check()
    print(f"{d.accepted / d.steps:.2f} of at most {4} drafted tokens accepted a step, "
          f"{d.cache.free_pages} of {d.cache.n_pages} pages free")
    for s in seqs:
        print(s.tokens)
    pair = [seqs[0], d.fork(seqs[0])]
    at = len(pair[0].tokens)
    for _ in range(4):
        d.step(pair)
    d.check()
    print("forked:", pair[0].tokens[at:], "and", pair[1].tokens[at:])
    for s in seqs + pair[1:]:
        d.cache.free(s)
    assert d.cache.free_pages == d.cache.n_pages


if __name__ == "__main__":
    main()
