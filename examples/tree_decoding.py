"""Sampled decoding with drafted token trees, end to end on random weights.

A small decoder (Q4_0 matrices) runs one batched forward over the trees of two
sequences a step, with the library's operators for everything that touches
weights, cache or vocabulary:

    prompt     PagedCache.append turns its rows by their positions into the cache,
               PagedCache.attend_prompt is their attention, in one piece
    draft      a tree a sequence from a bigram table (siblings drawn without
               replacement)
    forward    Matrix.verify for the projections, Rope.rotate for the positions,
               PagedCache.attend for the attention (every node sees the cached rows and
               its ancestors), residual_norm between the blocks
    verify     adjust_scores penalises repeated tokens, verify_sample walks each
               tree by rejection sampling, count_tokens counts what it emitted
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
        self.ones = torch.ones(HIDDEN, device="cuda")
        _, start = q.residual_norm(self.embed, weight=self.ones, dtype=torch.float32)
        self.bigram = start @ self.head.dequantize().t() + torch.randn(VOCAB, VOCAB, generator=g, device="cuda")
        self.rope = q.Rope(*q.rope_frequencies(HEAD_DIM), layout="interleaved")

    @staticmethod
    def product(w, x):
        """Of any number of rows, 16 at a time."""
        return torch.cat([w.verify(part) for part in x.split(16)])

    def blocks(self, tokens, attention):
        """The normed state [rows, HIDDEN] after all layers; attention(layer, qkv) of the rows'
        heads [rows, heads, HEAD_DIM]."""
        x = self.embed[tokens.long()].view(-1, HIDDEN)
        _, h = q.residual_norm(x, weight=self.ones)
        for i, w in enumerate(self.layers):
            att = attention(i, self.product(w["qkv"], h).view(len(x), -1, HEAD_DIM))
            x, h = q.residual_norm(x, self.product(w["out"], att.reshape(len(x), -1)), self.ones)
            up = self.product(w["up"], h)
            y = self.product(w["down"], (torch.nn.functional.silu(up[:, :MLP]) * up[:, MLP:]).bfloat16())
            x, h = q.residual_norm(x, y, self.ones)
        return h

    def forward(self, cache, tokens, depths, table, lens, mask):
        """Scores [B, T, V] after every node of tokens [B, T]."""
        B, T = tokens.shape
        positions = (lens[:, None] + depths).int()

        def attention(i, qkv):
            x = self.rope.rotate(qkv.view(B, T, -1, HEAD_DIM), positions, heads=HEADS + KV_HEADS, dtype=torch.bfloat16)
            return cache.attend(i, x[:, :, :HEADS], x[:, :, HEADS:HEADS + KV_HEADS], x[:, :, HEADS + KV_HEADS:], table, lens,
                                mask=mask)[0]

        return self.product(self.head, self.blocks(tokens, attention)).view(B, T, VOCAB)

    def prompt(self, cache, tokens, table, lens, starts):
        """Packed rows of prompts into the cache."""
        def attention(i, qkv):
            x, k, v = qkv.split([HEADS, KV_HEADS, KV_HEADS], 1)
            x = cache.append(i, x, k, v, table, lens, starts, rope=self.rope)
            return cache.attend_prompt(i, x, table, lens, starts)[0]

        self.blocks(tokens, attention)


class Decoder:
    """Sequences that are decoded together, a tree of nodes a step."""

    # node 0 is the last committed token; two branches from it, the first goes on
    PARENTS = [-1, 0, 0, 1, 1, 2, 3, 6]

    def __init__(self, model, nodes=8, pages=64, temperature=1.0, seed=1, repetition=1.0, presence=0.0):
        self.model, self.temperature = model, temperature
        self.repetition, self.presence = repetition, presence
        self.cache = q.PagedCache(LAYERS, pages, 16, HEADS, KV_HEADS, HEAD_DIM, max_batch=2)
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.parents = self.PARENTS[:nodes]
        self.accepted = self.steps = 0

    def start(self, prompt):
        """A sequence with all of the prompt but its last token in the cache."""
        seq = self.cache.new_sequence()
        seq.tokens = list(prompt)
        seq.counts = torch.zeros(VOCAB, dtype=torch.int32, device="cuda")  # what was emitted
        words = [0] * (-(-VOCAB // 32))
        for t in seq.tokens:
            words[t // 32] |= 1 << t % 32
        seq.prompt = torch.tensor([w - (w >> 31 << 32) for w in words], dtype=torch.int32, device="cuda")
        body = torch.tensor(seq.tokens[:-1], dtype=torch.int32, device="cuda")
        if len(body):
            self.cache.reserve([seq], len(body))
            self.model.prompt(self.cache, body, *self.cache.tables([seq]), self.cache.starts([len(body)]))
            self.cache.advance([seq], [len(body)])
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
        parents, counts = parents.cuda(), torch.stack([s.counts for s in seqs])
        scores = q.adjust_scores(scores, tokens, parents, counts=counts, prompt=torch.stack([s.prompt for s in seqs]),
                                 repetition=torch.full((B,), self.repetition, device="cuda"),
                                 presence=torch.full((B,), self.presence, device="cuda"), out=scores)
        accept, path = q.verify_sample(
            scores, drafted, tokens, torch.rand(B, T, generator=self.g, device="cuda"),
            torch.empty(B, VOCAB, device="cuda").exponential_(generator=self.g), parents=parents,
            temperature=torch.full((B,), self.temperature, device="cuda"))
        q.count_tokens(counts, tokens, path, accept)
        cache.commit(table, lens, path, accept)
        # the host learns what was kept
        kept, walk, tokens = accept.tolist(), path.tolist(), tokens.tolist()
        for b, s in enumerate(seqs):
            k, last = kept[b]
            s.tokens += [tokens[b][n] for n in walk[b][:k]] + [last]
            s.counts = counts[b]
            self.accepted += k
            self.steps += 1
        cache.advance(seqs, [k + 1 for k, _ in kept])

    def fork(self, seq):
        other = self.cache.fork(seq)
        other.tokens, other.counts, other.prompt = list(seq.tokens), seq.counts, seq.prompt
        return other

    def check(self):
        for status in [self.cache.sync_status()] + [w.sync_status() for layer in self.model.layers
                                                    for w in layer.values()]:
            if status != q.QMM_OK:
                raise RuntimeError(q.qmm_strerror(status))


def main():
    model = Model()
    d = Decoder(model, repetition=1.1, presence=0.2)
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
