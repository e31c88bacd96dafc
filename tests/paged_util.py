"""Plain 64-bit implementations of the paged-cache operators and the tolerance of
the attention tests (no library code)."""
from __future__ import annotations

import math

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# unit roundoff of the 16-bit types
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


class Attention:
    """Random inputs of one call; `lens`, `counts` are host lists."""

    def __init__(self, dtype, D, Hq, Hkv, T, page, lens, counts=None, tree=False, seed=0, layers=1, layer=0,
                 extra_pages=3, fill=None, sigma=1.0, strided=False):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = np.random.default_rng(seed)
        self.dtype, self.D, self.Hq, self.Hkv, self.T, self.page = TYPES[dtype], D, Hq, Hkv, T, page
        self.lens, self.layer = list(lens), layer
        B = self.B = len(lens)
        self.counts = [T] * B if counts is None else list(counts)
        need = [(n + T + page - 1) // page for n in lens]
        total = sum(need) + extra_pages
        ids = r.permutation(total)[:sum(need)]
        self.table = torch.zeros(B, max(need), dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = torch.from_numpy(ids[at:at + n].astype(np.int32))
            at += n
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        shape = (layers, total, Hkv, page, D)
        self.k_pool, self.v_pool = rnd(*shape).to(self.dtype), rnd(*shape).to(self.dtype)
        if fill is not None:  # what stale rows hold: everything past the cached rows
            for pool in (self.k_pool, self.v_pool):
                keep = torch.full_like(pool, fill)
                for b in range(B):
                    for j in range(self.lens[b]):
                        p = int(self.table[b, j // page])
                        keep[:, p, :, j % page] = pool[:, p, :, j % page]
                pool.copy_(keep)
        if strided:  # one buffer of queries, keys and values, and a wider output
            x = rnd(B, T + 1, Hq + 2 * Hkv + 1, D + 8)
            x[:, :, :Hq] *= sigma
            x = x.to(self.dtype)[:, :T, :, :D]
            self.q, self.k, self.v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:Hq + 2 * Hkv]
        else:
            self.q = (rnd(B, T, Hq, D) * sigma).to(self.dtype)
            self.k, self.v = rnd(B, T, Hkv, D).to(self.dtype), rnd(B, T, Hkv, D).to(self.dtype)
        self.scale = D ** -0.5
        self.seen = np.tril(np.ones((B, T, T), bool))
        self.mask = None
        if tree:
            seen = np.zeros((B, T, T), bool)
            for b in range(B):
                for i in range(T):
                    if i:
                        seen[b, i] = seen[b, r.integers(max(0, i - 5), i)]
                    seen[b, i, i] = True
            self.set_seen(seen)

    def set_seen(self, seen):
        self.seen = seen
        w = (seen.astype(np.uint64) << np.arange(self.T, dtype=np.uint64)).sum(-1, dtype=np.uint64)
        self.mask = torch.from_numpy(w.view(np.int64).copy())

    def call(self, cache, out=None, lse=None, stream=None, ragged=True):
        cuda = lambda x: x.cuda() if x is not None else None  # noqa: E731
        n = torch.tensor(self.counts, dtype=torch.int32).cuda() if ragged else None
        return cache.attend(self.layer, self.q, self.k, self.v, self.table.cuda(),
                            torch.tensor(self.lens, dtype=torch.int32).cuda(), mask=cuda(self.mask), n_tokens=n,
                            out=out, lse=lse, stream=stream)

    def make_cache(self, q):
        return q.PagedCache(self.k_pool.shape[0], self.k_pool.shape[1], self.page, self.Hq, self.Hkv, self.D,
                            dtype=self.dtype, max_batch=self.B, k_pool=self.k_pool, v_pool=self.v_pool)

    def rows(self, b):
        """Keys and values [Hkv, lens + counts, D] of sequence b, before the call."""
        out = []
        for pool, new in ((self.k_pool, self.k), (self.v_pool, self.v)):
            ids = self.table[b, :(self.lens[b] + self.page - 1) // self.page].long().cuda()
            old = pool[self.layer, ids].transpose(0, 1).reshape(self.Hkv, -1, self.D)[:, :self.lens[b]]
            out.append(torch.cat([old, new[b, :self.counts[b]].transpose(0, 1)], 1))
        return out

    def reference(self):
        """(out, lse, bound of out, bound of lse) in 64 bits.

        With u the 16-bit unit roundoff, A = sum p |v| / sum p and ds a bound of
        a score's fp32 error (products of 16-bit values are exact, D additions,
        each off by one unit in the last place at most, a 2-ulp exponential):
        |out - o| <= u (|o| + A) + 2 ds A, with u A for the rounded p.  In f16 p
        (at least 1 at a row's maximum) also loses up to 2^-25 each below the
        normal range, and an output below it as much: 2^-25 (sum |v| + 1).  The
        lse is off by ds, the sum's and the logarithm's roundings."""
        B, T, Hq, D, g = self.B, self.T, self.Hq, self.D, self.Hq // self.Hkv
        out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
        lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device="cuda")
        tol, ltol = torch.zeros_like(out), torch.zeros(B, T, Hq, dtype=torch.float64, device="cuda")
        u = ROUND[self.dtype]
        for b in range(B):
            n, L = self.counts[b], self.lens[b]
            if n == 0:
                continue
            k, v = self.rows(b)
            see = torch.ones(n, L + n, dtype=torch.bool)
            see[:, L:] = torch.from_numpy(self.seen[b, :n, :n])
            see = see.cuda()
            some = see.any(1)
            for h in range(Hq):
                kk, vv, qq = k[h // g].double(), v[h // g].double(), self.q[b, :n, h].double()
                # rows that a node does not see have no part in anything that follows
                s = torch.where(see, (qq[:, None] * kk).sum(-1) * self.scale, -math.inf)
                z = torch.where(some, torch.logsumexp(s, 1), 0.0)
                p = torch.exp(s - z[:, None])
                o, A = p @ vv, p @ vv.abs()
                size = torch.where(see, (qq.abs()[:, None] * kk.abs()).sum(-1), 0.0).amax(1) * self.scale
                ds = size * (D + 4) * 2.0 ** -23 + 2.0 ** -20
                e = 1.01 * u * (o.abs() + A) + 2 * ds[:, None] * A
                if self.dtype == torch.float16:
                    e += 2.0 ** -25 * (see.double() @ vv.abs() + 1)
                out[b, :n, h] = torch.where(some[:, None], o, 0.0)
                tol[b, :n, h] = torch.where(some[:, None], e, 0.0)
                lse[b, :n, h] = torch.where(some, z, -math.inf)
                ltol[b, :n, h] = torch.where(some, ds + 2.0 ** -20 * (1 + z.abs()), 0.0)
        return out, lse, tol, ltol

    def expect_pools(self):
        """The pools after the call."""
        pools = []
        for pool, new in ((self.k_pool, self.k), (self.v_pool, self.v)):
            want = pool.clone()
            for b in range(self.B):
                for t in range(self.counts[b]):
                    j = self.lens[b] + t
                    want[self.layer, int(self.table[b, j // self.page]), :, j % self.page] = new[b, t]
            pools.append(want)
        return pools


def assert_attention(a, cache, q, **kw):
    """One call against the 64-bit definition: outputs, lse and the written rows."""
    ref, lref, tol, ltol = a.reference()
    pools = a.expect_pools()
    out, lse = a.call(cache, **kw)
    torch.cuda.synchronize()
    assert cache.sync_status() == q.QMM_OK
    check(out, lse, ref, lref, tol, ltol)
    for got, want in zip((a.k_pool, a.v_pool), pools):
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), "rows of the cache"
    return out, lse


def check(out, lse, ref, lref, tol, ltol):
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(out.double()), torch.isnan(ref)), "NaN where the definition has none, or none"
    err = (out.double() - ref).abs()[fine]
    worst = (err - tol[fine]).max().item() if err.numel() else 0.0
    assert worst <= 0, f"out: {worst} above its bound"
    lfine = torch.isfinite(lref)
    assert torch.equal(lse.double()[~lfine].nan_to_num(nan=1.0), lref[~lfine].nan_to_num(nan=1.0)), "lse of empty rows"
    lerr = (lse.double() - lref).abs()[lfine]
    worst = (lerr - ltol[lfine]).max().item() if lerr.numel() else 0.0
    assert worst <= 0, f"lse: {worst} above its bound"


def sample_reference(target, draft, tokens, parents, u, noise, temperature, n_tokens):
    """The walk of one sequence in 64 bits, and the smallest relative margin of its
    decisions: (nodes, next token, margin).  numpy float64 [T, V].

    A relative rounding of P and Q grows by 1 / mass where max(P - Q, 0) of that
    mass is normalised, so later margins at the node count by the mass."""
    T, V = target.shape
    soft = lambda x: np.exp(x - x.max()) / np.exp(x - x.max()).sum()  # noqa: E731
    node, path, margin, mass = 0, [], math.inf, 1.0
    while True:
        with np.errstate(invalid="ignore"):
            p = soft(target[node] / temperature)
        kids = [i for i in range(node + 1, n_tokens) if parents[i] == node and 0 <= tokens[i] < V]
        qd = soft(draft[node] / temperature) if draft is not None and kids else None
        for c in kids:
            x = tokens[c]
            lhs, rhs = u[c] * (1.0 if draft is None else qd[x]), p[x]
            if max(lhs, rhs) > 0:
                margin = min(margin, mass * abs(lhs - rhs) / max(lhs, rhs))
            if lhs < rhs:
                path.append(c)
                node, mass = c, 1.0
                break
            left = p.copy()
            if draft is None:
                left[x] = 0
            else:
                left = np.maximum(p - qd, 0)
                qd[x] = 0
                if qd.sum() > 0:
                    qd = qd / qd.sum()
            mass *= min(1.0, left.sum())
            if left.sum() > 0:
                p = left / left.sum()
        else:
            break
    race = p / noise
    order = np.sort(race)
    if V > 1 and order[-1] > 0:
        margin = min(margin, mass * (order[-1] - order[-2]) / order[-1])
    return path, int(race.argmax()), margin
