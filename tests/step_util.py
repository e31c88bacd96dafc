"""Plain 64-bit implementations of the operators of a prompt and between the products,
with the bounds of the tests (no library code)."""
from __future__ import annotations

import math

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# unit roundoff: half a step
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half a step below the normal range
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


def rounding(x, dtype):
    """How far a value near x may move when it is rounded to dtype, with 1 % for the
    error that it has already."""
    return 1.01 * ROUND[dtype] * x.abs() + TINY[dtype]


def assert_close(got, want, bound, what="out"):
    fine = torch.isfinite(want)
    got = got.double()
    assert torch.equal(got[~fine].nan_to_num(nan=7.0), want[~fine].nan_to_num(nan=7.0)), f"{what}: infinities and NaN"
    err = (got - want).abs()[fine] - bound.expand_as(want)[fine]
    worst = err.max().item() if err.numel() else 0.0
    assert worst <= 0, f"{what}: {worst} above its bound"


# ------------------------------------------------------------------ rotary positions
def turn(x, positions, freq, half, amplitude=1.0, heads=None):
    """(values, bound of their error before rounding) of x [..., H, D] turned by
    positions [...], frequencies in radians.

    The kernel's angle is exact but for its rounding to 24 bits of at most half a
    turn, 2 pi 2^-26; sincospi is off by at most 2 ulp (2^-23), times the amplitude
    2^-24 more: below 2^-21 in all.  The two products and their sum add 2^-23 at
    most: (|x| + |y|) A 2^-20 holds them all."""
    x = x.double()
    m = len(freq)
    heads = x.shape[-2] if heads is None else heads
    w = (positions.double()[..., None] * freq)[..., None, :]
    c, s = amplitude * w.cos(), amplitude * w.sin()
    a = slice(0, m) if half else slice(0, 2 * m, 2)
    b = slice(m, 2 * m) if half else slice(1, 2 * m, 2)
    out, err = x.clone(), torch.zeros_like(x)
    u, v = x[..., :heads, a], x[..., :heads, b]
    out[..., :heads, a], out[..., :heads, b] = u * c - v * s, u * s + v * c
    e = (u.abs() + v.abs()) * abs(amplitude) * 2.0 ** -20
    err[..., :heads, a], err[..., :heads, b] = e, e
    return out, err


# ------------------------------------------------------------------ packed prompts
class Prompt:
    """Pools, tables and packed rows of one call; lens and counts are host lists."""

    def __init__(self, dtype, D, Hq, Hkv, page, lens, counts, seed=0, layers=1, layer=0, extra_pages=3, extra_rows=0,
                 fill=None, sigma=1.0, strided=False, extra_columns=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = np.random.default_rng(seed)
        self.dtype, self.D, self.Hq, self.Hkv, self.page = TYPES[dtype], D, Hq, Hkv, page
        self.lens, self.counts, self.layer, self.B = list(lens), list(counts), layer, len(lens)
        need = [-(-(n + k) // page) for n, k in zip(lens, counts)]
        total = sum(need) + extra_pages
        ids = r.permutation(total)[:sum(need)]
        table = np.zeros((self.B, max(1, max(need)) + extra_columns), np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        self.table = torch.from_numpy(table).cuda()
        shape = (layers, total, Hkv, page, D)
        self.k_pool, self.v_pool = (torch.randn(shape, generator=g, device="cuda").to(self.dtype) for _ in range(2))
        if fill is not None:  # what stale rows hold: all that no sequence has
            for pool in (self.k_pool, self.v_pool):
                keep = torch.full_like(pool, fill)
                for b in range(self.B):
                    for j in range(self.lens[b] + self.counts[b]):
                        keep[:, table[b, j // page], :, j % page] = pool[:, table[b, j // page], :, j % page]
                pool.copy_(keep)
        self.starts = [0]
        for n in counts:
            self.starts.append(self.starts[-1] + n)
        self.N = self.starts[-1] + extra_rows
        if strided:
            self.q = (torch.randn(self.N, Hq + 3, D + 8, generator=g, device="cuda") * sigma).to(self.dtype)[:, 1:1 + Hq, :D]
        else:
            self.q = (torch.randn(self.N, Hq, D, generator=g, device="cuda") * sigma).to(self.dtype)
        self.d_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.d_starts = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        self.scale = D ** -0.5

    def make_cache(self, q, max_batch=None):
        return q.PagedCache(self.k_pool.shape[0], self.k_pool.shape[1], self.page, self.Hq, self.Hkv, self.D,
                            dtype=self.dtype, max_batch=max_batch or self.B, k_pool=self.k_pool, v_pool=self.v_pool)

    def call(self, cache, **kw):
        return cache.attend_prompt(self.layer, self.q, self.table, self.d_lens, self.d_starts, **kw)

    def rows(self, b):
        """Keys and values [Hkv, lens + counts, D] of sequence b."""
        n = self.lens[b] + self.counts[b]
        ids = self.table[b, :-(-n // self.page)].long()
        return [p[self.layer, ids].transpose(0, 1).reshape(self.Hkv, -1, self.D)[:, :n] for p in (self.k_pool, self.v_pool)]

    def reference(self):
        """(out, lse, bound of out, bound of lse) in 64 bits, for the rows that belong to
        a sequence.

        With u the 16-bit unit roundoff, A = sum p |v| / sum p and ds a bound of a
        score's fp32 error (products of 16-bit values are exact, D additions, each
        off by one unit in the last place at most, a 2-ulp exponential): |out - o|
        <= u (|o| + A) + 2 ds A, with u A for the rounded p.  In f16 p (at least 1
        at a row's maximum) also loses up to 2^-25 each below the normal range, and
        an output below it as much: 2^-25 (sum |v| + 1).  The lse is off by ds, the
        sum's and the logarithm's roundings."""
        n, Hq, D, g = self.starts[-1], self.Hq, self.D, self.Hq // self.Hkv
        out = torch.zeros(n, Hq, D, dtype=torch.float64, device="cuda")
        lse = torch.zeros(n, Hq, dtype=torch.float64, device="cuda")
        tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
        u = ROUND[self.dtype]
        for b in range(self.B):
            L, k = self.lens[b], self.counts[b]
            if k == 0:
                continue
            rows = slice(self.starts[b], self.starts[b + 1])
            keys, values = self.rows(b)
            see = torch.ones(k, L + k, dtype=torch.bool, device="cuda").tril(L)
            for h in range(Hq):
                kk, vv, qq = keys[h // g].double(), values[h // g].double(), self.q[rows, h].double()
                s = torch.where(see, qq @ torch.where(torch.isfinite(kk), kk, 0.0).T * self.scale, -math.inf)
                bad = ~torch.isfinite(kk).all(1)
                if bad.any():  # a key that is not finite: for those that see it alone
                    s = torch.where(see & bad, (qq[:, None] * kk).sum(-1) * self.scale, s)
                z = torch.logsumexp(s, 1)
                p = torch.exp(s - z[:, None])
                # values that are not finite count for the rows that see them alone
                fine = torch.isfinite(vv)
                clean = torch.where(fine, vv, 0.0)
                o, A = p @ clean, p @ clean.abs()
                for j in (~fine).any(1).nonzero().flatten().tolist():
                    o = torch.where(see[:, j, None] & ~fine[j], o + p[:, j, None] * vv[j], o)
                size = torch.where(see, qq.abs() @ kk.abs().nan_to_num(nan=0.0, posinf=0.0).T, 0.0).amax(1) * self.scale
                ds = size * (D + 4) * 2.0 ** -23 + 2.0 ** -20
                e = 1.01 * u * (o.abs() + A) + 2 * ds[:, None] * A
                if self.dtype == torch.float16:
                    e += 2.0 ** -25 * (see.double() @ clean.abs() + 1)
                out[rows, h], tol[rows, h], lse[rows, h] = o, e, z
                ltol[rows, h] = ds + 2.0 ** -20 * (1 + z.abs())
        return out, lse, tol, ltol


def check_prompt(p, out, lse):
    ref, lref, tol, ltol = p.reference()
    n = p.starts[-1]
    assert_close(out[:n], ref, tol, "out")
    assert_close(lse[:n], lref, ltol, "lse")


# ------------------------------------------------------------------ norms
SUMS = 2.0 ** -18  # relative, see normed()


def normed(x, e, weight, bias, eps, centered):
    """(norm(x) weight + bias, bound) for x whose entries are off by up to e.

    A sum of N entries runs over at most 32 of a thread and 10 levels of a tree: 42
    roundings of 2^-24 of its terms' magnitudes, below 2^-18.  The factor of the norm is a
    square root's inverse: half the mean square's relative error, which is at most 2
    |e| / |x| + 2^-18, and rsqrtf's 2 ulp."""
    n = x.shape[-1]
    if centered:
        mean = x.mean(-1, keepdim=True)
        e = e + (e + SUMS * x.abs()).mean(-1, keepdim=True) + 2.0 ** -22 * (x.abs() + mean.abs())
        x = x - mean
    ms = x.square().mean(-1, keepdim=True) + eps
    f = ms.rsqrt()
    df = e.square().mean(-1, keepdim=True).sqrt() * f + SUMS
    y = x * f * weight.double()
    d = weight.double().abs() * (f * e + x.abs() * f * df) * 1.01 + 2.0 ** -22 * y.abs()
    if bias is not None:
        y = y + bias.double()
        d = d + 2.0 ** -23 * y.abs()
    return y, d


def residual_norm(r, y, weight, bias, post_weight, post_bias, gate, scale, eps, centered):
    """((r', bound), (h, bound)) before their rounding."""
    x = r.double()
    e = torch.zeros_like(x)
    if y is not None:
        z = y.double()
        if post_weight is not None:
            z, ez = normed(z, e, post_weight, post_bias, eps, centered)
        else:
            ez = torch.zeros_like(z)
        g = 1.0 if gate is None else gate.double()
        ga = 1.0 if gate is None else gate.double().abs()
        add = scale * g * z
        x = x + add
        e = abs(scale) * ga * ez + 2.0 ** -22 * (add.abs() + x.abs())
    return (x, e), (None if weight is None else normed(x, e, weight, bias, eps, centered))


# ------------------------------------------------------------------ scores
def words(bits):
    """Truth values [..., n] as int32 words, entry v in bit v % 32 of word v // 32."""
    n = bits.shape[-1]
    pad = np.zeros(bits.shape[:-1] + (-(-n // 32) * 32,), bool)
    pad[..., :n] = bits
    packed = np.packbits(pad, axis=-1, bitorder="little")
    return torch.from_numpy(packed.view("<u4").astype(np.int64).astype(np.uint32).view(np.int32)).cuda()


def adjust(scores, tokens, parents, counts, prompt, repetition, frequency, presence, bias, mask):
    """numpy: scores [T, V] of one sequence, adjusted in 64 bits, and a bound of the fp32
    error: each of the at most four operations rounds what it has by 2^-24, the inverse
    of the repetition penalty 2^-24 more."""
    T, V = scores.shape
    out, err = np.zeros((T, V)), np.zeros((T, V))
    for t in range(T):
        c = np.zeros(V) if counts is None else counts.astype(np.float64).copy()
        node = t
        while node > 0:
            x = -1 if tokens is None else tokens[node]
            if 0 <= x < V:
                c[x] += 1
            up = node - 1 if parents is None else parents[node]
            if up >= node:
                break
            node = up
        x = scores[t].astype(np.float64)
        seen = c > 0 if prompt is None else (c > 0) | prompt
        with np.errstate(invalid="ignore", over="ignore"):
            x = np.where(seen, np.where(x > 0, x / repetition, x * repetition), x)
            e = np.abs(x) + abs(frequency) * c + abs(presence)
            x = x - frequency * c - presence * (c > 0)
            if bias is not None:
                x = x + bias
                e = e + np.abs(bias)
        if mask is not None:
            x = np.where(mask[t], x, -np.inf)
        out[t], err[t] = x, np.where(np.isfinite(e), e, 0.0) * 2.0 ** -21
    return out, err
