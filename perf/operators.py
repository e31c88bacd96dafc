"""Workloads of the token-tree operators: tree attention over a paged cache,
verification of drafted tokens by rejection sampling, compaction of the cache
after it, and copies of cache pages.

Every case is one call of one operator.  With ``own`` false ``run`` computes it
with elementary torch operations in 32 bits; with ``own`` true it calls the
library.  The operators:

  attend  B sequences, T drafted nodes each.  Key/value rows of the nodes are
          written behind the ``lens[b]`` cached ones, and node t attends to all
          cached rows and to the nodes named by the bits of ``mask[b][t]``:
          out = softmax(scale q k^T) v, lse = log sum exp.  Nodes at or past
          ``n_tokens[b]`` give zeros and -inf.
  sample  Walk from node 0: with P, Q = softmax(target), softmax(draft) of the
          node over the temperature, its children c are tried in index order;
          c is accepted if u[c] Q(x) < P(x), x = tokens[c]; else
          P <- max(P - Q, 0) and Q <- Q without x, both normalised (P is kept
          where nothing is left).  Without draft scores Q is 1 at x.  The walk
          ends where no child is accepted, with the token argmax P / noise.
  commit  In every layer, rows lens[b] + path[b][j] move to lens[b] + 1 + j for
          j < accept[b][0]; the new length is lens[b] + 1 + accept[b][0].
  copy    In every layer, the first rows[i] rows of page src[i] go to dst[i].
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the smallest step: one sequence, one token, a short prompt; 40 query and 20 key/value
        # heads of 128 are what a 5120 -> 10240 qkv projection with a 5120-wide output holds
        dict(name="attend one token", op="attend", B=1, T=1, Hq=40, Hkv=20, D=128, L=512, page=16,
             type="bf16", tree=False, ragged=False),
        # plain decoding of a batch with mixed lengths, eight query heads to a key/value head
        dict(name="attend decode batch", op="attend", B=32, T=1, Hq=64, Hkv=8, D=128, L=8192, page=16,
             type="bf16", tree=False, ragged=True),
        # odd everything: 15 drafted nodes, three heads to a group, head size 64, mixed lengths and widths
        dict(name="attend odd trees", op="attend", B=13, T=15, Hq=24, Hkv=8, D=64, L=4097, page=32,
             type="f16", tree=True, ragged=True),
        # wide trees over long prompts: the products, not the cache, are the work
        dict(name="attend wide trees", op="attend", B=4, T=64, Hq=64, Hkv=8, D=128, L=16384, page=64,
             type="bf16", tree=True, ragged=False),
        # one very long sequence: the cache's length is split over the whole GPU
        dict(name="attend long context", op="attend", B=1, T=8, Hq=40, Hkv=20, D=128, L=131071, page=128,
             type="bf16", tree=True, ragged=False),
        # a drafted chain of one sequence on the 151,936-entry vocabulary: a call's latency
        dict(name="sample one chain", op="sample", B=1, T=8, V=151936, type="f32", tree=False, draft=True),
        # a served batch of drafted blocks of 16
        dict(name="sample chain batch", op="sample", B=32, T=16, V=151936, type="bf16", tree=False, draft=True),
        # wide trees, many siblings, an odd vocabulary
        dict(name="sample trees", op="sample", B=4, T=64, V=50257, type="f32", tree=True, draft=True),
        # one accepted branch of one sequence
        dict(name="commit one branch", op="commit", B=1, T=8, Hkv=20, D=128, layers=16, L=300, page=16,
             type="bf16"),
        # a batch of branches in every layer of a 64-layer model
        dict(name="commit batch", op="commit", B=64, T=32, Hkv=20, D=128, layers=64, L=100, page=16, type="bf16"),
        # forking one sequence: its last, partly filled page
        dict(name="copy fork", op="copy", n=3, Hkv=20, D=128, layers=16, page=16, type="bf16"),
        # moving whole sequences' pages apart
        dict(name="copy many pages", op="copy", n=255, Hkv=8, D=128, layers=64, page=32, type="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "sample", "sample", "commit", "copy"])
    if op == "attend":
        Hq, Hkv = rng.choice([(40, 20), (64, 8), (32, 4), (16, 16), (24, 8), (8, 1)])
        c = dict(op=op, B=_log(rng, 1, 64), T=_log(rng, 1, 64), Hq=Hq, Hkv=Hkv, D=rng.choice([64, 128]),
                 L=_log(rng, 1, 65536), page=rng.choice([16, 32, 64, 128]), type=rng.choice(["bf16", "f16"]),
                 tree=rng.random() < 0.6, ragged=rng.random() < 0.6)
        while c["B"] > 1 and (c["B"] * c["L"] * Hkv * c["D"] > 200e6 or c["B"] * c["L"] * Hq * c["T"] > 250e6):
            c["B"] -= 1
        while c["L"] * Hq * c["T"] > 250e6:
            c["L"] = c["L"] * 3 // 4
        return c
    if op == "sample":
        c = dict(op=op, B=_log(rng, 1, 48), T=_log(rng, 2, 64), V=_log(rng, 500, 260000),
                 type=rng.choice(["f32", "bf16", "f16"]), tree=rng.random() < 0.5, draft=rng.random() < 0.75)
        while c["B"] > 1 and c["B"] * c["T"] * c["V"] > 70e6:
            c["B"] -= 1
        return c
    if op == "commit":
        return dict(op=op, B=_log(rng, 1, 64), T=_log(rng, 4, 64), Hkv=rng.choice([1, 4, 8, 20]),
                    D=rng.choice([64, 128]), layers=_log(rng, 1, 64), L=_log(rng, 1, 200),
                    page=rng.choice([16, 32, 64, 128]), type=rng.choice(["bf16", "f16"]))
    c = dict(op=op, n=_log(rng, 1, 255), Hkv=rng.choice([1, 4, 8, 20]), D=rng.choice([64, 128]),
             layers=_log(rng, 1, 64), page=rng.choice([16, 32, 64, 128]), type=rng.choice(["bf16", "f16"]))
    while c["n"] > 1 and c["n"] * c["layers"] * c["Hkv"] * c["page"] * c["D"] > 500e6:
        c["n"] -= 1
    return c


def _lengths(c):
    """Cached rows and drafted nodes of every sequence (of the case, not of the seed)."""
    r = random.Random(c["B"] * 1000003 + c["L"])
    if not c.get("ragged"):
        return [c["L"]] * c["B"], [c["T"]] * c["B"]
    return ([r.randint(c["L"] // 4, c["L"]) for _ in range(c["B"])],
            [r.randint(max(1, c["T"] // 2), c["T"]) for _ in range(c["B"])])


def _accepted(c):
    """Accepted nodes of every sequence: at most half of them, so that a branch past them has room."""
    most = (c["T"] - 1) // 2
    return [(7 * b + most) % (most + 1) for b in range(c["B"])]


def _copied(c):
    """Rows of every copied page: half of them are full."""
    return [c["page"] if i % 2 else 1 + (5 * i + c["page"] // 2) % c["page"] for i in range(c["n"])]


def work(c):
    size = 4 if c["type"] == "f32" else 2
    if c["op"] == "attend":
        lens, counts = _lengths(c)
        row = c["Hkv"] * c["D"] * size * 2  # a key and a value row
        io = 2 * c["B"] * c["T"] * c["Hq"] * c["D"] * size + 4 * c["B"] * c["T"] * c["Hq"]
        return {"bytes": float(sum(lens) * row + 2 * sum(counts) * row + io),
                "flops": float(sum(4 * n * (L + n) * c["Hq"] * c["D"] for L, n in zip(lens, counts)))}
    if c["op"] == "sample":
        # what no outcome can do without: the root's scores and the random numbers of the last token
        per = c["V"] * (size * (2 if c["draft"] else 1) + 4)
        return {"bytes": float(c["B"] * per), "flops": float(c["B"] * c["V"] * 12)}
    row = c["Hkv"] * c["D"] * size * 2 * c["layers"]
    moved = sum(_accepted(c)) if c["op"] == "commit" else sum(_copied(c))
    return {"bytes": float(2 * max(1, moved) * row), "flops": 0.0}


# ------------------------------------------------------------------ inputs
def _pages(c, counts, g):
    """A page table that scatters every sequence's pages over the pool, and the pool's size."""
    need = [(n + c["page"] - 1) // c["page"] for n in counts]
    total = sum(need)
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    width = max(need)
    table = torch.zeros(len(need), width, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, total


def _pools(c, layers, n_pages, g):
    """Pages that were used before: whatever they hold is a row like any other."""
    shape = (layers, n_pages, c["Hkv"], c["page"], c["D"])
    return [torch.randn(shape, generator=g, device="cuda", dtype=TYPES[c["type"]]) for _ in range(2)]


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _parents(c, r):
    """Drafted trees: every node's parent comes before it, a few places back."""
    return [[-1] + [r.randint(max(0, i - 6), i - 1) if c["tree"] else i - 1 for i in range(1, c["T"])]
            for _ in range(c["B"])]


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = random.Random(seed)
    s = dict(c)
    if c["op"] == "attend":
        lens, counts = _lengths(c)
        B, T, Hq, Hkv, D = (c[k] for k in ("B", "T", "Hq", "Hkv", "D"))
        s["table"], n_pages = _pages(c, [n + T for n in lens], g)
        s["k_pool"], s["v_pool"] = _pools(c, 1, n_pages, g)
        # one projection's result holds queries, keys and values side by side
        qkv = torch.randn(B, T, Hq + 2 * Hkv, D, generator=g, device="cuda")
        qkv[:, :, :Hq] *= 1.5
        qkv = qkv.to(TYPES[c["type"]])
        s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        s["lens"], s["n_tokens"] = _int(lens), _int(counts)
        masks = []
        for par in _parents(c, r):
            m = [1]
            for i in range(1, T):
                m.append(m[par[i]] | 1 << i)
            masks.append([x - (1 << 64) if x >> 63 else x for x in m])
        s["mask"] = torch.tensor(masks, dtype=torch.int64, device="cuda")
        if own:
            s["cache"] = _cache(s, 1, n_pages)
    elif c["op"] == "sample":
        B, T, V = c["B"], c["T"], c["V"]
        target = torch.randn(B, T, V, generator=g, device="cuda").mul_(2)
        top = torch.randint(V, (B, T, min(16, V)), generator=g, device="cuda")
        lift = 13 - torch.arange(top.shape[2], device="cuda") * 0.6 + torch.randn(top.shape, generator=g, device="cuda")
        target.scatter_add_(2, top, lift)
        draft = target + torch.randn(B, T, V, generator=g, device="cuda").mul_(0.7)
        par = _parents(c, r)
        rank = [[sum(p[j] == p[i] for j in range(1, i)) for i in range(T)] for p in par]
        s["parents"] = _int(par)
        # siblings are drawn from their parent's draft scores without replacement
        noisy = draft - torch.empty_like(draft).exponential_(generator=g).log_() if c["draft"] else draft
        order = noisy.topk(min(V, 1 + max(map(max, rank))), dim=2).indices
        rows = torch.arange(B, device="cuda")[:, None]
        s["tokens"] = order[rows, s["parents"].long().clamp(min=0), _int(rank).long()].to(torch.int32).contiguous()
        s["target"] = target.to(TYPES[c["type"]])
        s["draft"] = draft.to(TYPES[c["type"]]) if c["draft"] else None
        s["u"] = torch.rand(B, T, generator=g, device="cuda")
        s["noise"] = torch.empty(B, V, device="cuda").exponential_(generator=g)
        s["temperature"] = 0.7 + 0.5 * torch.rand(B, generator=g, device="cuda")
        del target, draft, noisy
    elif c["op"] == "commit":
        B, T = c["B"], c["T"]
        lens = [c["L"] - (3 * b) % max(1, c["L"] // 2) for b in range(B)]
        s["table"], n_pages = _pages(c, [n + T for n in lens], g)
        s["k_pool"], s["v_pool"] = _pools(c, c["layers"], n_pages, g)
        k = _accepted(c)
        # a branch whose nodes lie past the places that they move to
        path = [sorted(r.sample(range(n + 1, T), n)) + [-1] * (T - n) for n in k]
        s["lens"], s["path"] = _int(lens), _int(path)
        s["accept"] = _int([[n, 5] for n in k])
        if own:
            s["cache"] = _cache(s, c["layers"], n_pages)
    else:
        n = c["n"]
        s["k_pool"], s["v_pool"] = _pools(c, c["layers"], 2 * n, g)
        ids = torch.randperm(2 * n, generator=g, device="cuda").to(torch.int32)
        s["src"], s["dst"], s["rows"] = ids[:n].contiguous(), ids[n:].contiguous(), _int(_copied(c))
        if own:
            s["cache"] = _cache(s, c["layers"], 2 * n)
    return s


def _cache(s, layers, n_pages):
    import speculative_decode_verification_qmm_gb300 as q
    return q.PagedCache(layers, n_pages, s["page"], s.get("Hq", s["Hkv"]), s["Hkv"], s["D"], dtype=TYPES[s["type"]],
                        max_batch=s.get("B", 1), k_pool=s["k_pool"], v_pool=s["v_pool"])


# ------------------------------------------------------------------ one pass
def run(s):
    if s["op"] == "attend":
        if own:
            out, lse = s["cache"].attend(0, s["q"], s["k"], s["v"], s["table"], s["lens"], mask=s["mask"],
                                         n_tokens=s["n_tokens"])
        else:
            out, lse = _attend(s)
        return out, lse, s["k_pool"], s["v_pool"]
    if s["op"] == "sample":
        if own:
            import speculative_decode_verification_qmm_gb300 as q
            return q.verify_sample(s["target"], s["draft"], s["tokens"], s["u"], s["noise"], parents=s["parents"],
                                   temperature=s["temperature"])
        return _sample(s)
    if s["op"] == "commit":
        lens = s["cache"].commit(s["table"], s["lens"], s["path"], s["accept"]) if own else _commit(s)
        return lens, s["k_pool"], s["v_pool"]
    if own:
        s["cache"].copy_pages(s["src"], s["dst"], s["rows"])
    else:
        _copy(s)
    return s["k_pool"], s["v_pool"]


def _attend(s):
    B, T, Hq, Hkv, D, page = (s[k] for k in ("B", "T", "Hq", "Hkv", "D", "page"))
    node = torch.arange(T, device="cuda")
    live = node < s["n_tokens"][:, None]
    pos = s["lens"][:, None] + node
    at = s["table"].long().gather(1, pos // page), pos.long() % page
    kv = []
    for pool, new in ((s["k_pool"][0], s["k"]), (s["v_pool"][0], s["v"])):
        pool[at[0], :, at[1]] = torch.where(live[:, :, None, None], new, pool[at[0], :, at[1]])
        kv.append(pool[s["table"].long()].transpose(1, 2).reshape(B, Hkv, -1, D).float())
    q = s["q"].float().reshape(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    scores = torch.matmul(q, kv[0].transpose(2, 3)).mul_(D ** -0.5).view(B, Hkv, Hq // Hkv, T, -1)
    j = torch.arange(scores.shape[-1], device="cuda")
    back = j - s["lens"][:, None]  # the key's node, where it is one
    bit = (s["mask"][:, :, None] >> back.clamp(0, 63)[:, None]) & 1
    seen = (back < 0)[:, None] | (bit.bool() & ((back >= 0) & (back < s["n_tokens"][:, None]))[:, None])
    seen = (seen & live[:, :, None])[:, None, None]
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = (scores - top.clamp(min=-3e38)).exp_()
    total = p.sum(-1)
    out = torch.matmul(p.view(B, Hkv, -1, p.shape[-1]), kv[1]).view(B, Hkv, Hq // Hkv, T, D)
    out = torch.where(total[..., None] > 0, out / total[..., None], 0.0)
    lse = top[..., 0] + total.log()
    return (out.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(s["q"].dtype),
            lse.permute(0, 3, 1, 2).reshape(B, T, Hq).contiguous())


def _softmax(x):
    e = (x - x.amax(1, keepdim=True)).exp()
    return e / e.sum(1, keepdim=True)


def _sample(s):
    B, T = s["B"], s["T"]
    t = s["temperature"][:, None]
    row = torch.arange(B, device="cuda")
    here = torch.zeros(B, dtype=torch.int64, device="cuda")
    count = torch.zeros(B, dtype=torch.int64, device="cuda")
    path = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    P = _softmax(s["target"][:, 0].float() / t)
    Q = _softmax(s["draft"][:, 0].float() / t) if s["draft"] is not None else torch.zeros_like(P)
    # every parent comes before its children, so one walk over the nodes meets them in order
    for i in range(1, T):
        x = s["tokens"][:, i].long()
        if s["draft"] is None:
            Q = torch.zeros_like(P).index_put_((row, x), torch.ones(B, device="cuda"))
        tried = s["parents"][:, i] == here
        yes = tried & (s["u"][:, i] * Q[row, x] < P[row, x])
        no = (tried & ~yes)[:, None]
        left = (P - Q).clamp(min=0)
        mass = left.sum(1, keepdim=True)
        P = torch.where(no & (mass > 0), left / mass, P)
        rest = Q.index_put((row, x), torch.zeros(B, device="cuda"))
        mass = rest.sum(1, keepdim=True)
        Q = torch.where(no, torch.where(mass > 0, rest / mass, rest), Q)
        P = torch.where(yes[:, None], _softmax(s["target"][:, i].float() / t), P)
        if s["draft"] is not None:
            Q = torch.where(yes[:, None], _softmax(s["draft"][:, i].float() / t), Q)
        path[row, count] = torch.where(yes, i, path[row, count])
        here = torch.where(yes, i, here)
        count = count + yes
    last = (P / s["noise"]).argmax(1)
    return torch.stack([count, last], 1).to(torch.int32), path


def _commit(s):
    page, T = s["page"], s["T"]
    j = torch.arange(T - 1, device="cuda")
    live = j < s["accept"][:, :1]
    old = s["lens"][:, None] + s["path"][:, :T - 1].clamp(min=0)
    new = s["lens"][:, None] + 1 + j
    table = s["table"].long()
    src = table.gather(1, old.long() // page), old.long() % page
    dst = table.gather(1, new // page), new % page
    for pool in (s["k_pool"], s["v_pool"]):
        pool[:, dst[0], :, dst[1]] = torch.where(live[:, :, None, None, None], pool[:, src[0], :, src[1]],
                                                 pool[:, dst[0], :, dst[1]])
    return s["lens"] + 1 + s["accept"][:, 0]


def _copy(s):
    live = (torch.arange(s["page"], device="cuda") < s["rows"][:, None])[None, :, None, :, None]
    src, dst = s["src"].long(), s["dst"].long()
    for pool in (s["k_pool"], s["v_pool"]):
        pool[:, dst] = torch.where(live, pool[:, src], pool[:, dst])


# ------------------------------------------------------------------ in 64 bits
def exact(c, seed):
    """The definition, sequence by sequence, in 64 bits.  Moves and copies compute
    nothing; the attended outputs and the sampled walks are returned."""
    global own
    if c["op"] in ("commit", "copy"):
        return None
    kept, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = kept
    return (_exact_attend if c["op"] == "attend" else _exact_sample)(c, s)


def _exact_attend(c, s):
    B, T, Hq, Hkv, D, page = (c[k] for k in ("B", "T", "Hq", "Hkv", "D", "page"))
    lens, counts = _lengths(c)
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        L, n = lens[b], counts[b]
        ids = s["table"][b, :(L + page - 1) // page].long()
        bits = [[m >> i & 1 for i in range(n)] for m in s["mask"][b, :n].tolist()]
        seen = torch.ones(n, L + n, dtype=torch.bool, device="cuda")
        seen[:, L:] = torch.tensor(bits, device="cuda").bool()
        for h in range(Hkv):
            k, v = (torch.cat([pool[0, ids, h].reshape(-1, D)[:L], new[b, :n, h]]).double()
                    for pool, new in ((s["k_pool"], s["k"]), (s["v_pool"], s["v"])))
            for a in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                z = s["q"][b, :n, a].double() @ k.T / math.sqrt(D)
                z[~seen] = -math.inf
                lse[b, :n, a] = torch.logsumexp(z, 1)
                out[b, :n, a] = torch.exp(z - lse[b, :n, a, None]) @ v
    return out, lse, None, None


def _exact_sample(c, s):
    accept, paths = [], []
    for b in range(c["B"]):
        t = float(s["temperature"][b])
        tokens, parents, u = s["tokens"][b].tolist(), s["parents"][b].tolist(), s["u"][b].tolist()
        node, path = 0, []
        while True:
            p = torch.softmax(s["target"][b, node].double() / t, 0)
            q = torch.softmax(s["draft"][b, node].double() / t, 0) if c["draft"] else None
            taken = None
            for k in (i for i in range(node + 1, c["T"]) if parents[i] == node):
                x = tokens[k]
                if u[k] * (1.0 if q is None else float(q[x])) < float(p[x]):
                    taken = k
                    break
                left = p.clone()
                if q is None:
                    left[x] = 0
                else:
                    left = (left - q).clamp_(min=0)
                    q[x] = 0
                    q /= max(float(q.sum()), 1e-300)
                if float(left.sum()) > 0:
                    p = left / left.sum()
            if taken is None:
                break
            node = taken
            path.append(taken)
        accept.append([len(path), int((p / s["noise"][b].double()).argmax())])
        paths.append(path + [-1] * (c["T"] - len(path)))
    return _int(accept), _int(paths)
