"""Workloads of the operators around a prompt's and a drafted step's products:
rotary positions, appending to the paged cache, attention of a prompt over it,
residual sums with their norms, and the adjustment of scores before sampling.

Every case is one call of one operator.  With ``own`` false ``run`` computes it
with elementary torch operations in 32 bits; with ``own`` true it calls the
library.  The operators:

  rotate  The first ``rotated`` of H heads are turned by their row's position:
          of each of the pairs of the first ``dims`` dimensions, (x, y) becomes
          a (x cos w - y sin w, x sin w + y cos w), w = position * frequency.
          What is not turned is converted to the output's type.
  append  Packed rows; row i of sequence b becomes row lens[b] + i of the paged
          cache, its key turned by that position; its queries come back turned.
  prompt  Packed queries of rows that the cache holds already: row i of sequence
          b attends to the cache's rows j <= lens[b] + i.
          out = softmax(q k^T / sqrt(D)) v, lse = log sum exp.
  norm    r' = r + scale gate z and h = norm(r') weight, with z = y or
          norm(y) post; norm(x) = x / sqrt(mean x^2 + eps), or, centered, the
          same of x - mean x, plus a bias.
  adjust  Scores after each node of a drafted tree.  c(v) is how often v was
          emitted, before the tree and on the node's own path after the root;
          where c(v) > 0 or v is in the prompt, x becomes x / r for x > 0 and
          x r otherwise; then x - f c - p [c > 0] + bias, and -inf where the
          node's grammar bit is 0.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one sequence's drafted block after the qkv product (5120 -> 10240: 40 + 20 + 20 heads of
        # 128 in fp32): latency counts
        dict(name="rotate one step", op="rotate", B=1, T=8, H=80, rotated=60, D=128, dims=128, src="f32", type="bf16",
             half=True, scaled=False, far=4096),
        # queries of a long prompt, a quarter of the head turned, frequencies scaled for long contexts
        dict(name="rotate part of the head", op="rotate", B=3, T=1367, H=36, rotated=33, D=96, dims=24, src="bf16",
             type="f16", half=False, scaled=True, far=131072),
        # single tokens of a served batch
        dict(name="append single tokens", op="append", B=16, n=1, L=1000, page=16, Hq=40, Hkv=20, D=128, dims=128,
             src="f32", type="bf16", half=True, scaled=False, ragged=True),
        # one prompt from the prefill product
        dict(name="append a prompt", op="append", B=1, n=8192, L=0, page=16, Hq=40, Hkv=20, D=128, dims=128,
             src="f32", type="bf16", half=True, scaled=False, ragged=False),
        # the smallest prompt: a question of some dozens of tokens
        dict(name="prompt of 75 tokens", op="prompt", B=1, n=75, L=0, page=16, Hq=40, Hkv=20, D=128, type="bf16",
             ragged=False),
        # mixed prompts in one call, odd lengths, some behind a shared prefix; 64-wide heads, seven to a group
        dict(name="prompt batch, ragged", op="prompt", B=9, n=1501, L=700, page=32, Hq=28, Hkv=4, D=64, type="f16",
             ragged=True),
        # one long prompt in one piece
        dict(name="prompt of 8192 tokens", op="prompt", B=1, n=8192, L=0, page=16, Hq=40, Hkv=20, D=128, type="bf16",
             ragged=False),
        # the last piece of a very long prompt: few rows over many cached ones
        dict(name="prompt piece behind 65536", op="prompt", B=1, n=512, L=65536, page=64, Hq=64, Hkv=8, D=128,
             type="bf16", ragged=False),
        # between two products of a drafted step
        dict(name="norm one step", op="norm", M=8, N=5120, res="f32", y="f32", type="bf16", post=False, gate=False,
             centered=False),
        # between two products of a prompt, norms on both sides of the block and a gate
        dict(name="norm a prompt", op="norm", M=8192, N=5120, res="bf16", y="f32", type="bf16", post=True, gate=True,
             centered=False),
        # penalties for one drafted tree on the 151,936-entry vocabulary
        dict(name="adjust one tree", op="adjust", B=1, T=8, V=151936, type="f32", tree=True, bias=False, mask=False),
        # a served batch of drafted blocks of 16 under grammars and biases
        dict(name="adjust a batch", op="adjust", B=32, T=16, V=151936, type="bf16", tree=False, bias=True, mask=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _some(rng, name, *choices):
    return {name: rng.choice(choices)}


def draw(rng):
    op = rng.choice(["rotate", "append", "append", "prompt", "prompt", "prompt", "norm", "norm", "adjust", "adjust"])
    c = dict(op=op)
    if op in ("append", "prompt"):
        c["Hq"], c["Hkv"] = rng.choice([(40, 20), (64, 8), (32, 4), (12, 12), (28, 4), (8, 1)])
        c |= dict(D=rng.choice([64, 128]), type=rng.choice(["bf16", "f16"]), page=rng.choice([16, 32, 64, 128]),
                  B=_log(rng, 1, 48), n=_log(rng, 1, 8192), L=rng.choice([0, _log(rng, 1, 60000)]),
                  ragged=rng.random() < 0.6)
    if op == "rotate":
        D = rng.choice([48, 64, 80, 96, 128, 256])
        c |= dict(B=_log(rng, 1, 64), T=_log(rng, 1, 4096), H=rng.randint(1, 96), D=D, dims=2 * rng.randint(D // 8, D // 2),
                  src=rng.choice(["f32", "f32", "bf16", "f16"]), type=rng.choice(["bf16", "f16", "f32"]))
        c |= dict(rotated=rng.randint((c["H"] + 1) // 2, c["H"]), half=rng.random() < 0.5, scaled=rng.random() < 0.5,
                  far=_log(rng, 100, 500000))
        while c["T"] > 1 and c["B"] * c["T"] * c["H"] * D > 60e6:
            c["T"] = c["T"] * 3 // 4
    elif op == "append":
        c |= dict(src=rng.choice(["f32", "f32", c["type"]]), half=rng.random() < 0.5, scaled=rng.random() < 0.5,
                  dims=rng.choice([c["D"], c["D"], c["D"] // 2, c["D"] // 4]))
        heads = (c["Hq"] + 2 * c["Hkv"]) * c["D"]
        while c["n"] > 1 and c["B"] * c["n"] * heads > 80e6:
            c["n"] = c["n"] * 3 // 4
        while c["B"] > 1 and c["B"] * c["L"] * c["Hkv"] * c["D"] > 100e6:
            c["B"] = c["B"] * 3 // 4
    elif op == "prompt":
        while c["B"] > 1 and (c["B"] * (c["L"] + c["n"]) * c["Hkv"] * c["D"] > 100e6 or c["B"] * c["n"] > 16384):
            c["B"] = c["B"] * 3 // 4
        while c["B"] * c["n"] * (c["L"] + c["n"]) * c["Hq"] * c["D"] > 2.7e11:
            c["n"], c["L"] = max(1, c["n"] * 3 // 4), c["L"] * 3 // 4
    elif op == "norm":
        c |= dict(M=_log(rng, 1, 20000), N=_log(rng, 32, 20000), post=rng.random() < 0.5, gate=rng.random() < 0.5,
                  centered=rng.random() < 0.3)
        c |= _some(rng, "res", "f32", "bf16", "f16") | _some(rng, "y", "f32", "bf16", "f16")
        c |= _some(rng, "type", "bf16", "f16", "f32")
        while c["M"] > 1 and c["M"] * c["N"] > 28e6:
            c["M"] = c["M"] * 3 // 4
    else:
        c |= dict(B=_log(rng, 1, 48), T=_log(rng, 1, 64), V=_log(rng, 500, 260000), type=rng.choice(["f32", "bf16", "f16"]),
                  tree=rng.random() < 0.5, bias=rng.random() < 0.5, mask=rng.random() < 0.5)
        while c["B"] > 1 and c["B"] * c["T"] * c["V"] > 48e6:
            c["B"] -= 1
    return c


def _lengths(c):
    """Cached and new rows of every sequence (of the case, not of the seed)."""
    if not c["ragged"]:
        return [c["L"]] * c["B"], [c["n"]] * c["B"]
    r = random.Random(c["B"] * 1000003 + c["L"] + c["n"])
    return ([r.randint(c["L"] // 4, c["L"]) for _ in range(c["B"])],
            [r.randint(max(1, c["n"] // 4), c["n"]) for _ in range(c["B"])])


def _size(t):
    return 4 if t == "f32" else 2


def work(c):
    if c["op"] == "rotate":
        n = c["B"] * c["T"] * c["H"] * c["D"]
        return {"bytes": float(n * (_size(c["src"]) + _size(c["type"])) + 4 * c["B"] * c["T"]),
                "flops": float(3 * c["B"] * c["T"] * c["rotated"] * c["dims"])}
    if c["op"] == "append":
        rows = sum(_lengths(c)[1])
        n = rows * (c["Hq"] + 2 * c["Hkv"]) * c["D"]
        return {"bytes": float(n * (_size(c["src"]) + 2)), "flops": float(3 * rows * (c["Hq"] + c["Hkv"]) * c["dims"])}
    if c["op"] == "prompt":
        lens, counts = _lengths(c)
        seen = sum(n * L + n * (n + 1) // 2 for L, n in zip(lens, counts))
        kv = sum(L + n for L, n in zip(lens, counts)) * c["Hkv"] * c["D"] * 4
        return {"bytes": float(kv + sum(counts) * c["Hq"] * (4 * c["D"] + 4)),
                "flops": float(4 * seen * c["Hq"] * c["D"])}
    if c["op"] == "norm":
        per = 2 * _size(c["res"]) + _size(c["y"]) + _size(c["type"])
        return {"bytes": float(c["M"] * c["N"] * per), "flops": float(c["M"] * c["N"] * (14 if c["post"] else 8))}
    rows = c["B"] * c["T"]
    per_row = 2 * _size(c["type"]) * c["V"] + (c["V"] / 8 if c["mask"] else 0)
    return {"bytes": float(rows * per_row + c["B"] * c["V"] * (4 + 1 / 8) + (4 * c["V"] if c["bias"] else 0)),
            "flops": float(rows * c["V"] * 6)}


# ------------------------------------------------------------------ inputs
def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _frequencies(c):
    """Radians a position, in 64 bits: base^(-2 i / dims), and for a context eight times the trained
    8,192 positions slow ones divided by 8, fast ones kept, those between blended."""
    freq = 10000.0 ** (-torch.arange(0, c["dims"], 2, dtype=torch.float64) / c["dims"])
    if not c["scaled"]:
        return freq.cuda(), 1.0
    turns = 8192 * freq / (2 * math.pi)
    keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
    return (freq * (keep + (1 - keep) / 8)).cuda(), 0.1 * math.log(8) + 1


def _rope(s):
    import speculative_decode_verification_qmm_gb300 as q
    return q.Rope(s["freq"], layout="half" if s["half"] else "interleaved", amplitude=s["amplitude"])


def _paged(s, g):
    """A page table that scatters every sequence's pages over pools that were used before."""
    s["page_counts"] = need = [max(1, -(-(L + n) // s["page"])) for L, n in zip(*_lengths(s))]
    ids = torch.randperm(sum(need) + 2, generator=g, device="cuda").to(torch.int32)
    s["table"] = torch.zeros(len(need), max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        s["table"][b, :n] = ids[at:at + n]
        at += n
    shape = (1, sum(need) + 2, s["Hkv"], s["page"], s["D"])
    s["k_pool"], s["v_pool"] = [torch.randn(shape, generator=g, device="cuda", dtype=TYPES[s["type"]]) for _ in range(2)]
    lens, counts = _lengths(s)
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    s["lens"], s["starts"], s["rows"] = _int(lens), _int(starts), starts[-1]
    if own:
        import speculative_decode_verification_qmm_gb300 as q
        s["cache"] = q.PagedCache(1, shape[1], s["page"], s["Hq"], s["Hkv"], s["D"], dtype=TYPES[s["type"]],
                                  max_batch=s["B"], k_pool=s["k_pool"], v_pool=s["v_pool"])


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = random.Random(seed)
    s = dict(c)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if c["op"] in ("rotate", "append"):
        s["freq"], s["amplitude"] = _frequencies(c)
        if own:
            s["rope"] = _rope(s)
    if c["op"] == "rotate":
        B, T = c["B"], c["T"]
        s["x"] = normal(B, T, c["H"], c["D"]).to(TYPES[c["src"]])
        first = torch.randint(c["far"], (B, 1), generator=g, device="cuda")
        # the nodes of a drafted tree, or a prompt's rows: one after the other, some side by side
        s["positions"] = (first + torch.arange(T, device="cuda") * 3 // 4).to(torch.int32)
    elif c["op"] == "append":
        _paged(s, g)
        # one product's result holds queries, keys and values side by side
        qkv = normal(s["rows"], c["Hq"] + 2 * c["Hkv"], c["D"]).to(TYPES[c["src"]])
        s["q"], s["k"], s["v"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], 1)
    elif c["op"] == "prompt":
        _paged(s, g)
        s["q"] = (1.5 * normal(s["rows"], c["Hq"], c["D"])).to(TYPES[c["type"]])
    elif c["op"] == "norm":
        M, N = c["M"], c["N"]
        # a stream whose rows differ in size and have a few large channels; a block's output
        s["r"] = (normal(M, N) * (0.5 + 2 * torch.rand(M, 1, generator=g, device="cuda"))).to(TYPES[c["res"]])
        s["r"][:, r.randrange(N)] *= 20
        s["v"] = (0.7 * normal(M, N)).to(TYPES[c["y"]])
        s["weight"], s["bias"] = 1 + 0.2 * normal(N), 0.1 * normal(N) if c["centered"] else None
        s["post"] = 1 + 0.2 * normal(N) if c["post"] else None
        s["gate"] = 1 + 0.3 * normal(N) if c["gate"] else None
        s["scale"] = r.uniform(0.2, 1.0) if c["gate"] else 1.0
    else:
        B, T, V = c["B"], c["T"], c["V"]
        s["scores"] = (4 * normal(B, T, V)).to(TYPES[c["type"]])
        parents = [[-1] + [r.randint(max(0, i - 6), i - 1) if c["tree"] else i - 1 for i in range(1, T)]
                   for _ in range(B)]
        s["parents"] = _int(parents)
        s["tokens"] = torch.randint(V, (B, T), generator=g, device="cuda", dtype=torch.int32)
        # some hundreds of emitted tokens, some of them often; a prompt's tokens as bits
        said = (torch.rand(B, 600, generator=g, device="cuda") ** 3 * V).long().clamp(max=V - 1)
        s["counts"] = torch.zeros(B, V, dtype=torch.int32, device="cuda")
        s["counts"].scatter_add_(1, said, torch.ones_like(said, dtype=torch.int32))
        asked = torch.zeros(B, -(-V // 32) * 32, dtype=torch.bool, device="cuda")
        asked.scatter_(1, torch.randint(V, (B, 900), generator=g, device="cuda"), True)
        s["prompt"] = _words(asked)
        s["repetition"], s["frequency"], s["presence"] = [
            lo + (hi - lo) * torch.rand(B, generator=g, device="cuda") for lo, hi in ((1.0, 1.4), (0.0, 0.5), (-0.2, 0.6))]
        s["bias"] = normal(V) * (torch.rand(V, generator=g, device="cuda") < 0.02) if c["bias"] else None
        # a grammar allows about a quarter of the vocabulary
        s["mask"] = (_words(torch.rand(B, T, -(-V // 32) * 32, generator=g, device="cuda") < 0.25)
                     if c["mask"] else None)
    return s


def _words(bits):
    """Truth values [..., 32 n] as int32 words [..., n], entry v in bit v % 32 of word v // 32."""
    weights = torch.tensor([1 << i for i in range(31)] + [-(1 << 31)], dtype=torch.int64, device="cuda")
    rows = bits.view(-1, bits.shape[-1] // 32, 32)
    step = max(1, (1 << 24) // rows.shape[1])
    return torch.cat([(part * weights).sum(-1).to(torch.int32) for part in rows.split(step)]).view(
        *bits.shape[:-1], -1)


def _bits(words, n):
    """The first n truth values of int32 words."""
    at = torch.arange(n, device="cuda")
    return (words[..., at // 32] >> (at % 32).to(torch.int32)) & 1 != 0


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _call(s)
    return {"rotate": _rotate_case, "append": _append, "prompt": _prompt, "norm": _norm, "adjust": _adjust}[s["op"]](s)


def _call(s):
    import speculative_decode_verification_qmm_gb300 as q
    if s["op"] == "rotate":
        return s["rope"].rotate(s["x"], s["positions"], heads=s["rotated"], dtype=TYPES[s["type"]])
    if s["op"] == "append":
        out = s["cache"].append(0, s["q"], s["k"], s["v"], s["table"], s["lens"], s["starts"], rope=s["rope"])
        return out, s["k_pool"], s["v_pool"]
    if s["op"] == "prompt":
        return s["cache"].attend_prompt(0, s["q"], s["table"], s["lens"], s["starts"])
    if s["op"] == "norm":
        return q.residual_norm(s["r"], s["v"], s["weight"], bias=s["bias"], post_weight=s["post"], gate=s["gate"],
                               scale=s["scale"], eps=EPS, centered=s["centered"], dtype=TYPES[s["type"]])
    return q.adjust_scores(s["scores"], tokens=s["tokens"], parents=s["parents"], counts=s["counts"], prompt=s["prompt"],
                           repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"],
                           bias=s["bias"], mask=s["mask"])


def _turn(s, x, positions):
    """x [..., heads, D] in 32 bits, turned by positions [...]; angles in 64 bits."""
    w = positions.double()[..., None, None] * s["freq"]
    cos, sin = (w.cos() * s["amplitude"]).float(), (w.sin() * s["amplitude"]).float()
    m, x = s["dims"] // 2, x.float()
    a, b = (x[..., :m], x[..., m:2 * m]) if s["half"] else (x[..., :2 * m:2], x[..., 1:2 * m:2])
    pair = a * cos - b * sin, a * sin + b * cos
    turned = torch.cat(pair, -1) if s["half"] else torch.stack(pair, -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * m:]], -1)


def _rotate_case(s):
    n = s["rotated"]
    out = torch.cat([_turn(s, s["x"][:, :, :n], s["positions"]), s["x"][:, :, n:].float()], 2)
    return out.to(TYPES[s["type"]])


def _places(s):
    """Sequence, position in it, page and row of the page of every packed row."""
    row = torch.arange(s["rows"], device="cuda")
    b = (row[:, None] >= s["starts"][1:]).sum(1)
    pos = s["lens"][b] + row - s["starts"][b]
    return b, pos, s["table"][b, pos // s["page"]].long(), pos % s["page"]


def _append(s):
    _, pos, page, at = _places(s)
    t = TYPES[s["type"]]
    s["k_pool"][0][page, :, at] = _turn(s, s["k"], pos).to(t)
    s["v_pool"][0][page, :, at] = s["v"].to(t)
    return _turn(s, s["q"], pos).to(t), s["k_pool"], s["v_pool"]


def _prompt(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    out = torch.empty(s["rows"], Hq, D, dtype=TYPES[s["type"]], device="cuda")
    lse = torch.empty(s["rows"], Hq, device="cuda")
    at = 0
    # a sequence at a time, and so many of its rows that their scores fit
    for b, (L, n) in enumerate(zip(*_lengths(s))):
        pages = s["table"][b, :s["page_counts"][b]].long()
        k, v = (pool[0, pages].transpose(0, 1).reshape(Hkv, -1, D)[:, :L + n].float() for pool in (s["k_pool"], s["v_pool"]))
        step = max(64, int(1e9) // (Hq * (L + n)))
        for i in range(0, n, step):
            m = min(step, n - i)
            end = L + i + m
            x = s["q"][at + i:at + i + m].float().view(m, Hkv, -1, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
            z = torch.matmul(x, k[:, :end].transpose(1, 2)).mul_(D ** -0.5).view(Hkv, -1, m, end)
            row = torch.arange(m, device="cuda")[:, None] + L + i
            z.masked_fill_(torch.arange(end, device="cuda") > row, -math.inf)
            top = z.amax(-1, keepdim=True)
            z.sub_(top).exp_()
            total = z.sum(-1, keepdim=True)
            o = torch.matmul(z.view(Hkv, -1, end), v[:, :end]).view(Hkv, -1, m, D) / total
            out[at + i:at + i + m] = o.permute(2, 0, 1, 3).reshape(m, Hq, D).to(out.dtype)
            lse[at + i:at + i + m] = (top + total.log()).squeeze(-1).permute(2, 0, 1).reshape(m, Hq)
        at += n
    return out, lse


def _normed(s, x, weight, bias=None):
    if s["centered"]:
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    return x if bias is None else x + bias


def _norm(s):
    z = s["v"].float()
    if s["post"] is not None:
        z = _normed(s, z, s["post"])
    if s["gate"] is not None:
        z = s["gate"] * z
    r = s["r"].float() + s["scale"] * z
    return r.to(s["r"].dtype), _normed(s, r, s["weight"], s["bias"]).to(TYPES[s["type"]])


def _ancestors(s):
    """[B, T, T]: whether node j lies on the path to node i, the root left out."""
    T = s["T"]
    up = torch.zeros(s["B"], T, T, dtype=torch.bool, device="cuda")
    row = torch.arange(s["B"], device="cuda")
    for i in range(1, T):
        up[:, i] = up[row, s["parents"][:, i].long()]
        up[:, i, i] = True
    return up


def _adjust(s):
    B, T, V = s["B"], s["T"], s["V"]
    c = s["counts"].float()[:, None].expand(B, T, V).contiguous()
    c.scatter_add_(2, s["tokens"].long()[:, None].expand(B, T, T), _ancestors(s).float())
    x = s["scores"].float()
    r, f, p = (s[k][:, None, None] for k in ("repetition", "frequency", "presence"))
    seen = (c > 0) | _bits(s["prompt"], V)[:, None]
    x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
    x = x - f * c - p * (c > 0)
    if s["bias"] is not None:
        x = x + s["bias"]
    if s["mask"] is not None:
        x = torch.where(_bits(s["mask"], V), x, -math.inf)
    return x.to(s["scores"].dtype)


# ------------------------------------------------------------------ in 64 bits
def exact(c, seed):
    """The definitions in 64 bits, a row, head or sequence at a time."""
    global own
    kept, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = kept
    return {"rotate": _exact_rotate, "append": _exact_append, "prompt": _exact_prompt, "norm": _exact_norm,
            "adjust": _exact_adjust}[c["op"]](s)


def _exact_turn(s, x, positions):
    """As complex numbers: x + i y times a e^(i w)."""
    m = s["dims"] // 2
    y = x.double().clone()
    w = torch.polar(torch.full_like(s["freq"], s["amplitude"])[None].expand(len(positions), m),
                    positions.double()[:, None] * s["freq"])[:, None]
    first = slice(0, m) if s["half"] else slice(0, 2 * m, 2)
    second = slice(m, 2 * m) if s["half"] else slice(1, 2 * m, 2)
    z = torch.complex(y[..., first].clone(), y[..., second].clone()) * w
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rotate(s):
    out = s["x"].double()
    for b in range(s["B"]):
        out[b, :, :s["rotated"]] = _exact_turn(s, s["x"][b, :, :s["rotated"]], s["positions"][b])
    return out


def _exact_append(s):
    lens, counts = _lengths(s)
    pos = torch.cat([torch.arange(L, L + n, device="cuda") for L, n in zip(lens, counts)])
    k = _exact_turn(s, s["k"], pos)
    pools = [s["k_pool"].double(), s["v_pool"].double()]
    at = 0
    for b, (L, n) in enumerate(zip(lens, counts)):
        ids = s["table"][b].tolist()
        for first in range(L // s["page"], (L + n - 1) // s["page"] + 1):
            lo, hi = max(L, first * s["page"]), min(L + n, (first + 1) * s["page"])
            into = slice(lo - first * s["page"], hi - first * s["page"])
            rows = slice(at + lo - L, at + hi - L)
            pools[0][0, ids[first], :, into] = k[rows].transpose(0, 1)
            pools[1][0, ids[first], :, into] = s["v"][rows].double().transpose(0, 1)
        at += n
    return _exact_turn(s, s["q"], pos), pools[0], pools[1]


def _exact_prompt(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    out = torch.empty(s["rows"], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["rows"], Hq, dtype=torch.float64, device="cuda")
    at = 0
    for b, (L, n) in enumerate(zip(*_lengths(s))):
        ids = s["table"][b, :s["page_counts"][b]].long()
        later = torch.ones(n, L + n, dtype=torch.bool, device="cuda").triu(L + 1)
        for h in range(Hq):
            k, v = (pool[0, ids, h * Hkv // Hq].reshape(-1, D)[:L + n].double() for pool in (s["k_pool"], s["v_pool"]))
            z = (s["q"][at:at + n, h].double() @ k.T / math.sqrt(D)).masked_fill_(later, -math.inf)
            lse[at:at + n, h] = torch.logsumexp(z, 1)
            out[at:at + n, h] = torch.exp(z - lse[at:at + n, h, None]) @ v
        at += n
    return out, lse


def _exact_norm(s):
    def normed(x, weight, bias):
        if s["centered"]:
            x = x - x.sum(1, keepdim=True) / s["N"]
        y = x / torch.sqrt((x * x).sum(1, keepdim=True) / s["N"] + EPS) * weight.double()
        return y if bias is None else y + bias.double()

    z = s["v"].double() if s["post"] is None else normed(s["v"].double(), s["post"], None)
    r = s["r"].double() + s["scale"] * (z if s["gate"] is None else z * s["gate"].double())
    return r, normed(r, s["weight"], s["bias"])


def _exact_adjust(s):
    B, T, V = s["B"], s["T"], s["V"]
    out = torch.empty(B, T, V, dtype=torch.float64, device="cuda")
    tokens, parents = s["tokens"].tolist(), s["parents"].tolist()
    asked = _bits(s["prompt"], V)
    for b in range(B):
        r, f, p = (float(s[k][b]) for k in ("repetition", "frequency", "presence"))
        for t in range(T):
            c = s["counts"][b].double()
            path, node = [], t
            while node > 0:
                path.append(tokens[b][node])
                node = parents[b][node]
            c = c + torch.bincount(torch.tensor(path, dtype=torch.int64, device="cuda"), minlength=V)
            x = s["scores"][b, t].double()
            x = torch.where((c > 0) | asked[b], torch.where(x > 0, x / r, x * r), x) - f * c - p * (c > 0).double()
            if s["bias"] is not None:
                x = x + s["bias"].double()
            if s["mask"] is not None:
                x[~_bits(s["mask"][b, t], V)] = -math.inf
            out[b, t] = x
    return out
