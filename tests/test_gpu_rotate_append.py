"""Rope.rotate and PagedCache.append against their definitions in 64 bits."""
import math

import pytest

import speculative_decode_verification_qmm_gb300 as q

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from step_util import TYPES, Prompt, assert_close, check_prompt, rounding, turn  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    q.load(build_if_missing=True)
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def frequencies(dims):
    return (10000.0 ** (-torch.arange(0, dims, 2, dtype=torch.float64) / dims)).cuda()


def check_rotate(x, positions, freq, half, heads=None, dtype=None, amplitude=1.0, **kw):
    rope = q.Rope(freq, amplitude=amplitude, layout="half" if half else "interleaved")
    want, err = turn(x, positions, freq, half, amplitude, heads)
    out = rope.rotate(x, positions, heads=heads, dtype=dtype, **kw)
    torch.cuda.synchronize()
    assert_close(out, want, err + rounding(want, out.dtype))
    if heads is not None and heads < x.shape[-2]:
        assert torch.equal(out[..., heads:, :], x[..., heads:, :].to(out.dtype))
    return out


def inputs(B, T, H, D, src, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(B, T, H, D, generator=g, device="cuda").to(TYPES[src])
    return x, torch.randint(0, 131072, (B, T), generator=g, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("src", TYPES)
@pytest.mark.parametrize("dst", TYPES)
@pytest.mark.parametrize("half", [True, False])
def test_types(src, dst, half):
    x, pos = inputs(2, 7, 5, 64, src)
    check_rotate(x, pos, frequencies(64), half, dtype=TYPES[dst], heads=4)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("B,T,H,D,dims,heads", [
    (1, 1, 1, 2, 2, 1), (1, 1, 80, 128, 128, 60), (3, 5, 7, 96, 24, 7), (2, 3, 4, 80, 30, 2), (1, 9, 3, 48, 46, 3),
    (2, 2, 2, 9, 4, 1), (1, 1, 2, 1024, 1024, 2), (5, 1, 33, 256, 64, 33), (1, 700, 3, 64, 64, 0), (1, 2, 1000, 6, 6, 999)])
def test_shapes(B, T, H, D, dims, heads, half):
    x, pos = inputs(B, T, H, D, "f32", seed=D)
    check_rotate(x, pos, frequencies(dims), half, heads=heads, dtype=torch.bfloat16)
    check_rotate(x.bfloat16(), pos, frequencies(dims), half, heads=heads, dtype=torch.float16, amplitude=1.3)


def test_far_and_negative_positions():
    """The angle is exact modulo a turn at any position."""
    freq = torch.tensor([1.0, 0.3, 1e-3, 7.5, -0.2], dtype=torch.float64)
    rope = q.Rope(freq)
    pos = [0, 1, -1, 131071, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 999999937]
    x = torch.zeros(len(pos), 1, 10, device="cuda")
    x[:, :, :5] = 1.0
    out = rope.rotate(x, torch.tensor(pos, dtype=torch.int32, device="cuda")).double().cpu()
    two_pi = 2 * 31415926535897932384626433832795028841972
    for i, p in enumerate(pos):
        for k, f in enumerate(freq.tolist()):
            num, den = f.as_integer_ratio()
            turns = p * num * 10 ** 40 % (two_pi * den)  # the remainder of a whole turn, exactly
            w = 2 * math.pi * (turns / (two_pi * den))
            # 2^-21 as for other positions, and 2^-64 of a turn for each of 2^31 positions
            assert abs(out[i, 0, k] - math.cos(w)) <= 2.0 ** -20, (p, f)
            assert abs(out[i, 0, 5 + k] - math.sin(w)) <= 2.0 ** -20, (p, f)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dims", [32, 30])
def test_strides_in_place_and_untouched_places(half, dims):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    big = torch.randn(3, 6, 9, 40, generator=g, device="cuda").bfloat16()
    pos = torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5)
    freq = frequencies(dims)
    for at in (4, 3):  # on a vector's boundary and not
        x = big[1:, :5, 2:8, at:at + 36]
        want, err = turn(x, pos, freq, half)
        kept = big.clone()
        rope = q.Rope(freq, layout="half" if half else "interleaved")
        wide = torch.full((2, 5, 7, 50), 3.0, dtype=torch.float32, device="cuda")
        rope.rotate(x, pos, dtype=torch.float32, out=wide[:, :, :6, 8:44])
        assert_close(wide[:, :, :6, 8:44], want, err + rounding(want, torch.float32))
        assert (wide[:, :, 6] == 3).all() and (wide[..., :8] == 3).all() and (wide[..., 44:] == 3).all()
        assert torch.equal(big, kept)
        again = big.clone()
        y = again[1:, :5, 2:8, at:at + 36]
        assert rope.rotate(y, pos, out=y) is y
        assert_close(y, want, err + rounding(want, torch.bfloat16))
        again[1:, :5, 2:8, at:at + 36] = x
        assert torch.equal(again, big)
    # transposed heads and rows, one row for all sequences
    x = big[:2, :6].transpose(1, 2)[:, :5]
    check_rotate(x, pos.new_zeros(2, 5) + 77, freq, half)
    check_rotate(big[:1, :1].expand(4, 3, 9, 40), torch.arange(12, dtype=torch.int32, device="cuda").view(4, 3), freq, half)


def test_packed_rows_streams_and_graphs():
    x, pos = inputs(1, 11, 4, 64, "f32", seed=2)
    freq = frequencies(64)
    a = check_rotate(x[0], pos[0], freq, True, dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rope = q.Rope(freq)
    b = rope.rotate(x[0], pos[0], dtype=torch.bfloat16, stream=side)
    side.synchronize()
    assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = rope.rotate(x[0], pos[0], dtype=torch.bfloat16)
    x.mul_(2)
    pos.add_(1)
    graph.replay()
    want, err = turn(x[0], pos[0], freq, True)
    assert_close(c, want, err + rounding(want, torch.bfloat16))


def test_values_that_are_not_finite_stay_in_their_pair():
    x, pos = inputs(1, 3, 2, 16, "f32", seed=3)
    x[0, 1, 0, 2] = math.nan
    x[0, 2, 1, 15] = math.inf
    out = q.Rope(frequencies(16)).rotate(x, pos, heads=1)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[0, 1, 0, [2, 10]] = True
    want[0, 2, 1, 15] = True  # a head that is not turned
    assert torch.equal(bad, want)


def test_offsets_past_32_bits():
    H, D = 64, 1024
    T = 2 ** 31 // (H * D) + 3
    x = torch.zeros(1, T, H, D, dtype=torch.bfloat16, device="cuda")
    x[0, -1] = 1.0
    x[0, 1] = 2.0
    pos = torch.full((1, T), 5, dtype=torch.int32, device="cuda")
    freq = frequencies(64)
    out = q.Rope(freq).rotate(x, pos, out=x)
    for row, value in ((T - 1, 1.0), (1, 2.0)):
        want, err = turn(torch.full((1, H, D), value, device="cuda"), pos[0, :1], freq, True)
        assert_close(out[0, row], want[0], (err + rounding(want, torch.bfloat16))[0])
    assert not out[0, 2].any()


def test_rotate_refusals():
    x, pos = inputs(2, 3, 4, 64, "f32")
    rope = q.Rope(frequencies(64))

    def refuse(error, *a, **kw):
        with pytest.raises(error):
            rope.rotate(*a, **kw)

    refuse(TypeError, x.double(), pos)
    refuse(TypeError, x.cpu(), pos)
    refuse(ValueError, x[0, 0], pos)
    refuse(ValueError, x, pos[:1])
    refuse(TypeError, x, pos.long())
    refuse(ValueError, x, pos.t().contiguous().t())
    refuse(ValueError, x.transpose(2, 3), pos)
    refuse(TypeError, x, pos, dtype=torch.int32)
    refuse(TypeError, x, pos, dtype=torch.bfloat16, out=x)
    refuse(ValueError, x, pos, out=x[:, :2])
    for heads in (-1, 5):
        with pytest.raises(q.QmmError) as e:
            rope.rotate(x, pos, heads=heads)
        assert e.value.code == q.QMM_ERR_SHAPE
    with pytest.raises(q.QmmError) as e:  # 64 turned dimensions of 32
        rope.rotate(x[..., :32], pos)
    assert e.value.code == q.QMM_ERR_SHAPE
    with pytest.raises(q.QmmError) as e:  # onto itself with other strides
        rope.rotate(x.view(2, 3, 4, 64).transpose(1, 2)[:, :3, :3], pos, out=x[:, :, :3])
    assert e.value.code == q.QMM_ERR_INVALID_ARG
    with pytest.raises(q.QmmError):
        rope.rotate(torch.empty(1, 1, 1, 1026, device="cuda"), pos[:1, :1])
    assert rope.rotate(x[:0], pos[:0]).shape == (0, 3, 4, 64)


# ------------------------------------------------------------------ appending
class Append(Prompt):
    def __init__(self, dtype, src, D, Hq, Hkv, page, lens, counts, dims, half, seed=0, amplitude=1.0, **kw):
        super().__init__(dtype, D, Hq, Hkv, page, lens, counts, seed=seed, **kw)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 1)
        qkv = torch.randn(self.N, Hq + 2 * Hkv, D, generator=g, device="cuda").to(TYPES[src])
        self.x, self.k, self.v = qkv.split([Hq, Hkv, Hkv], 1)
        self.freq, self.half, self.amplitude = frequencies(dims) if dims else None, half, amplitude
        self.rope = q.Rope(self.freq, amplitude, "half" if half else "interleaved") if dims else None

    def turned(self, x, positions):
        if self.freq is None:
            return x.double(), torch.zeros_like(x, dtype=torch.float64)
        return turn(x, positions, self.freq, self.half, self.amplitude)

    def check(self, cache, positions=None, **kw):
        pools = [self.k_pool.clone(), self.v_pool.clone()]
        out = cache.append(self.layer, self.x, self.k, self.v, self.table, self.d_lens, self.d_starts, rope=self.rope,
                           positions=positions, **kw)
        torch.cuda.synchronize()
        assert cache.sync_status() == q.QMM_OK
        n = self.starts[-1]
        pos = torch.cat([torch.arange(L, L + k, device="cuda") for L, k in zip(self.lens, self.counts)])
        at = pos if positions is None else positions[:n]
        want, err = self.turned(self.x[:n], at)
        assert_close(out[:n], want, err + rounding(want, self.dtype), "queries")
        want, err = self.turned(self.k[:n], at)
        err = err + rounding(want, self.dtype)
        r = 0
        for b in range(self.B):
            for i in range(self.counts[b]):
                j = self.lens[b] + i
                page, row = int(self.table[b, j // self.page]), j % self.page
                assert_close(self.k_pool[self.layer, page, :, row], want[r], err[r], "key")
                pools[0][self.layer, page, :, row] = self.k_pool[self.layer, page, :, row]
                pools[1][self.layer, page, :, row] = self.v[r].to(self.dtype)
                r += 1
        # every other row is as it was
        assert torch.equal(self.k_pool.view(torch.int16), pools[0].view(torch.int16))
        assert torch.equal(self.v_pool.view(torch.int16), pools[1].view(torch.int16))
        return out


@pytest.mark.parametrize("dtype,src", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16"), ("bf16", "f16")])
@pytest.mark.parametrize("D,dims,half", [(128, 128, True), (64, 64, False), (128, 32, True), (64, 10, True), (64, 6, False), (64, 0, True)])
def test_append(dtype, src, D, dims, half):
    a = Append(dtype, src, D, 6, 2, 16, [0, 5, 16, 31, 100], [40, 1, 16, 0, 3], dims, half, seed=dims, layers=2, layer=1)
    cache = a.make_cache(q)
    a.check(cache)
    cache.close()


def test_append_large_pages_positions_and_rows_behind():
    a = Append("bf16", "f32", 128, 5, 5, 1024, [1000, 0], [60, 7], 128, True, extra_rows=5, amplitude=0.5, seed=1)
    cache = a.make_cache(q)
    positions = torch.randint(-5, 500000, (a.N,), dtype=torch.int32, device="cuda")
    out = torch.full((a.N, 5, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    assert a.check(cache, positions=positions, out=out) is out
    assert (out[a.starts[-1]:] == 3).all()
    cache.close()


def test_append_strides_and_keys_alone():
    a = Append("f16", "f32", 64, 4, 2, 32, [10, 20], [30, 40], 64, True, seed=2)
    wide = torch.randn(a.N, 12, 70, device="cuda")
    a.x, a.k, a.v = wide[:, 1:5, 3:67], wide[:, 5:7, 5:69], wide[:, 8:10, 1:65]
    cache = a.make_cache(q)
    out = torch.empty(a.N, 5, 72, dtype=torch.float16, device="cuda")[:, :4, 4:68]
    a.check(cache, out=out)
    k, v = a.k_pool.clone(), a.v_pool.clone()
    a.k_pool.zero_(), a.v_pool.zero_()
    assert cache.append(0, None, a.k, a.v, a.table, a.d_lens, a.d_starts, rope=a.rope) is None
    ids = a.table[0, :2].long()
    for pool, old in ((a.k_pool, k), (a.v_pool, v)):
        assert torch.equal(pool[0, ids].transpose(0, 1).reshape(2, 64, 64)[:, 10:40], old[0, ids].transpose(0, 1).reshape(2, 64, 64)[:, 10:40])
    cache.close()


@pytest.mark.parametrize("src", ["f16", "bf16"])
def test_append_turns_queries_in_place(src):
    """With the queries' own strides, whatever 16-bit type they come in."""
    a = Append("f16", src, 128, 4, 2, 16, [10, 20], [30, 40], 128, True, seed=6)
    cache = a.make_cache(q)
    want = a.check(cache)
    x = a.x.clone()
    out = x.view(torch.float16)
    assert cache.append(0, x, a.k, a.v, a.table, a.d_lens, a.d_starts, rope=a.rope, out=out) is out
    assert torch.equal(out, want)
    other = a.x.clone()
    for bad in (other.view(torch.float16).view(-1).as_strided(other.shape, (other.stride(0) // 2, other.stride(1), 1)),
                other.view(torch.float16).view(-1).as_strided(other.shape, (other.stride(0), other.stride(1) - 8, 1))):
        with pytest.raises(q.QmmError) as e:
            cache.append(0, other, a.k, a.v, a.table, a.d_lens, a.d_starts, rope=a.rope, out=bad)
        assert e.value.code == q.QMM_ERR_INVALID_ARG
    cache.close()


def test_append_bad_places_are_skipped():
    a = Append("bf16", "f32", 64, 2, 1, 16, [20, 30, 40], [30, 20, 10], 64, True, seed=3)
    cache = a.make_cache(q)
    width = a.table.shape[1] * 16
    for change in (dict(lens=-1), dict(lens=width - 5), dict(lens=2 ** 31 - 1), dict(page=-1), dict(page=a.k_pool.shape[1])):
        lens, table = a.d_lens.clone(), a.table.clone()
        if "lens" in change:
            lens[1] = change["lens"]
        else:
            table[1, 2] = change["page"]
        before = a.k_pool.clone()
        cache.append(0, a.x, a.k, a.v, table, lens, a.d_starts, rope=a.rope)
        assert cache.sync_status() == q.QMM_ERR_INDEX
        assert cache.sync_status() == q.QMM_OK
        keep = [int(p) for p in a.table[1, :4]] + [p for p in range(a.k_pool.shape[1]) if p not in a.table.flatten().tolist()]
        if change.get("lens", 0) < 0 or change.get("lens", 0) == 2 ** 31 - 1:
            assert torch.equal(a.k_pool[0, keep], before[0, keep])
    a.check(cache)
    cache.close()


def test_append_refusals():
    a = Append("bf16", "f32", 64, 4, 2, 16, [20, 30], [30, 20], 64, True, seed=4)
    cache = a.make_cache(q)
    args = dict(layer=0, q=a.x, k=a.k, v=a.v, page_table=a.table, lens=a.d_lens, starts=a.d_starts, rope=a.rope)

    def refuse(error, **kw):
        with pytest.raises(error):
            cache.append(**(args | kw))

    refuse(ValueError, k=a.k[:10])
    refuse(TypeError, k=a.k.double())
    refuse(TypeError, v=a.v.bfloat16())
    refuse(ValueError, v=a.v[:, :1])
    refuse(ValueError, q=a.x[:, :3])
    refuse(ValueError, q=None, out=torch.empty(50, 4, 64, dtype=torch.bfloat16, device="cuda"))
    refuse(TypeError, out=torch.empty(50, 4, 64, device="cuda"))
    refuse(TypeError, positions=torch.zeros(50, device="cuda"))
    refuse(ValueError, positions=torch.zeros(49, dtype=torch.int32, device="cuda"))
    refuse(ValueError, starts=a.d_starts[:2])
    refuse(q.QmmError, layer=1)
    refuse(q.QmmError, rope=q.Rope(frequencies(66)))
    # no rows at all
    none = dict(q=a.x[:0], k=a.k[:0], v=a.v[:0], starts=a.d_starts * 0)
    assert cache.append(**(args | none)).shape == (0, 4, 64) and cache.append(**(args | none | dict(q=None))) is None
    one = a.make_cache(q, max_batch=1)
    with pytest.raises(q.QmmError):
        one.append(**args)
    one.close()
    a.check(cache)
    cache.close()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype,Hq,Hkv,D,half", [("bf16", 8, 2, 128, True), ("f16", 7, 1, 64, False)])
def test_prompts_in_pieces_and_drafted_steps(dtype, Hq, Hkv, D, half):
    """A prompt fed in pieces behind another's, its last rows again as a drafted chain
    through attend(): the same cache rows and outputs as in one piece."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    counts = [150, 37]
    n = sum(counts)
    qkv = torch.randn(n, Hq + 2 * Hkv, D, generator=g, device="cuda")
    rope = q.Rope(*q.rope_frequencies(D), layout="half" if half else "interleaved")

    def new():
        c = q.PagedCache(1, 40, 16, Hq, Hkv, D, dtype=TYPES[dtype], max_batch=2)
        c.k_pool.fill_(math.nan), c.v_pool.fill_(math.nan)  # pages of an uncleared pool
        return c, [c.new_sequence(), c.new_sequence()]

    def feed(c, seqs, rows, ns):
        c.reserve(seqs, max(ns))
        table, lens = c.tables(seqs)
        starts = c.starts(ns)
        x, k, v = rows.split([Hq, Hkv, Hkv], 1)
        x = c.append(0, x, k, v, table, lens, starts, rope=rope)
        out, lse = c.attend_prompt(0, x, table, lens, starts)
        c.advance(seqs, ns)
        return out, lse

    whole, ws = new()
    out, lse = feed(whole, ws, qkv, counts)
    a, s = new()
    first = feed(a, s, torch.cat([qkv[:100], qkv[150:151]]), [100, 1])
    second = feed(a, s, torch.cat([qkv[100:130], qkv[151:187]]), [30, 36])
    # the last 20 rows of the first sequence as a chain of nodes
    a.reserve(s[:1], 20)
    table, lens = a.tables(s[:1])
    pos = lens[:, None] + torch.arange(20, dtype=torch.int32, device="cuda")
    turned = rope.rotate(qkv[None, 130:150], pos, heads=Hq + Hkv, dtype=TYPES[dtype])
    x, k, v = turned.split([Hq, Hkv, Hkv], 2)
    third = a.attend(0, x, k, v, table, lens)
    a.advance(s[:1], [20])
    assert a.sync_status() == q.QMM_OK and whole.sync_status() == q.QMM_OK
    got = torch.cat([first[0][:100], second[0][:30], third[0][0], first[0][100:], second[0][30:]])
    got_lse = torch.cat([first[1][:100], second[1][:30], third[1][0], first[1][100:], second[1][30:]])
    for c, seqs in ((whole, ws), (a, s)):
        for b, m in enumerate(counts):
            rows = [p[0, seqs[b].pages].transpose(0, 1).reshape(Hkv, -1, D)[:, :m] for p in (c.k_pool, c.v_pool)]
            if c is whole:
                kept = rows if b == 0 else kept + rows
            else:
                assert torch.equal(rows[0], kept[2 * b]) and torch.equal(rows[1], kept[2 * b + 1])
    p = Prompt.__new__(Prompt)
    p.dtype, p.D, p.Hq, p.Hkv, p.page, p.layer, p.B = TYPES[dtype], D, Hq, Hkv, 16, 0, 2
    p.lens, p.counts, p.starts, p.scale = [0, 0], counts, [0, 150, n], D ** -0.5
    p.table, _ = whole.tables(ws)
    p.k_pool, p.v_pool = whole.k_pool, whole.v_pool
    pos = torch.cat([torch.arange(m, dtype=torch.int32, device="cuda") for m in counts])
    p.q = rope.rotate(qkv[:, :Hq], pos, dtype=TYPES[dtype])
    check_prompt(p, out, lse)
    check_prompt(p, got, got_lse)
    whole.close(), a.close()


# ------------------------------------------------------------------ places out of range
@pytest.mark.parametrize("change", [dict(lens=-1), dict(lens=-2 ** 31), dict(lens=59), dict(lens=64), dict(lens=2 ** 31 - 1),
                                    dict(column=2, page=-1), dict(column=3, page=-2 ** 31), dict(column=2, page="all"),
                                    dict(column=3, page=2 ** 31 - 1)])
@pytest.mark.parametrize("dtype,src,D,dims,half,aligned", [("bf16", "f32", 64, 64, True, True), ("f16", "f16", 128, 96, False, True),
                                                           ("bf16", "bf16", 64, 10, False, False)])
def test_append_writes_only_what_has_a_place(change, dtype, src, D, dims, half, aligned):
    """Both whole pools and the queries, bit for bit: rows without a place leave everything as it
    was, all others are written as in a call without bad places."""
    counts = [30, 20, 10]  # each sequence fills 50 rows of its four pages of 16
    a = Append(dtype, src, D, 4, 2, 16, [20, 30, 40], counts, dims, half, seed=21, layers=3, layer=1, extra_rows=4)
    assert a.table.shape == (3, 4)
    if not aligned:
        wide = torch.randn(a.N, 10, D + 1, device="cuda").to(TYPES[src])
        a.x, a.k, a.v = wide[:, :4, 1:], wide[:, 4:6, 1:], wide[:, 7:9, 1:]
    cache = a.make_cache(q)
    positions = torch.arange(100, 100 + a.N, dtype=torch.int32, device="cuda")  # so that keys do not depend on lens
    old = a.k_pool.clone(), a.v_pool.clone()
    good = torch.full((a.N, 4, D), 3.0, dtype=a.dtype, device="cuda")

    def call(out, lens, table):
        a.k_pool.copy_(old[0]), a.v_pool.copy_(old[1])
        cache.append(a.layer, a.x, a.k, a.v, table, lens, a.d_starts, rope=a.rope, positions=positions, out=out)
        return cache.sync_status()

    assert call(good, a.d_lens, a.table) == q.QMM_OK
    keys = [[pool[a.layer, a.table[b, j // 16], :, j % 16].clone() for b in range(3) for j in range(a.lens[b], 50)] for pool in (a.k_pool, a.v_pool)]
    lens, table = a.d_lens.clone(), a.table.clone()
    if "lens" in change:
        lens[1] = change["lens"]
    else:
        table[1, change["column"]] = a.k_pool.shape[1] if change["page"] == "all" else change["page"]
    out = torch.full_like(good, 3.0)
    assert call(out, lens, table) == q.QMM_ERR_INDEX
    assert cache.sync_status() == q.QMM_OK
    want, want_out, written = [p.clone() for p in old], torch.full_like(good, 3.0), 0
    r = 0
    for b in range(3):
        for i in range(counts[b]):
            j = int(lens[b]) + i
            if lens[b] >= 0 and j < 64 and 0 <= int(table[b, j // 16]) < a.k_pool.shape[1]:
                for pool, rows in zip(want, keys):
                    pool[a.layer, table[b, j // 16], :, j % 16] = rows[r]
                want_out[r] = good[r]
                written += 1
            r += 1
    assert written < r == 60
    for got, w in ((a.k_pool, want[0]), (a.v_pool, want[1]), (out, want_out)):
        assert torch.equal(got.view(torch.int16), w.view(torch.int16))
    cache.close()
