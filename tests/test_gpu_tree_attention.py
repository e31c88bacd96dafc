"""qmm_tree_attention against its definition in 64 bits: types, head layouts, page
sizes, lengths from nothing to long, trees, strides, and what rows that may not
be seen hold.  Tolerances are derived in paged_util.Attention.reference."""
import ctypes

import numpy as np
import pytest

import speculative_decode_verification_qmm_gb300 as q
from speculative_decode_verification_qmm_gb300 import _lib

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from paged_util import Attention, assert_attention, check  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    q.load(build_if_missing=True)
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


EDGES = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,T,page", [
    (8, 8, 1, 16),     # one row
    (8, 1, 1, 32),     # a decoding step, eight heads to one
    (6, 2, 5, 16),     # 15 rows
    (4, 2, 8, 64),     # 16 rows
    (4, 2, 16, 16),    # 32 rows
    (6, 2, 11, 32),    # 33 rows
    (8, 2, 16, 128),   # 64 rows
    (12, 3, 32, 16),   # 128 rows
    (8, 2, 33, 64),    # 132 rows
    (8, 1, 64, 16),    # 512 rows
])
def test_shapes_and_lengths(dtype, D, Hq, Hkv, T, page):
    rng = np.random.default_rng(T * 7 + Hq)
    lens = EDGES if T <= 16 else [0, 1, 63, 64, 129, 127]
    counts = [int(rng.integers(1, T + 1)) for _ in lens]
    a = Attention(dtype, D, Hq, Hkv, T, page, lens, counts, tree=True, seed=D + T, sigma=1.5)
    assert_attention(a, a.make_cache(q), q)


@pytest.mark.parametrize("T", [1, 7, 16, 40])
def test_chain_without_mask_or_counts(T):
    a = Attention("bf16", 128, 8, 2, T, 16, [0, 5, 300], seed=T)
    assert_attention(a, a.make_cache(q), q, ragged=False)


@pytest.mark.parametrize("T,Hq", [(3, 2), (20, 4), (30, 8)])
def test_long_sequence_is_split(T, Hq):
    """One sequence over the whole grid: every CTA leaves partials to join."""
    a = Attention("bf16", 128, Hq, 1, T, 64, [40001], [T - 1], tree=True, seed=3)
    cache = a.make_cache(q)
    first = assert_attention(a, cache, q)
    # a second call finds the tickets at zero and gives the same bits
    again = a.call(cache)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("T,Hq,Hkv", [(4, 8, 4), (16, 16, 4), (64, 8, 4)])
def test_many_short_sequences(T, Hq, Hkv):
    rng = np.random.default_rng(0)
    lens = [int(x) for x in rng.integers(0, 90, 70)]
    counts = [int(x) for x in rng.integers(0, T + 1, 70)]
    a = Attention("f16", 64, Hq, Hkv, T, 16, lens, counts, tree=True, seed=4)
    assert_attention(a, a.make_cache(q), q)


@pytest.mark.parametrize("T,Hq", [(4, 2), (16, 8)])
def test_rows_that_see_nothing(T, Hq):
    """Mask words of zero: nothing cached gives zeros and -inf, else the prefix alone."""
    a = Attention("bf16", 128, Hq, 2, T, 16, [0, 40], seed=5)
    seen = np.tril(np.ones((2, T, T), bool))
    seen[:, 1] = False
    seen[:, T - 1] = False
    seen[0, 0] = False
    a.set_seen(seen)
    out, lse = assert_attention(a, a.make_cache(q), q)
    assert (out[0, 1] == 0).all() and (lse[0, 1] == -np.inf).all()
    assert torch.isfinite(lse[1]).all()


@pytest.mark.parametrize("T,Hq", [(6, 2), (16, 8), (64, 4)])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf")])
def test_unseen_rows_hold_anything(T, Hq, fill):
    """Stale rows of the pages, and nodes that a row may not see, are NaN or
    infinite; only nodes that see a bad node get a bad result."""
    counts = [T - 1, T, T - 2]
    a = Attention("bf16", 128, Hq, 2, T, 32, [0, 37, 200], counts, tree=True, seed=6, fill=fill)
    bad = 2
    seen = a.seen.copy()
    seen[:, :, bad] = False  # nobody sees node 2 ...
    seen[:, bad, bad] = True  # ... but itself
    a.set_seen(seen)
    a.k[:, bad, :, 3] = fill
    a.v[:, bad, :, 5::7] = fill
    for b, n in enumerate(counts):
        a.q[b, n:] = fill
        a.k[b, n:] = fill
        a.v[b, n:] = fill
    out, lse = a.call(a.make_cache(q))
    a.k[:, bad], a.v[:, bad] = 0, 0
    for b, n in enumerate(counts):
        a.q[b, n:], a.k[b, n:], a.v[b, n:] = 0, 0, 0
    ref, lref, tol, ltol = a.reference()
    rows = [t for t in range(T) if t != bad]
    check(out[:, rows], lse[:, rows], ref[:, rows], lref[:, rows], tol[:, rows], ltol[:, rows])


@pytest.mark.parametrize("T,Hq", [(6, 2), (16, 8)])
def test_seen_nonfinite_values_arrive(T, Hq):
    """An infinite or NaN value element of a node reaches exactly the rows that see
    the node, and exactly its own column."""
    a = Attention("bf16", 128, Hq, 2, T, 16, [33, 8], tree=True, seed=7)
    a.v[:, 1, :, 9] = float("inf")
    a.v[:, 3, :, 20] = float("nan")
    out, _ = a.call(a.make_cache(q))
    sees1, sees3 = torch.from_numpy(a.seen[:, :, 1]).cuda(), torch.from_numpy(a.seen[:, :, 3]).cuda()
    assert torch.equal(torch.isinf(out[..., 9]), sees1[:, :, None].expand(-1, -1, Hq))
    assert torch.equal(torch.isnan(out[..., 20]), sees3[:, :, None].expand(-1, -1, Hq))
    other = [d for d in range(128) if d not in (9, 20)]
    assert torch.isfinite(out[..., other].float()).all()


def test_nan_scores_of_the_prefix_arrive():
    a = Attention("bf16", 64, 4, 2, 3, 16, [20, 20], seed=8)
    a.q[0, 1, 2, 7] = float("nan")
    out, lse = a.call(a.make_cache(q))
    bad = torch.zeros(2, 3, 4, dtype=torch.bool, device="cuda")
    bad[0, 1, 2] = True
    assert torch.equal(torch.isnan(out.float()).all(-1), bad)
    assert torch.equal(torch.isnan(lse), bad) and torch.equal(torch.isnan(out.float()).any(-1), bad)


@pytest.mark.parametrize("T,Hq,Hkv", [(5, 6, 2), (16, 8, 2)])
def test_strides(T, Hq, Hkv):
    a = Attention("f16", 64, Hq, Hkv, T, 16, [7, 130, 64], tree=True, seed=9, strided=True)
    assert not a.q.is_contiguous() and not a.v.is_contiguous()
    wide = torch.full((3, T, Hq + 1, 72), 7.0, dtype=torch.float16, device="cuda")
    out, _ = assert_attention(a, a.make_cache(q), q, out=wide[:, :, :Hq, :64])
    assert (wide[:, :, Hq] == 7).all() and (wide[:, :, :, 64:] == 7).all()


@pytest.mark.parametrize("sigma", [0.0, 30.0])
@pytest.mark.parametrize("T,Hq", [(4, 2), (32, 4)])
def test_flat_and_peaked_scores(sigma, T, Hq):
    """All scores equal, and scores of some hundreds whose running maximum climbs."""
    a = Attention("bf16", 128, Hq, 1, T, 16, [700, 0, 65], tree=True, seed=10, sigma=sigma)
    assert_attention(a, a.make_cache(q), q)


@pytest.mark.parametrize("T,Hq", [(4, 2), (32, 4)])
def test_rising_scores(T, Hq):
    """Every cached row scores higher than those before it, then the order turned."""
    for sign in (1, -1):
        a = Attention("f16", 64, Hq, 1, T, 16, [500], seed=11)
        a.q[:] = 1.0
        for j in range(500):
            a.k_pool[0, int(a.table[0, j // 16]), 0, j % 16] = sign * (j - 250) / 40
        assert_attention(a, a.make_cache(q), q)


def test_layers_and_offsets_past_32_bits():
    """Pools of more than 2^32 elements: the last layer's pages are addressed in 64 bits."""
    layers, page, Hkv, D = 9, 1024, 8, 128
    n_pages = (1 << 32) // (8 * page * Hkv * D) + 1
    k_pool = torch.zeros(layers, n_pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    v_pool = torch.zeros_like(k_pool)
    assert k_pool.numel() > 1 << 32
    a = Attention("bf16", D, 16, Hkv, 3, page, [700, 1030], [3, 2], tree=True, seed=12, layers=1, extra_pages=0)
    last = [n_pages - 1 - i for i in range(a.k_pool.shape[1])]
    k_pool[layers - 1, last] = a.k_pool[0]
    v_pool[layers - 1, last] = a.v_pool[0]
    ref, lref, tol, ltol = a.reference()
    cache = q.PagedCache(layers, n_pages, page, 16, Hkv, D, dtype=torch.bfloat16, max_batch=2, k_pool=k_pool,
                         v_pool=v_pool)
    a.table = n_pages - 1 - a.table
    a.layer = layers - 1
    out, lse = a.call(cache)
    check(out, lse, ref, lref, tol, ltol)
    written = k_pool[layers - 1, int(a.table[1, 1]), :, 1030 - 1024 + 1]
    assert torch.equal(written, a.k[1, 1])
    assert not k_pool[:layers - 1].any()


@pytest.mark.parametrize("T,Hq", [(4, 4), (48, 4)])
def test_side_stream_and_graph(T, Hq):
    a = Attention("bf16", 128, Hq, 2, T, 16, [100, 9], tree=True, seed=13)
    ref, lref, tol, ltol = a.reference()
    cache = a.make_cache(q)
    s = torch.cuda.Stream()
    args = (a.table.cuda(), torch.tensor(a.lens, dtype=torch.int32).cuda())
    mask = a.mask.cuda()
    torch.cuda.synchronize()
    out, lse = cache.attend(0, a.q, a.k, a.v, *args, mask=mask, stream=s)
    s.synchronize()
    check(out, lse, ref, lref, tol, ltol)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            gout, glse = cache.attend(0, a.q, a.k, a.v, *args, mask=mask)
    for _ in range(2):
        gout.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(gout, out) and torch.equal(glse, lse)


@pytest.mark.parametrize("T,Hq", [(2, 2), (40, 4)])
def test_bad_lengths_and_pages_are_reported(T, Hq):
    """Page ids and lengths out of range: nothing outside the pools is touched, the
    status says so, other sequences' results stand, and the handle works on."""
    a = Attention("bf16", 64, Hq, 2, T, 16, [50, 40, 30], seed=14)
    ref, lref, tol, ltol = a.reference()
    good_table, good_lens = a.table.clone(), list(a.lens)
    cache = a.make_cache(q)
    for table_edit, lens_edit in (((1, 0, 10 ** 6), None), ((1, 2, -1), None), (None, (1, -5)), (None, (1, 10 ** 6))):
        a.table, a.lens = good_table.clone(), list(good_lens)
        if table_edit:
            a.table[table_edit[0], table_edit[1]] = table_edit[2]
        if lens_edit:
            a.lens[lens_edit[0]] = lens_edit[1]
        out, lse = a.call(cache)
        torch.cuda.synchronize()
        assert cache.sync_status() == q.QMM_ERR_INDEX
        assert cache.sync_status() == q.QMM_OK
        check(out[::2], lse[::2], ref[::2], lref[::2], tol[::2], ltol[::2])


def _many(B, T, seed=20, **kw):
    """Sequences enough for every warp of the GPU to work alone: B * 8 heads of 128, 16 * B of 64."""
    rng = np.random.default_rng(seed)
    lens = [EDGES[i % len(EDGES)] for i in range(B)]
    counts = [int(x) for x in rng.integers(0, T + 1, B)]
    return Attention("bf16", 128, kw.pop("Hq", 8), 8, T, kw.pop("page", 16), lens, counts, tree=True, seed=seed, **kw)


@pytest.mark.parametrize("dtype,D,Hq,Hkv,T,page,B", [
    ("bf16", 128, 8, 8, 1, 16, 120),
    ("f16", 128, 16, 8, 8, 32, 120),    # 16 rows
    ("bf16", 128, 24, 8, 5, 64, 120),   # 15 rows
    ("f16", 128, 64, 8, 1, 128, 120),
    ("bf16", 64, 40, 20, 7, 16, 100),   # 14 rows
    ("f16", 64, 20, 20, 2, 16, 100),
])
def test_many_sequences(dtype, D, Hq, Hkv, T, page, B):
    rng = np.random.default_rng(T)
    lens = [EDGES[i % len(EDGES)] for i in range(B - 1)] + [900]
    counts = [int(x) for x in rng.integers(0, T + 1, B)]
    a = Attention(dtype, D, Hq, Hkv, T, page, lens, counts, tree=True, seed=D + T, sigma=1.5)
    cache = a.make_cache(q)
    first = assert_attention(a, cache, q)
    again = a.call(cache)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("dtype,D,Hq,Hkv,T,page,B", [
    ("bf16", 128, 24, 8, 7, 16, 120),   # 21 rows
    ("f16", 128, 16, 8, 16, 32, 120),   # 32 rows
    ("bf16", 64, 40, 20, 16, 16, 100),  # 32 rows
])
def test_many_sequences_two_row_tiles(dtype, D, Hq, Hkv, T, page, B):
    rng = np.random.default_rng(T)
    lens = [EDGES[i % len(EDGES)] for i in range(B - 1)] + [400]
    counts = [int(x) for x in rng.integers(0, T + 1, B)]
    a = Attention(dtype, D, Hq, Hkv, T, page, lens, counts, tree=True, seed=D + T, sigma=1.5)
    cache = a.make_cache(q)
    first = assert_attention(a, cache, q)
    again = a.call(cache)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("dtype,D,Hq,Hkv,T,B", [
    ("bf16", 128, 8, 8, 3, 160),    # 3 rows
    ("f16", 64, 24, 8, 16, 160),    # 48 rows
    ("bf16", 64, 12, 4, 50, 310),   # 150 rows: two row tiles
])
def test_one_long_among_many_sequences(dtype, D, Hq, Hkv, T, B):
    """More items than a CTA each, and one that is cut between many CTAs."""
    rng = np.random.default_rng(T)
    lens = [EDGES[i % len(EDGES)] for i in range(B)]
    lens[B // 2] = 30001
    counts = [int(x) for x in rng.integers(0, T + 1, B)]
    a = Attention(dtype, D, Hq, Hkv, T, 16, lens, counts, tree=True, seed=D + T)
    cache = a.make_cache(q)
    first = assert_attention(a, cache, q)
    again = a.call(cache)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("T,fill", [(6, float("nan")), (6, float("inf")), (6, -float("inf")), (20, float("nan"))])
def test_many_sequences_unseen_rows_hold_anything(T, fill):
    bad = 2
    a = _many(120, T, seed=21, fill=fill)
    seen = a.seen.copy()
    seen[:, :, bad] = False
    seen[:, bad, bad] = True
    seen[:, 3] = False  # a row that sees no node
    a.set_seen(seen)
    a.k[:, bad, :, 3] = fill
    a.v[:, bad, :, 5::7] = fill
    for b, n in enumerate(a.counts):
        a.q[b, n:], a.k[b, n:], a.v[b, n:] = fill, fill, fill
    out, lse = a.call(a.make_cache(q))
    a.k[:, bad], a.v[:, bad] = 0, 0
    for b, n in enumerate(a.counts):
        a.q[b, n:], a.k[b, n:], a.v[b, n:] = 0, 0, 0
    ref, lref, tol, ltol = a.reference()
    rows = [t for t in range(T) if t != bad]
    check(out[:, rows], lse[:, rows], ref[:, rows], lref[:, rows], tol[:, rows], ltol[:, rows])


def test_many_sequences_seen_nonfinite_values_arrive():
    a = _many(120, 6, seed=22)
    a.counts = [6] * 120
    a.v[:, 1, :, 9] = float("inf")
    a.v[:, 3, :, 20] = float("nan")
    out, _ = a.call(a.make_cache(q))
    sees1, sees3 = torch.from_numpy(a.seen[:, :, 1]).cuda(), torch.from_numpy(a.seen[:, :, 3]).cuda()
    assert torch.equal(torch.isinf(out[..., 9]), sees1[:, :, None].expand(-1, -1, 8))
    assert torch.equal(torch.isnan(out[..., 20]), sees3[:, :, None].expand(-1, -1, 8))


def test_many_sequences_strides():
    a = _many(120, 5, seed=23, Hq=16, page=32, strided=True)
    assert not a.q.is_contiguous() and not a.v.is_contiguous()
    wide = torch.full((120, 5, 17, 136), 7.0, dtype=torch.bfloat16, device="cuda")
    assert_attention(a, a.make_cache(q), q, out=wide[:, :, :16, :128])
    assert (wide[:, :, 16] == 7).all() and (wide[:, :, :, 128:] == 7).all()


def test_many_sequences_bad_lengths_and_pages_are_reported():
    a = _many(120, 3, seed=24)
    ref, lref, tol, ltol = a.reference()
    good_table, good_lens = a.table.clone(), list(a.lens)
    cache = a.make_cache(q)
    for table_edit, lens_edit in (((2, 0, 10 ** 6), None), ((4, 0, -1), None), (None, -5), (None, 10 ** 6)):
        a.table, a.lens = good_table.clone(), list(good_lens)
        at = table_edit[0] if table_edit else 1
        if table_edit:
            a.table[at, table_edit[1]] = table_edit[2]
        else:
            a.lens[at] = lens_edit
        out, lse = a.call(cache)
        assert cache.sync_status() == q.QMM_ERR_INDEX
        assert cache.sync_status() == q.QMM_OK
        keep = [b for b in range(120) if b != at]
        check(out[keep], lse[keep], ref[keep], lref[keep], tol[keep], ltol[keep])


@pytest.mark.parametrize("T,Hq", [(16, 8), (64, 8)])
def test_expired_waits_are_reported(T, Hq):
    """Waits that give up at once: the call ends, the status says so, and the
    handle works again."""
    a = Attention("bf16", 128, Hq, 2, T, 16, [3000, 9], tree=True, seed=16)
    ref, lref, tol, ltol = a.reference()
    cache = a.make_cache(q)
    q.qmm_debug_set_cache_wait_limit(cache.handle, 0)
    a.call(cache)
    assert cache.sync_status() == q.QMM_ERR_TIMEOUT
    assert cache.sync_status() == q.QMM_OK
    q.qmm_debug_set_cache_wait_limit(cache.handle, 2_000_000_000)
    out, lse = a.call(cache)
    assert cache.sync_status() == q.QMM_OK
    check(out, lse, ref, lref, tol, ltol)
    with pytest.raises(q.QmmError):
        q.qmm_debug_set_cache_wait_limit(cache.handle, -1)


def test_refusals():
    a = Attention("bf16", 64, 4, 2, 3, 16, [5, 6], seed=15)
    cache = a.make_cache(q)
    table, lens = a.table.cuda(), torch.tensor(a.lens, dtype=torch.int32).cuda()
    call = lambda **kw: cache.attend(**{**dict(layer=0, q=a.q, k=a.k, v=a.v, page_table=table, lens=lens), **kw})  # noqa: E731

    def code(**kw):
        with pytest.raises(q.QmmError) as e:
            call(**kw)
        return e.value.code

    assert code(layer=1) == q.QMM_ERR_SHAPE and code(layer=-1) == q.QMM_ERR_SHAPE
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert code(scale=scale) == q.QMM_ERR_INVALID_ARG
    odd = torch.zeros(2, 3, 4, 68, dtype=torch.bfloat16, device="cuda")
    assert code(q=odd[..., :64]) == q.QMM_ERR_ALIGN  # head stride 68
    assert code(q=odd.view(2, 3, -1)[:, :, 4:260].unflatten(2, (4, 64))) == q.QMM_ERR_ALIGN  # pointer
    three = torch.zeros(3, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    kv3 = torch.zeros(3, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert code(q=three, k=kv3, v=kv3, page_table=torch.zeros(3, 2, dtype=torch.int32, device="cuda"),
                lens=torch.zeros(3, dtype=torch.int32, device="cuda")) == q.QMM_ERR_SHAPE  # above max_batch
    long = torch.zeros(2, 65, 4, 64, dtype=torch.bfloat16, device="cuda")
    kvl = torch.zeros(2, 65, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert code(q=long, k=kvl, v=kvl) == q.QMM_ERR_SHAPE
    for kw in (dict(q=a.q.float()), dict(lens=lens.long()), dict(page_table=table.cpu()), dict(k=a.k.half())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(q=a.q[:, :, :3]), dict(lens=lens[:1]), dict(v=a.v[:, :2]), dict(mask=torch.zeros(2, 4, dtype=torch.int64, device="cuda")),
               dict(q=a.q.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError):
            call(**kw)
    L = q.load()
    args = _lib.qmm_attn_args()
    assert L.qmm_tree_attention(cache.handle, None, None) == q.QMM_ERR_INVALID_ARG
    assert L.qmm_tree_attention(cache.handle, ctypes.byref(args), None) == q.QMM_ERR_INVALID_ARG
    h = cache.handle
    cache.close()
    assert L.qmm_tree_attention(h, ctypes.byref(args), None) == q.QMM_ERR_STATE
    assert L.qmm_cache_destroy(h) == q.QMM_ERR_STATE


def test_allocation_failures_leave_nothing():
    pool = torch.zeros(1, 2, 1, 16, 64, dtype=torch.float16, device="cuda")
    for n in (1, 2):  # the workspace and the status word
        q.qmm_debug_fail_allocs(n)
        try:
            with pytest.raises(q.QmmError) as e:
                q.PagedCache(1, 2, 16, 1, 1, 64, dtype=torch.float16, k_pool=pool, v_pool=pool)
            assert e.value.code == q.QMM_ERR_CUDA
        finally:
            q.qmm_debug_fail_allocs(0)
    q.PagedCache(1, 2, 16, 1, 1, 64, dtype=torch.float16, k_pool=pool, v_pool=pool).close()
