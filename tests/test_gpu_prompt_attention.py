"""PagedCache.attend_prompt against its definition in 64 bits."""
import math

import pytest

import speculative_decode_verification_qmm_gb300 as q

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from step_util import Prompt, check_prompt  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    q.load(build_if_missing=True)
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def run(p, **kw):
    cache = p.make_cache(q)
    out, lse = p.call(cache, **kw)
    torch.cuda.synchronize()
    assert cache.sync_status() == q.QMM_OK
    check_prompt(p, out, lse)
    cache.close()
    return out, lse


SHAPES = [
    # dtype, D, Hq, Hkv, page, lens, counts
    ("bf16", 128, 2, 1, 16, [0], [1]),
    ("f16", 64, 1, 1, 16, [0], [1]),
    ("bf16", 128, 4, 2, 16, [0], [64]),
    ("bf16", 64, 4, 4, 64, [0], [129]),
    ("f16", 128, 4, 1, 128, [0, 1, 127, 128, 129, 5], [1, 127, 128, 129, 0, 31]),   # tile edges, nothing new
    ("f16", 64, 14, 2, 32, [3, 0, 700], [333, 1, 40]),                               # seven heads to a group
    ("bf16", 128, 6, 2, 16, [700], [600]),
    ("bf16", 64, 64, 1, 16, [10, 0], [5, 130]),                                      # two tokens a row tile
    ("bf16", 128, 43, 1, 16, [10], [23]),                                            # 86 or 215 rows of a tile
    ("f16", 128, 3, 3, 16, [0, 250], [300, 700]),                                    # 256 tokens a row tile
    ("bf16", 128, 8, 1, 16, [5000], [3]),                                            # few rows, many parts
    ("f16", 64, 8, 8, 1024, [4000, 0], [2, 1]),
    ("bf16", 64, 8, 2, 16, [17] * 40, [1] * 40),                                     # single tokens of a batch
    ("bf16", 128, 5, 5, 32, [0] * 20, [7, 0, 30] * 6 + [0, 0]),                      # empty ones in between and last
]


@pytest.mark.parametrize("dtype,D,Hq,Hkv,page,lens,counts", SHAPES)
def test_shapes(dtype, D, Hq, Hkv, page, lens, counts):
    run(Prompt(dtype, D, Hq, Hkv, page, lens, counts, seed=D + Hq))


# Row tiles are of 256 rows where sequences have more than 128 on average and the table has room for
# many cache tiles: here always.
WIDE = 400_000


@pytest.mark.parametrize("dtype,D,Hq,Hkv,page,lens,counts", [s for s in SHAPES if sum(s[6]) * s[2] // s[3] > 128 * len(s[6])] + [
    ("f16", 128, 8, 1, 16, [130, 0, 3], [77, 1, 33]), ("bf16", 64, 12, 4, 128, [1, 500], [90, 257]), ("bf16", 128, 7, 7, 64, [0], [1000])])
def test_row_tiles_of_256(dtype, D, Hq, Hkv, page, lens, counts):
    run(Prompt(dtype, D, Hq, Hkv, page, lens, counts, extra_columns=WIDE // page, seed=D + Hq + 1))


@pytest.mark.parametrize("dtype,D,Hq,Hkv,page,lens,counts", [
    ("bf16", 128, 8, 1, 16, [20000], [9]),                     # one item over all SMs
    ("bf16", 128, 16, 2, 64, [20000], [64]),                   # few items of 256 rows
    ("f16", 64, 16, 2, 128, [9000, 300], [40, 3]),
    ("f16", 64, 8, 1, 16, [30000], [70]),
    ("bf16", 64, 4, 2, 32, [6000, 0, 100, 9000], [1, 700, 0, 130]),
    ("f16", 128, 4, 4, 16, [(37 * i) % 300 for i in range(97)], [(11 * i) % 23 for i in range(97)]),  # sequences, 32 at a time
])
def test_long_chains_of_parts(dtype, D, Hq, Hkv, page, lens, counts):
    run(Prompt(dtype, D, Hq, Hkv, page, lens, counts, seed=D + len(lens)))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("sigma", [0.01, 6.0])
def test_flat_and_sharp_rows(dtype, sigma):
    """Scores of a hundredth and of dozens: maxima that grow along the row."""
    run(Prompt(dtype, 128, 4, 2, 16, [300, 0], [200, 500], sigma=sigma, seed=3))


@pytest.mark.parametrize("columns", [0, WIDE // 16])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64)])
def test_growing_scores(dtype, D, columns):
    """Every later key fits better: the running maximum moves in every tile."""
    p = Prompt(dtype, D, 2, 1, 16, [900], [300], extra_columns=columns, seed=4)
    n = 1200
    ids = p.table[0].long()
    grow = torch.linspace(0.1, 4.0, n, device="cuda")
    for j in range(n):
        p.k_pool[0, ids[j // 16], 0, j % 16] = grow[j] * torch.ones(D, device="cuda")
    p.q.fill_(1.0)
    run(p)


@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("counts", [[70, 1, 130], [3, 2, 1]])
def test_rows_that_no_sequence_has(fill, counts):
    """The rest of the last pages, and pages of nobody, hold anything."""
    run(Prompt("bf16", 64, 4, 2, 16, [0, 77, 130], counts, fill=fill, seed=5))
    run(Prompt("f16", 128, 2, 2, 32, [0, 77, 130], counts, fill=fill, seed=6))


@pytest.mark.parametrize("dtype,D,Hq,Hkv,L,n", [("bf16", 128, 2, 2, 100, 260), ("f16", 64, 8, 1, 3, 150), ("bf16", 64, 2, 1, 0, 40),
                                               ("f16", 128, 1, 1, 128, 400)])
@pytest.mark.parametrize("columns", [0, WIDE // 16])
def test_later_rows_that_are_not_finite(dtype, D, Hq, Hkv, L, n, columns):
    """A value or key of a new row that is infinite or NaN counts for the rows from it on."""
    p = Prompt(dtype, D, Hq, Hkv, 16, [L], [n], extra_columns=columns, seed=7)
    ids = p.table[0].long()
    for j, what, where, pool in ((L + 1, math.inf, 3, p.v_pool), (L + n // 2, -math.inf, D - 1, p.v_pool), (L + n // 2 + 1, math.nan, 5, p.v_pool),
                                 (L + n - 1, math.nan, 0, p.v_pool), (L + n - 2, math.nan, 1, p.k_pool)):
        pool[0, ids[j // 16], :, j % 16, where] = what
    run(p)
    # an earlier row's value counts for all
    if L:
        p.v_pool[0, ids[0], :, 0, 9] = math.inf
        run(p)


def test_strides_and_rows_behind_the_last_sequence():
    p = Prompt("bf16", 64, 6, 2, 16, [20, 0, 5], [30, 100, 1], strided=True, extra_rows=9, seed=8)
    wide = torch.full((p.N, p.Hq + 1, p.D + 16), 3.0, dtype=p.dtype, device="cuda")
    lse = torch.full((p.N, p.Hq), 5.0, device="cuda")
    out, _ = run(p, out=wide[:, 1:, 8:8 + p.D], lse=lse)
    n = p.starts[-1]
    assert (wide[n:] == 3).all() and (lse[n:] == 5).all()
    assert (wide[:, 0] == 3).all() and (wide[:, :, :8] == 3).all() and (wide[:, :, 8 + p.D:] == 3).all()


def test_scale_and_layers():
    p = Prompt("f16", 128, 2, 1, 16, [50], [60], layers=3, layer=1, seed=9)
    p.scale = 0.3
    run(p, scale=0.3)


def test_wide_table():
    """Columns that no sequence uses name pages that do not exist."""
    p = Prompt("bf16", 64, 4, 2, 16, [40, 0], [30, 300], extra_columns=70, seed=10)
    for b in range(2):
        p.table[b, -(-(p.lens[b] + p.counts[b]) // 16):] = 1 << 30
    run(p)


def test_offsets_past_32_bits():
    """The last layer's last pages of pools of 5.2 GB each."""
    D, page, Hkv, layers, n_pages = 128, 64, 8, 8, 5000
    assert layers * n_pages * Hkv * page * D > 2 ** 31
    p = Prompt("bf16", D, 16, Hkv, page, [100, 3], [80, 200], seed=11)
    k_pool, v_pool = (torch.zeros(layers, n_pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    have = p.k_pool.shape[1]
    k_pool[-1, -have:], v_pool[-1, -have:] = p.k_pool[0], p.v_pool[0]
    p.table += n_pages - have
    p.k_pool, p.v_pool, p.layer = k_pool, v_pool, layers - 1
    run(p)


@pytest.mark.parametrize("D,columns", [(128, 0), (128, WIDE // 16), (64, 0), (64, WIDE // 16)])
def test_equal_calls_give_equal_bits(D, columns):
    p = Prompt("bf16", D, 8, 2, 16, [1000, 0, 50], [200, 300, 7], extra_columns=columns, seed=12)
    cache = p.make_cache(q)
    a, la = p.call(cache)
    for _ in range(5):
        b, lb = p.call(cache)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)
    cache.close()


def test_stream_and_graph():
    p = Prompt("bf16", 128, 8, 2, 16, [600, 0], [100, 300], seed=13)
    cache = p.make_cache(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = p.call(cache, stream=side)
    side.synchronize()
    check_prompt(p, out, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = p.call(cache)
    for seed in (1, 2):
        new = Prompt("bf16", 128, 8, 2, 16, [600, 0], [100, 300], seed=13 + seed)
        p.q.copy_(new.q)
        graph.replay()
        torch.cuda.synchronize()
        check_prompt(p, out, lse)
    # other lengths in the same buffers
    p.lens, p.counts = [300, 150], [350, 20]
    p.starts = [0, 350, 370]
    p.d_lens.copy_(torch.tensor(p.lens, dtype=torch.int32))
    p.d_starts.copy_(torch.tensor(p.starts, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    check_prompt(p, out, lse)
    assert cache.sync_status() == q.QMM_OK
    cache.close()


def test_bad_sizes_and_pages_are_reported():
    p = Prompt("bf16", 64, 4, 2, 16, [20, 30, 40, 50], [30, 20, 10, 5], seed=14)
    cache = p.make_cache(q)
    width = p.table.shape[1] * 16
    good = p.call(cache)
    for change in (dict(lens=(1, -1)), dict(lens=(1, width - 19)), dict(lens=(1, 2 ** 31 - 1)), dict(starts=(4, p.N + 1)),
                   dict(starts=(2, 20)), dict(table=(1, p.k_pool.shape[1])), dict(table=(1, -1))):
        (name, (at, value)), = change.items()
        lens, starts, table = p.d_lens.clone(), p.d_starts.clone(), p.table.clone()
        if name == "table":
            table[at, 0] = value
        else:
            (lens if name == "lens" else starts)[at] = value
        out = torch.full_like(p.q, 3.0)
        cache.attend_prompt(0, p.q, table, lens, starts, out=out)
        assert cache.sync_status() == q.QMM_ERR_INDEX, change
        assert cache.sync_status() == q.QMM_OK
        # the first sequence is as it was, one that could not be placed is left alone
        assert torch.equal(out[:p.starts[1 if name != "starts" or at != 2 else 0]], good[0][:p.starts[1 if name != "starts" or at != 2 else 0]])
        if name == "lens":
            assert (out[p.starts[1]:p.starts[2]] == 3).all() and torch.equal(out[p.starts[2]:], good[0][p.starts[2]:])
    cache.close()


@pytest.mark.parametrize("counts", [[5], [400]])
@pytest.mark.parametrize("D,columns", [(128, 0), (128, WIDE // 16), (64, 0), (64, WIDE // 16)])
def test_expired_waits(counts, D, columns):
    p = Prompt("bf16", D, 4, 2, 16, [300], counts, extra_columns=columns, seed=15)
    cache = p.make_cache(q)
    q.qmm_debug_set_cache_wait_limit(cache.handle, 0)
    p.call(cache)
    assert cache.sync_status() == q.QMM_ERR_TIMEOUT
    q.qmm_debug_set_cache_wait_limit(cache.handle, 2_000_000_000)
    out, lse = p.call(cache)
    assert cache.sync_status() == q.QMM_OK
    check_prompt(p, out, lse)
    cache.close()


def test_no_rows():
    p = Prompt("bf16", 64, 2, 1, 16, [5, 3], [0, 0], seed=16)
    cache = p.make_cache(q)
    out, lse = p.call(cache)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    # rows, and none of a sequence's
    x = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(x, 3.0)
    cache.attend_prompt(0, x, p.table, p.d_lens, p.d_starts, out=out)
    assert cache.sync_status() == q.QMM_OK and (out == 3).all()
    cache.close()


def test_refusals():
    p = Prompt("bf16", 64, 4, 2, 16, [20, 0], [30, 10], seed=17)
    cache = p.make_cache(q)
    a = dict(layer=0, q=p.q, page_table=p.table, lens=p.d_lens, starts=p.d_starts)

    def refuse(error, **kw):
        with pytest.raises(error):
            cache.attend_prompt(**(a | kw))

    refuse(TypeError, q=p.q.float())
    refuse(TypeError, q=p.q.cpu())
    refuse(ValueError, q=p.q[:, :2])
    refuse(ValueError, q=p.q[None])
    refuse(ValueError, q=p.q.transpose(1, 2).contiguous().transpose(1, 2))
    refuse(ValueError, starts=p.d_starts[:2])
    refuse(TypeError, starts=p.d_starts.long())
    refuse(TypeError, lens=p.d_lens.long())
    refuse(ValueError, page_table=p.table[:1])
    refuse(ValueError, out=torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda"))
    refuse(ValueError, lse=torch.empty(40, 5, device="cuda"))
    for scale in (0.0, -1.0, math.inf, math.nan):
        refuse(q.QmmError, scale=scale)
    refuse(q.QmmError, out=p.q)
    refuse(q.QmmError, layer=1)
    refuse(q.QmmError, layer=-1)
    refuse(q.QmmError, q=torch.empty(40, 4, 72, dtype=torch.bfloat16, device="cuda")[:, :, 4:68])  # not on 16 bytes
    refuse(q.QmmError, q=torch.empty(40, 4, 68, dtype=torch.bfloat16, device="cuda")[:, :, :64])   # a stride of 68
    out, lse = cache.attend_prompt(**a)
    check_prompt(p, out, lse)
    cache.close()


def test_a_destroyed_cache():
    p = Prompt("bf16", 64, 4, 2, 16, [20], [30], seed=18)
    cache = p.make_cache(q)
    handle, cache.handle = cache.handle, None
    q.qmm_cache_destroy(handle)
    with pytest.raises(q.QmmError) as e:
        q.qmm_prompt_attention(handle, 0, p.q, p.table, p.d_lens, p.d_starts, torch.empty_like(p.q))
    assert e.value.code == q.QMM_ERR_STATE


# ------------------------------------------------------------------ both kernels, each by name
def tall(p, cache):
    return q.qmm_debug_prompt_rows(cache.handle, p.B, p.N, p.table.shape[1])


# a table that 1,000,000 rows fit in: 256 rows a tile wherever a sequence has more than 128 on average
FAR = 1_000_000


@pytest.mark.parametrize("dtype,D,Hq,Hkv,page,lens,counts", [s for s in SHAPES if sum(s[6]) * s[2] // s[3] > 128 * len(s[6])])
def test_tables_choose_the_kernel(dtype, D, Hq, Hkv, page, lens, counts):
    for columns, rows in ((0, 128), (FAR // page, 256)):
        p = Prompt(dtype, D, Hq, Hkv, page, lens, counts, extra_columns=columns, seed=D)
        cache = p.make_cache(q)
        assert tall(p, cache) == rows
        out, lse = p.call(cache)
        assert cache.sync_status() == q.QMM_OK
        check_prompt(p, out, lse)
        cache.close()


@pytest.mark.parametrize("columns,rows", [(0, 128), (FAR // 16, 256)])
@pytest.mark.parametrize("dtype,D,Hq,Hkv,L,n", [("bf16", 64, 2, 1, 0, 90), ("bf16", 64, 4, 1, 5, 40), ("f16", 128, 4, 1, 60, 33), ("bf16", 128, 1, 1, 3, 131)])
def test_few_rows_that_are_not_finite(dtype, D, Hq, Hkv, L, n, columns, rows):
    """Values and keys of new rows, of little more than a row tile of 128, by both kernels."""
    p = Prompt(dtype, D, Hq, Hkv, 16, [L], [n], extra_columns=columns, seed=19)
    ids = p.table[0].long()
    for j, what, where, pool in ((L + 1, math.inf, 3, p.v_pool), (L + n // 2, -math.inf, D - 1, p.v_pool), (L + n // 2 + 1, math.nan, 5, p.v_pool),
                                 (L + n - 1, math.nan, 0, p.v_pool), (L + n - 2, math.nan, 1, p.k_pool)):
        pool[0, ids[j // 16], :, j % 16, where] = what
    cache = p.make_cache(q)
    assert tall(p, cache) == rows
    cache.close()
    run(p)


@pytest.mark.parametrize("columns,rows", [(0, 128), (FAR // 16, 256)])
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("counts", [[70], [40, 120]])
def test_expired_waits_of_both_kernels(counts, D, columns, rows):
    p = Prompt("bf16", D, 4, 2, 16, [300] * len(counts), counts, extra_columns=columns, seed=20)
    cache = p.make_cache(q)
    assert tall(p, cache) == rows
    q.qmm_debug_set_cache_wait_limit(cache.handle, 0)
    p.call(cache)
    assert cache.sync_status() == q.QMM_ERR_TIMEOUT
    q.qmm_debug_set_cache_wait_limit(cache.handle, 2_000_000_000)
    out, lse = p.call(cache)
    assert cache.sync_status() == q.QMM_OK
    check_prompt(p, out, lse)
    cache.close()


def test_prompt_rows_refusals():
    p = Prompt("bf16", 64, 4, 2, 16, [20], [30], seed=21)
    cache = p.make_cache(q)
    assert tall(p, cache) == 128
    for sizes in ((0, 30, 4), (2, 30, 4), (1, -1, 4), (1, (1 << 24) + 1, 4), (1, 30, 0), (1, 30, 1 << 27)):
        with pytest.raises(q.QmmError) as e:
            q.qmm_debug_prompt_rows(cache.handle, *sizes)
        assert e.value.code == q.QMM_ERR_SHAPE
    handle = cache.handle
    cache.close()
    with pytest.raises(q.QmmError) as e:
        q.qmm_debug_prompt_rows(handle, 1, 30, 4)
    assert e.value.code == q.QMM_ERR_STATE


def test_two_caches_at_once():
    """Calls of two handles on two streams run side by side and give what they give alone."""
    shapes = [("bf16", 128, 8, 2, 16, [1000, 0], [100, 700]), ("f16", 64, 8, 2, 32, [0, 900], [500, 60])]
    ps = [Prompt(*s, extra_columns=c, seed=22 + i) for i, (s, c) in enumerate(zip(shapes, (0, FAR // 32)))]
    caches = [p.make_cache(q) for p in ps]
    alone = [p.call(c) for p, c in zip(ps, caches)]
    for p, (out, lse) in zip(ps, alone):
        check_prompt(p, out, lse)
    streams = [torch.cuda.Stream() for _ in ps]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    results = [[p.call(c, stream=s) for p, c, s in zip(ps, caches, streams)] for _ in range(20)]
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for both in results:
        for (out, lse), (want, want_lse) in zip(both, alone):
            assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, want_lse)
    for c in caches:
        assert c.sync_status() == q.QMM_OK
        c.close()
