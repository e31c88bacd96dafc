"""Tree attention where its other tests do not go: waits that give up at any
point, row coordinates past 32 bits in the tcgen05 kernel, long f16 tails, prompts
in chains of 64.  Bounds as in paged_util.Attention.reference unless a test derives
its own."""
import numpy as np
import pytest

import speculative_decode_verification_qmm_gb300 as q

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from paged_util import Attention, check  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    q.load(build_if_missing=True)
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("lens", [[100, 9], [300, 120, 250], [40000, 9]])
@pytest.mark.parametrize("D,T,Hq", [(128, 16, 8), (64, 16, 8), (128, 64, 8), (64, 64, 8)])
def test_waits_that_give_up_under_copies_in_flight(D, T, Hq, lens):
    """With no time to wait the products give up while the loading warps, which need
    no wait for the first tiles of their rings, still request copies, or have ended
    their loops.  Each call ends, its copies have landed before another CTA has the
    shared memory, and calls right behind it give what they should."""
    a = Attention("bf16", D, Hq, 2, T, 16, lens, tree=True, seed=17)
    ref, lref, tol, ltol = a.reference()
    cache = a.make_cache(q)
    for _ in range(10):
        q.qmm_debug_set_cache_wait_limit(cache.handle, 0)
        a.call(cache)
        a.call(cache)
        q.qmm_debug_set_cache_wait_limit(cache.handle, 2_000_000_000)
        out, lse = a.call(cache)
        assert cache.sync_status() == q.QMM_ERR_TIMEOUT
        assert cache.sync_status() == q.QMM_OK
        check(out, lse, ref, lref, tol, ltol)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,T,Hq", [(64, 64, 8), (128, 64, 8), (128, 43, 6)])
def test_two_row_tiles_over_many_cache_tiles(dtype, D, T, Hq):
    """129 rows a head and more: scores of a cache tile take the place of the tile
    before's probabilities, over long segments and from one segment to the next.
    Equal calls give equal bits."""
    a = Attention(dtype, D, Hq, 2, T, 32, [9000, 130, 2000, 0, 5000], tree=True, seed=18, sigma=1.5)
    ref, lref, tol, ltol = a.reference()
    cache = a.make_cache(q)
    out, lse = a.call(cache)
    check(out, lse, ref, lref, tol, ltol)
    for _ in range(10):
        again = a.call(cache)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("B,L,T,Hq,Hkv", [
    (1, 20000, 3, 2, 1),      # 6 rows a head
    (2, 20000, 16, 4, 2),     # 32 rows
    (1, 20000, 64, 8, 2),     # 256 rows
    (120, 900, 2, 16, 16),    # many short sequences
    (120, 400, 10, 32, 16),   # the same, 20 rows
])
def test_f16_tails_far_below_the_peaks(B, L, T, Hq, Hkv):
    """Every 16th cached row scores highest and has values of 0; all others weigh
    e^-17.5 = 2^-25.2 of it, with values of 1000: they alone make the output.  With
    a base at least 2^7 below a row's maximum, an f16 probability loses at most
    2^-25 of 2^7 of the largest, so the bound's term 2^-25 sum |v| becomes 2^-32
    sum |v| over the number of the largest."""
    a = Attention("f16", 64, Hq, Hkv, T, 32, [L] * B, seed=19)
    a.q.zero_(), a.k.zero_(), a.k_pool.zero_()
    a.q[..., 0] = 8.0  # scores are k[0]
    a.k_pool[..., 0], a.k[..., 0] = -17.5, -17.5
    a.v_pool.fill_(1000.0), a.v.fill_(1000.0)
    a.k_pool[:, :, :, ::16, 0], a.v_pool[:, :, :, ::16] = 0.0, 0.0
    ref, lref, tol, ltol = a.reference()
    assert ref.min() > 1000 * 14 * 2.0 ** -25.3
    peaks = (L + 15) // 16
    total = 1000.0 * (L - peaks + 1 + torch.arange(T, device="cuda"))[:, None, None].double()  # sum |v| of what node t sees
    tol -= 2.0 ** -25 * (total + 1)
    tol += 2.0 ** -32 * total / peaks + 2.0 ** -25
    out, lse = a.call(a.make_cache(q), ragged=False)
    check(out, lse, ref, lref, tol, ltol)


@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 5, 4, 2), (3, 1, 4, 2), (2, 3, 1, 1), (1, 1, 1, 1), (1, 20, 4, 1)])
def test_strides_that_are_never_used(B, T, Hq, Hkv):
    """A dimension of one entry has any stride: it is neither checked nor followed."""
    a = Attention("bf16", 64, Hq, Hkv, T, 16, [33, 5, 60][:B], tree=True, seed=24)
    ref, lref, tol, ltol = a.reference()
    cache = a.make_cache(q)

    def odd(x, stride=3):
        return x.as_strided(x.shape, [stride if n == 1 else s for n, s in zip(x.shape, x.stride())])

    table, lens, mask = a.table.cuda(), torch.tensor(a.lens, dtype=torch.int32).cuda(), a.mask.cuda()
    out = odd(torch.empty(B, T, Hq, 64, dtype=torch.bfloat16, device="cuda"))
    _, lse = cache.attend(0, odd(a.q), odd(a.k), odd(a.v), odd(table, 1), lens, mask=odd(mask, 1), out=out)
    check(out, lse, ref, lref, tol, ltol)
    path = torch.arange(1, T + 1, dtype=torch.int32, device="cuda").repeat(B, 1)
    accept = torch.tensor([[T - 1, 0]] * B, dtype=torch.int32, device="cuda")
    got = cache.commit(odd(table, 1), lens, odd(path, 1), accept)
    assert got.tolist() == [n + T for n in a.lens] and cache.sync_status() == q.QMM_OK
    if B > 1:  # and where there are several entries it is
        with pytest.raises(q.QmmError) as e:
            cache.commit(table.as_strided(table.shape, (1, 1)), lens, path, accept)
        assert e.value.code == q.QMM_ERR_ALIGN


def test_a_step_on_a_side_stream():
    """attend, fork, reserve (which copies the shared last page) and attend again, all
    on one stream that is behind the host and the current stream: the fork's copy
    holds the rows that the first call wrote."""
    g = torch.Generator(device="cuda")
    g.manual_seed(25)
    cache = q.PagedCache(2, 8, 16, 4, 2, 64)
    x = [torch.randn(1, 5, 8, 64, generator=g, device="cuda").bfloat16() for _ in range(2)]
    s = torch.cuda.Stream()

    def attend(seq, layer, part, stream):
        table, lens = cache.tables([seq], stream)
        return cache.attend(layer, part[:, :, :4], part[:, :, 4:6], part[:, :, 6:], table, lens, stream=stream)[0]

    def step(stream):
        a = cache.new_sequence()
        cache.reserve([a], 5, stream)
        for layer in range(2):
            attend(a, layer, x[0], stream)
        cache.advance([a], [5])
        b = cache.fork(a)
        cache.reserve([b], 5, stream)
        assert b.pages != a.pages
        return a, b, [attend(b, layer, x[1], stream) for layer in range(2)]

    a, b, want = step(None)
    pages, length = [a.pages[0], b.pages[0]], a.length
    torch.cuda.synchronize()
    rows = cache.k_pool[:, pages].clone()
    cache.free(a), cache.free(b)
    cache.k_pool.zero_(), cache.v_pool.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)  # some 50 ms
    a, b, got = step(s)
    s.synchronize()
    assert length == a.length == 5 and cache.sync_status() == q.QMM_OK
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert torch.equal(cache.k_pool[:, [a.pages[0], b.pages[0]]][:, :, :, :5], rows[:, :, :, :5])


@pytest.mark.parametrize("D,T,Hq", [(128, 1, 1), (64, 3, 2), (128, 9, 4)])
def test_one_item_over_most_of_the_grid_among_many(D, T, Hq):
    """More items than the join has CTAs for by item, and one that goes on through more
    workers than a warp has lanes."""
    B = 1300
    lens = [i % 19 for i in range(B)]
    lens[700] = 70001
    a = Attention("bf16", D, Hq, 1, T, 16, lens, tree=True, seed=26)
    ref, lref, tol, ltol = a.reference()
    out, lse = a.call(a.make_cache(q))
    check(out, lse, ref, lref, tol, ltol)


@pytest.mark.parametrize("T,Hq", [(16, 16), (48, 16), (64, 32)])
def test_offsets_past_32_bits_with_many_rows(T, Hq):
    """32, 96 and 256 rows a head in the last layer of pools of more than 2^32
    elements: copied rows and written nodes are addressed in 64 bits."""
    layers, page, Hkv, D = 9, 1024, 8, 128
    n_pages = (1 << 32) // (8 * page * Hkv * D) + 1
    k_pool = torch.zeros(layers, n_pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    v_pool = torch.zeros_like(k_pool)
    assert k_pool.numel() > 1 << 32
    a = Attention("bf16", D, Hq, Hkv, T, page, [700, 1010], [T, T - 1], tree=True, seed=27, extra_pages=0)
    last = [n_pages - 1 - i for i in range(a.k_pool.shape[1])]
    k_pool[layers - 1, last] = a.k_pool[0]
    v_pool[layers - 1, last] = a.v_pool[0]
    ref, lref, tol, ltol = a.reference()
    want = a.expect_pools()
    cache = q.PagedCache(layers, n_pages, page, Hq, Hkv, D, max_batch=2, k_pool=k_pool, v_pool=v_pool)
    a.table = n_pages - 1 - a.table
    a.layer = layers - 1
    out, lse = a.call(cache)
    assert cache.sync_status() == q.QMM_OK
    check(out, lse, ref, lref, tol, ltol)
    for pool, w in zip((k_pool, v_pool), want):
        assert torch.equal(pool[layers - 1, last], w[0])
        assert not pool[:layers - 1].any()


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2)])
def test_prompt_in_chains_of_64(Hq, Hkv):
    """A prompt of 150 tokens as chains of 64, 64 and 22: every chunk attends to those
    before it, which its own calls have written."""
    whole = Attention("bf16", 128, Hq, Hkv, 150, 16, [0], seed=28)
    cache = whole.make_cache(q)
    at = 0
    while at < 150:
        n = min(64, 150 - at)
        a = Attention("bf16", 128, Hq, Hkv, n, 16, [at], seed=29)
        a.table, a.k_pool, a.v_pool = whole.table, whole.k_pool, whole.v_pool
        a.q, a.k, a.v = (x[:, at:at + n] for x in (whole.q, whole.k, whole.v))
        out, lse = a.call(cache)
        check(out, lse, *a.reference())
        at += n
    for pool, new in ((whole.k_pool, whole.k), (whole.v_pool, whole.v)):
        ids = whole.table[0].long().cuda()
        assert torch.equal(pool[0, ids].transpose(0, 1).reshape(Hkv, -1, 128)[:, :150], new[0].transpose(0, 1))
