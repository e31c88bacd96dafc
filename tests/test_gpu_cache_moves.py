"""qmm_cache_commit and qmm_cache_copy move bits: the pools afterwards equal those
of a plain move, everywhere."""
import numpy as np
import pytest

import speculative_decode_verification_qmm_gb300 as q

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib_built():
    q.load(build_if_missing=True)
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


class Pools:
    def __init__(self, layers, n_pages, page, Hkv, D, max_batch=8, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        # bit patterns of every kind, NaN among them
        mk = lambda: torch.randint(-32768, 32767, (layers, n_pages, Hkv, page, D), generator=g, device="cuda",  # noqa: E731
                                   dtype=torch.int16).view(dtype)
        self.k, self.v, self.page = mk(), mk(), page
        self.cache = q.PagedCache(layers, n_pages, page, Hkv, Hkv, D, dtype=dtype, max_batch=max_batch,
                                  k_pool=self.k, v_pool=self.v)

    def bits(self):
        return self.k.view(torch.int16).clone(), self.v.view(torch.int16).clone()

    def equals(self, want):
        return all(torch.equal(a, b) for a, b in zip(self.bits(), want))


def tables(r, lens, T, page, extra=2):
    need = [(n + T + page - 1) // page for n in lens]
    ids = r.permutation(sum(need) + extra)
    table = np.zeros((len(lens), max(need) + 1), np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, len(ids)


@pytest.mark.parametrize("layers,page,Hkv,D,T", [(1, 16, 1, 64, 2), (3, 16, 5, 128, 9), (2, 32, 8, 64, 64),
                                                 (2, 1024, 3, 128, 40), (5, 64, 2, 128, 1)])
def test_commit(layers, page, Hkv, D, T):
    """Branches of every length: overlapping sources and destinations, first
    children that are in place already, the last node of all."""
    r = np.random.default_rng(T)
    lens = [0, 1, page - 1, page, page + 1, 3 * page - T if 3 * page > T else 5, 77, 130]
    table, n_pages = tables(r, lens, T, page)
    p = Pools(layers, n_pages, page, Hkv, D, seed=T)
    k = [min(T - 1, x) for x in (0, 1, T - 1, T // 2, T // 3, 2, T - 1, (T - 1) // 2)]
    path = np.full((8, T + 3), 12345, np.int32)  # what follows the branch is not looked at
    for b in range(8):
        path[b, :k[b]] = np.sort(r.choice(np.arange(1, T), k[b], replace=False)) if k[b] else []
    path[2, :k[2]] = np.arange(1, k[2] + 1)  # a chain: nothing moves
    want = p.bits()
    for pool in want:
        old = pool.clone()
        for b in range(8):
            for j in range(k[b]):
                s, d = lens[b] + path[b, j], lens[b] + 1 + j
                pool[:, table[b, d // page], :, d % page] = old[:, table[b, s // page], :, s % page]
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = p.cache.commit(dev(table), dev(lens), dev(path)[:, :T], dev([[x, 9] for x in k]))
    assert out.tolist() == [n + 1 + x for n, x in zip(lens, k)]
    assert p.equals(want)
    assert p.cache.sync_status() == q.QMM_OK


def test_commit_refuses_bad_branches():
    """Nodes out of order or range, counts, lengths and pages: the sequence stays as
    it is, its neighbours are committed."""
    page, T = 16, 6
    lens = [20, 20, 20]
    table, n_pages = tables(np.random.default_rng(0), lens, T, page)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    good = [2, 4, 5, -1, -1, -1]
    for bad in (dict(path=[3, 2, 5]), dict(path=[2, 2, 5]), dict(path=[2, 4, 6]), dict(path=[0, 4, 5]),
                dict(path=[-1, 4, 5]), dict(k=6), dict(k=-1), dict(len=10 ** 6), dict(len=-3), dict(page=-7),
                dict(page=n_pages)):
        p = Pools(2, n_pages, page, 2, 64)
        path, accept, tab, ln = [list(good) for _ in range(3)], [[3, 0]] * 3, table.copy(), list(lens)
        path[1][:3] = bad.get("path", good[:3])
        accept = [[3, 0], [bad.get("k", 3), 0], [3, 0]]
        ln[1] = bad.get("len", 20)
        if "page" in bad:
            tab[1, 20 // page] = bad["page"]
        want = p.bits()
        for pool in want:
            old = pool.clone()
            for b in (0, 2):
                for j, s in enumerate(good[:3]):
                    d, s = 21 + j, 20 + s
                    pool[:, table[b, d // page], :, d % page] = old[:, table[b, s // page], :, s % page]
        out = p.cache.commit(dev(tab), dev(ln), dev(path), dev(accept))
        assert out.tolist() == [24, ln[1], 24], bad
        assert p.equals(want), bad
        assert p.cache.sync_status() == q.QMM_ERR_INDEX and p.cache.sync_status() == q.QMM_OK


@pytest.mark.parametrize("layers,page,Hkv,D,n", [(1, 16, 1, 64, 1), (3, 16, 5, 128, 7), (2, 1024, 3, 64, 3),
                                                 (70, 32, 2, 128, 40)])
@pytest.mark.parametrize("partial", [True, False])
def test_copy(layers, page, Hkv, D, n, partial):
    r = np.random.default_rng(n)
    p = Pools(layers, 2 * n + 3, page, Hkv, D, seed=n)
    ids = r.permutation(2 * n + 3)
    src, dst = ids[:n].astype(np.int32), ids[n:2 * n].astype(np.int32)
    rows = r.integers(0, page + 1, n).astype(np.int32)
    rows[0] = page
    if n > 2:
        src[1] = src[0]  # one page to two places
        rows[2] = 0
        dst[2] = src[2]
    want = p.bits()
    for pool in want:
        old = pool.clone()
        for i in range(n):
            m = rows[i] if partial else page
            pool[:, dst[i], :, :m] = old[:, src[i], :, :m]
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    p.cache.copy_pages(dev(src), dev(dst), dev(rows) if partial else None)
    assert p.equals(want)
    assert p.cache.sync_status() == q.QMM_OK


def test_copy_refuses_bad_entries():
    p = Pools(2, 6, 16, 2, 64)
    want = p.bits()
    for pool in want:
        pool[:, 5, :, :4] = pool[:, 1, :, :4]
    dev = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    p.cache.copy_pages(dev(6, 0, 1, -1, 2, 2), dev(0, 6, 5, 3, -9, 4), dev(4, 4, 4, 4, 4, 17))
    assert p.equals(want)
    assert p.cache.sync_status() == q.QMM_ERR_INDEX and p.cache.sync_status() == q.QMM_OK
    p.cache.copy_pages(dev(), dev())
    assert p.equals(want)


def test_refusals():
    p = Pools(1, 4, 16, 2, 64, max_batch=2)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens, path, accept = dev([[0], [1]]), dev([3, 3]), dev([[1, -1], [-1, -1]]), dev([[1, 0], [0, 0]])
    with pytest.raises(q.QmmError) as e:
        p.cache.commit(table, lens, path, accept, lens_out=lens)
    assert e.value.code == q.QMM_ERR_INVALID_ARG
    with pytest.raises(q.QmmError) as e:
        p.cache.commit(dev([[0]] * 3), dev([1] * 3), dev([[-1, -1]] * 3), dev([[0, 0]] * 3))
    assert e.value.code == q.QMM_ERR_SHAPE
    with pytest.raises(q.QmmError) as e:
        p.cache.commit(table, lens, dev([[-1] * 65] * 2), accept)
    assert e.value.code == q.QMM_ERR_SHAPE
    for kw in (dict(path=path[:1]), dict(accept=accept[:, :1]), dict(lens_out=dev([1])), dict(accept=accept.t())):
        with pytest.raises(ValueError):
            p.cache.commit(**{**dict(page_table=table, lens=lens, path=path, accept=accept), **kw})
    with pytest.raises(TypeError):
        p.cache.copy_pages(lens.long(), lens)
    with pytest.raises(ValueError):
        p.cache.copy_pages(lens, lens[:1])
    pool = torch.zeros(1, 4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")

    def code(**kw):
        d = dict(dtype=q.QMM_DT_BF16, n_layers=1, n_pages=4, page_size=16, n_q_heads=2, n_kv_heads=2, head_dim=64,
                 max_batch=2, k_pool=pool, v_pool=pool)
        with pytest.raises(q.QmmError) as e:
            q.qmm_cache_create(**{**d, **kw})
        return e.value.code

    for kw in (dict(n_layers=0), dict(n_pages=0), dict(page_size=8), dict(page_size=24), dict(page_size=2048),
               dict(n_q_heads=3), dict(n_q_heads=130), dict(n_q_heads=1), dict(n_kv_heads=0), dict(head_dim=96),
               dict(max_batch=0), dict(max_batch=5000)):
        assert code(**kw) == q.QMM_ERR_SHAPE, kw
    assert code(dtype=q.QMM_DT_F32) == q.QMM_ERR_INVALID_ARG
    assert code(k_pool=pool.flatten()[4:]) == q.QMM_ERR_ALIGN
    L = q.load()
    h = p.cache.handle
    p.cache.close()
    assert L.qmm_cache_copy(h, 0, None, None, None, None) == q.QMM_ERR_STATE
    assert L.qmm_cache_sync_status(h, None) == q.QMM_ERR_STATE


def test_more_layers_than_a_grid_dimension_holds():
    """What qmm_cache_create accepts can be copied and committed: 40,000 layers, 80,000
    pools of a layer."""
    layers = 40000
    p = Pools(layers, 3, 16, 1, 64, seed=3)
    want = p.bits()
    for pool in want:
        pool[:, 2, :, :9] = pool[:, 0, :, :9]
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    p.cache.copy_pages(dev([0]), dev([2]), dev([9]))
    assert p.equals(want)
    for pool in want:
        pool[:, 2, :, 3] = pool[:, 2, :, 6]
    out = p.cache.commit(dev([[2]]), dev([2]), dev([[4, 0, 0, 0, 0]]), dev([[1, 0]]))
    assert out.tolist() == [4] and p.equals(want)
    assert p.cache.sync_status() == q.QMM_OK
