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
